// tree_mla_pair.cu -- the tree attention for more than 64 query rows (node, head) of a sequence:
// two CTAs of a cluster work on 128 query rows and 128 keys at a time with paired tensor-core
// instructions (cta_group::2, M = 128), which hold 64 rows x 512 outputs in half of each CTA's
// tensor memory and let each CTA keep only its half of every B operand:
//     S = Q K^T     A: this CTA's 64 rows of Q       B: K, this CTA's 64 keys x 512 dims
//     O += P V      A: this CTA's 64 rows of P       B: V, 128 keys x this CTA's 256 dims
// A key tile is thus widened one and a half times (K and V copies of its own quarter) for 128 query rows, where the
// one-CTA kernel (tree_mla.cu) widens it once for 64 and reads its operands from shared memory
// twice as often; shared-memory bandwidth is what bounds both. Roles of the 13 warps of a CTA:
//   * warps 4-11 (widening): K(t + 1) once S(t) is done, V(t) once O of t - 1 is done; the codes of
//     the tile after are in registers meanwhile;
//   * warp 12 of the first CTA (tensor cores): S(t + 1), then O of t, for both CTAs;
//   * warps 0-3 (softmax): one thread per row and half of the keys (tensor-memory lane = row, the
//     upper 64 lanes hold the tile's upper 64 keys): references, sums and P' as in tree_mla.cu, the
//     two halves of a row meeting only when a reference moves.
// K and V have one buffer each: while S(t + 1) runs V(t) is written, while O of t runs K(t + 2).
#include "tree_mla_common.cuh"

namespace glm {

namespace {

using namespace tree;

constexpr int kPrWarpWiden = 4;
constexpr int kPrWarpMma = 12;
constexpr int kPrThreads = 13 * 32;
constexpr int kPrRows = 64;                    // query rows of a CTA
constexpr int kPrKeys = 128;                   // keys of a tile
constexpr int kPrMeta = 3;                     // tiles whose scales are kept
constexpr uint32_t kPrSCol = 256;              // two score accumulators of 64 columns after the output's 256

enum PrBar { kPbQ = 0, kPbK, kPbV, kPbP, kPbSFree, kPbS = 6, kPbDone = 8, kPbMeta = 10, kPbCount = 13 };

struct PrLayout {
    static constexpr int kQ = 0;                                 // 8 row groups x 64 dim groups x 128 B
    static constexpr int kK = kQ + kPrRows * 1024;               // 8 key groups x 64 dim groups x 128 B
    static constexpr int kV = kK + 64 * 1024;                    // 16 key groups x 32 own dim groups x 128 B
    static constexpr int kP = kV + kPrKeys * 512;                // 8 row groups x 16 key groups x 128 B
    static constexpr int kScl = kP + kPrRows * kPrKeys * 2;      // [3][128] row scales
    static constexpr int kMax = kScl + kPrMeta * kPrKeys * 4;    // [3][16] largest finite scale of 8 keys
    static constexpr int kValid = kMax + kPrMeta * 16 * 4;       // [3][16] bytes: which rows are keys
    static constexpr int kRed = kValid + kPrMeta * 16;           // [128]
    static constexpr int kRowK = kRed + 128 * 4;                 // [64] score factors
    static constexpr int kBar = kRowK + kPrRows * 4;
    static constexpr int kTmem = kBar + kPbCount * 8;
    static constexpr int kBytes = kTmem + 8;
    static_assert(kBar % 8 == 0 && kScl % 16 == 0 && kValid % 16 == 0, "alignment");
    static_assert(kBytes <= 232448, "shared memory of one CTA");
};

__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// One arrival on a barrier of the pair's first CTA.
__device__ __forceinline__ void arrive_leader(uint32_t mbar) {
    asm volatile(
        "{\n\t.reg .b32 r;\n\t"
        "mapa.shared::cluster.u32 r, %0, 0;\n\t"
        "mbarrier.arrive.release.cluster.shared::cluster.b64 _, [r];\n\t}\n" ::"r"(mbar)
        : "memory");
}
__device__ __forceinline__ bool cluster_wait(uint32_t mbar, uint32_t parity, uint32_t limit) {
    for (uint32_t i = 0; i < limit; i++) {
        uint32_t ok;
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
            "selp.u32 %0, 1, 0, p;\n\t}\n"
            : "=r"(ok)
            : "r"(mbar), "r"(parity)
            : "memory");
        if (ok) return true;
    }
    return false;
}
__device__ __forceinline__ void mma_pair(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}\n" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(accumulate));
}
// Arrive on the barrier of this offset in both CTAs when the products issued so far are done.
__device__ __forceinline__ void commit_pair(uint32_t mbar) {
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(mbar),
        "h"(static_cast<uint16_t>(3))
        : "memory");
}

template <int kFmt>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kPrThreads, 1)
    tree_mla_pair_kernel(TreeArgs a, TreePlan plan, float *__restrict__ part_acc, float *__restrict__ part_ml) {
    using L = PrLayout;
    using R = Row<kFmt>;
    pdl_begin(a.q, a.cache, a.rows, a.row_len, a.draft, a.mask, a.n_tree);
    extern __shared__ __align__(128) unsigned char smem[];
    float *scl = reinterpret_cast<float *>(smem + L::kScl);
    float *smx = reinterpret_cast<float *>(smem + L::kMax);
    uint8_t *val = reinterpret_cast<uint8_t *>(smem + L::kValid);
    float *red = reinterpret_cast<float *>(smem + L::kRed);
    float *rowk = reinterpret_cast<float *>(smem + L::kRowK);
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + L::kTmem);
    const uint32_t bar0 = tc::smem_addr(smem + L::kBar);
    auto bar = [&](int i) { return bar0 + 8u * static_cast<uint32_t>(i); };

    const int cta = blockIdx.x & 1, qt = blockIdx.x >> 1, b = blockIdx.y, part = blockIdx.z;
    const int tid = threadIdx.x, lane = tid & 31;
    const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
    const int H = a.n_heads, n_rows_q = a.n_nodes * H;
    const int r0 = qt * 2 * kPrRows + cta * kPrRows;          // this CTA's first query row
    const int parts = plan.parts;
    const bool direct = parts == 1;

    // the sequence's tiles [0, tiles), those of the list first, and this part's [t0, t1)
    const int plen = list_len(a, b), tree_n = tree_len(a, b);
    const int prefix = (plen + kPrKeys - 1) / kPrKeys, tiles = prefix + (tree_n > 0 ? 1 : 0);
    const int run = direct ? tiles : run_tiles(a, plan, kPrKeys);
    const int t0 = static_cast<int>(min(static_cast<int64_t>(tiles), static_cast<int64_t>(part) * run));
    const int t1 = min(tiles, t0 + run);
    const int live = tree_n * H;                             // query rows of the tree
    const int n_tiles = qt * 2 * kPrRows < live ? t1 - t0 : 0;
    // where query row r goes: the output, or this part's partial
    auto row_at = [&](int r) -> int64_t {
        if (direct) return static_cast<int64_t>(b) * n_rows_q + r;
        const int node = r / H;
        return ((static_cast<int64_t>(b) * a.n_nodes + node) * parts + part) * H + (r - node * H);
    };
    if (n_tiles == 0) {   // no key for the pair, or no node of the tree
        if (direct)
            for (int i = tid; i < kPrRows * 64; i += kPrThreads) {
                const int r = r0 + (i >> 6);
                if (r < n_rows_q) reinterpret_cast<uint4 *>(a.out + row_at(r) * kLatent)[i & 63] = make_uint4(0u, 0u, 0u, 0u);
            }
        if (tid < kPrRows && r0 + tid < n_rows_q) {
            const int64_t o = row_at(r0 + tid);
            if (!direct) {
                part_ml[2 * o] = -INFINITY;
                part_ml[2 * o + 1] = 0.0f;
            } else if (a.lse) {
                a.lse[o] = -INFINITY;
            }
        }
        return;
    }
    if (warp == kPrWarpMma) {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(tc::smem_addr(tmem_slot))
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
        tc::fence_before_sync();
        if (lane == 0) {
            tc::mbar_init(bar(kPbQ), 8);                      // (both CTAs' warps arrive at the first's)
            tc::mbar_init(bar(kPbK), 16);
            tc::mbar_init(bar(kPbV), 16);
            tc::mbar_init(bar(kPbP), 8);
            for (int i = 0; i < 2; i++) {
                tc::mbar_init(bar(kPbSFree + i), 8);
                tc::mbar_init(bar(kPbS + i), 1);
                tc::mbar_init(bar(kPbDone + i), 1);
            }
            for (int i = 0; i < kPrMeta; i++) tc::mbar_init(bar(kPbMeta + i), 8);
            tc::mbar_fence_init();
        }
    }
    __syncthreads();
    cluster_sync();
    tc::fence_after_sync();
    const uint32_t tmem = *tmem_slot;
    bool ok = true;
    auto wait = [&](int i, int use) {
        if (ok && !cluster_wait(bar(i), static_cast<uint32_t>(use & 1), kWaitLimit)) ok = false;
    };

    if (warp >= kPrWarpWiden && warp < kPrWarpMma) {
        // ---------------- widening ----------------
        constexpr int kKp = R::kPieces / 4;                   // pieces of K of a thread
        constexpr int kVp = R::kPieces / 8;                   // pieces of V of a thread, in each of two rows
        const int w = warp - kPrWarpWiden, jl = lane & 7, part4 = lane >> 3;
        const int32_t *list = a.rows + static_cast<int64_t>(b) * a.width;
        // the row of key 64 half + 8 w + jl of tile t, -1: none
        auto row_of = [&](int t, int half) -> int64_t {
            if (t >= t1) return -1;
            const int k = half * 64 + w * 8 + jl;
            if (t < prefix) {
                const int j = t * kPrKeys + k;
                const int r = j < plen ? __ldg(list + j) : -1;
                return (r >= 0 && r < a.n_rows) ? r : -1;
            }
            return k < tree_n ? static_cast<int64_t>(b) * a.n_nodes + k : -1;
        };
        auto base_of = [&](int t) { return t < prefix ? a.cache : a.draft; };
        // pieces of the own 256 dims: the row's piece of own piece m
        auto own_piece = [&](int m) { return (m / (R::kPieces / 4)) * (R::kPieces / 2) + cta * (R::kPieces / 4) + m % (R::kPieces / 4); };
        uint4 kv[kKp], vv[2][kVp];
        uint32_t kes[R::kFp4 ? kKp : 1], ves[2][R::kFp4 ? kVp : 1];
        float sc[2];
        int64_t kr[2] = {-1, -1}, vr[2] = {-1, -1};                                 // rows of the tile held (K) and of V's, by half of the tile
        auto load_k = [&](int t) {
            const uint8_t *base = base_of(t);
            const int64_t own = cta ? kr[1] : kr[0];
#pragma unroll
            for (int h = 0; h < 2; h++) sc[h] = R::scale(base, kr[h]);
#pragma unroll
            for (int i = 0; i < kKp; i++) {
                kv[i] = R::codes(base, own, 4 * i + part4);
                if constexpr (R::kFp4) kes[i] = R::block_scales(base, own, 4 * i + part4);
            }
        };
        auto load_v = [&](int t) {
            const uint8_t *base = base_of(t);
#pragma unroll
            for (int h = 0; h < 2; h++)
#pragma unroll
                for (int i = 0; i < kVp; i++) {
                    const int k = own_piece(4 * i + part4);
                    vv[h][i] = R::codes(base, vr[h], k);
                    if constexpr (R::kFp4) ves[h][i] = R::block_scales(base, vr[h], k);
                }
        };
        auto store_k = [&](int t) {
            const int m = (t - t0) % kPrMeta;
            const bool drafts = t >= prefix;
            unsigned char *row = smem + L::kK + w * 8192 + jl * 16;
#pragma unroll
            for (int i = 0; i < kKp; i++)
#pragma unroll
                for (int u = 0; u < R::kLines; u++)
                    *reinterpret_cast<uint4 *>(row + (R::kLines * (4 * i + part4) + u) * 128) =
                        R::line(kv[i], R::kFp4 ? kes[R::kFp4 ? i : 0] : 0u, u, drafts);
#pragma unroll
            for (int h = 0; h < 2; h++) {
                // a drafted row with NaN codes: its scale makes every score with it NaN
                if (kFmt != kFmtInt8 && drafts) {
                    const unsigned nan = __ballot_sync(0xffffffffu, R::has_nan(a.draft, kr[h], part4));
                    if ((nan >> jl) & 0x01010101u) sc[h] = __int_as_float(0x7fc00000);
                }
                const unsigned valid = __ballot_sync(0xffffffffu, kr[h] >= 0) & 0xffu;
                float mx = fabsf(sc[h]) < INFINITY ? sc[h] : 0.0f;
#pragma unroll
                for (int o = 4; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
                if (lane < 8) scl[m * kPrKeys + h * 64 + w * 8 + lane] = sc[h];
                if (lane == 0) {
                    smx[m * 16 + h * 8 + w] = mx;
                    val[m * 16 + h * 8 + w] = static_cast<uint8_t>(valid);
                }
            }
            tc::fence_proxy_async();
            __syncwarp();
            if (lane == 0) {
                tc::mbar_arrive(bar(kPbMeta + m));
                arrive_leader(bar(kPbK));
            }
        };
        auto store_v = [&](int t) {
            const bool drafts = t >= prefix;
#pragma unroll
            for (int h = 0; h < 2; h++) {
                unsigned char *row = smem + L::kV + (h * 8 + w) * 4096 + jl * 16;
#pragma unroll
                for (int i = 0; i < kVp; i++)
#pragma unroll
                    for (int u = 0; u < R::kLines; u++)
                        *reinterpret_cast<uint4 *>(row + (R::kLines * (4 * i + part4) + u) * 128) =
                            R::line(vv[h][i], R::kFp4 ? ves[h][R::kFp4 ? i : 0] : 0u, u, drafts);
            }
            tc::fence_proxy_async();
            __syncwarp();
            if (lane == 0) arrive_leader(bar(kPbV));
        };
        int64_t next[2];
#pragma unroll
        for (int h = 0; h < 2; h++) vr[h] = kr[h] = row_of(t0, h);
        load_k(t0);
        load_v(t0);
#pragma unroll
        for (int h = 0; h < 2; h++) next[h] = row_of(t0 + 1, h);
        store_k(t0);
        // rows of tile t + 1 (K) are taken over by V one step later
#pragma unroll
        for (int h = 0; h < 2; h++) kr[h] = next[h];
        if (n_tiles > 1) load_k(t0 + 1);
#pragma unroll
        for (int h = 0; h < 2; h++) next[h] = row_of(t0 + 2, h);
        for (int i = 0; i < n_tiles; i++) {
            const int t = t0 + i;
            if (i + 1 < n_tiles) {
                wait(kPbS + (i & 1), i >> 1);                 // S(t) is done: K is free
                store_k(t + 1);
            }
#pragma unroll
            for (int h = 0; h < 2; h++) vr[h] = kr[h];        // the rows of t + 1
            if (i + 2 < n_tiles) {
#pragma unroll
                for (int h = 0; h < 2; h++) kr[h] = next[h];
                load_k(t + 2);
#pragma unroll
                for (int h = 0; h < 2; h++) next[h] = row_of(t + 3, h);
            }
            if (i > 0) wait(kPbDone + ((i - 1) & 1), (i - 1) >> 1);   // O of t - 1 is done: V is free
            store_v(t);
            if (i + 1 < n_tiles) load_v(t + 1);
        }
    } else if (warp == kPrWarpMma) {
        // ---------------- tensor cores (the first CTA's, for both) ----------------
        if (cta == 0) {
            constexpr uint32_t id_s = tc::idesc_f16(128, kPrKeys, false, false);
            constexpr uint32_t id_o = tc::idesc_f16(128, 256, false, true);
            const uint64_t dq = tc::desc(tc::smem_addr(smem + L::kQ), 128, 8192);
            const uint64_t dk = tc::desc(tc::smem_addr(smem + L::kK), 128, 8192);
            const uint64_t dv = tc::desc(tc::smem_addr(smem + L::kV), 4096, 128);
            const uint64_t dp = tc::desc(tc::smem_addr(smem + L::kP), 128, 2048);
            auto accumulate = [&](int i) {   // O += P(i) V(i): two products of 256 dims, K = 128 keys
                wait(kPbV, i);
                wait(kPbP, i);
                ok = __all_sync(0xffffffffu, ok);
                tc::fence_after_sync();
                if (tc::elect_one()) {
#pragma unroll
                    for (int ks = 0; ks < kPrKeys / 16; ks++)
#pragma unroll
                        for (int j = 0; j < 2; j++)
                            mma_pair(tmem + j * 128, dp + ((ks * 256) >> 4), dv + ((ks * 2 * 4096 + j * 2048) >> 4), id_o,
                                     (i > 0 || ks > 0) ? 1u : 0u);
                    commit_pair(bar(kPbDone + (i & 1)));
                }
                __syncwarp();
            };
            wait(kPbQ, 0);
            for (int i = 0; i < n_tiles; i++) {
                wait(kPbK, i);
                if (i >= 2) wait(kPbSFree + (i & 1), (i >> 1) - 1);
                ok = __all_sync(0xffffffffu, ok);
                tc::fence_after_sync();
                if (tc::elect_one()) {   // S(i) = Q K(i)^T: N = 128 keys, K = 512
#pragma unroll
                    for (int ks = 0; ks < kLatent / 16; ks++)
                        mma_pair(tmem + kPrSCol + (i & 1) * 64, dq + ((ks * 256) >> 4), dk + ((ks * 256) >> 4), id_s,
                                 ks > 0 ? 1u : 0u);
                    commit_pair(bar(kPbS + (i & 1)));
                }
                __syncwarp();
                if (i > 0) accumulate(i - 1);
            }
            accumulate(n_tiles - 1);
        }
    } else {
        // ---------------- softmax ----------------
        // the query rows as fp16 first: each warp two groups of 8 rows, four lanes a row
#pragma unroll 1
        for (int g = warp; g < kPrRows / 8; g += 4) {
            const int qr = g * 8 + (lane & 7);
            const bool real = r0 + qr < live;
            const uint4 *src = reinterpret_cast<const uint4 *>(
                a.q + (static_cast<int64_t>(b) * n_rows_q + (real ? r0 + qr : 0)) * kLatent);
            uint4 v[16];
            unsigned mx = 0u;
#pragma unroll
            for (int i = 0; i < 16; i++) {
                v[i] = real ? __ldg(src + 4 * i + (lane >> 3)) : make_uint4(0u, 0u, 0u, 0u);
                mx = max(mx, bf16_absmax(v[i]));
            }
            mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, 8));
            mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, 16));
            const int e = query_exponent(mx);
            const float f = pow2f_exact(e);
            if (lane < 8) rowk[qr] = a.sm_scale * 1.4426950408889634f * pow2f_exact(-e);
#pragma unroll
            for (int i = 0; i < 16; i++)
                *reinterpret_cast<uint4 *>(smem + L::kQ + g * 8192 + (4 * i + (lane >> 3)) * 128 + (lane & 7) * 16) =
                    bf16_to_f16x8(v[i], f);
        }
        tc::fence_proxy_async();
        __syncwarp();
        if (lane == 0) arrive_leader(bar(kPbQ));
        named_sync(1, 128);

        const int row = (warp & 1) * 32 + lane, half = warp >> 1;       // tensor-memory lane 32 warp + lane
        const uint32_t lanes = static_cast<uint32_t>(warp * 32) << 16;
        const int r = r0 + row;
        const float qk = rowk[row];
        const uint64_t seen = r < live ? a.mask[static_cast<int64_t>(b) * a.n_nodes + r / H] : 0ull;
        float ref = 0.0f, l = 0.0f, sigma = 0.0f;
        bool none = true;                                               // the row has seen no key
        unsigned char *prow = smem + L::kP + (row >> 3) * 2048 + half * 1024 + (row & 7) * 16;
        for (int i = 0; i < n_tiles; i++) {
            const int t = t0 + i, m = i % kPrMeta;
            wait(kPbMeta + m, i / kPrMeta);
            wait(kPbS + (i & 1), i >> 1);
            ok = __all_sync(0xffffffffu, ok);
            tc::fence_after_sync();
            float x[64];
            {
                uint32_t s0[32], s1[32];
                tc::tmem_ld32(tmem + lanes + kPrSCol + (i & 1) * 64, s0);
                tc::tmem_ld32(tmem + lanes + kPrSCol + (i & 1) * 64 + 32, s1);
                tc::tmem_wait_ld();
                tc::fence_before_sync();
                __syncwarp();
                if (lane == 0) arrive_leader(bar(kPbSFree + (i & 1)));
                const float4 *sc4 = reinterpret_cast<const float4 *>(scl + m * kPrKeys + half * 64);
#pragma unroll
                for (int e = 0; e < 64; e += 4) {
                    const float4 s = sc4[e >> 2];
                    const uint32_t *v = e < 32 ? &s0[e] : &s1[e - 32];
                    x[e] = fmaf(__uint_as_float(v[0]) * qk, s.x, -ref);
                    x[e + 1] = fmaf(__uint_as_float(v[1]) * qk, s.y, -ref);
                    x[e + 2] = fmaf(__uint_as_float(v[2]) * qk, s.z, -ref);
                    x[e + 3] = fmaf(__uint_as_float(v[3]) * qk, s.w, -ref);
                }
            }
            const uint2 vw = *reinterpret_cast<const uint2 *>(val + m * 16 + half * 8);
            uint64_t keys = (static_cast<uint64_t>(vw.y) << 32) | vw.x;
            if (t >= prefix) keys &= half == 0 ? seen : 0ull;        // what the node sees of the drafts
            if (keys != ~0ull) {
#pragma unroll
                for (int e = 0; e < 64; e++)
                    if (!((keys >> e) & 1ull)) x[e] = -INFINITY;
            }
            float mx = -INFINITY;
#pragma unroll
            for (int e = 0; e < 64; e++) mx = fmaxf(mx, x[e]);
            const float4 *m4 = reinterpret_cast<const float4 *>(smx + m * 16);
            float smax = 0.0f;
#pragma unroll
            for (int e = 0; e < 4; e++) {
                const float4 v = m4[e];
                smax = fmaxf(smax, fmaxf(fmaxf(v.x, v.y), fmaxf(v.z, v.w)));
            }
            const bool over = none ? mx > -INFINITY : mx > kGrow;
            const bool grow = smax > 16.0f * sigma;                     // (sigma 0: no scale yet)
            if (named_or(1, 128, over) || grow) {
                // the references and sigma move; what they scale is rescaled
                red[warp * 32 + lane] = mx;
                const float sig_new = grow ? pow2_ceil(smax) : sigma;
                const float beta = sigma == 0.0f ? 1.0f : sigma / sig_new;   // powers of two: exact
                sigma = sig_new;
                named_sync(1, 128);
                const float mr = fmaxf(mx, red[(warp ^ 2) * 32 + lane]);
                const float delta = mr > (none ? -INFINITY : kGrow) ? mr : 0.0f;
                const float alpha = none ? 0.0f : exp2f(-delta);
                none = none && !(mr > -INFINITY);
                ref += delta;
                l *= alpha;
#pragma unroll
                for (int e = 0; e < 64; e++) x[e] -= delta;
                if (i > 0) {
                    wait(kPbDone + ((i - 1) & 1), (i - 1) >> 1);
                    ok = __all_sync(0xffffffffu, ok);
                    tc::fence_after_sync();
                    const float f = alpha * beta;
#pragma unroll 1
                    for (int c = 0; c < 256; c += 16) {
                        uint32_t o[16];
                        tc::tmem_ld16(tmem + lanes + c, o);
                        tc::tmem_wait_ld();
#pragma unroll
                        for (int e = 0; e < 16; e++) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
                        tc::tmem_st16(tmem + lanes + c, o);
                    }
                    tc::tmem_wait_st();
                    tc::fence_before_sync();
                }
                named_sync(1, 128);                                     // (red is free again)
            }
            const float inv = sigma > 0.0f ? kBoost / sigma : 1.0f;     // (sigma 0: every finite scale is 0)
            uint32_t p[32];
            const float4 *sc4 = reinterpret_cast<const float4 *>(scl + m * kPrKeys + half * 64);
#pragma unroll
            for (int e = 0; e < 64; e += 4) {
                const float4 s = sc4[e >> 2];
                const float p0 = exp2_approx(x[e]), p1 = exp2_approx(x[e + 1]), p2 = exp2_approx(x[e + 2]), p3 = exp2_approx(x[e + 3]);
                l += (p0 + p1) + (p2 + p3);
                p[e >> 1] = f16x2_rn(p0 * (s.x * inv), p1 * (s.y * inv));
                p[(e >> 1) + 1] = f16x2_rn(p2 * (s.z * inv), p3 * (s.w * inv));
            }
            if (keys != ~0ull) {   // a key that is not one may have any scale: its weight is 0
#pragma unroll
                for (int e = 0; e < 64; e += 2) {
                    if (!((keys >> e) & 1ull)) p[e >> 1] &= 0xffff0000u;
                    if (!((keys >> (e + 1)) & 1ull)) p[e >> 1] &= 0x0000ffffu;
                }
            }
            if (i > 0) wait(kPbDone + ((i - 1) & 1), (i - 1) >> 1);     // P(t - 1) has been read
#pragma unroll
            for (int g = 0; g < 8; g++)
                *reinterpret_cast<uint4 *>(prow + g * 128) = make_uint4(p[4 * g], p[4 * g + 1], p[4 * g + 2], p[4 * g + 3]);
            tc::fence_proxy_async();
            __syncwarp();
            if (lane == 0) arrive_leader(bar(kPbP));
        }
        // the row's sum over both halves of the keys
        red[warp * 32 + lane] = l;
        named_sync(1, 128);
        l += red[(warp ^ 2) * 32 + lane];
        named_sync(1, 128);
        const bool empty = r >= live || l == 0.0f;
        const float scale = sigma * (1.0f / kBoost);
        if (half == 0) {
            red[row] = empty ? 0.0f : (direct ? scale / l : scale);
            red[64 + row] = empty ? 0.0f : 1.0f;
            if (r < n_rows_q) {
                const int64_t o = row_at(r);
                const float mn = ref * 0.6931471805599453f;
                if (!direct) {
                    part_ml[2 * o] = empty ? -INFINITY : mn;
                    part_ml[2 * o + 1] = empty ? 0.0f : l;
                } else if (a.lse) {
                    a.lse[o] = empty ? -INFINITY : mn + logf(l);
                }
            }
        }
    }
    // every product of the pair is done: the output
    wait(kPbDone + ((n_tiles - 1) & 1), (n_tiles - 1) >> 1);
    const bool all_ok = __syncthreads_and(ok);
    if (!all_ok) {   // a wait gave up: the status word, and a bounded wait for products still in flight
        if (tid == 0) atomicOr(a.status, 64);
        cluster_wait(bar(kPbDone + ((n_tiles - 1) & 1)), static_cast<uint32_t>(((n_tiles - 1) >> 1) & 1), kWaitLimit);
        __syncthreads();
    }
    tc::fence_after_sync();
    if (warp < 8) {
        // tensor-memory lane 32 (warp % 4) + lane: row, and the upper or lower 128 of the product's 256
        // dims; warps 0-3 the first product's dims, 4-7 the second's
        const int quad = warp & 3, j = warp >> 2;
        const int row = (quad & 1) * 32 + lane, r = r0 + row;
        const bool seen = red[64 + row] != 0.0f;
        const float f = red[row];
        const bool put = r < n_rows_q && (direct || seen);
        const int64_t o = put ? row_at(r) * kLatent + j * 256 + (quad >> 1) * 128 : 0;
#pragma unroll 1
        for (int c = 0; c < 128; c += 16) {
            uint32_t v[16];
            __syncwarp();
            tc::tmem_ld16(tmem + (static_cast<uint32_t>(quad * 32) << 16) + j * 128 + c, v);
            tc::tmem_wait_ld();
            float y[16];
#pragma unroll
            for (int e = 0; e < 16; e++) {
                y[e] = seen ? __uint_as_float(v[e]) * f : 0.0f;
                if (!all_ok) y[e] = __int_as_float(0x7fc00000);
            }
            if (put && direct) {
#pragma unroll
                for (int g = 0; g < 2; g++) {
                    uint32_t w4[4];
#pragma unroll
                    for (int e = 0; e < 4; e++) {
                        const __nv_bfloat162 h2 = __floats2bfloat162_rn(y[8 * g + 2 * e], y[8 * g + 2 * e + 1]);
                        w4[e] = *reinterpret_cast<const uint32_t *>(&h2);
                    }
                    *reinterpret_cast<uint4 *>(a.out + o + c + 8 * g) = make_uint4(w4[0], w4[1], w4[2], w4[3]);
                }
            } else if (put) {
#pragma unroll
                for (int e = 0; e < 16; e += 4)
                    *reinterpret_cast<float4 *>(part_acc + o + c + e) = make_float4(y[e], y[e + 1], y[e + 2], y[e + 3]);
            }
        }
        if (!all_ok && direct && a.lse && j == 0 && quad < 2 && r < n_rows_q) a.lse[row_at(r)] = __int_as_float(0x7fc00000);
    }
    tc::fence_before_sync();
    __syncthreads();
    cluster_sync();   // (the other CTA's arrivals here, and its reads of this CTA's operands, are over)
    if (warp == kPrWarpMma) {
        tc::fence_after_sync();
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");
    }
}

template <int kFmt>
cudaError_t launch_pair_t(const TreePlan &p, const TreeArgs &a, float *part_acc, float *part_ml, cudaStream_t stream) {
    auto kernel = tree_mla_pair_kernel<kFmt>;
    const int smem = PrLayout::kBytes;
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    e = launch_pdl(kernel, dim3(2 * p.q_tiles, a.batch, p.parts), dim3(kPrThreads), smem, stream, a, p, part_acc,
                   part_ml);
    return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace

cudaError_t launch_tree_pair(const TreePlan &p, const TreeArgs &a, int format, float *part_acc, float *part_ml,
                             cudaStream_t stream) {
    if (format == kFmtInt8) return launch_pair_t<kFmtInt8>(p, a, part_acc, part_ml, stream);
    if (format == kFmtFp8) return launch_pair_t<kFmtFp8>(p, a, part_acc, part_ml, stream);
    if (format == kFmtFp4) return launch_pair_t<kFmtFp4>(p, a, part_acc, part_ml, stream);
    return cudaErrorInvalidValue;
}

}  // namespace glm
