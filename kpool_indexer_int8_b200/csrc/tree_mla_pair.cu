// tree_mla_pair.cu -- the tree attention for more than 64 query rows (node, head) of a sequence:
// two CTAs of a cluster work on 128 query rows and 96 keys at a time with paired tensor-core
// instructions (cta_group::2, M = 128), which hold 64 rows x 512 outputs in half of each CTA's
// tensor memory and let each CTA keep only its half of every B operand:
//     S = Q K^T     A: this CTA's 64 rows of Q       B: K, this CTA's 48 keys x 512 dims
//     O += P V      A: this CTA's 64 rows of P       B: V, 96 keys x this CTA's 256 dims
// A key tile is thus widened twice over the pair (as K and as V) for 128 query rows, where the one-CTA
// kernel (tree_mla.cu) widens it once for 64 and reads its operands from shared memory twice as
// often. Roles of the 15 warps of a CTA, each with its own raw rows in shared memory, filled by
// asynchronous copies a tile ahead:
//   * warps 0-3 (softmax): one thread per row and half of the keys (tensor-memory lane = row, the
//     upper 64 lanes hold the tile's upper 48 keys): references, sigmas, sums and P' as in tree_mla.cu, the
//     two halves of a row meeting only when one of them may have to move;
//   * warps 4-9 (K): whole rows of the CTA's 48 keys as fp16 once S(t - 1) is done, and the scales of all 96;
//   * warps 10-13 (V): the CTA's 256 dims of the 96 keys once O of t - 1 is done;
//   * warp 14 of the first CTA (tensor cores): S(t + 1), then O of t, for both CTAs.
// K, V and P have one buffer each: shared memory holds no more beside Q.
//
// What bounds it: shared memory's 128 bytes a cycle. A tile takes 3,710 cycles of a CTA. The tensor cores read 172 KB of
// operands (Q 64, K 48, V 48, P 12), 1,380 cycles; the warps' own bytes (rows copied in and read, 49 KB each way, K
// and V 48 KB each and P 12 KB written) are 1,650, with scales, barriers and partials 1,870 wavefronts, and 320 more are
// counted as bank conflicts, whose cause is not known (the addresses here have none). Tensor pipe 42 % active,
// issue 47 %. 8 nodes of 64 heads over 262,144 int8 rows: 383 us a call back to back, under the power limit, 348 and
// 790 TFLOP/s one at a time, 0.48 of the measured bf16 rate. What was tried on top of it and did not pay (against 369 then):
// two teams of softmax warps on alternate tiles (410 us), eight softmax warps on one tile (386), rows read
// in rolled loops right before they are widened (390-404), one set of warps for K and V (391), P read for each of its
// two products (372), P' tested for fp16's range after the exponentials with the scores read again to move (389).
#include "tree_mla_common.cuh"

namespace glm {

namespace {

using namespace tree;

constexpr int kPrSoft = 4, kPrK = 6, kPrV = 4; // warps 0-3 softmax, 4-9 K, 10-13 V, 14 tensor cores
constexpr int kPrWarpV = kPrSoft + kPrK, kPrWarpMma = kPrWarpV + kPrV;
constexpr int kPrThreads = (kPrWarpMma + 1) * 32;
constexpr int kPrRows = 64;                    // query rows of a CTA
constexpr int kPrKeys = kTreePairKeys;         // keys of a tile
constexpr int kPrHalf = kPrKeys / 2;           // keys of a CTA's K
constexpr int kPrKn = kPrHalf / kPrK;          // keys of a K warp, of each half of a tile
constexpr int kPrVn = kPrKeys / kPrV;          // keys of a V warp
constexpr int kPrMeta = 3;                     // tiles whose scales are kept
constexpr uint32_t kPrSCol = 256;              // two score accumulators of 48 columns after the output's 256
constexpr uint32_t kPrSStep = 64;

enum PrBar { kPbK = 0, kPbV, kPbP, kPbS, kPbDone = 5, kPbMeta = 7, kPbEnd = 10, kPbCount };

struct PrLayout {
    static constexpr int kQ = 0;                                 // 8 row groups x 64 dim groups x 128 B
    static constexpr int kKBlock = kPrHalf * 128;                // a block of 64 dims of K, of V
    static constexpr int kVBlock = kPrKeys * 128;
    static constexpr int kK = kQ + kPrRows * 1024;               // 8 blocks of 64 dims x 48 keys x 128 B, swizzled
    static constexpr int kV = kK + 8 * kKBlock;                  // 4 blocks of 64 own dims x 96 keys x 128 B, swizzled
    static constexpr int kPGroup = kPrKeys * 16;                 // 8 rows of P'
    static constexpr int kP = kV + 4 * kVBlock;                  // 8 row groups x 12 key groups x 128 B
    static constexpr int kOutRow = kLatent * 2 + 16, kPartRow = kLatent * 4 + 16;   // rows of the epilogue
    static constexpr int kRawK = kP + 8 * kPGroup;               // the 48 own keys' rows: codes, then tails
    static constexpr int kRawV = kRawK + kPrHalf * kRowBytes;    // the own dims of 96 rows: codes, then tails of 4-bit rows
    static constexpr int kScl = kRawV + kPrKeys * 256;           // [3][96] row scales
    static constexpr int kMax = kScl + kPrMeta * kPrKeys * 4;    // [3][8] largest finite scale of a K warp's keys (6 used)
    static constexpr int kValid = kMax + kPrMeta * 8 * 4;       // [3][96] bytes: 1 where there is a key
    static constexpr int kFull = kValid + kPrMeta * kPrKeys;     // [3][2][8] bytes: 1 where a K warp's keys are all there
    static constexpr int kLog = kFull + kPrMeta * 16;            // [3][96] log2 of the row scales
    static constexpr int kRed = kLog + kPrMeta * kPrKeys * 4;    // [2][64] pairs
    static constexpr int kRowK = kRed + 128 * 8;                 // [64] score factors
    static constexpr int kBar = kRowK + kPrRows * 4;
    static constexpr int kTmem = kBar + kPbCount * 8;
    static constexpr int kBytes = kTmem + 8;
    static constexpr int kAlloc = kBytes + 1024;                 // from a 1024-byte aligned base
    static_assert(kPrRows == 16 * kPrSoft, "query rows of a softmax warp");
    static_assert(kBar % 8 == 0 && kScl % 16 == 0 && kValid % 8 == 0 && kFull % 16 == 0 && kLog % 16 == 0 && kMax % 16 == 0 && kK % 1024 == 0 &&
                      kV % 1024 == 0 && kKBlock % 1024 == 0 && kVBlock % 1024 == 0 && kRawK % 128 == 0 && kRawV % 128 == 0, "alignment");
    static_assert(kAlloc <= 232448 && kPrRows * kPartRow <= kP, "shared memory of one CTA");
};

__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// One arrival on a barrier of the pair's first CTA, whose tensor-core warp then issues products for both. It announces
// operands in the arriving CTA's own shared memory, made visible to that CTA's tensor core by the proxy fence before
// it, and tensor memory, behind a tcgen05 fence: neither goes through the other CTA, and the arrival follows both in the
// arriving warp. The memory model's own form of this is an arrival with release, and a wait with acquire, at cluster
// scope. Such an arrival waits 900 to 1,400 cycles for the warp's copies in flight, in each of the three a tile;
// passed on by the second CTA's idle tensor-core warp, 8 nodes over 262,144 rows take 399 us a call for 385, a batch
// of selected FP8 lists 75 for 66.6 (of which the hop itself 5).
__device__ __forceinline__ void arrive_leader(uint32_t mbar) {
    asm volatile(
        "{\n\t.reg .b32 r;\n\t"
        "mapa.shared::cluster.u32 r, %0, 0;\n\t"
        "mbarrier.arrive.shared::cluster.b64 _, [r];\n\t}\n" ::"r"(mbar)
        : "memory");
}
__device__ __forceinline__ void mma_pair(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}\n" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(accumulate));
}
// The two products of one A: the first keeps it beside the tensor core, the second takes it from there.
__device__ __forceinline__ void mma_pair_twice(uint32_t d0, uint32_t d1, uint64_t a, uint64_t b0, uint64_t b1, uint32_t idesc,
                                               uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %6, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f16.collector::a::fill [%0], %2, %3, %5, p;\n\t"
        "tcgen05.mma.cta_group::2.kind::f16.collector::a::lastuse [%1], %2, %4, %5, p;\n\t}\n" ::"r"(d0),
        "r"(d1), "l"(a), "l"(b0), "l"(b1), "r"(idesc), "r"(accumulate));
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
    extern __shared__ __align__(1024) unsigned char smem_raw[];
    unsigned char *smem = smem_raw + ((1024u - (tc::smem_addr(smem_raw) & 1023u)) & 1023u);
    float *scl = reinterpret_cast<float *>(smem + L::kScl);
    float *slog = reinterpret_cast<float *>(smem + L::kLog);
    float *smx = reinterpret_cast<float *>(smem + L::kMax);
    uint8_t *val = smem + L::kValid, *full = smem + L::kFull;
    float *red = reinterpret_cast<float *>(smem + L::kRed);
    float *rowk = reinterpret_cast<float *>(smem + L::kRowK);
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + L::kTmem);
    const uint32_t bar0 = tc::smem_addr(smem + L::kBar);
    auto bar = [&](int i) { return bar0 + 8u * static_cast<uint32_t>(i); };

    const int cta = blockIdx.x & 1, qt = blockIdx.x >> 1, b = blockIdx.z, part = blockIdx.y;
    const int tid = threadIdx.x, lane = tid & 31;
    const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
    const int H = a.n_heads, n_rows_q = a.n_nodes * H;
    const int r0 = qt * 2 * kPrRows + cta * kPrRows;          // this CTA's first query row
    const int parts = plan.parts;
    const bool direct = parts == 1;

    const Lengths own = load_lengths(a, b, true), mine = load_lengths(a, lane, !direct && lane < a.batch);
    if (warp < kPrSoft) {
        // The softmax warps: the query rows as fp16, each scaled by the power of two that puts its largest
        // magnitude in [2^14, 2^15), by way of shared memory where K and V will be (rows 16 bytes apart in the
        // banks), a warp two groups of 8 rows and four lanes a row. Rolled loops, and before the lengths are
        // there: held in registers, unrolled and after them, it took 12,000 cycles of a first call's 48,000.
        // (Rows that no node of the tree has are converted like the others; they are put out as empty.)
#pragma unroll 1
        for (int i = 0; i < 16 * 32; i += 32) {
            const int row = warp * 16 + i / 32;
            const uint16_t *from = a.q + (static_cast<int64_t>(b) * n_rows_q + min(r0 + row, n_rows_q - 1)) * kLatent;
            copy16(smem + L::kK + row * L::kOutRow + lane * 16, from + lane * 8, true);
            copy16(smem + L::kK + row * L::kOutRow + (lane + 32) * 16, from + (lane + 32) * 8, true);
        }
        copy_commit();
        copy_wait<0>();
#pragma unroll 1
        for (int g = 2 * warp; g < 2 * warp + 2; g++) {
            const int qr = g * 8 + (lane & 7);
            const unsigned char *from = smem + L::kK + qr * L::kOutRow + (lane >> 3) * 16;
            unsigned mx = 0u;
#pragma unroll 8
            for (int i = 0; i < 16; i++) mx = max(mx, bf16_absmax(*reinterpret_cast<const uint4 *>(from + 64 * i)));
            mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, 8));
            mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, 16));
            const int e = query_exponent(mx);
            const float f = pow2f_exact(e);
            if (lane < 8) rowk[qr] = a.sm_scale * 1.4426950408889634f * pow2f_exact(-e);
            unsigned char *to = smem + L::kQ + g * 8192 + (lane >> 3) * 128 + (lane & 7) * 16;
#pragma unroll 1
            for (int i = 0; i < 16; i += 4) {
                uint4 v[4];
#pragma unroll
                for (int k = 0; k < 4; k++) v[k] = *reinterpret_cast<const uint4 *>(from + 64 * (i + k));
#pragma unroll
                for (int k = 0; k < 4; k++) *reinterpret_cast<uint4 *>(to + 4 * (i + k) * 128) = bf16_to_f16x8(v[k], f);
            }
        }
        tc::fence_proxy_async();
    }
    // the sequence's tiles [0, tiles), those of the list first, and this part's [t0, t1)
    const int plen = list_len(a, own), tree_n = tree_len(a, own);
    const int n_keys = plen + tree_n, tiles = (n_keys + kPrKeys - 1) / kPrKeys;
    const int run = direct ? tiles : run_tiles(a, plan, kPrKeys, mine);
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
    if (tid < kPrMeta * 8) smx[tid] = 0.0f;                   // (what no K warp writes)
    if (tid < kPrMeta * 16) full[tid] = 1;
    if (warp == kPrWarpMma) {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(tc::smem_addr(tmem_slot))
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
        tc::fence_before_sync();
        if (lane == 0) {
            tc::mbar_init(bar(kPbK), 2 * kPrK);                         // (both CTAs' warps arrive at the first's)
            tc::mbar_init(bar(kPbV), 2 * kPrV);
            tc::mbar_init(bar(kPbP), 2 * kPrSoft);
            for (int i = 0; i < 2; i++) {
                tc::mbar_init(bar(kPbS + i), 1);
                tc::mbar_init(bar(kPbDone + i), 1);
            }
            for (int i = 0; i < kPrMeta; i++) tc::mbar_init(bar(kPbMeta + i), kPrK);
            tc::mbar_init(bar(kPbEnd), 1);
            tc::mbar_fence_init();
        }
    }
    // Every warp calls it once, before it first needs the query, the barriers or tensor memory of both CTAs
    // (it joins all threads of both).
    uint32_t tmem = 0;
    auto start = [&]() {
        __syncwarp();
        cluster_sync();
        tc::fence_after_sync();
        tmem = *tmem_slot;
    };
    bool ok = !a.give_up;
    auto wait = [&](int i, int use) {
        if (ok && !tc::mbar_wait(bar(i), static_cast<uint32_t>(use & 1), kWaitLimit)) ok = false;
    };

    const int32_t *list = a.rows + static_cast<int64_t>(b) * a.width;
    // the list's entry (or drafted row) of key `key` of tile t, and the row it means, -1: none. (An entry
    // is looked at only when its row is needed: a test right behind the load would hold the warp.)
    auto entry_of = [&](int t, int key) -> int {
        const int j = t * kPrKeys + key;
        if (t >= t1) return -1;
        if (j < plen) return __ldg(list + j);
        return j < n_keys ? draft_row(b * a.n_nodes + j - plen) : -1;
    };
    auto row_of = [&](int t, int key, int entry) {
        return t * kPrKeys + key >= plen || (entry >= 0 && entry < a.n_rows) ? entry : -1;
    };
    auto has_drafts = [&](int t) { return (t + 1) * kPrKeys > plen; };

    if (warp >= kPrSoft && warp < kPrWarpV) {
        // ---------------- K: keys 8 w .. 8 w + 7 of this CTA's half of each tile, whole rows ----------------
        // Lanes 0-7 hold their rows, lanes 16-23 those of the same keys of the other half, for the scales.
        constexpr int kN = kPrKn;
        constexpr unsigned kAll = (1u << kN) - 1;
        const int w = warp - kPrSoft, which = lane >> 4;
        const bool holds = (lane & 15) < kN;
        const int my_key = (which ? 1 - cta : cta) * kPrHalf + w * kN + (lane & 15);
        unsigned char *codes = smem + L::kRawK + w * kN * R::kCodes;
        unsigned char *tails = smem + L::kRawK + kPrHalf * R::kCodes + w * kN * R::kTail;
        auto entry = [&](int t) { return holds ? entry_of(t, my_key) : -1; };
        // the scale of a row of the other half (its own rows' scales come with them)
        auto other_scale = [&](int row) {
            return which && row != -1 ? __ldg(reinterpret_cast<const float *>(R::at(a, row) + R::kCodes + R::kSclAt)) : 0.0f;
        };
        int e1 = entry(t0 + 1);
        int rows = row_of(t0, my_key, entry(t0));
        R::template fetch<kN>(codes, tails, a, rows, 0, has_drafts(t0));
        copy_commit();
        float sc = other_scale(rows);
        for (int i = 0; i < n_tiles; i++) {
            const int t = t0 + i, m = i % kPrMeta;
            const bool drafts = has_drafts(t);
            const int e2 = entry(t + 2);
            copy_wait<0>();
            if (lane < kN) sc = R::scale(tails + lane * R::kTail);
            if (kFmt != kFmtInt8 && drafts) {   // a row with NaN codes: its scale makes every score with it NaN
                unsigned bad = 0u;
#pragma unroll 8
                for (int r = 0; r < 32; r++) {
                    const int row = __shfl_sync(0xffffffffu, rows, r);
                    const uint8_t *p = R::at(a, row);
                    if (row != -1 && R::nan_share(p, p + R::kCodes)) bad |= 1u << r;
                }
                if (__reduce_or_sync(0xffffffffu, bad) >> lane & 1u) sc = __int_as_float(0x7fc00000);
            }
            if (kFmt != kFmtInt8 && drafts) R::clean(R::kFp4 ? tails : codes, kN * (R::kFp4 ? R::kTail : R::kCodes));
            // (every read before the first write: the compiler keeps their order)
            typename R::Line v[kN][2];                         // lines lane and lane + 32 of each row
#pragma unroll
            for (int r = 0; r < kN; r++)
#pragma unroll
                for (int h = 0; h < 2; h++)
                    v[r][h] = R::line(codes + r * R::kCodes, tails + r * R::kTail, lane + 32 * h, lane / 2 + 16 * h);
            const unsigned bits = __ballot_sync(0xffffffffu, rows != -1);
            const float mx = finite_max(holds ? fabsf(sc) : 0.0f), lg = __log2f(fabsf(sc));
            // the next rows, into the slots just read
            const int nxt = row_of(t + 1, my_key, e1);
            if (i + 1 < n_tiles) R::template fetch<kN>(codes, tails, a, nxt, 0, has_drafts(t + 1));
            copy_commit();
            const float sc_next = other_scale(nxt);
            if (i > 0) wait(kPbS + ((i - 1) & 1), (i - 1) >> 1);   // S(t - 1) is done: K is free
            else start();
            if (holds) {
                scl[m * kPrKeys + my_key] = sc + (sc - sc);   // (an infinite scale: NaN, as 0 codes times it are)
                slog[m * kPrKeys + my_key] = lg;
                val[m * kPrKeys + my_key] = rows != -1 ? 1 : 0;
            }
            if (lane == 0) {
                smx[m * 8 + w] = mx;
                full[m * 16 + cta * 8 + w] = (bits & kAll) == kAll ? 1 : 0;
                full[m * 16 + (1 - cta) * 8 + w] = (bits >> 16 & kAll) == kAll ? 1 : 0;
            }
#pragma unroll
            for (int r = 0; r < kN; r++) {
                unsigned char *to = smem + L::kK + (lane >> 3) * L::kKBlock + swizzled(w * kN + r, lane & 7);
#pragma unroll
                for (int h = 0; h < 2; h++) *reinterpret_cast<uint4 *>(to + h * 4 * L::kKBlock) = R::widen(v[r][h]);
            }
            tc::fence_proxy_async();
            __syncwarp();
            if (lane == 0) {
                tc::mbar_arrive(bar(kPbMeta + m));
                arrive_leader(bar(kPbK));
            }
            rows = nxt;
            sc = sc_next;
            e1 = e2;
        }
    } else if (warp >= kPrWarpV && warp < kPrWarpMma) {
        // ---------------- V: keys 24 w .. 24 w + 23 of each tile, this CTA's 256 dims ----------------
        constexpr int kN = kPrVn;
        const int w = warp - kPrWarpV;
        unsigned char *codes = smem + L::kRawV + w * kN * (R::kCodes / 2);
        unsigned char *tails = smem + L::kRawV + kPrKeys * (R::kCodes / 2) + w * kN * R::kTail;   // (4-bit rows)
        const int my_key = w * kN + lane;
        auto entry = [&](int t) { return lane < kN ? entry_of(t, my_key) : -1; };
        const int block = (lane >> 4) * 16 + cta * 8 + (lane & 15) / 2;
        int e1 = entry(t0 + 1);
        R::template fetch_half<kN>(codes, tails, a, row_of(t0, my_key, entry(t0)), cta, has_drafts(t0));
        copy_commit();
        for (int i = 0; i < n_tiles; i++) {
            const int t = t0 + i;
            const bool drafts = has_drafts(t);
            const int e2 = entry(t + 2);
            copy_wait<0>();
            if (kFmt != kFmtInt8 && drafts) R::clean(R::kFp4 ? tails : codes, kN * (R::kFp4 ? R::kTail : R::kCodes / 2));
            typename R::Line v[kN];
#pragma unroll
            for (int r = 0; r < kN; r++) v[r] = R::line(codes + r * (R::kCodes / 2), tails + r * R::kTail, lane, block);
            const int nxt = row_of(t + 1, my_key, e1);
            __syncwarp();
            if (i + 1 < n_tiles) R::template fetch_half<kN>(codes, tails, a, nxt, cta, has_drafts(t + 1));
            copy_commit();
            if (i > 0) wait(kPbDone + ((i - 1) & 1), (i - 1) >> 1);   // O of t - 1 is done: V is free
            else start();
            unsigned char *to = smem + L::kV + (lane >> 3) * L::kVBlock;
#pragma unroll
            for (int r = 0; r < kN; r++)
                *reinterpret_cast<uint4 *>(to + swizzled(w * kN + r, lane & 7)) = R::widen(v[r]);
            tc::fence_proxy_async();
            __syncwarp();
            if (lane == 0) arrive_leader(bar(kPbV));
            e1 = e2;
        }
    } else if (warp == kPrWarpMma) {
        // ---------------- tensor cores (the first CTA's, for both) ----------------
        start();
        if (cta == 0) {
            constexpr uint32_t id_s = tc::idesc_f16(128, kPrKeys, false, false);
            constexpr uint32_t id_o = tc::idesc_f16(128, 256, false, true);
            const uint64_t dq = tc::desc(tc::smem_addr(smem + L::kQ), 128, 8192);
            const uint64_t dk = tc::desc_sw128(tc::smem_addr(smem + L::kK), 1024);
            const uint64_t dv = tc::desc_sw128_mn(tc::smem_addr(smem + L::kV), L::kVBlock, 1024);
            const uint64_t dp = tc::desc(tc::smem_addr(smem + L::kP), 128, L::kPGroup);
            auto accumulate = [&](int i) {   // O += P(i) V(i): two products of 256 dims, K = 96 keys
                wait(kPbV, i);
                wait(kPbP, i);
                ok = __all_sync(0xffffffffu, ok);
                tc::fence_after_sync();
                if (tc::elect_one()) {
#pragma unroll
                    for (int ks = 0; ks < kPrKeys / 16; ks++)
                        mma_pair_twice(tmem, tmem + 128, dp + ((ks * 256) >> 4), dv + ((ks * 2048) >> 4),
                                       dv + ((ks * 2048 + 2 * L::kVBlock) >> 4), id_o, (i > 0 || ks > 0) ? 1u : 0u);
                    commit_pair(bar(kPbDone + (i & 1)));
                }
                __syncwarp();
            };
            for (int i = 0; i < n_tiles; i++) {
                wait(kPbK, i);   // (S(i - 2), which this one is written over, has been read: O of it is issued, after P(i - 2))
                ok = __all_sync(0xffffffffu, ok);
                tc::fence_after_sync();
                if (tc::elect_one()) {   // S(i) = Q K(i)^T: N = 96 keys, K = 512
#pragma unroll
                    for (int ks = 0; ks < kLatent / 16; ks++)
                        mma_pair(tmem + kPrSCol + (i & 1) * kPrSStep, dq + ((ks * 256) >> 4),
                                 dk + (((ks >> 2) * L::kKBlock + (ks & 3) * 32) >> 4), id_s,
                                 ks > 0 ? 1u : 0u);
                    commit_pair(bar(kPbS + (i & 1)));
                }
                __syncwarp();
                if (i > 0) accumulate(i - 1);
            }
            accumulate(n_tiles - 1);
            if (tc::elect_one()) commit_pair(bar(kPbEnd));
            __syncwarp();
        }
    } else {
        // ---------------- softmax ----------------
        start();

        // tensor-memory lane 32 warp + lane: row, and the lower or upper 48 keys of a tile
        const int row = (warp & 1) * 32 + lane, half = warp >> 1, key0 = half * kPrHalf;
        const uint32_t lanes = static_cast<uint32_t>(warp * 32) << 16;
        const int r = r0 + row;
        const float qk = rowk[row];
        const uint64_t seen = r < live ? a.mask[static_cast<int64_t>(b) * a.n_nodes + r / H] : 0ull;
        Scaling scaling{0.0f, 0.0f, true};
        float l = 0.0f, inv = 1.0f;                                     // (1 / sigma)
        const int mine = half * 64 + row, other = (1 - half) * 64 + row;   // two threads share a row
        float2 *red2 = reinterpret_cast<float2 *>(red);
        unsigned char *prow = smem + L::kP + (row >> 3) * L::kPGroup + key0 * 16 + (row & 7) * 16;
        for (int i = 0; i < n_tiles; i++) {
            const int t = t0 + i, m = i % kPrMeta;
            wait(kPbMeta + m, i / kPrMeta);
            // What a score may be: its p at most 2^kTop, and its product with any scale of the tile (of all keys, seen or
            // not) at most 2^kTop sigma; of a row without a reference: none.
            const float4 ma = *reinterpret_cast<const float4 *>(smx + m * 8), mb = *reinterpret_cast<const float4 *>(smx + m * 8 + 4);
            const float smax = fmaxf(max3(ma.x, ma.y, max3(ma.z, ma.w, mb.x)), max3(mb.y, mb.z, mb.w));
            const int bits = max(0, static_cast<int>(__float_as_uint(smax * inv) >> 23) - 126);   // smax / sigma < 2^bits
            const float most = scaling.none ? -INFINITY : kTop - static_cast<float>(bits);
            wait(kPbS + (i & 1), i >> 1);
            ok = __all_sync(0xffffffffu, ok);
            tc::fence_after_sync();
            float x[kPrHalf];
            const ulonglong2 *sc4 = reinterpret_cast<const ulonglong2 *>(scl + m * kPrKeys + key0);
            {
                uint32_t s0[32], s1[16];
                tc::tmem_ld32(tmem + lanes + kPrSCol + (i & 1) * kPrSStep, s0);
                tc::tmem_ld16(tmem + lanes + kPrSCol + (i & 1) * kPrSStep + 32, s1);
                tc::tmem_wait_ld();
                tc::fence_before_sync();
                const uint64_t qk2 = pack2(qk, qk), ref2 = pack2(-scaling.ref, -scaling.ref);
#pragma unroll
                for (int e = 0; e < kPrHalf; e += 4) {
                    const ulonglong2 s = sc4[e >> 2];
                    const uint32_t *v = e < 32 ? &s0[e] : &s1[e - 32];
                    unpack2(fma2(mul2(pack2(v[0], v[1]), qk2), s.x, ref2), x[e], x[e + 1]);
                    unpack2(fma2(mul2(pack2(v[2], v[3]), qk2), s.y, ref2), x[e + 2], x[e + 3]);
                }
            }
            const uint2 fw = *reinterpret_cast<const uint2 *>(full + m * 16 + half * 8);
            bool partial = (fw.x & fw.y) != 0x01010101u || has_drafts(t);
            uint64_t keys = (1ull << kPrHalf) - 1;                      // this thread's keys
            if (partial) {
                const uint2 *vb = reinterpret_cast<const uint2 *>(val + m * kPrKeys + key0);
                keys = 0ull;
#pragma unroll
                for (int g = 0; g < kPrHalf / 8; g++) {
                    // eight bytes of 0 or 1 to eight bits
                    const uint2 v = vb[g];
                    keys |= static_cast<uint64_t>(((v.x * 0x10204080u) >> 28) | (((v.y * 0x10204080u) >> 28) << 4)) << (8 * g);
                }
                if (has_drafts(t)) {                                    // what the node sees of the drafts
                    const int n = plen - t * kPrKeys - key0;            // this thread's first draft
                    keys &= n >= kPrHalf ? ~0ull : (n > 0 ? ((1ull << n) - 1) | seen << n : (n > -64 ? seen >> -n : 0ull));
                }
#pragma unroll
                for (int e = 0; e < kPrHalf; e++)
                    if (!((keys >> e) & 1ull)) x[e] = -INFINITY;
            }
            float mx = -INFINITY;
#pragma unroll
            for (int e = 0; e < kPrHalf; e += 2) mx = max3(mx, x[e], x[e + 1]);
            if (named_or(1, 32 * kPrSoft, mx > most)) {
                // the scaling of the rows moves, where it has to, and what it scales is rescaled
                float my = -INFINITY;                                   // (of the scores less mx)
                const float4 *lg4 = reinterpret_cast<const float4 *>(slog + m * kPrKeys + key0);
#pragma unroll
                for (int e = 0; e < kPrHalf; e += 4) {
                    const float4 lg = lg4[e >> 2];
                    my = max3(max3(my, (x[e] - mx) + lg.x, (x[e + 1] - mx) + lg.y), (x[e + 2] - mx) + lg.z, (x[e + 3] - mx) + lg.w);
                }
                red2[mine] = make_float2(mx, my);
                named_sync(1, 32 * kPrSoft);
                const float2 o = red2[other];
                float fl, fo;
                const float delta = move_scaling(scaling, larger({mx, my}, {o.x, o.y}), fl, fo);
                inv = pow2f_exact(-static_cast<int>(scaling.log_sigma));
                l *= fl;
#pragma unroll
                for (int e = 0; e < kPrHalf; e++) x[e] -= delta;
                if (i > 0 && __any_sync(0xffffffffu, fo != 1.0f)) {
                    wait(kPbDone + ((i - 1) & 1), (i - 1) >> 1);
                    ok = __all_sync(0xffffffffu, ok);
                    tc::fence_after_sync();
#pragma unroll 1
                    for (int c = 0; c < 256; c += 32) {
                        uint32_t v[32];
                        tc::tmem_ld32(tmem + lanes + c, v);
                        tc::tmem_wait_ld();
#pragma unroll
                        for (int e = 0; e < 32; e++) v[e] = __float_as_uint(__uint_as_float(v[e]) * fo);
                        tc::tmem_st32(tmem + lanes + c, v);
                    }
                    tc::tmem_wait_st();
                    tc::fence_before_sync();
                }
            }
            if (!(smax * inv <= kFltMax)) {   // keys whose scale over sigma is not finite weigh nothing
                partial = true;
#pragma unroll 1
                for (int e = 0; e < kPrHalf; e++)
                    if (!(fabsf(scl[m * kPrKeys + key0 + e]) * inv <= kFltMax)) keys &= ~(1ull << e);
            }
            uint32_t p[kPrHalf / 2];
            const uint64_t inv2 = pack2(inv, inv);
            uint64_t l2[2] = {pack2(0.0f, 0.0f), pack2(0.0f, 0.0f)};
#pragma unroll
            for (int e = 0; e < kPrHalf; e += 4) {
                const ulonglong2 s = sc4[e >> 2];
                const uint64_t p0 = pack2(exp2_approx(x[e]), exp2_approx(x[e + 1]));
                const uint64_t p1 = pack2(exp2_approx(x[e + 2]), exp2_approx(x[e + 3]));
                l2[0] = add2(l2[0], p0);
                l2[1] = add2(l2[1], p1);
                float y0, y1, y2, y3;
                unpack2(mul2(p0, mul2(s.x, inv2)), y0, y1);
                unpack2(mul2(p1, mul2(s.y, inv2)), y2, y3);
                p[e >> 1] = f16x2_rn(y0, y1);
                p[(e >> 1) + 1] = f16x2_rn(y2, y3);
            }
            {
                float u0, u1;
                unpack2(add2(l2[0], l2[1]), u0, u1);
                l += u0 + u1;
            }
            if (partial) {   // a key that is not one may have any scale: its weight is 0
#pragma unroll
                for (int e = 0; e < kPrHalf; e += 2) {
                    if (!((keys >> e) & 1ull)) p[e >> 1] &= 0xffff0000u;
                    if (!((keys >> (e + 1)) & 1ull)) p[e >> 1] &= 0x0000ffffu;
                }
            }
            if (i > 0) wait(kPbDone + ((i - 1) & 1), (i - 1) >> 1);     // P(t - 1) has been read
#pragma unroll
            for (int g = 0; g < kPrHalf / 8; g++)
                *reinterpret_cast<uint4 *>(prow + g * 128) = make_uint4(p[4 * g], p[4 * g + 1], p[4 * g + 2], p[4 * g + 3]);
            tc::fence_proxy_async();
            __syncwarp();
            if (lane == 0) arrive_leader(bar(kPbP));
        }
        // the row's sum over its two threads
        named_sync(1, 32 * kPrSoft);                                    // (red is free)
        red[mine] = l;
        named_sync(1, 32 * kPrSoft);
        l += red[other];
        named_sync(1, 32 * kPrSoft);
        const float sigma = 1.0f / inv;
        const bool empty = r >= live || l == 0.0f;
        if (key0 == 0) {
            red[row] = empty ? 0.0f : (direct ? sigma / l : sigma * kUnhead);
            red[64 + row] = empty ? 0.0f : 1.0f;
            if (r < n_rows_q) {
                const int64_t o = row_at(r);
                if (!direct) {
                    part_ml[2 * o] = empty ? -INFINITY : scaling.ref + kHead;
                    part_ml[2 * o + 1] = empty ? 0.0f : l * kUnhead;
                } else if (a.lse) {
                    a.lse[o] = empty ? -INFINITY : scaling.ref * 0.6931471805599453f + logf(l);
                }
            }
        }
    }
    // Every product of the pair is done: the output. (A barrier of its own, used once and told to both CTAs: that of
    // a tile says nothing to a thread that gave up, whose products may be several phases behind.)
    if (!tc::mbar_wait(bar(kPbEnd), 0, kWaitLimit)) ok = false;
    const bool all_ok = __syncthreads_and(ok);
    if (!all_ok && tid == 0) atomicOr(a.status, 64);
    tc::fence_after_sync();
    // the output or partials go through shared memory (over Q, K and V, which no product reads any more;
    // rows 16 bytes apart in the banks), then, whole lines of them,
    // to memory
    const int stride = direct ? L::kOutRow : L::kPartRow;
    if (warp < 8) {
        // tensor-memory lane 32 (warp % 4) + lane: row, and the upper or lower 128 of the product's 256
        // dims; warps 0-3 the first product's dims, 4-7 the second's
        const int quad = warp & 3, j = warp >> 2;
        const int row = (quad & 1) * 32 + lane, r = r0 + row;
        const bool seen = red[64 + row] != 0.0f;
        const float f = red[row];
        const int dim0 = j * 256 + (quad >> 1) * 128;
#pragma unroll 1
        for (int c = 0; c < 128; c += 16) {
            uint32_t v[16];
            tc::tmem_ld16(tmem + (static_cast<uint32_t>(quad * 32) << 16) + j * 128 + c, v);
            tc::tmem_wait_ld();
            float y[16];
#pragma unroll
            for (int e = 0; e < 16; e++) {
                y[e] = seen ? __uint_as_float(v[e]) * f : 0.0f;
                if (!all_ok) y[e] = __int_as_float(0x7fc00000);
            }
            unsigned char *to = smem + row * stride + (dim0 + c) * (direct ? 2 : 4);
            if (direct) {
#pragma unroll
                for (int g = 0; g < 2; g++) {
                    uint32_t w4[4];
#pragma unroll
                    for (int e = 0; e < 4; e++) {
                        const __nv_bfloat162 h2 = __floats2bfloat162_rn(y[8 * g + 2 * e], y[8 * g + 2 * e + 1]);
                        w4[e] = *reinterpret_cast<const uint32_t *>(&h2);
                    }
                    *reinterpret_cast<uint4 *>(to + 16 * g) = make_uint4(w4[0], w4[1], w4[2], w4[3]);
                }
            } else {
#pragma unroll
                for (int e = 0; e < 16; e += 4)
                    *reinterpret_cast<float4 *>(to + 4 * e) = make_float4(y[e], y[e + 1], y[e + 2], y[e + 3]);
            }
        }
        if (!all_ok && direct && a.lse && j == 0 && quad < 2 && r < n_rows_q) a.lse[row_at(r)] = __int_as_float(0x7fc00000);
    }
    __syncthreads();
    for (int row = warp; row < kPrRows; row += kPrThreads / 32) {
        if (r0 + row >= n_rows_q || (!direct && red[64 + row] == 0.0f)) continue;
        const uint4 *from = reinterpret_cast<const uint4 *>(smem + row * stride) + lane;
        const int64_t o = row_at(r0 + row) * kLatent;
        uint4 *to = (direct ? reinterpret_cast<uint4 *>(a.out + o) : reinterpret_cast<uint4 *>(part_acc + o)) + lane;
        for (int c = 0; c < (direct ? 64 : 128); c += 64) {
            const uint4 u = from[c], v = from[c + 32];
            to[c] = u;
            to[c + 32] = v;
        }
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
    const int smem = PrLayout::kAlloc;
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    // (The query tiles of a run side by side, for its rows in L2; the runs that a sequence does not have behind
    // its own: with the runs slowest, they were before the last runs of all, 52.2 us for short ragged
    // lists, 47.7 so.)
    e = launch_pdl(kernel, dim3(2 * p.q_tiles, p.parts, a.batch), dim3(kPrThreads), smem, stream, a, p, part_acc,
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
