// tree_mla.cu -- attention of a tree of drafted tokens over latent cache rows, on the sm_100a
// tensor cores: node i of sequence b attends to the rows of its sequence's index list and to the
// drafted rows whose bit is set in its mask,
//     s = sm_scale q . c,   out = sum softmax(s) c,   lse = log sum exp(s),   c = code * scale,
// the latent row being key and value. Every (node, head) of a sequence is a row of one query
// matrix, so that a widened tile of keys serves all of them.
//
// One CTA per (tile of NQ query rows, range of the sequence's keys, sequence) walks its range 64
// keys at a time, the drafted rows being the last tile. Keys are the MMA M dimension, query rows
// the N dimension (as in the sparse attention); 13 warps in three roles:
//   * warps 8-11 (widening): each thread holds the pieces of two key rows of the next tile in
//     registers while the tile before is worked on, then writes them as fp16 (exact: int8 and E4M3
//     codes, E2M1 code times block scale) to one of two tiles C[64 x 512] of 8x8 core matrices;
//   * warp 12 (tensor cores): S^T(t) = C(t) . Q^T into one of two accumulators, then O^T += C(t-1)^T
//     P(t-1)^T, so that the next scores are computed while the softmax of the tile before runs;
//   * warps 0-7 (softmax): x = S scale_row qk - ref in log2 units, P' = 2^x scale_row / sigma as fp16.
//     The reference of a query row moves only when a score passes it by 2^8 (a vote of the eight
//     warps per tile), and sigma, a power of two, only when a row scale passes 16 sigma: then the
//     accumulator in tensor memory is rescaled, otherwise no maximum is taken. Sums stay in
//     registers, one per thread and query row, until the end.
// P' is one fp16 term: a weight is off by at most 2^-11 of itself (an eighth of the bf16 output's
// 2^-8), or by 2^-28 of the largest once it is below 2^-17 of it.
//
// A sequence's keys are cut into ranges so that the CTAs fill the SMs; the combine kernel of the
// sparse attention merges the partials. Every wait is bounded; one that gives up sets the status
// word and the CTA writes NaN.
#include "common.cuh"
#include "row_codes.cuh"
#include "tc.cuh"
#include "tree_mla.cuh"

namespace glm {

namespace {

constexpr int kTrWarpWiden = 8;                // warps 0-7 softmax, 8-11 widening, 12 tensor cores: 13 warps
constexpr int kTrWarpMma = 12;                 // leave 128 registers a thread
constexpr int kTrThreads = 13 * 32;
constexpr int kTrKeys = 64;                    // keys of a tile
constexpr uint32_t kTrWaitLimit = 1u << 22;
constexpr float kTrNone = -1e30f;              // reference of a query row that has seen no key
constexpr float kTrGrow = 8.0f;                // a score passes its reference by at most 2^8
constexpr float kTrBoost = 8.0f;               // P' <= 2^8 * 16 * 8 = 2^15 < 65504

enum TrBar { kTbFull = 0, kTbDone = 2, kTbSFull = 4, kTbSFree = 6, kTbPFull = 8, kTbQ = 10, kTbCount = 11 };

template <int NQ>
struct TrLayout {
    static constexpr int kCBytes = kTrKeys * 1024;
    static constexpr int kC = 0;                                 // [2] tiles
    static constexpr int kQ = kC + 2 * kCBytes;                  // NQ/8 x 64 x 128 B
    static constexpr int kPBytes = kTrKeys * 2 * NQ;
    static constexpr int kP = kQ + NQ * 1024;                    // [2] P', core matrices of 8 keys x 8 query rows
    static constexpr int kFac = kP + 2 * kPBytes;                // [NQ] (qk, reference) pairs
    static constexpr int kMask = kFac + NQ * 8;                  // [NQ] visibility words
    static constexpr int kOut = kMask + NQ * 8;                  // [NQ] row of the output or partial, -1: none
    static constexpr int kRed = kOut + NQ * 8;                   // [4 quadrants][NQ]
    static constexpr int kAlpha = kRed + 4 * NQ * 4;             // [NQ] factors of a rescale; at the end 1 / l
    static constexpr int kScl = kAlpha + NQ * 4;                 // [2][64] row scales
    static constexpr int kMax = kScl + 2 * kTrKeys * 4;          // [2][8] largest finite scale of 8 rows
    static constexpr int kValid = kMax + 2 * 8 * 4;              // [2][8] bytes: which rows are keys
    static constexpr int kQmax = kValid + 16;                    // [NQ] |q| maxima (bf16 bits)
    static constexpr int kBar = kQmax + NQ * 4;
    static constexpr int kTmem = kBar + kTbCount * 8;
    static constexpr int kBytes = kTmem + 8;
    static_assert(kQ % 128 == 0 && kP % 128 == 0 && kFac % 16 == 0 && kBar % 8 == 0 && kMask % 8 == 0, "alignment");
    static_assert(kBytes <= 232448, "shared memory of one CTA");
};

// Rows of the output and of the partials of a query tile's columns, and where its keys end.
struct TrRange {
    int plen;      // entries of the index list
    int tree;      // drafted rows
    int tiles;     // tiles of 64 keys: the list's, then one of drafted rows
    int t0, t1;    // this CTA's
};
__device__ __forceinline__ TrRange tr_range(const TreeArgs &a, int b, int part, int parts) {
    TrRange r;
    r.plen = a.row_len ? min(max(a.row_len[b], 0), a.width) : a.width;
    r.tree = a.n_tree ? min(max(a.n_tree[b], 0), a.n_nodes) : a.n_nodes;
    r.tiles = (r.plen + kTrKeys - 1) / kTrKeys + (r.tree > 0 ? 1 : 0);
    const int per = (r.tiles + parts - 1) / parts;
    r.t0 = min(r.tiles, part * per);
    r.t1 = min(r.tiles, r.t0 + per);
    return r;
}

// The 16-byte pieces of one key row that a widening thread holds: pieces 4 it + (lane >> 3) of the
// row 8 w + (lane & 7) of the tile (four lanes read 64 contiguous bytes of a row, eight lanes write
// 128 contiguous bytes of a core matrix).
template <int kFmt>
struct TrRow {
    static constexpr bool kFp4 = kFmt == kFmtFp4;
    static constexpr int kRowB = kFp4 ? kFp4RowBytes : kRowBytes;
    static constexpr int kSclAt = kFp4 ? kFp4RowScaleAt : kLatent;
    static constexpr int kPieces = kFp4 ? 4 : 8;
    uint4 v[kPieces];
    uint32_t es[kFp4 ? kPieces : 1];
    float scale;
    bool valid;

    __device__ __forceinline__ void load(const uint8_t *base, int64_t r, int part) {
        valid = r >= 0;
        const uint8_t *p = base + (valid ? r : 0) * kRowB;
        scale = valid ? __ldg(reinterpret_cast<const float *>(p + kSclAt)) : 0.0f;
#pragma unroll
        for (int it = 0; it < kPieces; it++) {
            v[it] = valid ? __ldg(reinterpret_cast<const uint4 *>(p) + 4 * it + part) : make_uint4(0u, 0u, 0u, 0u);
            if constexpr (kFp4) es[it] = valid ? __ldg(reinterpret_cast<const uint16_t *>(p + kFp4ScalesAt) + 4 * it + part) : 0u;
        }
    }
    // row: the row's line in the first core matrix of its row group. clean: NaN codes become zeros
    // (returns whether there was one), so that a row that a node does not see cannot reach its sums.
    __device__ __forceinline__ bool store(unsigned char *row, int part, bool clean) const {
        bool nan = false;
        auto put = [&](int dim_group, uint32_t (&o)[4]) {
            if (clean) {
#pragma unroll
                for (int i = 0; i < 4; i++) {
                    const __half2 h = *reinterpret_cast<const __half2 *>(&o[i]);
                    if (__hisnan(__low2half(h))) { o[i] &= 0xffff0000u; nan = true; }
                    if (__hisnan(__high2half(h))) { o[i] &= 0x0000ffffu; nan = true; }
                }
            }
            *reinterpret_cast<uint4 *>(row + dim_group * 128) = make_uint4(o[0], o[1], o[2], o[3]);
        };
#pragma unroll
        for (int it = 0; it < kPieces; it++) {
            const int k = 4 * it + part;
            const uint32_t w[4] = {v[it].x, v[it].y, v[it].z, v[it].w};
            if constexpr (kFp4) {   // 32 codes: dim groups 4 k .. 4 k + 3
                const __half2_raw sc = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(es[it]), __NV_E4M3);
#pragma unroll
                for (int u = 0; u < 4; u++) {
                    uint32_t o[4];
                    fp4_to_f16x8(w[u], static_cast<uint32_t>(u < 2 ? sc.x : sc.y) * 0x10001u, o);
                    put(4 * k + u, o);
                }
            } else {
#pragma unroll
                for (int u = 0; u < 2; u++) {
                    uint32_t o[4];
                    if constexpr (kFmt == kFmtFp8) {
                        fp8_to_f16x4(w[2 * u], o[0], o[1]);
                        fp8_to_f16x4(w[2 * u + 1], o[2], o[3]);
                    } else {
                        codes_to_f16x4(w[2 * u], o[0], o[1]);
                        codes_to_f16x4(w[2 * u + 1], o[2], o[3]);
                    }
                    put(2 * k + u, o);
                }
            }
        }
        return nan;
    }
};

__device__ __forceinline__ void named_sync(int id, int threads) {
    asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}
__device__ __forceinline__ bool named_or(int id, int threads, bool p) {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.u32 p, %1, 0;\n\t"
        "bar.red.or.pred q, %2, %3, p;\n\t"
        "selp.u32 %0, 1, 0, q;\n\t}\n"
        : "=r"(r)
        : "r"(p ? 1u : 0u), "r"(id), "r"(threads)
        : "memory");
    return r != 0;
}

// 2^x to 2 ulp; 0 for x below -126.
__device__ __forceinline__ float tr_exp2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

template <int V>
__device__ __forceinline__ void tr_tmem_ld(uint32_t taddr, uint32_t (&r)[V]) {
    if constexpr (V == 8) tc::tmem_ld8(taddr, r);
    else if constexpr (V == 16) tc::tmem_ld16(taddr, r);
    else tc::tmem_ld32(taddr, r);
}

template <int NQ, int kFmt>
__global__ void __launch_bounds__(kTrThreads, 1) tree_mla_kernel(TreeArgs a, int parts, int q_tiles,
                                                                 float *__restrict__ part_acc,
                                                                 float *__restrict__ part_ml) {
    using L = TrLayout<NQ>;
    constexpr int V = NQ / 2;                                 // query rows of a softmax thread
    constexpr int kLboP = 16 * NQ;                            // P': bytes between groups of 8 keys
    constexpr uint32_t kSCol = 4 * NQ;                        // two score accumulators after the output's 4 tiles
    constexpr int kCols = 6 * NQ <= 128 ? 128 : (6 * NQ <= 256 ? 256 : 512);
    constexpr int kLow = (V == 32) ? 0 : (V == 16) ? 1 : 3;   // lane bits that repeat a query row in butterfly()
    constexpr int kShift = (V == 32) ? 0 : (V == 16) ? 1 : 2;
    pdl_begin(a.q, a.cache, a.rows, a.row_len, a.draft, a.mask, a.n_tree);
    extern __shared__ __align__(128) unsigned char smem[];
    float2 *fac = reinterpret_cast<float2 *>(smem + L::kFac);
    uint64_t *mask = reinterpret_cast<uint64_t *>(smem + L::kMask);
    int64_t *orow = reinterpret_cast<int64_t *>(smem + L::kOut);
    float *red = reinterpret_cast<float *>(smem + L::kRed);
    float *alpha = reinterpret_cast<float *>(smem + L::kAlpha);
    float *scl = reinterpret_cast<float *>(smem + L::kScl);
    float *smx = reinterpret_cast<float *>(smem + L::kMax);
    uint8_t *val = reinterpret_cast<uint8_t *>(smem + L::kValid);
    unsigned *qmax = reinterpret_cast<unsigned *>(smem + L::kQmax);
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + L::kTmem);
    const uint32_t bar0 = tc::smem_addr(smem + L::kBar);
    auto bar = [&](int i) { return bar0 + 8u * static_cast<uint32_t>(i); };

    const int b = blockIdx.z, part = blockIdx.y, qt = blockIdx.x;
    const int tid = threadIdx.x, lane = tid & 31;
    const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
    const TrRange rg = tr_range(a, b, part, parts);
    const int H = a.n_heads, r0 = qt * NQ;
    const int n_rows_q = a.n_nodes * H;                       // query rows of the sequence
    const int live = rg.tree * H;                             // those of its tree
    const bool direct = parts == 1;
    const int n_tiles = r0 < live ? rg.t1 - rg.t0 : 0;

    // where each query row of the tile goes, and what it sees of the drafts
    if (tid < NQ) {
        const int r = r0 + tid, node = r / H;
        int64_t o = -1;
        if (r < n_rows_q) {
            o = static_cast<int64_t>(b) * n_rows_q + r;
            if (!direct) o = ((static_cast<int64_t>(b) * a.n_nodes + node) * parts + part) * H + (r - node * H);
        }
        orow[tid] = o;
        mask[tid] = r < live ? a.mask[static_cast<int64_t>(b) * a.n_nodes + node] : 0ull;
        qmax[tid] = 0u;
    }
    if (n_tiles == 0) {   // no key in the range, or no node of the tree in the tile
        __syncthreads();
        if (!direct) {
            if (tid < NQ && orow[tid] >= 0) {
                part_ml[2 * orow[tid]] = -INFINITY;
                part_ml[2 * orow[tid] + 1] = 0.0f;
            }
            return;
        }
        for (int i = tid; i < NQ * 64; i += kTrThreads)
            if (orow[i >> 6] >= 0) reinterpret_cast<uint4 *>(a.out + orow[i >> 6] * kLatent)[i & 63] = make_uint4(0u, 0u, 0u, 0u);
        if (tid < NQ && orow[tid] >= 0 && a.lse) a.lse[orow[tid]] = -INFINITY;
        return;
    }
    if (warp == kTrWarpMma) {
        tc::tmem_alloc(tc::smem_addr(tmem_slot), kCols);
        tc::tmem_relinquish();
        tc::fence_before_sync();
        if (lane == 0) {
            for (int i = 0; i < 2; i++) {
                tc::mbar_init(bar(kTbFull + i), 4);
                tc::mbar_init(bar(kTbDone + i), 1);
                tc::mbar_init(bar(kTbSFull + i), 1);
                tc::mbar_init(bar(kTbSFree + i), 8);
                tc::mbar_init(bar(kTbPFull + i), 8);
            }
            tc::mbar_init(bar(kTbQ), 8);
            tc::mbar_fence_init();
        }
    }
    __syncthreads();
    tc::fence_after_sync();
    const uint32_t tmem = *tmem_slot;
    // a wait that gives up marks the thread, which skips its later waits; the output is then NaN
    bool ok = true;
    auto wait = [&](int i, int use) {
        if (ok && !tc::mbar_wait(bar(i), static_cast<uint32_t>(use & 1), kTrWaitLimit)) ok = false;
    };

    if (warp >= kTrWarpWiden && warp < kTrWarpMma) {
        // ---------------- widening: rows 8 w + (lane & 7) of each half of a tile ----------------
        const int w = warp - kTrWarpWiden, jl = lane & 7, piece = lane >> 3;
        const int32_t *list = a.rows + static_cast<int64_t>(b) * a.width;
        const int prefix = (rg.plen + kTrKeys - 1) / kTrKeys;
        // the cache row (or drafted row) of key 32 h + 8 w + jl of tile t, -1: none
        auto row_of = [&](int t, int h) -> int64_t {
            if (t >= rg.t1) return -1;
            const int k = h * 32 + w * 8 + jl;
            if (t < prefix) {
                const int j = t * kTrKeys + k;
                const int r = j < rg.plen ? __ldg(list + j) : -1;
                return (r >= 0 && r < a.n_rows) ? r : -1;
            }
            return k < rg.tree ? static_cast<int64_t>(b) * a.n_nodes + k : -1;
        };
        auto base_of = [&](int t) { return t < prefix ? a.cache : a.draft; };
        TrRow<kFmt> row[2];
        int64_t next[2];
#pragma unroll
        for (int h = 0; h < 2; h++) row[h].load(base_of(rg.t0), row_of(rg.t0, h), piece);
#pragma unroll
        for (int h = 0; h < 2; h++) next[h] = row_of(rg.t0 + 1, h);
        for (int i = 0; i < n_tiles; i++) {
            const int t = rg.t0 + i, buf = i & 1;
            if (i >= 2) wait(kTbDone + buf, (i >> 1) - 1);
#pragma unroll
            for (int h = 0; h < 2; h++) {
                const int g = h * 4 + w;   // group of 8 rows
                const bool nan = row[h].store(smem + L::kC + buf * L::kCBytes + g * 8192 + jl * 16, piece, t >= prefix);
                // a drafted row with NaN codes: its scale makes every score with it NaN
                float sc = row[h].scale;
                if (t >= prefix && ((__ballot_sync(0xffffffffu, nan) >> jl) & 0x01010101u)) sc = __int_as_float(0x7fc00000);
                const unsigned valid = __ballot_sync(0xffffffffu, row[h].valid) & 0xffu;
                float m = fabsf(sc) < INFINITY ? sc : 0.0f;
#pragma unroll
                for (int o = 4; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
                if (lane < 8) scl[buf * kTrKeys + g * 8 + lane] = sc;
                if (lane == 0) {
                    smx[buf * 8 + g] = m;
                    val[buf * 8 + g] = static_cast<uint8_t>(valid);
                }
            }
            tc::fence_proxy_async();
            __syncwarp();
            if (lane == 0) tc::mbar_arrive(bar(kTbFull + buf));
            if (i + 1 < n_tiles) {
#pragma unroll
                for (int h = 0; h < 2; h++) row[h].load(base_of(t + 1), next[h], piece);
#pragma unroll
                for (int h = 0; h < 2; h++) next[h] = row_of(t + 2, h);
            }
        }
    } else if (warp == kTrWarpMma) {
        // ---------------- tensor cores ----------------
        constexpr uint32_t id_s = tc::idesc_f16(kTrKeys, NQ, false, false);
        constexpr uint32_t id_o = tc::idesc_f16(128, NQ, true, true);
        const uint64_t dq = tc::desc(tc::smem_addr(smem + L::kQ), 128, 8192);
        const uint64_t dc = tc::desc(tc::smem_addr(smem + L::kC), 128, 8192);
        const uint64_t dct = tc::desc(tc::smem_addr(smem + L::kC), 8192, 128);
        const uint64_t dp = tc::desc(tc::smem_addr(smem + L::kP), kLboP, 128);
        auto accumulate = [&](int i) {   // O^T += C(i)^T P(i)^T: M = 128 latent dims of 4 tiles, K = 64 keys
            const int buf = i & 1;
            wait(kTbPFull + buf, i >> 1);
            ok = __all_sync(0xffffffffu, ok);
            tc::fence_after_sync();
            if (tc::elect_one()) {
                const uint64_t ca = dct + ((buf * L::kCBytes) >> 4), pa = dp + ((buf * L::kPBytes) >> 4);
#pragma unroll
                for (int ks = 0; ks < kTrKeys / 16; ks++)
#pragma unroll
                    for (int mt = 0; mt < kLatent / 128; mt++)
                        tc::mma_bf16(tmem + mt * NQ, ca + ((ks * 2 * 8192 + mt * 2048) >> 4), pa + ((ks * 2 * kLboP) >> 4),
                                     id_o, (i > 0 || ks > 0) ? 1u : 0u);
                tc::mma_commit(bar(kTbDone + buf));
            }
            __syncwarp();
        };
        wait(kTbQ, 0);
        for (int i = 0; i < n_tiles; i++) {
            const int buf = i & 1;
            wait(kTbFull + buf, i >> 1);
            if (i >= 2) wait(kTbSFree + buf, (i >> 1) - 1);
            ok = __all_sync(0xffffffffu, ok);
            tc::fence_after_sync();
            if (tc::elect_one()) {   // S^T = C(i) . Q^T: M = 64 keys, K = 512
                const uint64_t ca = dc + ((buf * L::kCBytes) >> 4);
#pragma unroll
                for (int ks = 0; ks < kLatent / 16; ks++)
                    tc::mma_bf16(tmem + kSCol + buf * NQ, ca + ((ks * 256) >> 4), dq + ((ks * 256) >> 4), id_s,
                                 ks > 0 ? 1u : 0u);
                tc::mma_commit(bar(kTbSFull + buf));
            }
            __syncwarp();
            if (i > 0) accumulate(i - 1);
        }
        accumulate(n_tiles - 1);
    } else {
        // ---------------- softmax ----------------
        // the query rows as fp16, each scaled by the power of two that puts its largest magnitude in
        // [2^14, 2^15) (exact: bf16 mantissas fit fp16)
        {
            constexpr int kGroups = NQ / 8;                       // groups of 8 query rows
            constexpr int kStride = 32 / kGroups;                 // threads of a row: its pieces interleave
            constexpr int kP = 64 / kStride;
            const int qr = (warp % kGroups) * 8 + (lane & 7), p0 = (warp / kGroups) * 4 + (lane >> 3);
            const bool real = r0 + qr < live;
            const uint4 *src = reinterpret_cast<const uint4 *>(a.q + (static_cast<int64_t>(b) * n_rows_q + (real ? r0 + qr : 0)) * kLatent);
            uint4 v[kP];
            unsigned mx = 0u;
#pragma unroll
            for (int i = 0; i < kP; i++) {
                v[i] = real ? __ldg(src + p0 + i * kStride) : make_uint4(0u, 0u, 0u, 0u);
                const uint32_t w4[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
#pragma unroll
                for (int e = 0; e < 4; e++) mx = max(mx, max(w4[e] & 0x7fffu, (w4[e] >> 16) & 0x7fffu));
            }
            mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, 8));
            mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, 16));
            if (lane < 8) atomicMax(&qmax[qr], mx);
            named_sync(1, 256);
            auto exponent = [](unsigned m) { return m == 0u ? 0 : min(120, max(-120, 14 - (static_cast<int>(m >> 7) - 127))); };
            const float f = __uint_as_float(static_cast<uint32_t>(exponent(qmax[qr]) + 127) << 23);
            if (tid < NQ)
                fac[tid] = make_float2(a.sm_scale * 1.4426950408889634f *
                                           __uint_as_float(static_cast<uint32_t>(127 - exponent(qmax[tid])) << 23), kTrNone);
#pragma unroll
            for (int i = 0; i < kP; i++) {
                const uint32_t w4[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
                uint32_t o[4];
#pragma unroll
                for (int k = 0; k < 4; k++)
                    o[k] = f16x2_rn(__uint_as_float(w4[k] << 16) * f, __uint_as_float(w4[k] & 0xffff0000u) * f);
                *reinterpret_cast<uint4 *>(smem + L::kQ + (qr >> 3) * 8192 + (p0 + i * kStride) * 128 + (qr & 7) * 16) =
                    make_uint4(o[0], o[1], o[2], o[3]);
            }
            tc::fence_proxy_async();
            named_sync(1, 256);
            if (lane == 0) tc::mbar_arrive(bar(kTbQ));
        }
        const int quad = warp & 3, hh = warp >> 2, c0 = hh * V;
        const uint32_t lanes = static_cast<uint32_t>(quad * 32) << 16;
        const int j = quad * 16 + (lane & 15);                    // this thread's key of a tile (M = 64: lanes 0-15)
        const bool has_key = lane < 16;
        const int draft_tile = rg.tree > 0 ? rg.tiles - 1 : -1;
        float l[V];
#pragma unroll
        for (int e = 0; e < V; e++) l[e] = 0.0f;
        float sigma = 0.0f;
        for (int i = 0; i < n_tiles; i++) {
            const int buf = i & 1, t = rg.t0 + i;
            wait(kTbFull + buf, i >> 1);                          // (the tile's scales and valid rows)
            wait(kTbSFull + buf, i >> 1);
            ok = __all_sync(0xffffffffu, ok);
            tc::fence_after_sync();
            uint32_t r[V];
            tr_tmem_ld<V>(tmem + lanes + kSCol + buf * NQ + c0, r);
            tc::tmem_wait_ld();
            tc::fence_before_sync();
            __syncwarp();
            if (lane == 0) tc::mbar_arrive(bar(kTbSFree + buf));
            const bool key = has_key && ((val[buf * 8 + (j >> 3)] >> (j & 7)) & 1);
            const float sc = key ? scl[buf * kTrKeys + j] : 0.0f;
            float smax = smx[buf * 8];
#pragma unroll
            for (int w = 1; w < 8; w++) smax = fmaxf(smax, smx[buf * 8 + w]);
            float x[V];
            const float4 *f4 = reinterpret_cast<const float4 *>(fac + c0);
            auto scores = [&]() {   // the score of this thread's key with each query row, less its reference
#pragma unroll
                for (int e = 0; e < V; e += 2) {
                    const float4 f = f4[e >> 1];
                    x[e] = key ? fmaf(__uint_as_float(r[e]) * sc, f.x, -f.y) : -INFINITY;
                    x[e + 1] = key ? fmaf(__uint_as_float(r[e + 1]) * sc, f.z, -f.w) : -INFINITY;
                }
                if (t == draft_tile) {   // what each node sees of the drafts
#pragma unroll
                    for (int e = 0; e < V; e++)
                        if (!((mask[c0 + e] >> j) & 1ull)) x[e] = -INFINITY;
                }
            };
            scores();
            bool over = false;
#pragma unroll
            for (int e = 0; e < V; e++) over |= x[e] > kTrGrow;
            const bool grow = smax > 16.0f * sigma;               // (sigma 0: no scale yet)
            if (named_or(1, 256, over) || grow) {
                // move the references and sigma, and rescale what they scale
                float m[V];
#pragma unroll
                for (int e = 0; e < V; e++)
                    m[e] = x[e] == -INFINITY ? -INFINITY : __uint_as_float(r[e]) * sc * fac[c0 + e].x;
                const float bm = butterfly<V, true>(m);
                if ((lane & kLow) == 0) red[quad * NQ + c0 + ((lane >> kShift) & (V - 1))] = bm;
                const float sig_new = grow ? pow2_ceil(smax) : sigma;
                const float beta = sigma == 0.0f ? 1.0f : sigma / sig_new;   // powers of two: exact
                sigma = sig_new;
                named_sync(1, 256);
                if (tid < NQ) {
                    const float mc = fmaxf(fmaxf(red[tid], red[NQ + tid]), fmaxf(red[2 * NQ + tid], red[3 * NQ + tid]));
                    const float old = fac[tid].y, ref = mc > old + kTrGrow ? mc : old;
                    alpha[tid] = exp2f(old - ref);
                    fac[tid].y = ref;
                }
                named_sync(1, 256);
#pragma unroll
                for (int e = 0; e < V; e++) l[e] *= alpha[c0 + e];
                if (i > 0) {
                    wait(kTbDone + ((i - 1) & 1), (i - 1) >> 1);
                    ok = __all_sync(0xffffffffu, ok);
                    tc::fence_after_sync();
                    constexpr int CH = NQ < 32 ? NQ : 32;
#pragma unroll 1
                    for (int mt = hh; mt < kLatent / 128; mt += 2) {
#pragma unroll 1
                        for (int cb = 0; cb < NQ; cb += CH) {
                            uint32_t o[CH];
                            tr_tmem_ld<CH>(tmem + lanes + mt * NQ + cb, o);
                            tc::tmem_wait_ld();
#pragma unroll
                            for (int e = 0; e < CH; e++)
                                o[e] = __float_as_uint(__uint_as_float(o[e]) * (alpha[cb + e] * beta));
                            if constexpr (CH == 16) tc::tmem_st16(tmem + lanes + mt * NQ + cb, o);
                            else tc::tmem_st32(tmem + lanes + mt * NQ + cb, o);
                        }
                    }
                    tc::tmem_wait_st();
                    tc::fence_before_sync();
                }
                scores();
            }
            const float ratio = sigma > 0.0f ? sc * (kTrBoost / sigma) : sc;   // (sigma 0: every finite scale is 0)
            if (i >= 2) wait(kTbDone + buf, (i >> 1) - 1);        // P(i - 2) has been read
            unsigned char *line = smem + L::kP + buf * L::kPBytes + (j >> 3) * kLboP + (c0 >> 3) * 128 + (j & 7) * 16;
#pragma unroll
            for (int g = 0; g < V / 8; g++) {
                uint32_t p4[4];
#pragma unroll
                for (int e = 0; e < 8; e += 2) {
                    const float p0 = tr_exp2(x[8 * g + e]), p1 = tr_exp2(x[8 * g + e + 1]);
                    l[8 * g + e] += p0;
                    l[8 * g + e + 1] += p1;
                    p4[e >> 1] = f16x2_rn(p0 * ratio, p1 * ratio);
                }
                if (has_key) *reinterpret_cast<uint4 *>(line + g * 128) = make_uint4(p4[0], p4[1], p4[2], p4[3]);
            }
            tc::fence_proxy_async();
            __syncwarp();
            if (lane == 0) tc::mbar_arrive(bar(kTbPFull + buf));
        }
        // the sums of the tile's query rows, and what their accumulators are multiplied by
        wait(kTbDone + ((n_tiles - 1) & 1), (n_tiles - 1) >> 1);
        const float bl = butterfly<V, false>(l);
        if ((lane & kLow) == 0) red[quad * NQ + c0 + ((lane >> kShift) & (V - 1))] = bl;
        named_sync(1, 256);
        if (tid < NQ) {
            const float sum = (red[tid] + red[NQ + tid]) + (red[2 * NQ + tid] + red[3 * NQ + tid]);
            const bool none = r0 + tid >= live || sum == 0.0f;    // (a node past the tree's, or no visible key)
            const float m = fac[tid].y * 0.6931471805599453f;
            const float scale = sigma * (1.0f / kTrBoost);
            alpha[tid] = none ? 0.0f : (direct ? scale / sum : scale);
            mask[tid] = none ? 0ull : 1ull;
            if (orow[tid] >= 0) {
                if (!direct) {
                    part_ml[2 * orow[tid]] = none ? -INFINITY : m;
                    part_ml[2 * orow[tid] + 1] = none ? 0.0f : sum;
                } else if (a.lse) {
                    a.lse[orow[tid]] = none ? -INFINITY : m + logf(sum);
                }
            }
        }
    }
    const bool all_ok = __syncthreads_and(ok);
    if (!all_ok) {   // a wait gave up: the status word, and a bounded wait for products still in flight
        if (tid == 0) atomicOr(a.status, 32);
        tc::mbar_wait(bar(kTbDone + ((n_tiles - 1) & 1)), static_cast<uint32_t>(((n_tiles - 1) >> 1) & 1), kTrWaitLimit);
        __syncthreads();
    }
    tc::fence_after_sync();
    if (warp < 8) {
        // O^T: tile mt of 128 latent dims, lane quadrant warp % 4 (dim 128 mt + 32 quad + lane)
        constexpr int CH = 16;
#pragma unroll 1
        for (int mt = warp >> 2; mt < kLatent / 128; mt += 2) {
            const int dim = mt * 128 + (warp & 3) * 32 + lane;
            const uint32_t ta = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16) + mt * NQ;
#pragma unroll 1
            for (int cb = 0; cb < NQ; cb += CH) {
                uint32_t o[CH];
                tr_tmem_ld<CH>(ta + cb, o);
                tc::tmem_wait_ld();
#pragma unroll
                for (int e = 0; e < CH; e++) {
                    const int64_t at = orow[cb + e];
                    const bool seen = mask[cb + e] != 0ull;
                    float v = seen ? __uint_as_float(o[e]) * alpha[cb + e] : 0.0f;
                    if (!all_ok) v = __int_as_float(0x7fc00000);
                    if (at >= 0) {
                        if (direct) a.out[at * kLatent + dim] = __bfloat16_as_ushort(__float2bfloat16_rn(v));
                        else if (seen) part_acc[at * kLatent + dim] = v;
                    }
                }
            }
        }
        if (!all_ok && tid < NQ && orow[tid] >= 0) {
            if (direct && a.lse) a.lse[orow[tid]] = __int_as_float(0x7fc00000);
        }
    }
    tc::fence_before_sync();
    __syncthreads();
    if (warp == kTrWarpMma) {
        tc::fence_after_sync();
        tc::tmem_dealloc(tmem, kCols);
    }
}

template <int NQ, int kFmt>
cudaError_t launch_tree_t(const TreePlan &p, const TreeArgs &a, float *part_acc, float *part_ml, cudaStream_t stream) {
    auto kernel = tree_mla_kernel<NQ, kFmt>;
    const int smem = TrLayout<NQ>::kBytes;
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    e = launch_pdl(kernel, dim3(p.q_tiles, p.parts, a.batch), dim3(kTrThreads), smem, stream, a, p.parts, p.q_tiles,
                   part_acc, part_ml);
    return e != cudaSuccess ? e : cudaGetLastError();
}

constexpr int kTrMaxParts = 1024;              // partials of one query that the combine kernel merges

}  // namespace

TreePlan tree_plan(int batch, int n_nodes, int n_heads, int width, int num_sms) {
    TreePlan p{};
    const int rows = n_nodes * n_heads;
    p.nq = rows <= 16 ? 16 : (rows <= 32 ? 32 : 64);
    p.q_tiles = (rows + p.nq - 1) / p.nq;
    p.parts = 1;
    const long long tiles = (width + kTrKeys - 1) / kTrKeys + 1, base = static_cast<long long>(batch) * p.q_tiles;
    // ranges: the count that minimises waves x (tiles per range + about three tiles of set-up and
    // output), a combine counting as four more; at most two waves of CTAs, so that the partials
    // stay within the workspace
    long long best = -1;
    for (long long n = 1; n <= tiles && n <= kTrMaxParts && (n == 1 || base * n <= 2ll * num_sms); n++) {
        const long long waves = (base * n + num_sms - 1) / num_sms;
        const long long cost = waves * ((tiles + n - 1) / n + 3) + (n > 1 ? 4 : 0);
        if (best < 0 || cost < best) {
            best = cost;
            p.parts = static_cast<int>(n);
        }
    }
    return p;
}

size_t tree_partials(int batch, int n_nodes, int n_heads, int width, int num_sms) {
    // a plan of more than one range has at most two waves of CTAs of at most 64 query rows
    const long long rows = static_cast<long long>(batch) * n_nodes * n_heads;
    long long tiles = (width + kTrKeys - 1) / kTrKeys + 1;
    if (tiles > kTrMaxParts) tiles = kTrMaxParts;
    const long long cap = 2ll * num_sms * 64;
    return static_cast<size_t>(rows * tiles < cap ? rows * tiles : cap);
}

cudaError_t launch_tree_mla(const TreePlan &p, const TreeArgs &a, int format, float *part_acc, float *part_ml,
                            cudaStream_t stream) {
#define GLM_TREE_LAUNCH(N, F) \
    if (p.nq == N && format == F) return launch_tree_t<N, F>(p, a, part_acc, part_ml, stream);
    GLM_TREE_LAUNCH(16, kFmtInt8)
    GLM_TREE_LAUNCH(32, kFmtInt8)
    GLM_TREE_LAUNCH(64, kFmtInt8)
    GLM_TREE_LAUNCH(16, kFmtFp8)
    GLM_TREE_LAUNCH(32, kFmtFp8)
    GLM_TREE_LAUNCH(64, kFmtFp8)
    GLM_TREE_LAUNCH(16, kFmtFp4)
    GLM_TREE_LAUNCH(32, kFmtFp4)
    GLM_TREE_LAUNCH(64, kFmtFp4)
#undef GLM_TREE_LAUNCH
    return cudaErrorInvalidValue;
}

}  // namespace glm
