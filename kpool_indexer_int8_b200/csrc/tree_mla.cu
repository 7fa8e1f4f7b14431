// tree_mla.cu -- attention of a tree of drafted tokens over latent cache rows, on the sm_100a
// tensor cores: node i of sequence b attends to the rows of its sequence's index list and to the
// drafted rows whose bit is set in its mask,
//     s = sm_scale q . c,   out = sum softmax(s) c,   lse = log sum exp(s),   c = code * scale,
// the latent row being key and value. Every (node, head) of a sequence is a row of one query
// matrix, so that a widened tile of keys serves all of them. This file: tiles of at most 64 query rows;
// tree_mla_pair.cu: of 128.
//
// One CTA per (sequence, tile of query rows, run of keys) walks its run 64 keys at a time, the drafted
// rows behind those of the list. Keys are the MMA M dimension, the NQ query rows the N dimension (as in the
// sparse attention); 17 warps in three roles:
//   * warps 8-15 (widening): eight rows of each tile each. Rows come into slots of the warp's own by
//     asynchronous copies, four at a time and (16 query rows) two tiles ahead, and are written as fp16
//     (exact: int8 and E4M3 codes, E2M1 code times block scale) to one of two tiles C[64 x 512], rows of
//     128 bytes in the 128-byte swizzle, which the tensor cores read both as keys and, transposed, as values;
//   * warp 16 (tensor cores): S^T(t) = C(t) . Q^T into one of two accumulators, O^T += C(t)^T P(t)^T,
//     whichever is ready first;
//   * warps 0-7 (softmax): x = S scale_row qk - ref in log2 units, P' = 2^x scale_row / sigma as fp16, with a
//     reference and a sigma for each query row. They move only when a weight of the row would pass 2^15 (a
//     vote of the eight warps per tile): then the accumulator in tensor memory is rescaled, otherwise no
//     maximum is taken. Sums stay in registers, one per thread and query row, until the end.
// P' is one fp16 term: a weight is off by at most 2^-11 of itself (an eighth of the bf16 output's 2^-8), or,
// once P' is below 2^-14, by 2^-24 - kHead of the row's largest weight times scale. Tiles of 16 query rows carry what it
// leaves as a second term, as the sparse attention does (2^-22): 16 more columns of N, 73.7 us for 71.6 over
// 262,144 4-bit rows. With 32 rows that takes 93 us for 87, with 64 shared memory has no room for it, and in a
// pair, where it doubles the products with the values, those alone take 58 us more than its 379.
//
// A sequence's keys are cut into runs so that the CTAs fill the SMs; tree_combine.cu merges the
// partials. Every wait is bounded; one that gives up sets the status word and the CTA writes NaN.
//
// What bounds it: with 16 query rows and a long list, the chain from a free C tile through widening
// (about 700 cycles), S (32 products of 23, 1,100 with their latency), softmax (1,700) and O (900), of which
// two are in flight: a 64-key tile takes 3,300 cycles, where shared memory (C written once and read twice)
// would allow 2,000. 262,144 4-bit rows, 16 query rows: 74 us a call with the merge, 1.1 TB/s; the rows at
// the copy rate would take 12. A small call is bound by the latencies of its start, two tiles and end (35 % of
// the warps' time waits for loads, 6 % for instructions): 67 int8 keys and 64 query rows take 9.7 us of the GPU.
#include <algorithm>

#include "tree_mla_common.cuh"

namespace glm {

namespace {

using namespace tree;

constexpr int kTrSoft = 8;                     // warps 0-7 softmax, then the widening warps and one for the tensor cores
constexpr int kTrKeys = 64;                    // keys of a tile

enum TrBar { kTbFull = 0, kTbDone = 2, kTbS = 4, kTbP = 6, kTbEnd = 8, kTbCount };

template <int NQ>
struct TrLayout {
    static constexpr int kCBytes = kTrKeys * 1024;
    static constexpr int kC = 0;                                 // [2] tiles: 8 blocks of 64 dims x 64 keys x 128 B, swizzled
    static constexpr int kQ = kC + 2 * kCBytes;                  // NQ/8 row groups x 64 dim groups x 128 B
    static constexpr int kTerms = NQ == 16 ? 2 : 1;               // fp16 numbers of a weight: columns of P' beside each other
    static constexpr int kNP = kTerms * NQ;
    static constexpr int kPBytes = kTrKeys * 2 * kNP;
    static constexpr int kPBufs = NQ == 64 ? 1 : 2;              // (what else shared memory holds of 64 rows)
    static constexpr int kP = kQ + NQ * 1024;                    // [kPBufs] P', core matrices of 8 keys x 8 query rows
    static constexpr int kWiden = 8;                              // widening warps
    static constexpr int kThreads = (kTrSoft + kWiden + 1) * 32;
    static constexpr int kGroups = NQ == 16 ? 4 : (NQ == 32 ? 2 : 1);            // groups of 4 rows a widening warp has in flight
    static constexpr int kRaw = kP + kPBufs * kPBytes;           // cache rows: codes, then tails, [kWiden warps][groups][4]
    static constexpr int kFac = kRaw + kWiden * kGroups * 4 * kRowBytes;                // [NQ] (score factor, reference) pairs
    static constexpr int kMask = kFac + NQ * 8;                  // [NQ] visibility words
    static constexpr int kOut = kMask + NQ * 8;                  // [NQ] row of the output or partial, -1: none
    static constexpr int kRed = kOut + NQ * 8;                   // [2][4 quadrants][NQ]
    static constexpr int kAlpha = kRed + 2 * 4 * NQ * 4;         // [NQ] factors of a rescale, at the end of the output
    static constexpr int kSigma = kAlpha + NQ * 4;               // [NQ] 1 / sigma
    static constexpr int kLog = kSigma + NQ * 4;                 // [NQ] log2 sigma, -infinity: no reference yet
    static constexpr int kScl = kLog + NQ * 4;                   // [2][64] row scales
    static constexpr int kValid = kScl + 2 * kTrKeys * 4;        // [2][64] bytes: 1 where there is a key
    static constexpr int kQmax = kValid + 2 * kTrKeys;                    // [NQ] |q| maxima (bf16 bits)
    static constexpr int kBar = kQmax + NQ * 4;
    static constexpr int kTmem = kBar + kTbCount * 8;
    static constexpr int kBytes = kTmem + 8;
    static constexpr int kAlloc = kBytes + 1024;                 // from a 1024-byte aligned base
    static_assert(kQ % 128 == 0 && kP % 128 == 0 && kFac % 16 == 0 && kBar % 8 == 0 && kMask % 8 == 0 && kSigma % 16 == 0 && kLog % 16 == 0,
                  "alignment");
    static_assert(kAlloc <= 232448, "shared memory of one CTA");
};

template <int V>
__device__ __forceinline__ void tr_tmem_ld(uint32_t taddr, uint32_t (&r)[V]) {
    if constexpr (V == 8) tc::tmem_ld8(taddr, r);
    else if constexpr (V == 16) tc::tmem_ld16(taddr, r);
    else tc::tmem_ld32(taddr, r);
}

// The largest over a warp's keys, one a lane with scores x of V query rows and log2 scale lg, for the row that butterfly()
// leaves in this lane.
template <int V>
__device__ __forceinline__ Largest largest_of(const float (&x)[V], float lg) {
    const int lane = threadIdx.x & 31;
    auto get = [](Largest v, int bit) { return Largest{__shfl_xor_sync(0xffffffffu, v.x, bit), __shfl_xor_sync(0xffffffffu, v.y, bit)}; };
    Largest t[V / 2];
    {
        const bool up = (lane & 16) != 0;
        const float other = __shfl_xor_sync(0xffffffffu, lg, 16);
#pragma unroll
        for (int i = 0; i < V / 2; i++) {
            const float send = up ? x[i] : x[i + V / 2], keep = up ? x[i + V / 2] : x[i];
            t[i] = larger({keep, lg}, {__shfl_xor_sync(0xffffffffu, send, 16), other});
        }
    }
#pragma unroll
    for (int half = V / 4, bit = 8; half >= 1; half >>= 1, bit >>= 1) {
        const bool up = (lane & bit) != 0;
#pragma unroll
        for (int i = 0; i < half; i++) {
            const Largest send = up ? t[i] : t[i + half], keep = up ? t[i + half] : t[i];
            t[i] = larger(keep, get(send, bit));
        }
    }
    constexpr int kRest = (V == 32) ? 0 : (V == 16) ? 1 : 2;
#pragma unroll
    for (int k = 0; k < kRest; k++) t[0] = larger(t[0], get(t[0], 1 << (kRest - 1 - k)));
    return t[0];
}

template <int NQ, int kFmt>
__global__ void __launch_bounds__(TrLayout<NQ>::kThreads, 1) tree_mla_kernel(TreeArgs a, TreePlan plan, float *__restrict__ part_acc,
                                                                 float *__restrict__ part_ml) {
    using L = TrLayout<NQ>;
    using R = Row<kFmt>;
    constexpr int kThreads = L::kThreads, kTrWarpMma = kTrSoft + L::kWiden;
    constexpr int V = NQ / 2;                                 // query rows of a softmax thread
    constexpr int NP = L::kNP, kLboP = 16 * NP;               // P': bytes between groups of 8 keys
    constexpr uint32_t kSCol = 4 * NP;                        // two score accumulators after the output's 4 tiles
    constexpr int kCols = 4 * NP + 2 * NQ <= 256 ? 256 : 512;   // (160, 192, 384)
    constexpr int kLow = (V == 32) ? 0 : (V == 16) ? 1 : 3;   // lane bits that repeat a query row in butterfly()
    constexpr int kShift = (V == 32) ? 0 : (V == 16) ? 1 : 2;
    pdl_begin(a.q, a.cache, a.rows, a.row_len, a.draft, a.mask, a.n_tree);
    extern __shared__ __align__(1024) unsigned char smem_raw[];
    unsigned char *smem = smem_raw + ((1024u - (tc::smem_addr(smem_raw) & 1023u)) & 1023u);
    float2 *fac = reinterpret_cast<float2 *>(smem + L::kFac);
    uint64_t *mask = reinterpret_cast<uint64_t *>(smem + L::kMask);
    int64_t *orow = reinterpret_cast<int64_t *>(smem + L::kOut);
    float *red = reinterpret_cast<float *>(smem + L::kRed);
    float *alpha = reinterpret_cast<float *>(smem + L::kAlpha);
    float *scl = reinterpret_cast<float *>(smem + L::kScl);
    float *inv = reinterpret_cast<float *>(smem + L::kSigma);
    float *log_sigma = reinterpret_cast<float *>(smem + L::kLog);
    uint8_t *val = reinterpret_cast<uint8_t *>(smem + L::kValid);
    unsigned *qmax = reinterpret_cast<unsigned *>(smem + L::kQmax);
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + L::kTmem);
    const uint32_t bar0 = tc::smem_addr(smem + L::kBar);
    auto bar = [&](int i) { return bar0 + 8u * static_cast<uint32_t>(i); };

    const int r0 = blockIdx.x * NQ, part = blockIdx.y, b = blockIdx.z, parts = plan.parts;
    const int tid = threadIdx.x, lane = tid & 31;
    const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
    const int H = a.n_heads;
    const int n_rows_q = a.n_nodes * H;                       // query rows of the sequence; this CTA's: r0 .. r0 + NQ - 1
    const bool direct = parts == 1;
    const Lengths own = load_lengths(a, b, true), mine = load_lengths(a, lane, !direct && lane < a.batch);
    for (int i = tid; i < min(NQ, n_rows_q - r0) * 8; i += kThreads)   // (read when the lengths are there)
        prefetch_line(a.q + (static_cast<int64_t>(b) * n_rows_q + r0) * kLatent + i * 64);
    // the sequence's tiles [0, tiles), those of the list first, and this part's [t0, t1)
    const int plen = list_len(a, own), tree_n = tree_len(a, own);
    const int n_keys = plen + tree_n, tiles = (n_keys + kTrKeys - 1) / kTrKeys;
    const int run = direct ? tiles : run_tiles(a, plan, kTrKeys, mine);
    const int t0 = static_cast<int>(min(static_cast<int64_t>(tiles), static_cast<int64_t>(part) * run));
    const int t1 = min(tiles, t0 + run);
    const int live = tree_n * H - r0;                         // of this CTA's query rows, those of the tree
    const int n_tiles = live > 0 ? t1 - t0 : 0;

    // where each query row goes, and what it sees of the drafts
    if (tid < NQ) {
        const int r = r0 + tid, node = r / H;
        int64_t o = -1;
        if (r < n_rows_q) {
            o = static_cast<int64_t>(b) * n_rows_q + r;
            if (!direct) o = ((static_cast<int64_t>(b) * a.n_nodes + node) * parts + part) * H + (r - node * H);
        }
        orow[tid] = o;
        mask[tid] = tid < live ? a.mask[static_cast<int64_t>(b) * a.n_nodes + node] : 0ull;
        qmax[tid] = 0u;
    }
    if (n_tiles == 0) {   // no key in the run, or no tree
        __syncthreads();
        if (!direct) {
            if (tid < NQ && orow[tid] >= 0) {
                part_ml[2 * orow[tid]] = -INFINITY;
                part_ml[2 * orow[tid] + 1] = 0.0f;
            }
            return;
        }
        for (int i = tid; i < NQ * 64; i += kThreads)
            if (orow[i >> 6] >= 0) reinterpret_cast<uint4 *>(a.out + orow[i >> 6] * kLatent)[i & 63] = make_uint4(0u, 0u, 0u, 0u);
        if (tid < NQ && orow[tid] >= 0 && a.lse) a.lse[orow[tid]] = -INFINITY;
        return;
    }
    // The warp's rows come into slots of its own in groups of four, each group refilled as soon as it
    // is read; lanes 0 .. kN - 1 hold the entries of a tile's keys.
    const bool widening = warp >= kTrSoft && warp < kTrWarpMma;
    constexpr int kN = kTrKeys / L::kWiden, kGt = kN / 4, kG = L::kGroups;   // keys and groups of a tile
    const int w = warp - kTrSoft;
    unsigned char *codes = smem + L::kRaw + w * kG * 4 * R::kCodes;
    unsigned char *tails = smem + L::kRaw + L::kWiden * kG * 4 * R::kCodes + w * kG * 4 * R::kTail;
    const int32_t *list = a.rows + static_cast<int64_t>(b) * a.width;
    // (An entry is looked at only when its row is needed: a test right behind the load would hold
    // the warp until it is there.)
    const int k = w * kN + lane;
    auto entry_of = [&](int t) -> int {
        if (t >= t1 || lane >= kN) return -1;
        const int j = t * kTrKeys + k;
        if (j < plen) return __ldg(list + j);
        return j < n_keys ? draft_row(b * a.n_nodes + j - plen) : -1;
    };
    auto row_of = [&](int t, int entry) { return t * kTrKeys + k >= plen || (entry >= 0 && entry < a.n_rows) ? entry : -1; };
    // starts copying group g (of four rows; kGt groups a tile, counted from the run's first); `rows`:
    // what the lanes hold of its tile
    auto request = [&](int g, int rows) {
        if (g < kGt * n_tiles)
            R::template fetch<4>(codes + g % kG * 4 * R::kCodes, tails + g % kG * 4 * R::kTail, a, rows, g % kGt * 4,
                                 (t0 + g / kGt + 1) * kTrKeys > plen);
        copy_commit();
    };
    // rows of tiles i .. i + 2, entries of the one after; the first copies go out before the barriers are there
    int rows[3] = {-1, -1, -1}, entry = -1;
    if (widening) {
        int e[3];
#pragma unroll
        for (int u = 0; u < 3; u++) e[u] = entry_of(t0 + u);
        entry = entry_of(t0 + 3);
#pragma unroll
        for (int u = 0; u < 3; u++) rows[u] = row_of(t0 + u, e[u]);
#pragma unroll
        for (int g = 0; g < kG; g++) request(g, rows[g / kGt]);
    }
    if (warp < kTrSoft) {
        // the query rows as fp16, each scaled by the power of two that puts its largest magnitude in
        // [2^14, 2^15): groups of 8 rows, the warps of a group and four lanes each sharing a row's pieces
        constexpr int kGroups = NQ / 8;
        constexpr int kStride = 32 / kGroups;                 // threads of a row
        constexpr int kN = 64 / kStride;
        const int qr = (warp % kGroups) * 8 + (lane & 7), p0 = (warp / kGroups) * 4 + (lane >> 3);
        const bool real = qr < live;
        const uint4 *src = reinterpret_cast<const uint4 *>(a.q + (static_cast<int64_t>(b) * n_rows_q + r0 + (real ? qr : 0)) * kLatent);
        named_sync(1, 256);                                   // (qmax is set)
        uint4 v[kN];
        unsigned mx = 0u;
#pragma unroll
        for (int i = 0; i < kN; i++) {
            v[i] = real ? __ldg(src + p0 + i * kStride) : make_uint4(0u, 0u, 0u, 0u);
            mx = max(mx, bf16_absmax(v[i]));
        }
        mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, 8));
        mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, 16));
        if (lane < 8) atomicMax(&qmax[qr], mx);
        named_sync(1, 256);
        const float f = pow2f_exact(query_exponent(qmax[qr]));
        if (tid < NQ) {
            fac[tid] = make_float2(a.sm_scale * 1.4426950408889634f * pow2f_exact(-query_exponent(qmax[tid])), 0.0f);
            inv[tid] = 1.0f;
            log_sigma[tid] = -INFINITY;
        }
#pragma unroll
        for (int i = 0; i < kN; i++)
            *reinterpret_cast<uint4 *>(smem + L::kQ + (qr >> 3) * 8192 + (p0 + i * kStride) * 128 + (qr & 7) * 16) =
                bf16_to_f16x8(v[i], f);
        tc::fence_proxy_async();
    }
    if (warp == kTrWarpMma) {
        tc::tmem_alloc(tc::smem_addr(tmem_slot), kCols);
        tc::tmem_relinquish();
        tc::fence_before_sync();
        if (lane == 0) {
            for (int i = 0; i < 2; i++) {
                tc::mbar_init(bar(kTbFull + i), L::kWiden);
                tc::mbar_init(bar(kTbDone + i), 1);
                tc::mbar_init(bar(kTbS + i), 1);
                tc::mbar_init(bar(kTbP + i), 8);
            }
            tc::mbar_init(bar(kTbEnd), 1);
            tc::mbar_fence_init();
        }
    }
    __syncthreads();
    tc::fence_after_sync();
    const uint32_t tmem = *tmem_slot;
    // a wait that gives up marks the thread, which skips its later waits; the output is then NaN
    bool ok = !a.give_up;
    auto wait = [&](int i, int use) {
        if (ok && !tc::mbar_wait(bar(i), static_cast<uint32_t>(use & 1), kWaitLimit)) ok = false;
    };

    if (widening) {
        // ---------------- widening: keys kN w .. kN w + kN - 1 of each tile ----------------
        for (int i = 0; i < n_tiles; i++) {
            const int t = t0 + i, buf = i & 1;
            const bool drafts = (t + 1) * kTrKeys > plen;     // some of its keys are
            const bool valid = rows[0] != -1;
            float sc = 0.0f;
#pragma unroll
            for (int h = 0; h < kGt; h++) {
                const int g = kGt * i + h;
                copy_wait<kG - 1>();                          // the group is there
                unsigned char *first = codes + g % kG * 4 * R::kCodes, *tail = tails + g % kG * 4 * R::kTail;
                if (valid && lane / 4 == h) sc = R::scale(tail + (lane & 3) * R::kTail);
                if (kFmt != kFmtInt8 && drafts) {   // a row with NaN codes: its scale makes every score with it NaN
                    for (int r = 0; r < 4; r++)
                        if (R::has_nan(first + r * R::kCodes, tail + r * R::kTail) && lane == h * 4 + r && valid) sc = __int_as_float(0x7fc00000);
                    R::clean(R::kFp4 ? tail : first, 4 * (R::kFp4 ? R::kTail : R::kCodes));
                }
                // the lines of the group, then the next group's copies into its slots, then the wait: what
                // follows Done(i - 2) is on the path from it to S(i)
                typename R::Line v[4][2];                     // lines lane and lane + 32 of each row
#pragma unroll
                for (int r = 0; r < 4; r++)
#pragma unroll
                    for (int u = 0; u < 2; u++)
                        v[r][u] = R::line(first + r * R::kCodes, tail + r * R::kTail, lane + 32 * u, lane / 2 + 16 * u);
                __syncwarp();
                request(g + kG, rows[(h + kG) / kGt]);
                if (h == 0 && i >= 2) wait(kTbDone + buf, (i >> 1) - 1);   // C(i - 2) has been read
#pragma unroll
                for (int r = 0; r < 4; r++) {
                    unsigned char *to = smem + L::kC + buf * L::kCBytes + (lane >> 3) * 8192 + swizzled(w * kN + h * 4 + r, lane & 7);
#pragma unroll
                    for (int u = 0; u < 2; u++) *reinterpret_cast<uint4 *>(to + u * 4 * 8192) = R::widen(v[r][u]);
                }
            }
            if (lane < kN) {
                scl[buf * kTrKeys + k] = sc + (sc - sc);   // (an infinite scale: NaN, as 0 codes times it are)
                val[buf * kTrKeys + k] = valid ? 1 : 0;
            }
            tc::fence_proxy_async();
            __syncwarp();
            if (lane == 0) tc::mbar_arrive(bar(kTbFull + buf));
            rows[0] = rows[1];
            rows[1] = rows[2];
            rows[2] = row_of(t + 3, entry);
            entry = entry_of(t + 4);
        }
    } else if (warp == kTrWarpMma) {
        // ---------------- tensor cores ----------------
        constexpr uint32_t id_s = tc::idesc_f16(kTrKeys, NQ, false, false);
        constexpr uint32_t id_o = tc::idesc_f16(128, NP, true, true);
        const uint64_t dq = tc::desc(tc::smem_addr(smem + L::kQ), 128, 8192);
        const uint64_t dc = tc::desc_sw128(tc::smem_addr(smem + L::kC), 1024);
        const uint64_t dct = tc::desc_sw128_mn(tc::smem_addr(smem + L::kC), 8192, 1024);
        const uint64_t dp = tc::desc(tc::smem_addr(smem + L::kP), kLboP, 128);
        auto accumulate = [&](int i) {   // O^T += C(i)^T P(i)^T: M = 128 latent dims of 4 tiles, K = 64 keys
            const int buf = i & 1;
            wait(kTbP + buf, i >> 1);
            ok = __all_sync(0xffffffffu, ok);
            tc::fence_after_sync();
            if (tc::elect_one()) {
                const uint64_t ca = dct + ((buf * L::kCBytes) >> 4), pa = dp + (((i % L::kPBufs) * L::kPBytes) >> 4);
#pragma unroll
                for (int ks = 0; ks < kTrKeys / 16; ks++)
#pragma unroll
                    for (int mt = 0; mt < kLatent / 128; mt++)
                        tc::mma_bf16(tmem + mt * NP, ca + ((ks * 2048 + mt * 2 * 8192) >> 4), pa + ((ks * 2 * kLboP) >> 4),
                                     id_o, (i > 0 || ks > 0) ? 1u : 0u);
                tc::mma_commit(bar(kTbDone + buf));
            }
            __syncwarp();
        };
        for (int i = 0; i < n_tiles; i++) {
            const int buf = i & 1;
            // whichever comes first, P(i - 1) or C(i): with two tiles in flight C(i) often waits for Done(i - 2)
            bool early = false;
            for (uint32_t k = 0; i > 0 && ok && k < kWaitLimit; k++) {
                early = __all_sync(0xffffffffu, tc::mbar_test(bar(kTbP + (buf ^ 1)), ((i - 1) >> 1) & 1));
                if (early || __all_sync(0xffffffffu, tc::mbar_test(bar(kTbFull + buf), (i >> 1) & 1))) break;
            }
            if (early) accumulate(i - 1);
            wait(kTbFull + buf, i >> 1);
            ok = __all_sync(0xffffffffu, ok);
            tc::fence_after_sync();
            // (S(i - 2), which this one is written over, has been read: O of it was issued above, after P(i - 2))
            if (tc::elect_one()) {   // S^T = C(i) . Q^T: M = 64 keys, K = 512
                const uint64_t ca = dc + ((buf * L::kCBytes) >> 4);
#pragma unroll
                for (int ks = 0; ks < kLatent / 16; ks++)
                    tc::mma_bf16(tmem + kSCol + buf * NQ, ca + (((ks >> 2) * 8192 + (ks & 3) * 32) >> 4),
                                 dq + ((ks * 256) >> 4), id_s,
                                 ks > 0 ? 1u : 0u);
                tc::mma_commit(bar(kTbS + buf));
            }
            __syncwarp();
            if (i > 0 && !early) accumulate(i - 1);
        }
        accumulate(n_tiles - 1);
        if (tc::elect_one()) tc::mma_commit(bar(kTbEnd));
        __syncwarp();
    } else {
        // ---------------- softmax ----------------
        const int quad = warp & 3, hh = warp >> 2, c0 = hh * V;
        const uint32_t lanes = static_cast<uint32_t>(quad * 32) << 16;
        const int j = quad * 16 + (lane & 15);                    // this thread's key of a tile (M = 64: lanes 0-15)
        float l[V];
#pragma unroll
        for (int e = 0; e < V; e++) l[e] = 0.0f;
        const float4 *f4 = reinterpret_cast<const float4 *>(fac + c0), *log4 = reinterpret_cast<const float4 *>(log_sigma + c0);
        const float4 *inv4 = reinterpret_cast<const float4 *>(inv + c0);
        for (int i = 0; i < n_tiles; i++) {
            const int buf = i & 1, t = t0 + i;
            wait(kTbFull + buf, i >> 1);                          // (the tile's scales and valid rows)
            const bool key = lane < 16 && val[buf * kTrKeys + j] != 0;
            const float sc = key ? scl[buf * kTrKeys + j] : 0.0f;
            // What a row's score may be beyond kTop: its p, and p scale / sigma, at most 2^kTop (a row without a reference:
            // none). And scale / sigma: a scale far above sigma, or a NaN, has a weight of 0, or the score is NaN; the
            // product of the weight with it must be 0 too. With 16 query rows while S is being made; with 32 the
            // registers for it spill (92.5 us for 89.3 over 262,144 int8 rows).
            float most[V], over[V];
            const float mag = fabsf(sc), lg = mag > 0.0f ? __log2f(mag) : -150.0f;
            const uint32_t sign = sc < 0.0f ? 0x80008000u : 0u;   // (unwritten drafts, that nobody sees, may have any)
            auto load_most = [&]() {
#pragma unroll
                for (int e = 0; e < V; e += 4) {
                    const float4 f = log4[e >> 2];
                    most[e] = fminf(0.0f, f.x - lg);
                    most[e + 1] = fminf(0.0f, f.y - lg);
                    most[e + 2] = fminf(0.0f, f.z - lg);
                    most[e + 3] = fminf(0.0f, f.w - lg);
                }
            };
            auto load_over = [&](int e0, int n) {
#pragma unroll
                for (int e = 0; e < V; e += 4) {
                    if (e < e0 || e >= e0 + n) continue;
                    const float4 f = inv4[e >> 2];
                    over[e] = fminf(mag * f.x, kFltMax);
                    over[e + 1] = fminf(mag * f.y, kFltMax);
                    over[e + 2] = fminf(mag * f.z, kFltMax);
                    over[e + 3] = fminf(mag * f.w, kFltMax);
                }
            };
            constexpr bool kEarly = V <= 8;
            if constexpr (kEarly) {
                load_most();
                load_over(0, V);
            }
            wait(kTbS + buf, i >> 1);
            ok = __all_sync(0xffffffffu, ok);
            tc::fence_after_sync();
            // the scores of this thread's key less the references
            float x[V];
            {
                uint32_t r[V];
                tr_tmem_ld<V>(tmem + lanes + kSCol + buf * NQ + c0, r);
                tc::tmem_wait_ld();
                tc::fence_before_sync();
#pragma unroll
                for (int e = 0; e < V; e += 2) {
                    const float4 f = f4[e >> 1];
                    x[e] = fmaf(__uint_as_float(r[e]) * f.x, sc, -f.y);
                    x[e + 1] = fmaf(__uint_as_float(r[e + 1]) * f.z, sc, -f.w);
                }
            }
            const int draft = t * kTrKeys + j - plen;             // which of the drafts the key is, if any
            const bool drafts = (t + 1) * kTrKeys > plen;
            if (!key || drafts) {
#pragma unroll
                for (int e = 0; e < V; e++)   // what each node sees of the drafts
                    if (!key || (draft >= 0 && !((mask[c0 + e] >> (draft & 63)) & 1ull))) x[e] = -INFINITY;
            }
            if constexpr (!kEarly) load_most();
            float past = -INFINITY;                               // (the maximum passes over what is NaN)
#pragma unroll
            for (int e = 0; e < V; e += 2) past = max3(past, x[e] - most[e], x[e + 1] - most[e + 1]);
            if (named_or(1, 256, past > kTop)) {
                // move the references and sigmas that have to, and rescale what they scale
                const int at = quad * NQ + c0 + ((lane >> kShift) & (V - 1));
                const Largest most_here = largest_of<V>(x, mag > 0.0f ? lg : -INFINITY);
                if ((lane & kLow) == 0) {
                    red[at] = most_here.x;
                    red[4 * NQ + at] = most_here.y;
                }
                named_sync(1, 256);
                float fo = 1.0f;
                if (tid < NQ) {
                    const float *rx = red + tid, *ry = red + 4 * NQ + tid;
                    const Largest t = larger(larger({rx[0], ry[0]}, {rx[NQ], ry[NQ]}), larger({rx[2 * NQ], ry[2 * NQ]}, {rx[3 * NQ], ry[3 * NQ]}));
                    Scaling s{fac[tid].y, log_sigma[tid], log_sigma[tid] == -INFINITY};
                    float fl;
                    red[tid] = move_scaling(s, t, fl, fo);
                    fac[tid].y = s.ref;
                    log_sigma[tid] = s.log_sigma;
                    if (!s.none) inv[tid] = pow2f_exact(-static_cast<int>(s.log_sigma));
                    alpha[tid] = fo;
                    red[4 * NQ + tid] = fl;
                }
                const bool rescale = named_or(1, 256, fo != 1.0f);
#pragma unroll
                for (int e = 0; e < V; e++) {
                    l[e] *= red[4 * NQ + c0 + e];
                    x[e] -= red[c0 + e];
                }
                if constexpr (kEarly) load_over(0, V);
                if (rescale && i > 0) {
                    wait(kTbDone + ((i - 1) & 1), (i - 1) >> 1);
                    ok = __all_sync(0xffffffffu, ok);
                    tc::fence_after_sync();
                    constexpr int CH = 16;
#pragma unroll 1
                    for (int mt = hh; mt < kLatent / 128; mt += 2) {
#pragma unroll 1
                        for (int cb = 0; cb < NP; cb += CH) {
                            uint32_t o[CH];
                            tr_tmem_ld<CH>(tmem + lanes + mt * NP + cb, o);
                            tc::tmem_wait_ld();
#pragma unroll
                            for (int e = 0; e < CH; e++) o[e] = __float_as_uint(__uint_as_float(o[e]) * alpha[cb % NQ + e]);
                            tc::tmem_st16(tmem + lanes + mt * NP + cb, o);
                        }
                    }
                    tc::tmem_wait_st();
                    tc::fence_before_sync();
                }
            }
            if (i >= L::kPBufs)                                   // P(i - kPBufs) has been read
                wait(kTbDone + ((i - L::kPBufs) & 1), (i - L::kPBufs) >> 1);
            unsigned char *line = smem + L::kP + (i % L::kPBufs) * L::kPBytes + (j >> 3) * kLboP + (c0 >> 3) * 128 + (j & 7) * 16;
#pragma unroll
            for (int g = 0; g < V / 8; g++) {
                uint32_t p4[4], r4[4];                            // P' as fp16, and what that leaves of it
                if constexpr (!kEarly) load_over(8 * g, 8);
#pragma unroll
                for (int e = 0; e < 8; e += 2) {
                    const float p0 = exp2_approx(x[8 * g + e]), p1 = exp2_approx(x[8 * g + e + 1]);
                    l[8 * g + e] += p0;
                    l[8 * g + e + 1] += p1;
                    const float w0 = p0 * over[8 * g + e], w1 = p1 * over[8 * g + e + 1];
                    const uint32_t h = f16x2_rn(w0, w1);
                    p4[e >> 1] = h ^ sign;
                    if constexpr (L::kTerms == 2) r4[e >> 1] = f16x2_rn(w0 - f16_lo_f(h), w1 - f16_hi_f(h)) ^ sign;
                }
                if (lane < 16) {
                    *reinterpret_cast<uint4 *>(line + g * 128) = make_uint4(p4[0], p4[1], p4[2], p4[3]);
                    if constexpr (L::kTerms == 2)
                        *reinterpret_cast<uint4 *>(line + 16 * NQ + g * 128) = make_uint4(r4[0], r4[1], r4[2], r4[3]);
                }
            }
            tc::fence_proxy_async();
            __syncwarp();
            if (lane == 0) tc::mbar_arrive(bar(kTbP + buf));
        }
        // the sums of the query rows, and what their accumulators are multiplied by
        named_sync(1, 256);                                       // (the arrays are free)
        const float bl = butterfly<V, false>(l);
        if ((lane & kLow) == 0) red[quad * NQ + c0 + ((lane >> kShift) & (V - 1))] = bl;
        named_sync(1, 256);
        if (tid < NQ) {
            const float sum = (red[tid] + red[NQ + tid]) + (red[2 * NQ + tid] + red[3 * NQ + tid]);
            const bool none = tid >= live || sum == 0.0f;         // (a node past the tree's, or no visible key)
            // (scores that are all NaN set no reference: theirs is 0)
            const float ref = fac[tid].y, sigma = 1.0f / inv[tid];
            alpha[tid] = none ? -1.0f : (direct ? sigma / sum : sigma * kUnhead);   // (-1: not a factor)
            if (orow[tid] >= 0) {
                if (!direct) {
                    part_ml[2 * orow[tid]] = none ? -INFINITY : ref + kHead;
                    part_ml[2 * orow[tid] + 1] = none ? 0.0f : sum * kUnhead;
                } else if (a.lse) {
                    a.lse[orow[tid]] = none ? -INFINITY : ref * 0.6931471805599453f + logf(sum);
                }
            }
        }
    }
    // Every product is done. (A barrier of its own, used once: that of a tile says nothing to a thread that
    // gave up, whose products may be several phases behind.)
    if (!tc::mbar_wait(bar(kTbEnd), 0, kWaitLimit)) ok = false;
    const bool all_ok = __syncthreads_and(ok);
    if (!all_ok && tid == 0) atomicOr(a.status, 32);
    tc::fence_after_sync();
    if (warp < 16) {
        // O^T: tile mt of 128 latent dims, lane quadrant warp % 4 (dim 128 mt + 32 quad + lane); rows of the
        // output or partials in shared memory, over the C tiles, then one copy a row: stored from the
        // registers, 4 bytes a lane, 64 rows took 6,300 cycles
        constexpr int CH = 16;
        const int mt = warp >> 2, dim = mt * 128 + (warp & 3) * 32 + lane;
        const uint32_t ta = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16) + mt * NP;
#pragma unroll 1
        for (int cb = 0; cb < NQ; cb += CH) {
            float f[CH];                                      // (read before the first write: the compiler keeps the order)
#pragma unroll
            for (int e = 0; e < CH; e += 4) *reinterpret_cast<float4 *>(f + e) = *reinterpret_cast<const float4 *>(alpha + cb + e);
            uint32_t o[CH];
            tr_tmem_ld<CH>(ta + cb, o);
            if constexpr (L::kTerms == 2) {
                uint32_t more[CH];
                tr_tmem_ld<CH>(ta + NQ + cb, more);
                tc::tmem_wait_ld();
#pragma unroll
                for (int e = 0; e < CH; e++) o[e] = __float_as_uint(__uint_as_float(o[e]) + __uint_as_float(more[e]));
            } else {
                tc::tmem_wait_ld();
            }
#pragma unroll
            for (int e = 0; e < CH; e++) {
                float v = f[e] == -1.0f ? 0.0f : __uint_as_float(o[e]) * f[e];
                if (!all_ok) v = __int_as_float(0x7fc00000);
                if (direct) reinterpret_cast<uint16_t *>(smem + L::kC)[(cb + e) * kLatent + dim] = __bfloat16_as_ushort(__float2bfloat16_rn(v));
                else reinterpret_cast<float *>(smem + L::kC)[(cb + e) * kLatent + dim] = v;
            }
        }
        if (!all_ok && direct && a.lse && tid < NQ && orow[tid] >= 0) a.lse[orow[tid]] = __int_as_float(0x7fc00000);
    }
    tc::fence_proxy_async();
    __syncthreads();
    if (lane == 0) {   // (a copy takes about 75 cycles to issue: every warp a few)
        for (int r = warp; r < NQ; r += kThreads / 32) {
            if (orow[r] < 0 || (!direct && alpha[r] == -1.0f)) continue;
            if (direct) bulk_store(a.out + orow[r] * kLatent, smem + L::kC + r * kLatent * 2, kLatent * 2);
            else bulk_store(part_acc + orow[r] * kLatent, smem + L::kC + r * kLatent * 4, kLatent * 4);
        }
        bulk_wait();
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
    const int smem = TrLayout<NQ>::kAlloc;
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    e = launch_pdl(kernel, dim3(p.q_tiles, p.parts, a.batch), dim3(TrLayout<NQ>::kThreads), smem, stream, a, p, part_acc, part_ml);
    return e != cudaSuccess ? e : cudaGetLastError();
}

constexpr int kTrMaxParts = 1024;              // partials of one query that the combine kernel merges
constexpr int kTrLevels = 4;                   // waves of runs to balance lists of different lengths

// Waves of runs that a batch of long lists may be cut into: so many that its (sequence, tile of query rows) pairs have three
// runs each or more, where one wave has two or three for some of them and none to balance with (8 sequences of 16
// nodes of 64 heads, 64 tiles of query rows for 74 pairs of SMs, lists of 4,000 to 32,768 rows: 654 us with one wave, 469
// with two, 487 with three, 514 with four; of 32,768 to 262,144: 5,050, 3,016, 2,912, 2,890). Where one wave
// has enough, more only write and merge more partials (8 sequences of 4 nodes, up to 60,000 rows: 220 us with one,
// 242, 268 and 305; 16 single tokens of 16 heads, 1,000 to 65,536 4-bit rows: 153, 183, 213, 247).
int tree_levels(long long base, int units) {
    const long long n = (3 * base + units - 1) / std::max(units, 1);
    return static_cast<int>(std::min(std::max(n, 1ll), static_cast<long long>(kTrLevels)));
}
long long tree_tiles(long long width, int keys) { return (width + keys - 1) / keys + 1; }

}  // namespace

TreePlan tree_plan(int batch, int n_nodes, int n_heads, int width, int num_sms) {
    TreePlan p{};
    const int rows = n_nodes * n_heads;
    // Few tiles: 16 query rows a CTA while each tile can have an SM of its own (64 rows over 67 keys:
    // 22.5 us a call as one CTA a tile, 12.7 as four).
    const bool small = static_cast<long long>(batch) * ((rows + 15) / 16) * tree_tiles(width, kTrKeys) <= num_sms;
    const bool pair = rows > 64 && !small;
    p.nq = rows <= 16 || small ? 16 : (rows <= 32 ? 32 : (pair ? 128 : 64));
    p.q_tiles = (rows + p.nq - 1) / p.nq;
    p.units = pair ? num_sms / 2 : num_sms;
    const long long tiles = tree_tiles(width, pair ? kTreePairKeys : kTrKeys), base = static_cast<long long>(batch) * p.q_tiles;
    // One wave of runs when the lists are short, up to 32 tiles an SM, or there is one (4 sequences of 13 nodes, up to 4,096
    // rows, 17 tiles a pair: 48.3 us a call, 75.5 with two waves); else the kernel weighs up to so many
    // against the lists' lengths.
    p.levels = batch > 1 && base * tiles > 32ll * p.units ? tree_levels(base, p.units) : 1;
    long long parts = base >= static_cast<long long>(p.levels) * p.units ? 1 : p.levels * static_cast<long long>(p.units) / base;
    // twice as many, for a list longer than the mean (those sequences: 48.3 us a call, 73 without, 70 with four times;
    // 16 of up to 100,000 rows, 64 query rows: 359, 588 and 376)
    if (batch > 1 && parts > 1) parts *= 2;
    if (parts > tiles) parts = tiles;
    if (parts > kTrMaxParts) parts = kTrMaxParts;
    // A few tiles (of this bound, one more than the list has) are one run, without a merge: 64 query rows over
    // 67 keys 9.8 us a call, 11.9 cut; 512 rows over 367 keys, five tiles, 18.2 and 16.7.
    if (tiles <= 3) parts = 1;
    p.parts = static_cast<int>(parts < 1 ? 1 : parts);
    return p;
}

size_t tree_partials(int batch, int n_nodes, int n_heads, int width, int num_sms) {
    // A plan of more than one part has at most as many runs as waves of its units, of nq query rows each (128 a pair
    // of SMs is 64 an SM), and at most one for each tile. Every factor grows with the shape, or stays.
    const long long rows = static_cast<long long>(n_nodes) * n_heads, all = tree_tiles(width, kTrKeys);
    const long long tiles = all > kTrMaxParts ? kTrMaxParts : all;
    const int nq = rows <= 16 ? 16 : (rows <= 32 ? 32 : 64);
    const long long base = batch * ((rows + 127) / 128);
    int waves = batch > 1 ? 2 : 1;
    if (batch > 1 && base * all > 32ll * (num_sms / 2)) waves *= tree_levels(base, num_sms / 2);
    const long long cap = static_cast<long long>(waves) * num_sms * nq;
    return static_cast<size_t>(batch * rows * tiles < cap ? batch * rows * tiles : cap);
}

cudaError_t launch_tree_mla(const TreePlan &p, const TreeArgs &a, int format, float *part_acc, float *part_ml,
                            cudaStream_t stream) {
    if (p.nq == 128) return launch_tree_pair(p, a, format, part_acc, part_ml, stream);
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
