// tree_mla_common.cuh -- pieces shared by the two tree attention kernels.
#pragma once

#include "common.cuh"
#include "row_codes.cuh"
#include "tc.cuh"
#include "tree_mla.cuh"

namespace glm {
namespace tree {

constexpr uint32_t kWaitLimit = 1u << 22;
// The softmax weights of a query row. It keeps a reference ref and log2 sigma, whole numbers in log2 units:
// p = 2^(s - ref) goes to the sum, P' = p scale / sigma as fp16 to the product with the codes. When they are set,
// from the keys that the row sees, the largest p and the largest P' are at most 2^kHead and above half of that;
// they move when a P' would pass fp16's range, so that rescales are rare and, by powers of two, exact. A
// row's sigma is its own, and follows what its keys weigh times their scale: a large scale in a key that
// the row does not see, or that weighs nothing, costs the others none of fp16's range.
// kHead: fp16 has no bits below 2^-24, so a weight is off by at most 2^-24 - kHead of the row's largest (each times its
// scale) beside its 2^-11; with 8, over 2^20 rows, that is 2^-12, an eighth of half a step of the bf16 output. Above
// it there is room for scores that grow by 2^7.9. 8 nodes over 262,144 rows, us a call: 364 with 2, 371 with
// 8 (338 and 341 one at a time: rescales cost next to nothing, bits that are not 0 take power); 373 and, with 10, 384
// on another chip.
constexpr float kHead = 8.0f, kUnhead = 0x1p-8f;   // (2^-kHead)
constexpr float kTop = 15.9f;                  // log2 of the largest P' (fp16: 65,504)
constexpr float kFltMax = 3.402823466e38f;

// The keys of a sequence: those of the index list, then the drafted rows, in tiles. The lengths as they are
// in memory are asked for first of all in a kernel and used as late as can be.
struct Lengths {
    int list, tree;
};
__device__ __forceinline__ Lengths load_lengths(const TreeArgs &a, int b, bool there) {
    return {there && a.row_len ? a.row_len[b] : a.width, there && a.n_tree ? a.n_tree[b] : a.n_nodes};
}
__device__ __forceinline__ int list_len(const TreeArgs &a, Lengths n) { return min(max(n.list, 0), a.width); }
__device__ __forceinline__ int tree_len(const TreeArgs &a, Lengths n) { return min(max(n.tree, 0), a.n_nodes); }
__device__ __forceinline__ int tile_count(const TreeArgs &a, Lengths n, int keys) {
    return (list_len(a, n) + tree_len(a, n) + keys - 1) / keys;
}
// A key's row: a cache row, or one of `draft` as -2 - its index there; -1: none.
__device__ __forceinline__ int draft_row(int index) { return -2 - index; }
// The tiles of a part: every sequence is cut into runs of as many, the length for which the busiest
// of `units` SMs (or pairs) is done first, a run costing about six tiles more than its own (set-up,
// output; 8 sequences of 8 nodes, up to 32,768 rows: 259 us with 6 or 2, 286 with 12; 16 nodes, up to 262,144: 2,900 with
// 6, 2,913 with 2, 2,947 with 12): up to `levels` waves of runs are tried, one when there is nothing to balance. A run counts once
// for each tile of query rows that the sequence's tree fills (4 trees of 8 to 13 nodes: 53.6 us a call, 54.3
// with all counted as full). Computed by every warp for itself from the device's lengths (mine: those
// of sequence `lane`).
__device__ __forceinline__ int run_tiles(const TreeArgs &a, const TreePlan &p, int keys, Lengths mine) {
    const int lane = threadIdx.x & 31;
    auto reduce = [](int v) {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
        return v;
    };
    auto weight = [&](Lengths n) { return (tree_len(a, n) * a.n_heads + p.nq - 1) / p.nq; };
    const int first = lane < a.batch ? tile_count(a, mine, keys) : 0, first_w = lane < a.batch ? weight(mine) : 0;
    // f(tiles, weight) over all sequences, this lane's share
    auto each = [&](auto f) {
        if (lane < a.batch) f(first, first_w);
        for (int s = lane + 32; s < a.batch; s += 32) {
            const Lengths n = load_lengths(a, s, true);
            f(tile_count(a, n, keys), weight(n));
        }
    };
    int sum = 0, most = 0;
    each([&](int tiles, int w) {
        sum += tiles * w;
        most = max(most, tiles);
    });
    sum = reduce(sum);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) most = max(most, __shfl_xor_sync(0xffffffffu, most, o));
    const int low = max(1, (most + p.parts - 1) / p.parts);
    int best = low, best_cost = 0x7fffffff;
    for (int k = 1; k <= p.levels; k++) {
        const int target = k * p.units;
        int run = max(low, (sum + target - 1) / target), n = 0;
        for (int it = 0; it < 8; it++) {
            n = 0;
            each([&](int tiles, int w) { n += (tiles + run - 1) / run * w; });
            n = reduce(n);
            if (n <= target || run >= most) break;
            run = max(run + 1, static_cast<int>(static_cast<int64_t>(run) * n / target));
        }
        const int cost = (n + p.units - 1) / p.units * (run + 6);
        if (cost < best_cost) {
            best_cost = cost;
            best = run;
        }
    }
    return best;
}

// Starts copying 16 bytes to shared memory, or zeroes them there (`there` false: nothing is read).
__device__ __forceinline__ void copy16(void *to_smem, const void *from, bool there) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(tc::smem_addr(to_smem)), "l"(from), "r"(there ? 16 : 0)
                 : "memory");
}
// Copies `bytes` (a multiple of 16) of shared memory, written through the generic proxy before a proxy
// fence and a barrier, to global memory; both 16-byte aligned. bulk_wait: the thread's
// copies have read the shared memory (their writes are done when the kernel is).
__device__ __forceinline__ void bulk_store(void *to, const void *from_smem, int bytes) {
    asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(to), "r"(tc::smem_addr(from_smem)), "r"(bytes)
                 : "memory");
}
__device__ __forceinline__ void bulk_wait() {
    asm volatile("cp.async.bulk.commit_group;\n\tcp.async.bulk.wait_group.read 0;" ::: "memory");
}
// Asks for a line of 128 bytes ahead of its use.
__device__ __forceinline__ void prefetch_line(const void *p) { asm volatile("prefetch.global.L2 [%0];" ::"l"(p)); }
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
// Waits until at most kNewer of the groups committed last are still in flight; for the whole warp.
template <int kNewer>
__device__ __forceinline__ void copy_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(kNewer) : "memory");
    __syncwarp();
}
// 0x80 in each byte that is an E4M3 NaN (0x7f, 0xff).
__device__ __forceinline__ uint32_t nan_bytes(uint32_t w) { return ((w & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u; }
// Cache rows of one of the formats, as a widening warp takes them. A row is copied whole into shared
// memory by one asynchronous 16-byte copy per lane (eight warps gather rows at 21 to 27 bytes a cycle
// and SM this way, 21 to 24 by bulk copies, whose issue takes 90 cycles a row, 19 to 24 by loads into
// registers); then each lane widens lines of 8 dims of it to fp16 (exact): 8 bytes of int8 or E4M3
// codes, 4 bytes of E2M1 codes with the block scale of their 16 dims.
template <int kFmt>
struct Row {
    static constexpr bool kFp4 = kFmt == kFmtFp4;
    static constexpr int kBytes = kFp4 ? kFp4RowBytes : kRowBytes;
    static constexpr int kCodes = kFp4 ? 256 : 512;         // bytes of codes, then the tail with the scales
    static constexpr int kTail = kBytes - kCodes;
    static constexpr int kSclAt = (kFp4 ? kFp4RowScaleAt : kLatent) - kCodes;   // the row scale in the tail

    __device__ __forceinline__ static const uint8_t *at(const TreeArgs &a, int row) {
        return (row >= 0 ? a.cache : a.draft) + static_cast<int64_t>(row >= 0 ? row : max(-2 - row, 0)) * kBytes;
    }
    // One warp starts copying the NR rows that lanes lane0 .. lane0 + NR - 1 hold (-1: zeros) to codes
    // [NR][kCodes] and tails [NR][kTail] in shared memory; mixed: some may be drafts (a tile in a list, and a
    // rolled loop: looking for them in every tile cost 3 % of a long call). No branch on a row, so that the
    // copies go out back to back.
    template <int NR>
    __device__ __forceinline__ static void fetch(unsigned char *codes, unsigned char *tails, const TreeArgs &a, int rows,
                                                 int lane0, bool mixed) {
        constexpr int kPer = 512 / kCodes, kTp = kTail / 16;      // rows of a copy, pieces of a tail
        static_assert(NR % kPer == 0 && NR <= 32, "rows of a group");
        const int lane = threadIdx.x & 31, piece = (lane * 16) % kCodes;
        auto code = [&](int i, auto from) {
            const int r = __shfl_sync(0xffffffffu, rows, lane0 + i * kPer + lane * 16 / kCodes);
            copy16(codes + i * 512 + lane * 16, from(r) + piece, r != -1);
        };
        auto tail = [&](int i, auto from) {
            const int p = i + lane, r = __shfl_sync(0xffffffffu, rows, lane0 + min(p / kTp, NR - 1));
            if (p < NR * kTp) copy16(tails + p * 16, from(r) + kCodes + p % kTp * 16, r != -1);
        };
        if (mixed) {
            auto from = [&](int r) { return at(a, r); };
#pragma unroll 1
            for (int i = 0; i < NR / kPer; i++) code(i, from);
#pragma unroll 1
            for (int i = 0; i < NR * kTp; i += 32) tail(i, from);
        } else {
            auto from = [&](int r) { return a.cache + static_cast<int64_t>(max(r, 0)) * kBytes; };
#pragma unroll
            for (int i = 0; i < NR / kPer; i++) code(i, from);
#pragma unroll
            for (int i = 0; i < NR * kTp; i += 32) tail(i, from);
        }
    }
    // The same for the codes of dims 128 part + [0, 128) of each 256 (half a row: 256 or 128 bytes of
    // codes, both parts of a row behind each other), and the whole tails of 4-bit rows.
    template <int NR>
    __device__ __forceinline__ static void fetch_half(unsigned char *codes, unsigned char *tails, const TreeArgs &a, int rows,
                                                      int part, bool mixed) {
        constexpr int kHalf = kCodes / 2, kPer = 512 / kHalf, kSeg = kHalf / 2;
        static_assert(NR % kPer == 0 && NR <= 32, "rows of a group");
        const int lane = threadIdx.x & 31, in = (lane * 16) % kHalf;
        const int piece = (in / kSeg) * kHalf + part * kSeg + in % kSeg;
        auto code = [&](int i, auto from) {
            const int r = __shfl_sync(0xffffffffu, rows, i * kPer + lane * 16 / kHalf);
            copy16(codes + i * 512 + lane * 16, from(r) + piece, r != -1);
        };
        auto tail = [&](int i, auto from) {
            const int p = i + lane, r = __shfl_sync(0xffffffffu, rows, min(p / 3, NR - 1));
            if (p < NR * 3) copy16(tails + p * 16, from(r) + kCodes + p % 3 * 16, r != -1);
        };
        constexpr int kTails = kFp4 ? NR * 3 : 0;
        if (mixed) {
            auto from = [&](int r) { return at(a, r); };
#pragma unroll 1
            for (int i = 0; i < NR / kPer; i++) code(i, from);
#pragma unroll 1
            for (int i = 0; i < kTails; i += 32) tail(i, from);
        } else {
            auto from = [&](int r) { return a.cache + static_cast<int64_t>(max(r, 0)) * kBytes; };
#pragma unroll
            for (int i = 0; i < NR / kPer; i++) code(i, from);
#pragma unroll
            for (int i = 0; i < kTails; i += 32) tail(i, from);
        }
    }
    __device__ __forceinline__ static float scale(const unsigned char *tail) { return *reinterpret_cast<const float *>(tail + kSclAt); }

    // Line `l` of codes as it lies there (block: which 16 dims of the row it belongs to), and as 8 fp16
    // values.
    struct Line {
        uint2 codes;
        uint32_t es;
    };
    __device__ __forceinline__ static Line line(const unsigned char *codes, const unsigned char *tail, int l, int block) {
        Line v;
        if constexpr (kFp4) {
            v.codes = make_uint2(reinterpret_cast<const uint32_t *>(codes)[l], 0u);
            v.es = tail[block];
        } else {
            v.codes = reinterpret_cast<const uint2 *>(codes)[l];
            v.es = 0u;
        }
        return v;
    }
    __device__ __forceinline__ static uint4 widen(const Line &v) {
        uint32_t o[4];
        if constexpr (kFp4) {
            const __half_raw sc = __nv_cvt_fp8_to_halfraw(static_cast<__nv_fp8_storage_t>(v.es), __NV_E4M3);
            fp4_to_f16x8(v.codes.x, static_cast<uint32_t>(sc.x) * 0x10001u, o);
        } else if constexpr (kFmt == kFmtFp8) {
            fp8_to_f16x4(v.codes.x, o[0], o[1]);
            fp8_to_f16x4(v.codes.y, o[2], o[3]);
        } else {
            codes_to_f16x4(v.codes.x, o[0], o[1]);
            codes_to_f16x4(v.codes.y, o[2], o[3]);
        }
        return make_uint4(o[0], o[1], o[2], o[3]);
    }
    // One warp makes zeros of the NaN codes of n bytes (a multiple of 16) of rows in shared memory: of E4M3
    // codes, or of 4-bit rows' tails, [rows][kTail], whose first 32 bytes are block scales.
    __device__ __forceinline__ static void clean(unsigned char *bytes, int n) {
        const int lane = threadIdx.x & 31;
        __syncwarp();
#pragma unroll 1
        for (int i = lane * 4; i < n; i += 128) {
            if (kFp4 && i % kTail >= 32) continue;
            uint32_t *w = reinterpret_cast<uint32_t *>(bytes + i);
            const uint32_t m = nan_bytes(*w);
            if (m) *w &= ~((m >> 7) * 0xffu);
        }
        __syncwarp();
    }
    // Whether this lane's share of a row holds a NaN code (E4M3 codes or block scales of 0x7f / 0xff).
    // Int8 codes have none.
    __device__ __forceinline__ static bool nan_share(const unsigned char *codes, const unsigned char *tail) {
        if constexpr (kFmt == kFmtInt8) return false;
        const int lane = threadIdx.x & 31;
        auto bad = [](uint32_t x) { return nan_bytes(x) != 0u; };
        bool nan;
        if constexpr (kFp4) {
            nan = lane < 8 && bad(reinterpret_cast<const uint32_t *>(tail)[lane]);
        } else {
            const uint4 v = reinterpret_cast<const uint4 *>(codes)[lane];
            nan = bad(v.x) || bad(v.y) || bad(v.z) || bad(v.w);
        }
        return nan;
    }
    __device__ __forceinline__ static bool has_nan(const unsigned char *codes, const unsigned char *tail) {
        return __any_sync(0xffffffffu, nan_share(codes, tail));
    }
};
// Where line c (of 8) of row r goes in a block of 64 dims, rows of 128 bytes in the 128-byte swizzle:
// eight lanes that write the lines of a row write eight different banks.
__device__ __forceinline__ int swizzled(int r, int c) { return r * 128 + ((c ^ (r & 7)) << 4); }

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
__device__ __forceinline__ float exp2_approx(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// Two fp32 values in one 64-bit register, and the packed operations on them.
__device__ __forceinline__ uint64_t pack2(float a, float b) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ uint64_t pack2(uint32_t a, uint32_t b) { return pack2(__uint_as_float(a), __uint_as_float(b)); }
__device__ __forceinline__ void unpack2(uint64_t v, float &a, float &b) { asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v)); }
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}
// The largest finite value >= 0 of a warp (row scales; 0 if there is none).
__device__ __forceinline__ float finite_max(float v) {
    return __uint_as_float(__reduce_max_sync(0xffffffffu, v > 0.0f && v < INFINITY ? __float_as_uint(v) : 0u));
}
// The power of two that puts a bf16 magnitude (its bits) in [2^14, 2^15): bf16 values so scaled are
// exact in fp16 (those below 2^-17 of the range aside).
__device__ __forceinline__ int query_exponent(unsigned bits) {
    return bits == 0u ? 0 : min(120, max(-120, 14 - (static_cast<int>(bits >> 7) - 127)));
}
__device__ __forceinline__ float pow2f_exact(int e) { return __uint_as_float(static_cast<uint32_t>(e + 127) << 23); }
// 2^d of a whole number d <= 127; 0 below -126.
__device__ __forceinline__ float pow2_whole(float d) { return d < -126.0f ? 0.0f : pow2f_exact(static_cast<int>(d)); }
// A query row's reference and log2 sigma, [-126, 126].
struct Scaling {
    float ref, log_sigma;
    bool none;                                 // it has seen no key
};
// What a tile's keys are to a query row: the largest score x, and y, the largest score plus log2 scale less x
// (a sum of both would lose the logarithm beside a score past 2^20). A key: its score and log2 scale; -infinity, or
// a score that is NaN: none that the row sees (y is then anything, NaN too, and passed over).
struct Largest {
    float x, y;
};
__device__ __forceinline__ Largest larger(Largest a, Largest b) {
    const float x = fmaxf(a.x, b.x);
    return {x, fmaxf(a.y + (a.x - x), b.y + (b.x - x))};
}
// The scaling moves for them. Returns by how much the reference does, and what the sum so far and the output have
// to be multiplied by.
__device__ __forceinline__ float move_scaling(Scaling &s, Largest t, float &l_factor, float &o_factor) {
    l_factor = o_factor = 1.0f;
    if (!(t.x > -INFINITY)) return 0.0f;
    const float delta = s.none || t.x > kHead ? ceilf(t.x - kHead) : 0.0f, y = t.y + (t.x - delta);
    float sigma = fminf(fmaxf(ceilf(y - kHead), -126.0f), 126.0f);
    if (!s.none) {
        sigma = delta == 0.0f && y - s.log_sigma <= kTop ? s.log_sigma : fmaxf(s.log_sigma - delta, sigma);
        l_factor = pow2_whole(-delta);
        o_factor = pow2_whole(s.log_sigma - sigma - delta);
    }
    s = {s.ref + delta, sigma, false};
    return delta;
}
// 8 bf16 values times f as 8 fp16 values.
__device__ __forceinline__ uint4 bf16_to_f16x8(const uint4 &v, float f) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    uint32_t o[4];
#pragma unroll
    for (int k = 0; k < 4; k++) o[k] = f16x2_rn(__uint_as_float(w[k] << 16) * f, __uint_as_float(w[k] & 0xffff0000u) * f);
    return make_uint4(o[0], o[1], o[2], o[3]);
}
__device__ __forceinline__ unsigned bf16_absmax(const uint4 &v) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    unsigned m = 0u;
#pragma unroll
    for (int e = 0; e < 4; e++) m = max(m, max(w[e] & 0x7fffu, (w[e] >> 16) & 0x7fffu));
    return m;
}

}  // namespace tree
}  // namespace glm
