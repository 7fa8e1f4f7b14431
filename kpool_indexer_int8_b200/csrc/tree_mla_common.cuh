// tree_mla_common.cuh -- pieces shared by the two tree attention kernels.
#pragma once

#include "common.cuh"
#include "row_codes.cuh"
#include "tc.cuh"
#include "tree_mla.cuh"

namespace glm {
namespace tree {

constexpr uint32_t kWaitLimit = 1u << 22;
constexpr float kGrow = 8.0f;                  // a score passes its reference by at most 2^8
constexpr float kBoost = 8.0f;                 // P' <= 2^8 * 16 * 8 = 2^15 < 65504

// The keys of a sequence in tiles: the index list's, then one tile of drafted rows.
__device__ __forceinline__ int list_len(const TreeArgs &a, int b) {
    return a.row_len ? min(max(a.row_len[b], 0), a.width) : a.width;
}
__device__ __forceinline__ int tree_len(const TreeArgs &a, int b) {
    return a.n_tree ? min(max(a.n_tree[b], 0), a.n_nodes) : a.n_nodes;
}
__device__ __forceinline__ int tile_count(const TreeArgs &a, int b, int keys) {
    return (list_len(a, b) + keys - 1) / keys + (tree_len(a, b) > 0 ? 1 : 0);
}
// The tiles of a part: every sequence is cut into runs of as many, the length for which the busiest
// of `units` SMs (or pairs) is done first, a run costing about six tiles more than its own (set-up,
// output): up to `levels` waves of runs are tried, one when there is nothing to balance. Computed
// by every warp for itself from the device's list lengths.
__device__ __forceinline__ int run_tiles(const TreeArgs &a, const TreePlan &p, int keys) {
    const int lane = threadIdx.x & 31;
    auto reduce = [](int v) {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
        return v;
    };
    const int first = lane < a.batch ? tile_count(a, lane, keys) : 0;
    int sum = 0, most = 0;
    for (int s = lane; s < a.batch; s += 32) {
        const int n = s < 32 ? first : tile_count(a, s, keys);
        sum += n;
        most = max(most, n);
    }
    sum = reduce(sum);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) most = max(most, __shfl_xor_sync(0xffffffffu, most, o));
    const int low = max(1, (most + p.parts - 1) / p.parts);
    int best = max(low, 1), best_cost = 0x7fffffff;
    for (int k = 1; k <= p.levels; k++) {
        const int target = max(1, k * p.units / p.q_tiles);   // runs of one query tile over all sequences
        int run = max(low, (sum + target - 1) / target), n = 0;
        for (int it = 0; it < 8; it++) {
            n = 0;
            for (int s = lane; s < a.batch; s += 32) n += ((s < 32 ? first : tile_count(a, s, keys)) + run - 1) / run;
            n = reduce(n);
            if (n <= target || run >= most) break;
            run = max(run + 1, static_cast<int>(static_cast<int64_t>(run) * n / target));
        }
        const int cost = (n * p.q_tiles + p.units - 1) / p.units * (run + 6);
        if (cost < best_cost) {
            best_cost = cost;
            best = run;
        }
    }
    return best;
}

// 16-byte pieces of a cache row of one of the formats, widened to fp16 (exact): 16 int8 or E4M3
// codes are two lines of 8 dims, 32 E2M1 codes (with two block scales) four.
template <int kFmt>
struct Row {
    static constexpr bool kFp4 = kFmt == kFmtFp4;
    static constexpr int kBytes = kFp4 ? kFp4RowBytes : kRowBytes;
    static constexpr int kSclAt = kFp4 ? kFp4RowScaleAt : kLatent;
    static constexpr int kPieces = kFp4 ? 16 : 32;          // of a row
    static constexpr int kLines = kFp4 ? 4 : 2;             // lines of 8 dims of a piece

    __device__ __forceinline__ static const uint8_t *at(const uint8_t *base, int64_t r) { return base + r * kBytes; }
    __device__ __forceinline__ static float scale(const uint8_t *base, int64_t r) {
        return r >= 0 ? __ldg(reinterpret_cast<const float *>(at(base, r) + kSclAt)) : 0.0f;
    }
    __device__ __forceinline__ static uint4 codes(const uint8_t *base, int64_t r, int k) {
        return r >= 0 ? __ldg(reinterpret_cast<const uint4 *>(at(base, r)) + k) : make_uint4(0u, 0u, 0u, 0u);
    }
    __device__ __forceinline__ static uint32_t block_scales(const uint8_t *base, int64_t r, int k) {
        return r >= 0 ? __ldg(reinterpret_cast<const uint16_t *>(at(base, r) + kFp4ScalesAt) + k) : 0u;
    }
    // Line u of piece v (block scales es) as 8 fp16 values; clean: NaN codes become zeros.
    __device__ __forceinline__ static uint4 line(const uint4 &v, uint32_t es, int u, bool clean) {
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
        uint32_t o[4];
        if constexpr (kFp4) {
            const __half2_raw sc = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(es), __NV_E4M3);
            fp4_to_f16x8(w[u], static_cast<uint32_t>(u < 2 ? sc.x : sc.y) * 0x10001u, o);
        } else if constexpr (kFmt == kFmtFp8) {
            fp8_to_f16x4(w[2 * u], o[0], o[1]);
            fp8_to_f16x4(w[2 * u + 1], o[2], o[3]);
        } else {
            codes_to_f16x4(w[2 * u], o[0], o[1]);
            codes_to_f16x4(w[2 * u + 1], o[2], o[3]);
        }
        if constexpr (kFmt != kFmtInt8) {
            if (clean) {
#pragma unroll
                for (int i = 0; i < 4; i++) {
                    if ((o[i] & 0x7fffu) > 0x7c00u) o[i] &= 0xffff0000u;
                    if ((o[i] & 0x7fff0000u) > 0x7c000000u) o[i] &= 0x0000ffffu;
                }
            }
        }
        return make_uint4(o[0], o[1], o[2], o[3]);
    }
    // Whether a row holds a NaN code (E4M3 codes or block scales of 0x7f / 0xff), looked for by the
    // four lanes that share it (part 0 .. 3); int8 codes have none.
    __device__ __forceinline__ static bool has_nan(const uint8_t *base, int64_t r, int part) {
        if constexpr (kFmt == kFmtInt8) return false;
        if (r < 0) return false;
        bool nan = false;
        const uint32_t *w = reinterpret_cast<const uint32_t *>(at(base, r) + (kFp4 ? kFp4ScalesAt : 0));
        for (int i = part; i < (kFp4 ? 8 : 128); i += 4) {
            const uint32_t v = __ldg(w + i) & 0x7f7f7f7fu;
            nan |= ((v + 0x01010101u) & 0x80808080u) != 0u;
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
__device__ __forceinline__ float exp2_approx(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// The power of two that puts a bf16 magnitude (its bits) in [2^14, 2^15): bf16 values so scaled are
// exact in fp16 (those below 2^-17 of the range aside).
__device__ __forceinline__ int query_exponent(unsigned bits) {
    return bits == 0u ? 0 : min(120, max(-120, 14 - (static_cast<int>(bits >> 7) - 127)));
}
__device__ __forceinline__ float pow2f_exact(int e) { return __uint_as_float(static_cast<uint32_t>(e + 127) << 23); }
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
