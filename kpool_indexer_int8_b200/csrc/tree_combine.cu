// tree_combine.cu -- the merge of the tree attention's partial softmax states.
//
// A query row's partials hold, over the keys of their run, acc = sum 2^(..) v, the sum l of the weights and
// their reference m (log2 units, a whole number); with M = max m over the partials with l > 0 the row is
//     out = sum 2^(m - M) acc / sum 2^(m - M) l,    lse = M log 2 + log(sum 2^(m - M) l),
// all of it in fp32, in the same order every time. It is bound by the partials' 2 KB each, which the
// attention has just written and L2 holds, and for few rows by the number of loads in flight. With as many
// rows as SMs, a row is one CTA of 128 threads, a thread four dims, eight partials in flight (3,328 rows
// of 4 partials: 26 us less a call than four CTAs of four warps a row, 512 of 18: 1.5); with fewer, a row is
// four CTAs of 128 dims and eight warps, each an eighth of the partials (16 rows of 148: 23 us less
// than one CTA a row). A row that saw a NaN has l = NaN in a partial, and is NaN.
#include "common.cuh"
#include "tree_mla.cuh"

namespace glm {

namespace {

constexpr int kTcWarps = 8;                    // of a CTA when there are few rows

template <bool kFew>
__global__ void __launch_bounds__(kFew ? 32 * kTcWarps : 128) tree_combine_kernel(const float *__restrict__ part_acc,
                                                                                  const float *__restrict__ part_ml, int n_heads,
                                                                                  int parts, uint16_t *__restrict__ out,
                                                                                  float *__restrict__ lse) {
    pdl_begin(part_acc, part_ml);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t row = kFew ? blockIdx.x / 4 : blockIdx.x, node = row / n_heads;
    const int64_t first = node * parts * n_heads + (row - node * n_heads);   // partial p: first + p n_heads
    const int dim = kFew ? (blockIdx.x & 3) * 128 + 4 * lane : 4 * threadIdx.x;
    const float2 *ml = reinterpret_cast<const float2 *>(part_ml);
    const float *acc = part_acc + dim;
    float top = -INFINITY;
    for (int p = lane; p < parts; p += 32) top = fmaxf(top, ml[first + static_cast<int64_t>(p) * n_heads].x);
    top = warp_max(top);
    float4 sum = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    float l = 0.0f;
    // this thread's partials: p = off + step j, j < mine
    constexpr int step = kFew ? kTcWarps : 1;
    const int off = kFew ? warp : 0, mine = (parts - off + step - 1) / step;
    for (int j0 = 0; j0 < mine; j0 += 32) {
        // lane j: the weight of partial j0 + j; a partial without a key (m = -inf) was never written
        const bool real = j0 + lane < mine;
        const float2 s = real ? ml[first + static_cast<int64_t>(off + (j0 + lane) * step) * n_heads] : make_float2(-INFINITY, 0.0f);
        const bool there = s.x > -INFINITY;
        const float w = there ? exp2f(s.x - top) : 0.0f;
        l += there ? w * s.y : 0.0f;
        const unsigned live = __ballot_sync(0xffffffffu, there);
        const int n = min(32, mine - j0);
        for (int k = 0; k < n; k += 8) {
            float4 v[8];
#pragma unroll
            for (int i = 0; i < 8; i++)
                v[i] = live >> (k + i) & 1u
                           ? __ldg(reinterpret_cast<const float4 *>(acc + (first + static_cast<int64_t>(off + (j0 + k + i) * step) * n_heads) * kLatent))
                           : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
            for (int i = 0; i < 8; i++) {
                const float f = __shfl_sync(0xffffffffu, w, k + i);
                sum.x = fmaf(f, v[i].x, sum.x);
                sum.y = fmaf(f, v[i].y, sum.y);
                sum.z = fmaf(f, v[i].z, sum.z);
                sum.w = fmaf(f, v[i].w, sum.w);
            }
        }
    }
    l = warp_sum(l);
    if constexpr (kFew) {
        __shared__ float4 sums[kTcWarps][32];
        __shared__ float ls[kTcWarps];
        sums[warp][lane] = sum;
        if (lane == 0) ls[warp] = l;
        __syncthreads();
        if (warp != 0) return;
        for (int i = 1; i < kTcWarps; i++) {
            const float4 v = sums[i][lane];
            sum.x += v.x;
            sum.y += v.y;
            sum.z += v.z;
            sum.w += v.w;
            l += ls[i];
        }
    }
    const bool none = !(top > -INFINITY);
    const float inv = none ? 0.0f : 1.0f / l;
    const __nv_bfloat162 lo = __floats2bfloat162_rn(sum.x * inv, sum.y * inv), hi = __floats2bfloat162_rn(sum.z * inv, sum.w * inv);
    *reinterpret_cast<uint2 *>(out + row * kLatent + dim) =
        make_uint2(*reinterpret_cast<const uint32_t *>(&lo), *reinterpret_cast<const uint32_t *>(&hi));
    if (lse && dim == 0) lse[row] = none ? -INFINITY : top * 0.6931471805599453f + logf(l);
}

}  // namespace

cudaError_t launch_tree_combine(const float *part_acc, const float *part_ml, int n_rows, int n_heads, int parts, int num_sms,
                                uint16_t *out, float *lse, cudaStream_t stream) {
    cudaError_t e;
    if (n_rows < num_sms)
        e = launch_pdl(tree_combine_kernel<true>, dim3(4 * n_rows), dim3(32 * kTcWarps), 0, stream, part_acc, part_ml, n_heads,
                       parts, out, lse);
    else
        e = launch_pdl(tree_combine_kernel<false>, dim3(n_rows), dim3(128), 0, stream, part_acc, part_ml, n_heads, parts, out, lse);
    return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace glm
