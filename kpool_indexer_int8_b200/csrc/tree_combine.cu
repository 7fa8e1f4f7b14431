// tree_combine.cu -- the merge of the tree attention's partial softmax states.
//
// A query row's partials hold, over the keys of their run, acc = sum 2^(..) v, the sum l of the weights and
// their reference m (natural units); with M = max m over the partials with l > 0 the row is
//     out = sum e^(m - M) acc / sum e^(m - M) l,    lse = M + log(sum e^(m - M) l),
// all of it in fp32, in the order of the partials. It is bound by the partials' 2 KB each, which the
// attention has just written and L2 holds. One CTA of 128 threads a row, a thread four dims, eight partials
// in flight. (The other attentions' merge spreads a row over four CTAs of four warps each, which is
// faster for a few rows of many partials but took 37 us for 3,328 rows of 4.)
#include "common.cuh"
#include "tree_mla.cuh"

namespace glm {

namespace {

constexpr int kTcThreads = 128;

__global__ void __launch_bounds__(kTcThreads) tree_combine_kernel(const float *__restrict__ part_acc,
                                                                  const float *__restrict__ part_ml, int n_heads, int parts,
                                                                  uint16_t *__restrict__ out, float *__restrict__ lse) {
    pdl_begin(part_acc, part_ml);
    const int lane = threadIdx.x & 31;
    const int64_t row = blockIdx.x, node = row / n_heads;
    const int64_t first = node * parts * n_heads + (row - node * n_heads);   // partial p: first + p n_heads
    const float2 *ml = reinterpret_cast<const float2 *>(part_ml);
    const float *acc = part_acc + 4 * threadIdx.x;
    float top = -INFINITY;
    for (int p = lane; p < parts; p += 32) top = fmaxf(top, ml[first + static_cast<int64_t>(p) * n_heads].x);
    top = warp_max(top);
    float4 sum = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    float l = 0.0f;
    for (int p0 = 0; p0 < parts; p0 += 32) {
        // lane p: the weight of partial p0 + p; a partial without a key (m = -inf) was never written
        const int64_t mine = first + static_cast<int64_t>(min(p0 + lane, parts - 1)) * n_heads;
        const float2 s = p0 + lane < parts ? ml[mine] : make_float2(-INFINITY, 0.0f);
        const bool there = s.x > -INFINITY;
        const float w = there ? expf(s.x - top) : 0.0f;
        l += there ? w * s.y : 0.0f;
        const unsigned live = __ballot_sync(0xffffffffu, there);
        const int n = min(32, parts - p0);
        for (int k = 0; k < n; k += 8) {
            float4 v[8];
#pragma unroll
            for (int i = 0; i < 8; i++)
                v[i] = live >> (k + i) & 1u
                           ? __ldg(reinterpret_cast<const float4 *>(acc + (first + static_cast<int64_t>(p0 + k + i) * n_heads) * kLatent))
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
    const bool none = !(top > -INFINITY);
    const float inv = none ? 0.0f : 1.0f / l;
    const __nv_bfloat162 lo = __floats2bfloat162_rn(sum.x * inv, sum.y * inv), hi = __floats2bfloat162_rn(sum.z * inv, sum.w * inv);
    *reinterpret_cast<uint2 *>(out + row * kLatent + 4 * threadIdx.x) =
        make_uint2(*reinterpret_cast<const uint32_t *>(&lo), *reinterpret_cast<const uint32_t *>(&hi));
    if (lse && threadIdx.x == 0) lse[row] = none ? -INFINITY : top + logf(l);
}

}  // namespace

cudaError_t launch_tree_combine(const float *part_acc, const float *part_ml, int n_rows, int n_heads, int parts, uint16_t *out,
                                float *lse, cudaStream_t stream) {
    const cudaError_t e = launch_pdl(tree_combine_kernel, dim3(n_rows), dim3(kTcThreads), 0, stream, part_acc, part_ml, n_heads,
                                     parts, out, lse);
    return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace glm
