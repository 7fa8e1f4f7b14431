// block_tables.cu -- block tables, slots and slot maps from request lengths, and the copy of
// accepted drafts into the slots so made. Both are bound by latency at decode sizes, so each is one
// launch: every CTA of the tables kernel scans the requests for itself (a few microseconds' worth
// of loads that all CTAs do at once) instead of waiting for a scan kernel. On the GPU a call takes 4.7 us
// for 8 requests with a token each, 5.4 for 200 with up to 8, 7.9 for 16 prompts of up to 32,768 tokens
// (6.8 MB of slots, positions and maps: 1.0 at the copy rate); the commit 1.9 for 4 tokens or 380. From
// Python the host's call is longer than either: 9.1 and 8.1 us.
#include <algorithm>

#include "block_tables.cuh"
#include "common.cuh"

namespace glm {

namespace {

constexpr int kBtThreads = 512;
constexpr int kBtWarps = kBtThreads / 32;

__device__ __forceinline__ int sat32(int64_t v) { return static_cast<int>(v < 0x7fffffffll ? v : 0x7fffffffll); }

// Exclusive sum over the CTA of one value per thread; *total receives the sum. scratch: kBtWarps.
__device__ __forceinline__ int64_t block_scan(int64_t v, int64_t *scratch, int64_t *total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int64_t s = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t u = __shfl_up_sync(0xffffffffu, s, o);
        if (lane >= o) s += u;
    }
    if (lane == 31) scratch[warp] = s;
    __syncthreads();
    int64_t w = lane < kBtWarps ? scratch[lane] : 0;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t u = __shfl_up_sync(0xffffffffu, w, o);
        if (lane >= o) w += u;
    }
    *total = __shfl_sync(0xffffffffu, w, 31);
    const int64_t before = __shfl_sync(0xffffffffu, w, warp > 0 ? warp - 1 : 0);
    __syncthreads();
    return s - v + (warp > 0 ? before : 0);
}

// One request's numbers. add: tokens to append; back: blocks it returns; room: everything but the
// free list allows it (its packed tokens end at `end`); need: blocks it takes.
struct BtRequest {
    int64_t len, add, held, pad, back;
    bool sound;
};
__device__ __forceinline__ BtRequest bt_load(const BlockTableArgs &a, int b) {
    BtRequest r;
    const int n = a.n_new[b];
    r.len = a.len[b];
    r.held = a.n_blocks[b];
    r.pad = a.pad ? a.pad[b] : 0;
    r.add = n > 0 ? n : 0;
    r.sound = n >= 0 && r.pad >= 0 && r.held >= 0 && r.held <= a.ld_blocks && r.len >= 0 && r.len <= r.held * a.block_size;
    const int64_t held = r.held < 0 ? 0 : (r.held < a.ld_blocks ? r.held : a.ld_blocks);
    r.back = n < 0 ? held : 0;
    return r;
}
__device__ __forceinline__ int64_t bt_need(const BlockTableArgs &a, const BtRequest &r, int64_t end) {
    const int64_t want = (r.len + r.add + a.block_size - 1) / a.block_size;
    const bool room = r.sound && want <= a.ld_blocks && end <= a.n_cap && r.pad + r.len + r.add <= 0x7fffffffll &&
                      (!a.slot_map || r.pad + r.len + r.add <= a.ld_slot);
    return room ? (want > r.held ? want - r.held : 0) : -1;   // -1: refused
}

__global__ void __launch_bounds__(kBtThreads) block_tables_kernel(BlockTableArgs a) {
    pdl_begin(a.len, a.n_new, a.n_blocks, a.pad, a.table, a.free_list, a.n_free);
    extern __shared__ int smem_bt[];
    int *cu = smem_bt;                       // [batch + 1] packed offsets
    int *off = cu + a.batch + 1;             // [batch] offset of the request's new blocks, -1: refused
    int *need_s = off + a.batch;             // [batch] blocks it takes
    int *roff = need_s + a.batch;            // [batch] offset of the blocks it returns, -1: none
    __shared__ int64_t scratch[kBtWarps];
    __shared__ int s_taken;
    const int tid = threadIdx.x, lane = tid & 31;
    const int n_free = min(max(*a.n_free, 0), a.free_cap);
    if (tid == 0) s_taken = 0;

    // 1. packed offsets and returned blocks
    const int per = (a.batch + kBtThreads - 1) / kBtThreads;
    const int b0 = min(a.batch, tid * per), b1 = min(a.batch, b0 + per);
    int64_t sum = 0, ret = 0;
    for (int b = b0; b < b1; b++) {
        const BtRequest r = bt_load(a, b);
        sum += r.add;
        ret += r.back;
    }
    int64_t n_tok, returned;
    int64_t at = block_scan(sum, scratch, &n_tok);
    int64_t rat = block_scan(ret, scratch, &returned);
    const int64_t first = at;
    // 2. blocks needed, in request order
    int64_t needs = 0;
    for (int b = b0; b < b1; b++) {
        const BtRequest r = bt_load(a, b);
        cu[b] = sat32(at);
        at += r.add;
        roff[b] = r.back > 0 ? sat32(rat) : -1;
        rat += r.back;
        const int64_t need = bt_need(a, r, at);
        needs += need > 0 ? need : 0;
    }
    if (tid == 0) cu[a.batch] = sat32(n_tok);
    int64_t total_need;
    int64_t o = block_scan(needs, scratch, &total_need);
    at = first;
    int taken = 0;
    for (int b = b0; b < b1; b++) {
        const BtRequest r = bt_load(a, b);
        at += r.add;
        const int64_t need = bt_need(a, r, at);
        const bool granted = need == 0 || (need > 0 && o + need <= n_free);
        off[b] = granted ? (need > 0 ? static_cast<int>(o) : 0) : -1;
        need_s[b] = granted ? static_cast<int>(need) : 0;
        if (granted && need > 0) taken = max(taken, static_cast<int>(o + need));
        o += need > 0 ? need : 0;
    }
    if (taken > 0) atomicMax(&s_taken, taken);
    __syncthreads();
    const int left = n_free - s_taken;       // granted requests take a prefix of the needs

    // 3. this CTA's share of the outputs
    const int64_t stride = static_cast<int64_t>(gridDim.x) * kBtThreads;
    const int64_t t0 = static_cast<int64_t>(blockIdx.x) * kBtThreads + tid;
    // packed tokens: the request of token i by bisection of the offsets
    for (int64_t i = t0; i < a.n_cap; i += stride) {
        int64_t slot = -1;
        int seq = -1, pos_out = -1;
        if (i < cu[a.batch]) {
            int lo = 0, hi = a.batch;        // the last request whose tokens start at or before i
            while (hi - lo > 1) {
                const int mid = (lo + hi) >> 1;
                if (cu[mid] <= i) lo = mid;
                else hi = mid;
            }
            if (off[lo] >= 0) {
                const int64_t held = a.n_blocks[lo], pos = a.len[lo] + (i - cu[lo]);
                const int64_t k = pos / a.block_size, pad = a.pad ? a.pad[lo] : 0;
                const int64_t blk = k < held ? a.table[lo * a.ld_blocks + k]
                                             : a.free_list[n_free - 1 - off[lo] - static_cast<int>(k - held)];
                seq = lo;
                pos_out = static_cast<int>(pad + pos);
                if (blk >= 0 && blk < a.pool_blocks) slot = blk * a.block_size + (pos - k * a.block_size);
                if (a.slot_map) a.slot_map[lo * a.ld_slot + pad + pos] = slot;
            }
        }
        a.slots[i] = slot;
        a.q_seq[i] = seq;
        a.q_pos[i] = pos_out;
    }
    // what is left of the free list
    for (int64_t i = t0; i < left; i += stride) a.free_out[i] = a.free_list[i];
    // one warp per request: its new blocks into the table, or its returned blocks onto the free list
    for (int64_t w = t0 >> 5; w < a.batch; w += stride >> 5) {
        const int b = static_cast<int>(w);
        for (int j = lane; j < need_s[b]; j += 32)
            a.table[b * a.ld_blocks + a.n_blocks[b] + j] = a.free_list[n_free - 1 - off[b] - j];
        if (roff[b] >= 0) {
            const int64_t n = min(static_cast<int64_t>(max(a.n_blocks[b], 0)), a.ld_blocks);
            for (int64_t j = lane; j < n; j += 32) {
                const int64_t d = static_cast<int64_t>(left) + roff[b] + j;
                if (d < a.free_cap) a.free_out[d] = a.table[b * a.ld_blocks + j];
            }
        }
        if (lane == 0) {
            const bool ended = a.n_new[b] < 0;
            const int n = a.len[b];
            a.len_out[b] = ended ? 0 : (off[b] >= 0 ? n + max(a.n_new[b], 0) : n);
            a.n_blocks_out[b] = ended ? 0 : a.n_blocks[b] + need_s[b];
        }
    }
    for (int64_t i = t0; i <= a.batch; i += stride) a.cu_new[i] = cu[i];
    if (t0 == 0) *a.n_free_out = static_cast<int>(min(static_cast<int64_t>(a.free_cap), left + returned));
}

// ------------------------------------------------------------------------------------------------
// accepted drafts: one warp per packed token
// ------------------------------------------------------------------------------------------------
constexpr int kTcWarps = 4;

__global__ void __launch_bounds__(32 * kTcWarps) tree_commit_kernel(TreeCommitArgs a) {
    pdl_begin(a.draft, a.path, a.slots, a.q_seq, a.q_pos, a.cu_new, a.draft_k, a.draft_gate);
    const int lane = threadIdx.x & 31;
    const int64_t warps = static_cast<int64_t>(gridDim.x) * kTcWarps;
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * kTcWarps + (threadIdx.x >> 5); i < a.n_cap; i += warps) {
        const int b = a.q_seq[i];
        const int64_t slot = a.slots[i];
        const int64_t pos = a.q_pos[i];
        if (b < 0 || b >= a.batch) continue;
        const int64_t j = i - a.cu_new[b];
        if (j < 0 || j >= a.ld_path) continue;
        const int node = a.path[static_cast<int64_t>(b) * a.ld_path + j];
        if (node < 0 || node >= a.n_nodes) continue;
        const int64_t src = static_cast<int64_t>(b) * a.n_nodes + node;
        const int pieces = a.row_bytes / 16;                       // 33, or 19 for 4-bit rows
        const bool put = slot >= 0 && slot < a.n_rows;
        const uint4 *from = reinterpret_cast<const uint4 *>(a.draft + src * a.row_bytes);
        uint4 v = make_uint4(0u, 0u, 0u, 0u), last = v, s = v;
        if (put && lane < pieces) v = from[lane];
        if (put && lane == 0 && pieces > 32) last = from[32];
        const bool state = a.k && pos >= 0 && pos < a.ld_tokens;   // lanes 0-15: k, 16-31: gate
        if (state)
            s = reinterpret_cast<const uint4 *>((lane < 16 ? a.draft_k : a.draft_gate) + src * kIdxDim)[lane & 15];
        uint4 *to = reinterpret_cast<uint4 *>(a.cache + slot * a.row_bytes);
        if (put && lane < pieces) to[lane] = v;
        if (put && lane == 0 && pieces > 32) to[32] = last;
        if (state)
            reinterpret_cast<uint4 *>((lane < 16 ? a.k : a.gate) + (b * a.ld_tokens + pos) * kIdxDim)[lane & 15] = s;
    }
}

}  // namespace

cudaError_t launch_block_tables(const BlockTableArgs &a, cudaStream_t stream, int num_sms) {
    // CTAs for the tokens, the free list (four entries a thread) and the requests (a warp each)
    int64_t ctas = (a.n_cap + kBtThreads - 1) / kBtThreads;
    ctas = std::max(ctas, (static_cast<int64_t>(a.free_cap) + 4 * kBtThreads - 1) / (4 * kBtThreads));
    ctas = std::max(ctas, (static_cast<int64_t>(a.batch) + kBtWarps - 1) / kBtWarps);
    ctas = std::min(std::max(ctas, static_cast<int64_t>(1)), static_cast<int64_t>(num_sms));
    const int smem = (4 * a.batch + 1) * 4;
    cudaError_t e = cudaSuccess;
    if (smem > 47 * 1024)                       // (48 KB, less its own, need no asking)
        e = cudaFuncSetAttribute(block_tables_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (4 * kBtMaxBatch + 1) * 4);
    if (e != cudaSuccess) return e;
    e = launch_pdl(block_tables_kernel, dim3(static_cast<unsigned>(ctas)), dim3(kBtThreads), smem, stream, a);
    return e != cudaSuccess ? e : cudaGetLastError();
}

cudaError_t launch_tree_commit(const TreeCommitArgs &a, cudaStream_t stream, int num_sms) {
    int64_t ctas = (a.n_cap + kTcWarps - 1) / kTcWarps;
    ctas = std::min(ctas, static_cast<int64_t>(num_sms) * 16);
    cudaError_t e = launch_pdl(tree_commit_kernel, dim3(static_cast<unsigned>(ctas)), dim3(32 * kTcWarps), 0, stream, a);
    return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace glm
