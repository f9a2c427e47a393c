// The two row operators beside the grouped products: rows grouped by expert id
// (lq_group_rows) and the experts' rows joined per token (lq_combine_rows).
#include "lq_debug.cuh"
#include "lq_epilogue.cuh"
#include "lq_internal.h"

namespace lq {
namespace {

constexpr int kThreads = 256;

// One CTA per expert: counts the ids of smaller experts (its offset), then walks
// the ids in order and gives its own the next slots. Stable and deterministic.
__global__ void __launch_bounds__(kThreads)
    group_kernel(const int* __restrict__ ids, int n, int topk, int experts, int* __restrict__ offsets,
                 int* __restrict__ rows, int* __restrict__ slots) {
    __shared__ int warp_sum[kThreads / 32];
    __shared__ int total;
    const int e = blockIdx.x, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    int less = 0, kept = 0;
    for (int i = tid; i < n; i += kThreads) {
        const int id = __ldg(ids + i);
        less += id >= 0 && id < e;
        kept += id >= 0 && id < experts;
    }
    auto block_sum = [&](int v) {
        for (int d = 16; d; d >>= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
        __syncthreads();
        if (lane == 0) warp_sum[warp] = v;
        __syncthreads();
        if (tid == 0) {
            int t = 0;
            for (int w = 0; w < kThreads / 32; ++w) t += warp_sum[w];
            total = t;
        }
        __syncthreads();
        return total;
    };
    const int base = block_sum(less), all = block_sum(kept);
    if (tid == 0) {
        offsets[e] = base;
        if (e == experts - 1) offsets[experts] = all;
    }
    int next = base;
    for (int i0 = 0; i0 < n; i0 += kThreads) {
        const int i = i0 + tid;
        const int id = i < n ? __ldg(ids + i) : -1;
        const unsigned mine = __ballot_sync(0xffffffffu, i < n && id == e);
        __syncthreads();
        if (lane == 0) warp_sum[warp] = __popc(mine);
        __syncthreads();
        int before = 0, chunk = 0;
        for (int w = 0; w < kThreads / 32; ++w) {
            if (w < warp) before += warp_sum[w];
            chunk += warp_sum[w];
        }
        if (i < n && id == e) {
            const int slot = next + before + __popc(mine & ((1u << lane) - 1u));
            if (LQ_IN_BOUNDS(slot, n)) {
                rows[slot] = i / topk;
                slots[i] = slot;
            }
        }
        if (e == 0 && i < n && (id < 0 || id >= experts)) slots[i] = -1;
        if (e == 0 && i < n && i >= all) rows[i] = -1;
        next += chunk;
    }
}

__global__ void __launch_bounds__(kThreads)
    combine_kernel(const void* __restrict__ y, bool bf16, int n, int width, const int* __restrict__ slots,
                   const float* __restrict__ weights, int tokens, int topk, const void* __restrict__ residual,
                   void* __restrict__ o) {
    const long long count = (long long)tokens * width;
    for (long long i = (long long)blockIdx.x * kThreads + threadIdx.x; i < count; i += (long long)gridDim.x * kThreads) {
        const long long t = i / width, c = i - t * width;
        float acc = 0.f;
        for (int j = 0; j < topk; ++j) {
            const int slot = __ldg(slots + t * topk + j);
            if (slot < 0 || slot >= n) continue;
            acc += __ldg(weights + t * topk + j) * load_elem(y, (long long)slot * width + c, bf16);
        }
        if (residual) acc += load_elem(residual, i, bf16);
        store_elem(o, i, bf16, acc);
    }
}

}  // namespace

cudaError_t launch_group_rows(const int* ids, int tokens, int topk, int experts, int* offsets, int* rows, int* slots,
                              cudaStream_t st) {
    group_kernel<<<experts, kThreads, 0, st>>>(ids, tokens * topk, topk, experts, offsets, rows, slots);
    return cudaGetLastError();
}

cudaError_t launch_combine_rows(const void* y, bool bf16, int n, int width, const int* slots, const float* weights,
                                int tokens, int topk, const void* residual, void* o, cudaStream_t st) {
    const long long blocks = ((long long)tokens * width + kThreads - 1) / kThreads;
    combine_kernel<<<(int)(blocks < 16384 ? blocks : 16384), kThreads, 0, st>>>(y, bf16, n, width, slots, weights,
                                                                              tokens, topk, residual, o);
    return cudaGetLastError();
}

}  // namespace lq

LQ_DEBUG_FLAG_TAKE(debug_take_rows)
