// The two row operators beside the grouped products: rows grouped by expert id
// (lq_group_rows) and the experts' rows joined per token (lq_combine_rows).
#include <cooperative_groups.h>

#include "lq_debug.cuh"
#include "lq_epilogue.cuh"
#include "lq_internal.h"

namespace lq {
namespace {

namespace cg = cooperative_groups;

// ---- lq_group_rows: a stable counting sort of the ids, in one launch
//
// One cluster (of 1, 8 or 16 CTAs) cuts the ids into one contiguous run per
// warp. Each warp counts its run's ids per expert in shared memory of its own (32 ids at a time:
// lanes with equal ids find one another by ballots, their lowest lane adds). Prefix sums over the warps,
// over the cluster's CTAs (distributed shared memory) and over the experts give every warp the
// first slot of its ids of each expert; walking its run again, it hands them out in order. So
// slots do not depend on timing and no global scratch is needed. Latency bounds it (131072 ids of
// 128 experts 17.5 us, 90 GB/s; 32 ids 3.9 us): loads of eight rounds are issued together, and each round is a chain
// of ballots and shared memory.
constexpr int kMaxWarps = 32, kRounds = 8, kCluster = 16;

// Lanes of the warp with this id (below 2^bits), and this lane's place among them: one ballot a bit. (A match
// instruction takes the SM ~64 clocks, which bounded the kernel: 35 us for 131072 ids of 128 experts.)
__device__ __forceinline__ int rank_among_equals(unsigned id, int bits, int lane, unsigned& peers) {
    peers = 0xffffffffu;
    for (int b = 0; b < bits; ++b) {
        const bool set = (id >> b) & 1u;
        const unsigned v = __ballot_sync(0xffffffffu, set);
        peers &= set ? v : ~v;
    }
    return __popc(peers & ((1u << lane) - 1u));
}

__global__ void __launch_bounds__(32 * kMaxWarps)
    group_kernel(const int* __restrict__ ids, int n, int topk, int experts, int bits, int* __restrict__ offsets,
                 int* __restrict__ rows, int* __restrict__ slots) {
    extern __shared__ int smem[];
    cg::cluster_group cluster = cg::this_cluster();
    const int ctas = (int)cluster.num_blocks(), cta = (int)cluster.block_rank();
    const int warps = blockDim.x >> 5, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    int* total = smem;                         // [experts] ids of each expert in this CTA
    int* base = smem + experts;                // [experts] first slot of this CTA's ids
    int* partial = base + experts;             // [32] for the scan over experts
    int* count = partial + 32;                 // [warps][experts]
    int* mine = count + warp * experts;
    const long long per = ((long long)n + ctas * warps - 1) / (ctas * warps);
    const int lo = (int)min((long long)n, per * (cta * warps + warp)), hi = (int)min((long long)n, (long long)lo + per);

    for (int i = threadIdx.x; i < warps * experts; i += blockDim.x) count[i] = 0;
    __syncthreads();
    for (long long i0 = lo; i0 < hi; i0 += 32 * kRounds) {
        unsigned id[kRounds];  // experts: left out
#pragma unroll
        for (int r = 0; r < kRounds; ++r) {
            const long long i = i0 + 32 * r + lane;
            id[r] = i < hi && LQ_IN_BOUNDS(i, n) ? min((unsigned)__ldg(ids + i), (unsigned)experts) : experts;
        }
#pragma unroll
        for (int r = 0; r < kRounds; ++r) {
            if (i0 + 32 * r >= hi) break;
            unsigned peers;
            const int rank = rank_among_equals(id[r], bits, lane, peers);
            if (rank == 0 && id[r] < (unsigned)experts) mine[id[r]] += __popc(peers);
            __syncwarp();
        }
    }
    __syncthreads();
    for (int e = threadIdx.x; e < experts; e += blockDim.x) {
        int sum = 0;
        for (int w = 0; w < warps; ++w) {
            const int c = count[w * experts + e];
            count[w * experts + e] = sum;
            sum += c;
        }
        total[e] = sum;
    }
    cluster.sync();
    // first slot of each expert: a run of experts per thread, runs summed over the block
    const int run = (experts + blockDim.x - 1) / blockDim.x;
    const int e0 = min(experts, (int)threadIdx.x * run), e1 = min(experts, e0 + run);
    int sum = 0;
    for (int e = e0; e < e1; ++e) {
        int all = 0, before = 0;
        for (int r = 0; r < ctas; ++r) {
            const int c = *cluster.map_shared_rank(total + e, r);
            all += c;
            if (r < cta) before += c;
        }
        base[e] = sum + before;  // from the run's start
        if (cta == 0) offsets[e] = sum;
        sum += all;
    }
    int upto = sum;
    for (int d = 1; d < 32; d <<= 1) {
        const int x = __shfl_up_sync(0xffffffffu, upto, d);
        if (lane >= d) upto += x;
    }
    if (lane == 31) partial[warp] = upto;
    __syncthreads();
    int start = upto - sum, kept = 0;
    for (int w = 0; w < warps; ++w) {
        if (w < warp) start += partial[w];
        kept += partial[w];
    }
    for (int e = e0; e < e1; ++e) {
        base[e] += start;
        if (cta == 0) offsets[e] += start;
    }
    if (cta == 0 && threadIdx.x == 0) offsets[experts] = kept;
    __syncthreads();
    for (long long i0 = lo; i0 < hi; i0 += 32 * kRounds) {
        unsigned id[kRounds];  // experts: left out
#pragma unroll
        for (int r = 0; r < kRounds; ++r) {
            const long long i = i0 + 32 * r + lane;
            id[r] = i < hi && LQ_IN_BOUNDS(i, n) ? min((unsigned)__ldg(ids + i), (unsigned)experts) : experts;
        }
#pragma unroll
        for (int r = 0; r < kRounds; ++r) {
            const long long i = i0 + 32 * r + lane;
            if (i0 + 32 * r >= hi) break;
            unsigned peers;
            const int rank = rank_among_equals(id[r], bits, lane, peers);
            const bool there = id[r] < (unsigned)experts;
            const int first = there ? mine[id[r]] : 0;
            __syncwarp();
            if (there && rank == 0) mine[id[r]] = first + __popc(peers);
            __syncwarp();
            if (i < hi) {
                const int slot = there ? base[id[r]] + first + rank : -1;
                slots[i] = slot;
                if (there && LQ_IN_BOUNDS(slot, n)) rows[slot] = (unsigned)i / (unsigned)topk;
            }
        }
    }
    for (long long i = kept + (long long)cta * blockDim.x + threadIdx.x; i < n; i += (long long)ctas * blockDim.x) rows[i] = -1;
    cluster.sync();  // no CTA leaves while others read its totals
}

// ---- lq_combine_rows
//
// A thread owns 16 bytes of a token's row (one element where rows are not 16-byte
// aligned) and adds the token's slots in order, the loads of four issued together. Bound by
// reading the y rows and writing o: 4096 tokens of four slots of 4096 bf16 37.5 us, 5.4 TB/s (83% of the measured copy).
// An element a thread takes 129 us for a width of 4095 (1.6 TB/s in loads of two bytes).
template <bool BF16, int N>
struct Chunk {
    typename Elem<BF16>::T v[N];
};

template <bool BF16, int N>
__device__ __forceinline__ Chunk<BF16, N> load_chunk(const void* p, long long i) {
    Chunk<BF16, N> c;
    using T = typename Elem<BF16>::T;
    if constexpr (N == 1)
        c.v[0] = __ldg(static_cast<const T*>(p) + i);
    else
        *reinterpret_cast<uint4*>(&c) = __ldg(reinterpret_cast<const uint4*>(static_cast<const T*>(p) + i));
    return c;
}

template <bool BF16, int N>
__global__ void __launch_bounds__(256)
    combine_kernel(const void* __restrict__ y, int n, int width, const int* __restrict__ slots,
                   const float* __restrict__ weights, int tokens, int topk, const void* __restrict__ residual,
                   void* __restrict__ o) {
    using T = typename Elem<BF16>::T;
    const long long extent = (long long)n * width;
    (void)extent;
    for (long long t = (long long)blockIdx.y * blockDim.y + threadIdx.y; t < tokens; t += (long long)gridDim.y * blockDim.y)
        for (long long c = ((long long)blockIdx.x * blockDim.x + threadIdx.x) * N; c < width; c += (long long)gridDim.x * blockDim.x * N) {
            float acc[N] = {};
            Chunk<BF16, N> res;
            if (residual) res = load_chunk<BF16, N>(residual, t * width + c);
            for (int j0 = 0; j0 < topk; j0 += 4) {
                Chunk<BF16, N> v[4];
                float w[4];
                bool there[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int slot = j0 + j < topk ? __ldg(slots + t * topk + j0 + j) : -1;
                    there[j] = slot >= 0 && slot < n && LQ_IN_BOUNDS((long long)slot * width + c + N - 1, extent);
                    if (there[j]) {
                        w[j] = __ldg(weights + t * topk + j0 + j);
                        v[j] = load_chunk<BF16, N>(y, (long long)slot * width + c);
                    }
                }
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    if (there[j])
#pragma unroll
                        for (int i = 0; i < N; ++i) acc[i] = fmaf(w[j], Elem<BF16>::to_float(v[j].v[i]), acc[i]);
            }
            Chunk<BF16, N> out;
#pragma unroll
            for (int i = 0; i < N; ++i)
                out.v[i] = Elem<BF16>::from_float(residual ? acc[i] + Elem<BF16>::to_float(res.v[i]) : acc[i]);
            if (!LQ_IN_BOUNDS(t * width + c + N - 1, (long long)tokens * width)) continue;
            if constexpr (N == 1)
                static_cast<T*>(o)[t * width + c] = out.v[0];
            else
                *reinterpret_cast<uint4*>(static_cast<T*>(o) + t * width + c) = *reinterpret_cast<uint4*>(&out);
        }
}

template <bool BF16, int N>
cudaError_t launch_combine(const void* y, int n, int width, const int* slots, const float* weights, int tokens, int topk,
                           const void* residual, void* o, cudaStream_t st) {
    const int chunks = (width + N - 1) / N;
    int x = 32;
    while (x < 256 && x < chunks) x *= 2;
    const dim3 block(x, 256 / x);
    const long long bx = (chunks + x - 1) / x, by = ((long long)tokens + block.y - 1) / block.y;
    combine_kernel<BF16, N><<<dim3((unsigned)(bx < 65535 ? bx : 65535), (unsigned)(by < 65535 ? by : 65535)), block, 0, st>>>(
        y, n, width, slots, weights, tokens, topk, residual, o);
    return cudaGetLastError();
}

constexpr size_t kGroupSmem = 200 * 1024;

// Whether clusters of sixteen CTAs (more than the portable eight) of the largest size fit on the device.
signed char sixteen_run(signed char (&known)[64]) {
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev >= 64) return -1;
    if (known[dev]) return known[dev];
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(kCluster);
    cfg.blockDim = dim3(32 * kMaxWarps);
    cfg.dynamicSmemBytes = kGroupSmem;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = kCluster;
    attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    int clusters = 0;
    const bool ok = cudaFuncSetAttribute(group_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kGroupSmem) == cudaSuccess &&
                    cudaFuncSetAttribute(group_kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) == cudaSuccess &&
                    cudaOccupancyMaxActiveClusters(&clusters, group_kernel, &cfg) == cudaSuccess && clusters > 0;
    if (!ok) cudaGetLastError();
    return known[dev] = ok ? 1 : -1;
}

}  // namespace

cudaError_t launch_group_rows(const int* ids, int tokens, int topk, int experts, int* offsets, int* rows, int* slots,
                              cudaStream_t st) {
    const int n = tokens * topk;
    // One CTA up to 512 ids (a cluster's start and two barriers cost more than they save: 32 ids 3.7 us, 2048 ids
    // 8.4 us against 6 for eight CTAs), sixteen from 16384 on (131072 ids: 17.5 us against 28); as many warps
    // as have 64 ids each, and as their counts fit in shared memory
    static signed char sixteen[64];  // per device: 0 not asked yet, 1 clusters of sixteen run, -1 they do not
    const int ctas = n <= 512 ? 1 : n <= 16384 || sixteen_run(sixteen) < 0 ? 8 : kCluster;
    const int room = 160 * 1024 / (4 * experts);
    int warps = (n + 64 * ctas - 1) / (64 * ctas);
    warps = warps > kMaxWarps ? kMaxWarps : warps;
    warps = warps > room ? room : warps;
    warps = warps < 4 ? 4 : warps;
    int bits = 0;  // of ids 0..experts, the last for those left out
    while (experts >> bits) ++bits;
    const size_t smem = ((size_t)(warps + 2) * experts + 32) * 4;
    static bool attr_set[64] = {};
    int dev = 0;
    cudaGetDevice(&dev);
    if (dev >= 64 || !attr_set[dev]) {
        cudaError_t e = cudaFuncSetAttribute(group_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kGroupSmem);
        if (e != cudaSuccess) return e;
        if (dev < 64) attr_set[dev] = true;
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(ctas);
    cfg.blockDim = dim3(32 * warps);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = ctas;
    attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, group_kernel, ids, n, topk, experts, bits, offsets, rows, slots);
}

cudaError_t launch_combine_rows(const void* y, bool bf16, int n, int width, const int* slots, const float* weights,
                                int tokens, int topk, const void* residual, void* o, cudaStream_t st) {
    if (bf16)
        return width % 8 == 0 ? launch_combine<true, 8>(y, n, width, slots, weights, tokens, topk, residual, o, st)
                              : launch_combine<true, 1>(y, n, width, slots, weights, tokens, topk, residual, o, st);
    return width % 4 == 0 ? launch_combine<false, 4>(y, n, width, slots, weights, tokens, topk, residual, o, st)
                          : launch_combine<false, 1>(y, n, width, slots, weights, tokens, topk, residual, o, st);
}

}  // namespace lq

LQ_DEBUG_FLAG_TAKE(debug_take_rows)
