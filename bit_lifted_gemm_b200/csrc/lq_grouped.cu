// Matrix products grouped by expert, with the fused epilogue (lq_gemm_grouped;
// lq_gemm_epilogue and lq_gemv_epilogue are its one-expert case):
//
//   z[i][r] = s_e[r] sum_k sigma_e[r][k] u[rows[i]][k] + bias_e[r],  offsets[e] <= i < offsets[e+1]
//   o[i][r] = act(z[i][r]) + residual[i][r], or gated
//   o[i][j] = act(z[i][2j]) z[i][2j+1] + residual[i][j]
//
// One warp per output element (two weight rows when gated); lanes stride over
// the sign words, fp32 sums.
#include "lq_debug.cuh"
#include "lq_epilogue.cuh"
#include "lq_internal.h"

namespace lq {
namespace {

constexpr int kWarps = 8;

__device__ __forceinline__ float dot_row(const uint32_t* w, const void* u, bool u_bf16, long long u0, int kw, int lane) {
    float acc = 0.f;
    for (int x = lane; x < kw; x += 32) {
        const uint32_t bits = __ldg(w + x);
        for (int j = 0; j < 32; ++j) {
            const float v = load_elem(u, u0 + 32ll * x + j, u_bf16);
            acc += (bits >> j) & 1u ? v : -v;
        }
    }
    for (int d = 16; d; d >>= 1) acc += __shfl_xor_sync(0xffffffffu, acc, d);
    return acc;
}

__global__ void __launch_bounds__(32 * kWarps) grouped_kernel(const GroupedCall c) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int kw = c.K >> 5, width = c.glu ? c.out / 2 : c.out;
    const int j = blockIdx.x * kWarps + warp;
    if (j >= width) return;
    for (long long i = blockIdx.y; i < c.n; i += gridDim.y) {
        int e = 0;
        if (c.offsets) {  // the expert whose range holds slot i
            for (e = 0; e < c.experts; ++e)
                if (i >= __ldg(c.offsets + e) && i < __ldg(c.offsets + e + 1)) break;
            if (e == c.experts) continue;
        }
        const long long row = c.rows ? (long long)__ldg(c.rows + i) : i;
        const bool there = row >= 0 && row < c.tokens;
        float z[2];
        for (int h = 0; h < (c.glu ? 2 : 1); ++h) {
            const long long r = (long long)e * c.out + (c.glu ? 2 * j + h : j);
            const float acc = there ? dot_row(c.packed + r * kw, c.u, c.u_bf16, row * c.K, kw, lane) : 0.f;
            z[h] = __ldg(c.s + r) * acc + (c.bias ? __ldg(c.bias + r) : 0.f);
        }
        if (lane == 0) {
            const float y = c.glu ? activate(z[0], c.act) * z[1] : activate(z[0], c.act);
            store_elem(c.o, i * width + j, c.o_bf16,
                       c.residual ? y + load_elem(c.residual, i * width + j, c.o_bf16) : y);
        }
    }
}

}  // namespace

size_t grouped_workspace_size(const GroupedCall& c) {
    const size_t planes = grouped_mma_workspace_size(c.K, c.n, c.u_bf16);
    return planes > 256 ? planes : 256;
}

cudaError_t launch_grouped(const GroupedCall& c, void* ws, unsigned* status, cudaStream_t st) {
    int dev = 0, sms = 148;
    cudaGetDevice(&dev);
    cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    const int active = c.n < c.experts ? c.n : c.experts;
    if (!c.u_bf16 || (c.n + active - 1) / active <= 32) return launch_grouped_mma(c, ws, status, st, sms);
    const int width = c.glu ? c.out / 2 : c.out;
    const dim3 grid((width + kWarps - 1) / kWarps, c.n < 16384 ? c.n : 16384);
    grouped_kernel<<<grid, 32 * kWarps, 0, st>>>(c);
    return cudaGetLastError();
}

}  // namespace lq
