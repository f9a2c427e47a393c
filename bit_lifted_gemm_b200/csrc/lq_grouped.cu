// Routing of the products grouped by expert with the fused epilogue (lq_gemm_grouped;
// lq_gemm_epilogue and lq_gemv_epilogue are its one-expert case):
//
//   z[i][r] = s_e[r] sum_k sigma_e[r][k] u[rows[i]][k] + bias_e[r],  offsets[e] <= i < offsets[e+1]
//   o[i][r] = act(z[i][r]) + residual[i][r], or gated
//   o[i][j] = act(z[i][2j]) z[i][2j+1] + residual[i][j]
//
// The sizes of the groups are known to the device alone, so the host goes by the rows an
// expert has on average if they spread over as many experts as they can; both kernels
// are right for any sizes.
#include "lq_internal.h"

namespace lq {

size_t grouped_workspace_size(const GroupedCall& c) {
    const size_t planes = grouped_mma_workspace_size(c.K, c.n, c.u_bf16);
    return planes > 256 ? planes : 256;
}

cudaError_t launch_grouped(const GroupedCall& c, void* ws, unsigned* status, cudaStream_t st) {
    int dev = 0, sms = 148;
    cudaGetDevice(&dev);
    cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    const int active = c.n < c.experts ? c.n : c.experts;
    const int each = (int)(((long long)c.n + active - 1) / active);
    if (!c.u_bf16 || each <= 32) return launch_grouped_mma(c, ws, status, st, sms);
    return launch_grouped_tc(c, status, st, sms, each);
}

}  // namespace lq
