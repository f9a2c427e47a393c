// Routing of the products grouped by expert with the fused epilogue (lq_gemm_grouped;
// lq_gemm_epilogue is its one-expert case):
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

namespace {

// Slots of an expert on average, and whether the kernel for few of them takes the call.
int slots_each(const GroupedCall& c) {
    const int active = c.n < c.experts ? c.n : c.experts;
    return (int)(((long long)c.n + active - 1) / active);
}
bool few_rows(const GroupedCall& c) { return slots_each(c) <= 8; }

}  // namespace

size_t grouped_workspace_size(const GroupedCall& c) {
    const size_t need = !few_rows(c) && c.offsets ? grouped_tc_workspace_size(c.K, c.n) : 0;
    return need > 256 ? need : 256;
}

cudaError_t launch_grouped(const GroupedCall& c, void* ws, unsigned* status, cudaStream_t st) {
    int dev = 0, sms = 148;
    cudaGetDevice(&dev);
    cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (few_rows(c)) return launch_grouped_mma(c, status, st, sms);
    return launch_grouped_tc(c, ws, status, st, sms, slots_each(c));
}

}  // namespace lq
