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
#include "lq_decode.h"
#include "lq_internal.h"

namespace lq {

namespace {

// Slots of an expert on average, if they spread over as many experts as they can.
int slots_each(const GroupedCall& c) {
    const int active = c.n < c.experts ? c.n : c.experts;
    return (int)(((long long)c.n + active - 1) / active);
}

// One or two tokens through one layer: the decode GEMV on u made fp32, unless its plan does not fit.
size_t decode_workspace(const GroupedCall& c) {
    return c.experts == 1 && !c.offsets && c.n <= 2 ? gemv_epilogue_bf16_workspace_size(c.out, c.K, c.n) : 0;
}

// Up to eight slots an expert, one pass of the mma.sync kernel, which reads the weights once for all of them.
bool few_rows(const GroupedCall& c) { return slots_each(c) <= 8; }

}  // namespace

size_t grouped_workspace_size(const GroupedCall& c) {
    size_t need = decode_workspace(c);
    if (!need && !few_rows(c) && c.offsets) need = grouped_tc_workspace_size(c.K, c.n);
    return need > 256 ? need : 256;
}

cudaError_t launch_grouped(const GroupedCall& c, void* ws, unsigned* status, cudaStream_t st) {
    if (decode_workspace(c)) {
        const DecodeEpilogue epi{c.bias, c.residual, c.o, nullptr, c.act, c.glu, c.o_bf16};
        return launch_gemv_epilogue_bf16(c.packed, c.s, c.out, c.K, c.u, c.n, epi, ws, status, st);
    }
    int dev = 0, sms = 148;
    cudaGetDevice(&dev);
    cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (few_rows(c)) return launch_grouped_mma(c, status, st, sms);
    return launch_grouped_tc(c, ws, status, st, sms, slots_each(c));
}

}  // namespace lq
