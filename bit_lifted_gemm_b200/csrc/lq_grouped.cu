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

// Tokens of one layer that take the decode GEMV on u made fp32 (1.5 us), unless its plan does not fit: one or two,
// and nine to sixteen where the tcgen05 kernel's 128-row tiles exceed the 148 SMs. Measured in us, this path
// against the kernel that would take them else: 13824 x 12288 at 1 / 2 / 16 tokens 12.8 / 14.6 / 42 against
// 18.7 / 18.3 / 37 to 43, 28672 x 20480 26.3 / 36.4 / 82 against 52 / 52 / 134, 4096 x 10240 8.7 / 10.6 / 34 against
// 9.7 / 10.1 / 17.
size_t decode_workspace(const GroupedCall& c) {
    if (c.experts != 1 || c.offsets || c.n > 16 || (c.n > 2 && (c.n <= 8 || c.out <= 148 * 128))) return 0;
    return gemv_epilogue_bf16_workspace_size(c.out, c.K, c.n);
}

// Slots of experts that take the same GEMV one by one, a share of the SMs each: up to two an expert, if the shares
// suffice and rows of words are 16-byte aligned. us against the mma.sync kernel: 2 slots of 8 experts of 11008 x 10240
// 15 against 27, of 4096 x 10240 one slot to each of 16 experts 30 against 62, of 128 188 against 393, two to each of
// 8 29 against 34; four to each of 4 28 against 20.
size_t slots_workspace(const GroupedCall& c) {
    if (!c.offsets || slots_each(c) > 2 || c.n > 148 || c.K % 128 != 0) return 0;
    return gemv_slots_workspace_size(c.out, c.K, c.n);
}

// Up to eight slots an expert, one pass of the mma.sync kernel, which reads the weights once for all of them (us at 8
// and 9 to 16 tokens of 13824 x 12288: 20 and, in two passes, 38; the tcgen05 kernel 37 to 43 for either).
bool few_rows(const GroupedCall& c) { return slots_each(c) <= 8; }

}  // namespace

size_t grouped_workspace_size(const GroupedCall& c) {
    size_t need = decode_workspace(c);
    if (!need) need = slots_workspace(c);
    if (!need && !few_rows(c)) need = grouped_tc_workspace_size(c, slots_each(c));
    return need > 256 ? need : 256;
}

cudaError_t launch_grouped(const GroupedCall& c, void* ws, unsigned* status, cudaStream_t st) {
    if (decode_workspace(c)) {
        const DecodeEpilogue epi{c.bias, c.residual, c.o, nullptr, c.act, c.glu, c.o_bf16};
        return launch_gemv_epilogue_bf16(c.packed, c.s, c.out, c.K, c.u, c.n, epi, ws, status, st);
    }
    if (slots_workspace(c)) return launch_gemv_slots(c, ws, status, st);
    int dev = 0, sms = 148;
    cudaGetDevice(&dev);
    cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (few_rows(c)) return launch_grouped_mma(c, status, st, sms);
    return launch_grouped_tc(c, ws, status, st, sms, slots_each(c));
}

}  // namespace lq
