// Epilogue arithmetic shared by the kernels of lq_gemm_epilogue,
// lq_gemv_epilogue and lq_gemm_grouped: activation, gate, residual and the one
// rounding of the result. Everything is fp32 until the final store.
#pragma once

#include <cuda_bf16.h>
#include <stdint.h>

#include "lq.h"

namespace lq {

// act(z) in fp32. The forms avoid cancellation for negative z: gelu as
// z/2 erfc(-z/sqrt 2), gelu_tanh through 1/2 (1 + tanh y) = 1 / (1 + e^(-2y)).
// relu keeps NaN.
__device__ __forceinline__ float activate(float z, int act) {
    switch (act) {
        case LQ_ACT_RELU: return z < 0.f ? 0.f : z;
        case LQ_ACT_GELU: return 0.5f * z * erfcf(-0.70710678118654752f * z);
        case LQ_ACT_GELU_TANH: {
            const float y = 0.79788456080286536f * (z + 0.044715f * z * z * z);
            return z / (1.f + expf(-2.f * y));
        }
        case LQ_ACT_SILU: return z / (1.f + expf(-z));
        default: return z;
    }
}

__device__ __forceinline__ float bf16_to_float(uint16_t b) { return __uint_as_float((uint32_t)b << 16); }

// Element i of an fp32 or bf16 array.
__device__ __forceinline__ float load_elem(const void* p, long long i, bool bf16) {
    return bf16 ? bf16_to_float(__ldg(static_cast<const uint16_t*>(p) + i)) : __ldg(static_cast<const float*>(p) + i);
}

// Round to nearest even once, at the store (bf16: off by at most 2^-8 of the value).
__device__ __forceinline__ void store_elem(void* p, long long i, bool bf16, float v) {
    if (bf16)
        static_cast<__nv_bfloat16*>(p)[i] = __float2bfloat16_rn(v);
    else
        static_cast<float*>(p)[i] = v;
}

}  // namespace lq
