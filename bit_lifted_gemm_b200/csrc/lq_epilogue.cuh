// Epilogue arithmetic shared by the kernels of lq_gemm_epilogue,
// lq_gemv_epilogue and lq_gemm_grouped: activation, gate, residual and the one
// rounding of the result. Everything is fp32 until the final store.
#pragma once

#include <cuda_bf16.h>
#include <stdint.h>

#include "lq.h"
#include "lq_debug.cuh"
#include "lq_decode.h"

namespace lq {

// a / b to two steps of fp32 without the branches of the rounded division, which keep a
// warp from overlapping one element's with the next one's. Denominators above 2^126 give 0, where a
// gate of such a denominator (e^-z, z < -87) is below 10^-36.
__device__ __forceinline__ float quotient(float a, float b) { return __fdividef(a, b); }

// act(z) in fp32. The forms avoid cancellation for negative z: gelu as
// z/2 erfc(-z/sqrt 2), gelu_tanh through 1/2 (1 + tanh y) = 1 / (1 + e^(-2y)).
// relu keeps NaN.
__device__ __forceinline__ float activate(float z, int act) {
    switch (act) {
        case LQ_ACT_RELU: return z < 0.f ? 0.f : z;
        case LQ_ACT_GELU: return 0.5f * z * erfcf(-0.70710678118654752f * z);
        case LQ_ACT_GELU_TANH: {
            const float y = 0.79788456080286536f * (z + 0.044715f * z * z * z);
            return quotient(z, 1.f + expf(-2.f * y));
        }
        case LQ_ACT_SILU: return quotient(z, 1.f + expf(-z));
        default: return z;
    }
}

// act on N values, the choice made once.
template <int N>
__device__ __forceinline__ void activate_all(float (&z)[N], int act) {
    switch (act) {
#define LQ_ACT_CASE(A)                                     \
    case A:                                                \
        _Pragma("unroll") for (int j = 0; j < N; ++j) z[j] = activate(z[j], A); \
        break;
        LQ_ACT_CASE(LQ_ACT_RELU)
        LQ_ACT_CASE(LQ_ACT_GELU)
        LQ_ACT_CASE(LQ_ACT_GELU_TANH)
        LQ_ACT_CASE(LQ_ACT_SILU)
#undef LQ_ACT_CASE
        default: break;
    }
}

__device__ __forceinline__ float bf16_to_float(uint16_t b) { return __uint_as_float((uint32_t)b << 16); }

// An fp32 or bf16 element as it is stored, and its conversions.
template <bool BF16>
struct Elem {
    using T = uint16_t;
    static __device__ __forceinline__ float to_float(T v) { return bf16_to_float(v); }
    static __device__ __forceinline__ T from_float(float v) { return __bfloat16_as_ushort(__float2bfloat16_rn(v)); }
};
template <>
struct Elem<false> {
    using T = float;
    static __device__ __forceinline__ float to_float(T v) { return v; }
    static __device__ __forceinline__ T from_float(float v) { return v; }
};

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

// The decode kernels' epilogue of weight row r of `count` columns from column 0 on, z with the scale applied and
// no bias yet. Called by the lanes of rows 2i and 2i + 1 together, which are neighbours, when gated. The
// choices are made outside the loops over the columns. `columns`: rows of o and of the residual, for the debug build.
template <int N>
__device__ __forceinline__ void finish_row(const DecodeEpilogue& e, int out, int columns, int c0, int count, int r, float (&z)[N],
                                           int lane) {
    const long long extent = (long long)columns * (e.glu ? out / 2 : out);
    (void)extent;
    const float bias = e.bias ? __ldg(e.bias + r) : 0.f;
#pragma unroll
    for (int c = 0; c < N; ++c) z[c] += bias;
    long long at = (long long)c0 * out + r, step = out;  // of column c0, and from one to the next
    if (e.glu) {
        float other[N];
#pragma unroll
        for (int c = 0; c < N; ++c) other[c] = __shfl_xor_sync(3u << (lane & 30), z[c], 1);
        if (r & 1) return;
        activate_all(z, e.act);
#pragma unroll
        for (int c = 0; c < N; ++c) z[c] *= other[c];
        step = out / 2;
        at = c0 * step + r / 2;
    } else {
        activate_all(z, e.act);
    }
    if (e.residual) {
        float res[N];
#pragma unroll
        for (int c = 0; c < N; ++c) res[c] = c < count && LQ_IN_BOUNDS(at + c * step, extent) ? load_elem(e.residual, at + c * step, e.o_bf16) : 0.f;
#pragma unroll
        for (int c = 0; c < N; ++c) z[c] += res[c];
    }
#pragma unroll
    for (int c = 0; c < N; ++c)
        if (c < count && LQ_IN_BOUNDS(at + c * step, extent)) store_elem(e.o, at + c * step, e.o_bf16, z[c]);
}

}  // namespace lq
