// The arithmetic of dq_w8a8_linear after its integer sum, shared by its kernels.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <stdint.h>

#include "dq.h"
#include "dq_device.cuh"

namespace dq {

struct LinearArgs {
  const int8_t* a;
  const int8_t* b;
  const float* a_scale;
  const float* b_scale;
  const void* bias;      // [n] of bias_dtype, or nullptr
  const void* residual;  // [m, n] of the output type, or nullptr (may be `out`)
  void* out;
  int64_t m, n, k;
  int bias_dtype;
  int out_kind;  // kOutF32 / kOutF16 / kOutBF16
  int vec_out;   // rows of out (and residual) start 16-byte aligned
};

// exp(-u) by the hardware's base-2 exponential: a few 2^-22 relative for the
// |u| that leave a trace in the result, far below the 16-bit outputs' rounding.
template <int ACT>
__device__ __forceinline__ float activate(float x) {
  if (ACT == DQ_ACT_RELU) return x < 0.0f ? 0.0f : x;
  if (ACT == DQ_ACT_GELU) return 0.5f * x * erfcf(-0.70710678118654752f * x);  // 1 + erf(z) = erfc(-z), no cancellation
  if (ACT == DQ_ACT_GELU_TANH) {
    // 0.5 (1 + tanh u) = 1 / (1 + exp(-2u))
    const float u = 1.5957691216057308f * fmaf(0.044715f * x * x, x, x);
    return __fdiv_rn(x, 1.0f + __expf(-u));
  }
  if (ACT == DQ_ACT_SILU) return __fdiv_rn(x, 1.0f + __expf(-x));
  return x;
}

// float(acc) * (a_scale * b_scale) + bias, then the activation.
template <int ACT>
__device__ __forceinline__ float linear_value(int acc, float sa, float sb, float bias, bool has_bias) {
  float t = __fmul_rn(__int2float_rn(acc), __fmul_rn(sa, sb));
  if (has_bias) t = __fadd_rn(t, bias);
  return activate<ACT>(t);
}

__device__ __forceinline__ float load_out(const void* p, int kind, int64_t e) {
  if (kind == kOutF32) return static_cast<const float*>(p)[e];
  if (kind == kOutF16) return __half2float(static_cast<const __half*>(p)[e]);
  return __bfloat162float(static_cast<const __nv_bfloat16*>(p)[e]);
}

__device__ __forceinline__ void store_one(void* p, int kind, int64_t e, float t) {
  if (kind == kOutF32) {
    static_cast<float*>(p)[e] = t;
  } else if (kind == kOutF16) {
    static_cast<__half*>(p)[e] = __float2half_rn(t);
  } else {
    static_cast<__nv_bfloat16*>(p)[e] = __float2bfloat16_rn(t);
  }
}

}  // namespace dq
