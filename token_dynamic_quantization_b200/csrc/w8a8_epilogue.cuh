// The arithmetic of dq_w8a8_linear after its integer sum, shared by its kernels.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <stdint.h>

#include "decoder_device.cuh"
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
  int pair_out;  // two neighbouring even columns lie in one aligned access, in every row
};

// The activations at a cost that the epilogue hides: on 4096^3 with bias and
// residual 128 values per thread and tile share the issue slots of 16384
// tensor-core cycles. The argument of an exponential is rounded, which costs |u| 2^-24 of
// the result (GELU: x^2 2^-24): next to zero a few units in the last place of
// binary32, 17 at GELU(-6) and 63 at GELU(-12). A quotient whose denominator passes 2^126
// is zero (SILU from -87.3 on, whose value there is 2^-119).
//   GELU  x Phi(x). With z = |x| / sqrt 2 and t = 1 / (1 + z / 2),
//         erfc(z) / 2 = t 2^(-z^2 log2(e) + Q(t)); Q is a degree-9 minimax fit of
//         log2(erfcx(z) / (2 t)) on 0 <= z <= 10.5 (within 1.8e-7; beyond, the
//         result has underflowed), so negative tails keep their relative accuracy.
//   GELU_TANH, SILU  x / (1 + exp(-u)) with u = 2 sqrt(2/pi) (x + 0.044715 x^3), or x.
template <int ACT>
__device__ __forceinline__ float activate(float x) {
  if (ACT == DQ_ACT_RELU) return x < 0.0f ? 0.0f : x;
  if (ACT == DQ_ACT_GELU) {
    const float t = rcp_approx(fmaf(fabsf(x), 0.35355339f, 1.0f));
    float q = 0.21028874814510345f;
    q = fmaf(q, t, -0.989096999168396f);
    q = fmaf(q, t, 1.6859502792358398f);
    q = fmaf(q, t, -1.0288206338882446f);
    q = fmaf(q, t, -0.09418636560440063f);
    q = fmaf(q, t, -0.010599673725664616f);
    q = fmaf(q, t, 0.05451582372188568f);
    q = fmaf(q, t, 0.5567557215690613f);
    q = fmaf(q, t, 1.440855860710144f);
    q = fmaf(q, t, -2.825662612915039f);
    const float h = t * exp2_approx(fmaf(x * x, -0.72134752f, q));  // Phi(-|x|)
    return x * (x < 0.0f ? h : 1.0f - h);
  }
  if (ACT == DQ_ACT_GELU_TANH)
    return __fdividef(x, 1.0f + exp2_approx(x * fmaf(x * x, -0.10294324f, -2.3022082f)));  // -u log2(e)
  if (ACT == DQ_ACT_SILU) return __fdividef(x, 1.0f + exp2_approx(-1.44269504f * x));
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

// Two 16-bit outputs in a word.
__device__ __forceinline__ float2 unpack2(uint32_t w, int kind) {
  if (kind == kOutF16) return __half22float2(*reinterpret_cast<const __half2*>(&w));
  return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
}
__device__ __forceinline__ uint32_t pack2(float x, float y, int kind) {
  if (kind == kOutF16) {
    const __half2 h = __floats2half2_rn(x, y);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
  const __nv_bfloat162 h = __floats2bfloat162_rn(x, y);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// Four neighbouring output columns from n on: what they need of the weights'
// side, held in registers from before the sum is ready.
struct Columns {
  int64_t n;
  int count;  // columns that exist
  bool whole;  // one access per row serves all four
  bool has_bias;
  float scale[4], bias[4];

  __device__ __forceinline__ Columns(const LinearArgs& a, int64_t first) : n(first) {
    count = first >= a.n ? 0 : (first + 4 <= a.n ? 4 : static_cast<int>(a.n - first));
    whole = count == 4 && a.vec_out;
    has_bias = a.bias != nullptr;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      scale[i] = i < count ? a.b_scale[n + i] : 0.0f;
      bias[i] = i < count && has_bias ? load_param(a.bias, a.bias_dtype, n + i) : 0.0f;
    }
  }

  // The residual of row m as it lies in memory, for finish(): nothing here waits
  // for the load.
  __device__ __forceinline__ uint4 residual(const LinearArgs& a, int64_t m) const {
    uint4 r = make_uint4(0u, 0u, 0u, 0u);
    if (a.residual == nullptr || count == 0) return r;
    const int64_t e = m * a.n + n;
    if (a.out_kind == kOutF32) {
      const uint32_t* p = static_cast<const uint32_t*>(a.residual) + e;
      if (whole) return *reinterpret_cast<const uint4*>(p);
      r.x = p[0];
      if (count > 1) r.y = p[1];
      if (count > 2) r.z = p[2];
      if (count > 3) r.w = p[3];
      return r;
    }
    const uint16_t* p = static_cast<const uint16_t*>(a.residual) + e;
    if (whole) {
      const uint2 w = *reinterpret_cast<const uint2*>(p);
      return make_uint4(w.x, w.y, 0u, 0u);
    }
    r.x = p[0];
    if (count > 1) r.y = p[1];
    if (count > 2) r.z = p[2];
    if (count > 3) r.w = p[3];
    return r;
  }
  __device__ __forceinline__ float4 widen(const LinearArgs& a, uint4 r) const {
    if (a.out_kind == kOutF32)
      return make_float4(__uint_as_float(r.x), __uint_as_float(r.y), __uint_as_float(r.z), __uint_as_float(r.w));
    const float2 x = unpack2(whole ? r.x : r.x | r.y << 16, a.out_kind), y = unpack2(whole ? r.y : r.z | r.w << 16, a.out_kind);
    return make_float4(x.x, x.y, y.x, y.y);
  }

  // Row m's outputs. `broken`: the sum is incomplete (a bounded wait ran out), NaN
  // marks it.
  template <int ACT>
  __device__ __forceinline__ void finish(const LinearArgs& a, int64_t m, float sa, int4 sum, uint4 raw, bool broken) const {
    if (count == 0) return;
    float x[4] = {linear_value<ACT>(sum.x, sa, scale[0], bias[0], has_bias), linear_value<ACT>(sum.y, sa, scale[1], bias[1], has_bias),
                  linear_value<ACT>(sum.z, sa, scale[2], bias[2], has_bias), linear_value<ACT>(sum.w, sa, scale[3], bias[3], has_bias)};
    if (a.residual != nullptr) {
      const float4 res = widen(a, raw);
      x[0] = __fadd_rn(x[0], res.x), x[1] = __fadd_rn(x[1], res.y), x[2] = __fadd_rn(x[2], res.z), x[3] = __fadd_rn(x[3], res.w);
    }
    if (broken) x[0] = x[1] = x[2] = x[3] = __int_as_float(0x7fc00000);
    const int64_t e = m * a.n + n;
    if (!whole) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (i < count) store_one(a.out, a.out_kind, e + i, x[i]);
      }
    } else if (a.out_kind == kOutF32) {
      *reinterpret_cast<float4*>(static_cast<float*>(a.out) + e) = make_float4(x[0], x[1], x[2], x[3]);
    } else {
      *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.out) + e) =
          make_uint2(pack2(x[0], x[1], a.out_kind), pack2(x[2], x[3], a.out_kind));
    }
  }
};

}  // namespace dq
