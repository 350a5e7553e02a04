// W8A8 product with bias, activation and residual in its epilogue
// (dq_w8a8_linear).
#include "dq.h"
#include "dq_launch.cuh"
#include "w8a8_epilogue.cuh"

namespace dq {

// Any shape and alignment: one output per thread, integer dot product on CUDA
// cores.
template <int ACT>
__global__ void __launch_bounds__(256) w8a8_linear_generic_kernel(const LinearArgs a) {
  pdl_launch_dependents();
  pdl_wait_primary();
  const int64_t total = a.m * a.n;
  for (int64_t e = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x; e < total;
       e += static_cast<int64_t>(gridDim.x) * blockDim.x) {
    const int64_t i = e / a.n, j = e - i * a.n;
    const int8_t* ar = a.a + i * a.k;
    const int8_t* br = a.b + j * a.k;
    int acc = 0;
    for (int64_t kk = 0; kk < a.k; ++kk) acc += static_cast<int>(ar[kk]) * static_cast<int>(br[kk]);
    const bool has_bias = a.bias != nullptr;
    float t = linear_value<ACT>(acc, a.a_scale[i], a.b_scale[j], has_bias ? load_param(a.bias, a.bias_dtype, j) : 0.0f,
                                has_bias);
    if (a.residual != nullptr) t = __fadd_rn(t, load_out(a.residual, a.out_kind, e));
    store_one(a.out, a.out_kind, e, t);
  }
}

}  // namespace dq

namespace {

using dq_host::aligned;

template <int ACT>
dq_status launch_generic(const dq::LinearArgs& a, cudaStream_t stream) {
  void (*fn)(const dq::LinearArgs) = dq::w8a8_linear_generic_kernel<ACT>;
  const int64_t want = (a.m * a.n + 255) / 256;
  const int64_t most = static_cast<int64_t>(dq_host::sm_count(dq_host::current_device())) * 64;
  return dq_host::launch_programmatic(fn, a, static_cast<int>(want < most ? want : most), 256, 0, stream);
}

template <int ACT>
dq_status dispatch(const dq::LinearArgs& a, cudaStream_t stream) {
  return launch_generic<ACT>(a, stream);
}

}  // namespace

extern "C" dq_status dq_w8a8_linear(const int8_t* a, const int8_t* b, int64_t m, int64_t n, int64_t k,
                                    const float* a_scale, const float* b_scale, const void* bias, dq_dtype bias_dtype,
                                    dq_activation activation, const void* residual, void* out, dq_dtype out_dtype,
                                    cudaStream_t stream) {
  // k < 2^17: |sum| <= k * 128 * 128 < 2^31 for any int8 codes (-128 included)
  if (m < 0 || n < 0 || k < 1 || k >= (int64_t(1) << 17) || m > (int64_t(1) << 31) || n > (int64_t(1) << 31))
    return DQ_ERR_BAD_SHAPE;
  const auto is_float = [](dq_dtype t) { return t == DQ_F32 || t == DQ_F16 || t == DQ_BF16; };
  if (!is_float(out_dtype) || (bias != nullptr && !is_float(bias_dtype))) return DQ_ERR_BAD_DTYPE;
  if (activation < DQ_ACT_NONE || activation > DQ_ACT_SILU) return DQ_ERR_BAD_ARGUMENT;
  if (m == 0 || n == 0) return DQ_OK;
  if (a == nullptr || b == nullptr || a_scale == nullptr || b_scale == nullptr || out == nullptr)
    return DQ_ERR_NULL_POINTER;
  const size_t os = out_dtype == DQ_F32 ? 4 : 2;
  if (!aligned(a_scale, 4) || !aligned(b_scale, 4) || !aligned(out, os) || (residual && !aligned(residual, os)) ||
      (bias && !aligned(bias, bias_dtype == DQ_F32 ? 4 : 2)))
    return DQ_ERR_MISALIGNED;
  dq::LinearArgs args{};
  args.a = a;
  args.b = b;
  args.a_scale = a_scale;
  args.b_scale = b_scale;
  args.bias = bias;
  args.residual = residual;
  args.out = out;
  args.m = m;
  args.n = n;
  args.k = k;
  args.bias_dtype = static_cast<int>(bias_dtype);
  args.out_kind = out_dtype == DQ_F32 ? dq::kOutF32 : (out_dtype == DQ_F16 ? dq::kOutF16 : dq::kOutBF16);
  args.vec_out = aligned(out, 16) && (residual == nullptr || aligned(residual, 16)) &&
                 (n * static_cast<int64_t>(os)) % 16 == 0;
  switch (activation) {
    case DQ_ACT_RELU: return dispatch<DQ_ACT_RELU>(args, stream);
    case DQ_ACT_GELU: return dispatch<DQ_ACT_GELU>(args, stream);
    case DQ_ACT_GELU_TANH: return dispatch<DQ_ACT_GELU_TANH>(args, stream);
    case DQ_ACT_SILU: return dispatch<DQ_ACT_SILU>(args, stream);
    default: return dispatch<DQ_ACT_NONE>(args, stream);
  }
}
