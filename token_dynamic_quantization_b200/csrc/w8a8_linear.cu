// W8A8 product with bias, activation and residual in its epilogue
// (dq_w8a8_linear).
#include <atomic>

#include "decoder_launch.cuh"
#include "dq.h"
#include "dq_launch.cuh"
#include "w8a8_epilogue.cuh"
#include "w8a8_linear_few.cuh"
#include "w8a8_linear_pair.cuh"
#include "w8a8_linear_split.cuh"

namespace dq {

// Any shape and alignment: one output per thread, integer dot product on CUDA
// cores, byte by byte (1 x 4096 x 1000: 52 us, 512 x 1024 x 1000: 684; with k = 1008 the
// latter takes 9 on the tensor cores).
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

constexpr int kMaxSplit = 8;  // the portable cluster size

// Clusters of 1 .. kMaxSplit CTAs of a kernel that fit the device at once (a
// cluster stays within one GPC, so it is fewer than slots / size); asked once
// per kernel and device. The answers are plain numbers that any thread would
// write alike.
template <typename Kernel>
const int* resident_clusters(Kernel kernel, int device, int block, size_t smem, std::atomic<int> (&known)[kMaxSplit + 1],
                             int (&out)[kMaxSplit + 1]) {
  for (int s = 1; s <= kMaxSplit; ++s) {
    int n = known[s].load(std::memory_order_relaxed);
    if (n == 0) {
      cudaLaunchConfig_t cfg = {};
      cfg.gridDim = dim3(static_cast<unsigned>(s) * 4096);
      cfg.blockDim = dim3(block);
      cfg.dynamicSmemBytes = smem;
      cudaLaunchAttribute attr[1];
      attr[0].id = cudaLaunchAttributeClusterDimension;
      attr[0].val.clusterDim.x = s;
      attr[0].val.clusterDim.y = 1;
      attr[0].val.clusterDim.z = 1;
      cfg.attrs = attr;
      cfg.numAttrs = 1;
      if (cudaOccupancyMaxActiveClusters(&n, kernel, &cfg) != cudaSuccess || n < 1) {
        cudaGetLastError();
        n = dq_host::sm_count(device) / s;
      }
      known[s].store(n, std::memory_order_relaxed);
    }
    out[s] = n;
  }
  return out;
}

// CTAs of a cluster among which K is split: the number whose clusters take the
// least time, in waves of resident clusters with K / split each; a larger one
// has to gain 5 %.
int best_split(int64_t tiles, int64_t pieces, const int* resident) {
  int split = 1;
  double best = 0.0;
  for (int s = 1; s <= kMaxSplit && s <= pieces; ++s) {
    const double time = static_cast<double>((tiles + resident[s] - 1) / resident[s]) *
                        (static_cast<double>((pieces + s - 1) / s) / static_cast<double>(pieces));
    if (s == 1 || time < 0.95 * best) {
      best = time;
      split = s;
    }
  }
  return split;
}

// Up to 8 tokens: a CTA for every 16 weight rows.
template <int ACT>
dq_status launch_few(const dq::LinearArgs& a, cudaStream_t stream) {
  void (*fn)(const dq::LinearArgs) = dq::w8a8_linear_few_kernel<ACT>;
  if (!dq_host::allow_smem_bytes(reinterpret_cast<const void*>(fn), dq_host::current_device(), dq::kFewSmem))
    return dq_host::kNotLaunchable;
  return dq_host::launch_programmatic(fn, a, static_cast<int>((a.n + dq::kFewRows - 1) / dq::kFewRows), dq::kFewThreads,
                                      dq::kFewSmem, stream);
}

// 9 to 128 tokens, up to TOK: tiles of 128 weight rows, K split over the CTAs of
// a cluster.
template <int ACT, int TOK>
dq_status launch_split(const dq::LinearArgs& a, cudaStream_t stream) {
  using Shape = dq::SplitShape<TOK>;
  auto fn = dq::w8a8_linear_split_kernel<ACT, TOK>;
  const int device = dq_host::current_device();
  CUtensorMap w, x;
  if (!dq_host::make_map(&w, a.b, a.n, a.k, 128) || !dq_host::make_map(&x, a.a, a.m, a.k, TOK) ||
      !dq_host::allow_smem_bytes(reinterpret_cast<const void*>(fn), device, Shape::kSmem))
    return dq_host::kNotLaunchable;
  const int64_t blocks = (a.n + 127) / 128;
  static std::atomic<int> known[dq_host::kMaxDevices][kMaxSplit + 1];
  int resident[kMaxSplit + 1];
  if (device < 0 || device >= dq_host::kMaxDevices) return dq_host::kNotLaunchable;
  const int split = best_split(blocks, (a.k + 127) / 128,
                               resident_clusters(fn, device, dq::kSplitThreads, Shape::kSmem, known[device], resident));
  return dq_host::launch_dependent(fn, dim3(static_cast<unsigned>(blocks * split)), dq::kSplitThreads, Shape::kSmem, split, stream, w,
                        x, a, split);
}

// Many tokens: one pair of CTAs for every two SMs over the list of tiles.
template <int ACT, bool TURN>
dq_status launch_pair(const dq::LinearArgs& a, cudaStream_t stream) {
  auto fn = dq::w8a8_linear_pair_kernel<ACT, TURN>;
  const int device = dq_host::current_device();
  CUtensorMap ma, mb128, mb64;
  if (!dq_host::make_map(&ma, a.a, a.m, a.k, 128) || !dq_host::make_map(&mb128, a.b, a.n, a.k, 128) ||
      !dq_host::make_map(&mb64, a.b, a.n, a.k, 64) ||
      !dq_host::allow_smem_bytes(reinterpret_cast<const void*>(fn), device, dq::PairShape<TURN>::kSmem))
    return dq_host::kNotLaunchable;
  const int64_t pairs = dq_host::sm_count(device) / 2;
  dq::PairSched ps;
  ps.n_tiles = (a.n + 255) / 256;
  const int64_t tiles = (a.m + 255) / 256 * ps.n_tiles, rest = tiles % pairs;
  const int64_t split = 2 * rest <= pairs ? rest : 0;  // halve the last ones when every half gets its own pair
  ps.wide = tiles - split;
  ps.items = tiles + split;
  const int64_t clusters = ps.items < pairs ? ps.items : pairs;
  return dq_host::launch_dependent(fn, dim3(static_cast<unsigned>(2 * clusters)), dq::kPairThreads, dq::PairShape<TURN>::kSmem, 1, stream, ma,
                        mb128, mb64, a, ps);
}

template <int ACT>
dq_status dispatch(const dq::LinearArgs& a, cudaStream_t stream) {
  // 16-byte pieces of K
  const bool pieces = a.k % 16 == 0 && aligned(a.a, 16) && aligned(a.b, 16);
  if (pieces) {
    // By the number of tokens, measured at n = k = 4096 to bf16 with bias and
    // residual: 8 tokens take 6.2 us with the first kernel and 8.2 with the second; 16
    // take 9.0 with the second and 10.6 with the first; 128 take 16.4 with the second
    // and 17.4 with the third, 200 19.3 and 17.6.
    dq_status st;
    if (a.m <= dq::kFewTokens) {
      st = launch_few<ACT>(a, stream);
    } else if (a.m <= 16) {
      st = launch_split<ACT, 16>(a, stream);
    } else if (a.m <= 32) {
      st = launch_split<ACT, 32>(a, stream);
    } else if (a.m <= 64) {
      st = launch_split<ACT, 64>(a, stream);
    } else if (a.m <= 128) {
      st = launch_split<ACT, 128>(a, stream);
    } else {
      st = a.vec_out && a.n % 32 == 0 ? launch_pair<ACT, false>(a, stream) : launch_pair<ACT, true>(a, stream);
    }
    if (st != dq_host::kNotLaunchable) return st;
  }
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
  args.pair_out = n % 2 == 0 && aligned(out, 2 * os) && (residual == nullptr || aligned(residual, 2 * os));
  switch (activation) {
    case DQ_ACT_RELU: return dispatch<DQ_ACT_RELU>(args, stream);
    case DQ_ACT_GELU: return dispatch<DQ_ACT_GELU>(args, stream);
    case DQ_ACT_GELU_TANH: return dispatch<DQ_ACT_GELU_TANH>(args, stream);
    case DQ_ACT_SILU: return dispatch<DQ_ACT_SILU>(args, stream);
    default: return dispatch<DQ_ACT_NONE>(args, stream);
  }
}
