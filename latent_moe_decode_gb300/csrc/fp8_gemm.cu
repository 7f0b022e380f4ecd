// Matrix product of E4M3 codes with a scale for each block of 128, dense and grouped by
// expert: argument checks and the choice of kernel.
//   out[m, n] = sum_b sa[m, b] * sw[n / 128, b] * sum_{k in b} a[m, k] * w[n, k]
#include "fp8_gemm.cuh"

namespace moe {
namespace {

using fp8_impl::GemmArgs;

int check(const GemmArgs& a, int out_dtype) {
  if (a.M < 0 || a.N < 0 || a.K < 16 || a.K % 16 != 0) return MOE_ERR_INVALID_ARGUMENT;
  if (out_dtype != MOE_DTYPE_F32 && out_dtype != MOE_DTYPE_BF16) return MOE_ERR_INVALID_ARGUMENT;
  if (a.M == 0 || a.N == 0) return MOE_OK;
  if (!a.a || !a.sa || !a.w || !a.sw || !a.out) return MOE_ERR_INVALID_ARGUMENT;
  if (!aligned(a.a, 16) || !aligned(a.w, 16) || !aligned(a.sa, 4) || !aligned(a.sw, 4) || !aligned(a.out, a.f32 ? 4 : 2))
    return MOE_ERR_ALIGNMENT;
  return MOE_OK;
}

int launch(GemmArgs& a, cudaStream_t stream) {
  if ((long long)a.E * a.N > 0x7FFFFFFFLL - 128 || a.a_rows > 0x7FFFFFFFLL) return MOE_ERR_CAPACITY;  // (TMA coordinates)
  a.nbk = (a.K - 1) / FP8_BLOCK + 1, a.nbn = (a.N - 1) / FP8_BLOCK + 1;
  DeviceInfo dev;
  int st = current_device(&dev);
  if (st != MOE_OK) return st;
  a.err = dev.error_word;
  const bool wide = a.offsets ? (long long)a.M >= 96LL * a.E : a.M >= 256;
  return wide ? fp8_impl::launch_wide(a, dev.sm_count, stream) : fp8_impl::launch_narrow(a, dev.sm_count, stream);
}

}  // namespace
}  // namespace moe

extern "C" int fp8_block_gemm(const uint8_t* a, const float* a_scales, const uint8_t* w, const float* w_scales,
                              void* out, int out_dtype, int M, int N, int K, moe_stream_t stream) {
  using namespace moe;
  GemmArgs g = {};
  g.a = a, g.sa = a_scales, g.w = w, g.sw = w_scales, g.out = out, g.f32 = out_dtype == MOE_DTYPE_F32;
  g.M = M, g.N = N, g.K = K, g.E = 1, g.a_rows = M;
  const int st = check(g, out_dtype);
  if (st != MOE_OK || M == 0 || N == 0) return st;
  return launch(g, as_cuda(stream));
}

extern "C" int moe_expert_gemm(const uint8_t* a, const float* a_scales, int64_t a_rows, const uint8_t* w,
                               const float* w_scales, const int32_t* offsets, const int32_t* pairs, int n_pairs,
                               int topk, int in_rows, int out_rows, void* out, int out_dtype, int E, int N, int K,
                               moe_stream_t stream) {
  using namespace moe;
  GemmArgs g = {};
  g.a = a, g.sa = a_scales, g.w = w, g.sw = w_scales, g.out = out, g.f32 = out_dtype == MOE_DTYPE_F32;
  g.M = n_pairs, g.N = N, g.K = K, g.E = E;
  g.offsets = offsets, g.pairs = pairs, g.a_rows = a_rows, g.topk = topk, g.in_rows = in_rows, g.out_rows = out_rows;
  if (E < 1 || topk < 1 || a_rows < 1) return MOE_ERR_INVALID_ARGUMENT;
  if (in_rows != MOE_ROWS_TOKEN && in_rows != MOE_ROWS_LIST && in_rows != MOE_ROWS_PAIR) return MOE_ERR_INVALID_ARGUMENT;
  if (out_rows != MOE_ROWS_LIST && out_rows != MOE_ROWS_PAIR) return MOE_ERR_INVALID_ARGUMENT;
  const int st = check(g, out_dtype);
  if (st != MOE_OK || n_pairs == 0 || N == 0) return st;
  if (!offsets || !pairs) return MOE_ERR_INVALID_ARGUMENT;
  if (E > MOE_MAX_EXPERTS) return MOE_ERR_CAPACITY;
  if (!aligned(offsets, 4) || !aligned(pairs, 4)) return MOE_ERR_ALIGNMENT;
  return launch(g, as_cuda(stream));
}
