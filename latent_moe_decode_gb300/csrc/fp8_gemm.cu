// Matrix product of E4M3 codes with a scale for each block of 128, dense and grouped by
// expert:
//   out[m, n] = sum_b sa[m, b] * sw[n / 128, b] * sum_{k in b} a[m, k] * w[n, k]
//
// CUDA-core form: 64 x 64 outputs per CTA, the codes of 32 columns at a time decoded to
// FP32 in shared memory, a block's 128 products summed before its scale is applied.
#include "fp8_block.cuh"

namespace moe {
namespace {

constexpr int kTile = 64, kCols = 32, kThreads = 256;

struct GemmArgs {
  const uint8_t* a;
  const float* sa;
  const uint8_t* w;
  const float* sw;
  void* out;
  int f32, M, N, K, nbk, nbn;
  // grouped (offsets != nullptr): E experts, M = the list's length
  const int32_t *offsets, *pairs;
  long long a_rows;
  int E, topk, in_rows, out_rows;
  uint32_t* err;
};

__device__ __forceinline__ float e4m3_value(uint32_t c) {
  uint32_t h;  // two FP16 values
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)c));
  float f;
  asm("{\n .reg .b16 l, u;\n mov.b32 {l, u}, %1;\n cvt.f32.f16 %0, l;\n}\n" : "=f"(f) : "r"(h));
  return f;
}

__device__ __forceinline__ int clamp_offset(int v, int n) { return min(max(v, 0), n); }

// Row tile `t` of the grouped product: its expert and first list position, by a scan
// over the experts' tile counts. False past the last.
__device__ bool find_tile(const GemmArgs& a, int t, int* expert, int* pos, int* end) {
  __shared__ int part[kThreads], found[3];
  const int per = (a.E + kThreads - 1) / kThreads, e0 = threadIdx.x * per, e1 = min(e0 + per, a.E);
  int n = 0;
  for (int e = e0; e < e1; ++e)
    n += (max(clamp_offset(a.offsets[e + 1], a.M) - clamp_offset(a.offsets[e], a.M), 0) + kTile - 1) / kTile;
  part[threadIdx.x] = n;
  if (threadIdx.x == 0) found[0] = -1;
  __syncthreads();
  int base = 0;
  for (int i = 0; i < (int)threadIdx.x; ++i) base += part[i];
  if (t >= base && t < base + n) {
    for (int e = e0; e < e1; ++e) {
      const int lo = clamp_offset(a.offsets[e], a.M), hi = clamp_offset(a.offsets[e + 1], a.M);
      const int c = (max(hi - lo, 0) + kTile - 1) / kTile;
      if (t < base + c) {
        found[0] = e, found[1] = lo + (t - base) * kTile, found[2] = hi;
        break;
      }
      base += c;
    }
  }
  __syncthreads();
  *expert = found[0], *pos = found[1], *end = found[2];
  return found[0] >= 0;
}

__global__ void __launch_bounds__(kThreads) gemm_kernel(const GemmArgs a) {
  __shared__ float as[kCols][kTile + 1], ws[kCols][kTile + 1];
  __shared__ long long in_row[kTile], out_row[kTile];
  grid_launch_dependents();
  grid_wait();
  int e = 0, pos = blockIdx.x * kTile, end = a.M;
  if (a.offsets && !find_tile(a, blockIdx.x, &e, &pos, &end)) return;
  if (threadIdx.x < kTile) {
    const int i = pos + threadIdx.x;
    long long in = -1, out = -1;
    if (i < end) {
      in = out = i;
      if (a.offsets) {
        const int p = a.pairs[i];
        in = a.in_rows == MOE_ROWS_TOKEN ? p / a.topk : (a.in_rows == MOE_ROWS_LIST ? i : p);
        out = a.out_rows == MOE_ROWS_LIST ? i : p;
        if (p < 0 || p >= a.M || in >= a.a_rows) {
          in = out = -1;
          set_error(a.err, MOE_DEVERR_ROW_INDEX);
        }
      }
    }
    in_row[threadIdx.x] = in, out_row[threadIdx.x] = out;
  }
  __syncthreads();
  const int n0 = blockIdx.y * kTile;
  const uint8_t* w = a.w + (long long)e * a.N * a.K;
  const float* sw = a.sw + (long long)e * a.nbn * a.nbk;
  const int tm = threadIdx.x >> 4, tn = threadIdx.x & 15;  // rows tm + 16 i, columns tn + 16 j
  float acc[4][4] = {}, part[4][4] = {};
  for (int k0 = 0; k0 < a.K; k0 += kCols) {
    for (int i = threadIdx.x; i < kTile * kCols; i += kThreads) {
      const int r = i / kCols, c = i % kCols;
      as[c][r] = in_row[r] >= 0 && k0 + c < a.K ? e4m3_value(a.a[in_row[r] * a.K + k0 + c]) : 0.f;
      ws[c][r] = n0 + r < a.N && k0 + c < a.K ? e4m3_value(w[(long long)(n0 + r) * a.K + k0 + c]) : 0.f;
    }
    __syncthreads();
    for (int c = 0; c < kCols; ++c)
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) part[i][j] = __fmaf_rn(as[c][tm + 16 * i], ws[c][tn + 16 * j], part[i][j]);
    __syncthreads();
    if ((k0 + kCols) % FP8_BLOCK == 0 || k0 + kCols >= a.K) {
      const int b = k0 / FP8_BLOCK;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const long long r = in_row[tm + 16 * i];
        const float s = r >= 0 ? a.sa[r * a.nbk + b] : 0.f;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int n = n0 + tn + 16 * j;
          if (n < a.N) acc[i][j] = __fmaf_rn(part[i][j], __fmul_rn(s, sw[(long long)(n / FP8_BLOCK) * a.nbk + b]), acc[i][j]);
          part[i][j] = 0.f;
        }
      }
    }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const long long r = out_row[tm + 16 * i];
    if (r < 0) continue;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int n = n0 + tn + 16 * j;
      if (n >= a.N) continue;
      if (a.f32)
        static_cast<float*>(a.out)[r * a.N + n] = acc[i][j];
      else
        static_cast<uint16_t*>(a.out)[r * a.N + n] = f32_to_bf16(acc[i][j]);
    }
  }
}

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
  a.nbk = (a.K + FP8_BLOCK - 1) / FP8_BLOCK, a.nbn = (a.N + FP8_BLOCK - 1) / FP8_BLOCK;
  DeviceInfo dev;
  int st = current_device(&dev);
  if (st != MOE_OK) return st;
  a.err = dev.error_word;
  const long long rows = ((long long)a.M + kTile - 1) / kTile + (a.offsets ? (a.E < a.M ? a.E : a.M) : 0);
  const long long cols = ((long long)a.N + kTile - 1) / kTile;
  if (cols > 65535) return MOE_ERR_CAPACITY;
  return launch_pdl(gemm_kernel, dim3((unsigned)rows, (unsigned)cols), dim3(kThreads), 0, stream, a);
}

}  // namespace
}  // namespace moe

extern "C" int fp8_block_gemm(const uint8_t* a, const float* a_scales, const uint8_t* w, const float* w_scales,
                              void* out, int out_dtype, int M, int N, int K, moe_stream_t stream) {
  using namespace moe;
  GemmArgs g = {};
  g.a = a, g.sa = a_scales, g.w = w, g.sw = w_scales, g.out = out, g.f32 = out_dtype == MOE_DTYPE_F32;
  g.M = M, g.N = N, g.K = K, g.E = 1;
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
