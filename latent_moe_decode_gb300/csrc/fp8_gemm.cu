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

// The kernel: 0 for the wide one, else the narrow one's rows a tile.
// Grouped, by the lists' average length, for tiles that hold all but the fullest lists. Times
// in us of 256 experts of 1024 x 1024 / 64 of 4096 x 3584, the rows copied first from 32 on:
//   average    16 rows     32 rows     64 rows      wide
//         8    46 / 145    47 / 146    58 / 153    78 / 188
//        16    54 / 154    53 / 155    63 / 156    82 / 190
//        32    78 / 218    61 / 164    72 / 160    89 / 192
//        48   104 / 307    76 / 198    85 / 172    88 / 194
//        64   131 / 395    94 / 246    99 / 184    91 / 196
//        80   159 / 479   110 / 288   113 / 208    94 / 198
// Dense, up to 64 rows: the narrowest tile that holds them. Above, whatever is estimated to
// end first, in ns for w tiles one after the other (per SM, for the wide kernel per pair) of b
// blocks each (of its split): wide 2700 + w (2250 + 350 b); 64 rows 5200 + w (2000 + 225 b),
// split 7300 + 440 b; 128 rows w (5400 + 305 b), split 6700 + 360 b. (Fitted to 70 sizes, M
// 128 to 2304, N 576 to 7168, K 400 to 7168, within 15 % of most; us wide / 64 / 128: 1024 x
// 1024 x 400 6.5 / 9.0 / 8.3, x 3584 14.4 / 13.7 / 11.9; 2304 x 2304 x 1296 15.3 / 26.6 /
// 27.5. Splitting K over pairs of a wide tile, too, measured slower: 15 us for 128 x 7168 x
// 3584, 29 for 333 x 2016 x 7184, the sum of 128 KB of partials a CTA and clusters of four or
// eight whole SMs costing more than the blocks saved.)
int choose_listed(int n_pairs, int E) {
  if (n_pairs > 72LL * E) return 0;
  return n_pairs > 40LL * E ? 64 : n_pairs > 10LL * E ? 32 : 16;
}
int choose(const GemmArgs& a, int sm_count) {
  if (a.offsets) return choose_listed(a.M, a.E);
  if (a.M <= 64) return a.M <= 16 ? 16 : a.M <= 32 ? 32 : 64;
  const long long M = a.M, tiles0 = ((M - 1) / 256 + 1) * ((a.nbn + 1) / 2), pairs = sm_count / 2;
  const long long w0 = (tiles0 - 1) / pairs + 1, ns0 = 2700 + w0 * (2250 + a.nbk * 350);
  const long long tiles64 = ((M - 1) / 64 + 1) * a.nbn, tiles128 = ((M - 1) / 128 + 1) * a.nbn;
  const int s64 = fp8_impl::narrow_splits(64, tiles64, a.nbk, sm_count), s128 = fp8_impl::narrow_splits(128, tiles128, a.nbk, sm_count);
  const long long w64 = (tiles64 - 1) / sm_count + 1, w128 = (tiles128 - 1) / sm_count + 1;
  const long long ns64 = s64 > 1 ? 7300 + ((a.nbk - 1) / s64 + 1) * 440 : 5200 + w64 * (2000 + a.nbk * 225);
  const long long ns128 = s128 > 1 ? 6700 + ((a.nbk - 1) / s128 + 1) * 360 : w128 * (5400 + a.nbk * 305);
  if (ns0 <= ns64 && ns0 <= ns128) return 0;
  return ns64 <= ns128 ? 64 : 128;
}

size_t align256(size_t n) { return (n + 255) / 256 * 256; }

// Whether rows that do not lie in list order are copied there before the product: always for
// the wide kernel, which reads boxes of them. The narrow one has a warp that looks up a tile's
// rows and fetches them singly, at 16 a tile as fast as HBM brings the weights. At 32 that
// costs more than the copies' launch from some hundred fetches an SM on (64 experts of 32 rows,
// N = 1280, K = 512, 20480 fetches: 25.6 us, 21.6 with the copies; of 16 rows, 10240 fetches:
// 34 and 38 at K = 2048); at 64, always (48 rows of 256 experts: 129 and 85; of 32: 24 and 25).
bool copies(int n_pairs, int E, int N, int in_rows) {
  const int bn = choose_listed(n_pairs, E);
  return in_rows != MOE_ROWS_LIST && (bn == 0 || bn == 64 || (bn == 32 && (long long)n_pairs * ((N - 1) / FP8_BLOCK + 1) > 16000));
}

// Copies of the listed pairs' rows and scales in list order.
size_t list_copy_bytes(int n_pairs, int K) {
  return align256((size_t)n_pairs * K) + align256((size_t)n_pairs * ((K - 1) / FP8_BLOCK + 1) * sizeof(float));
}

constexpr int kCopyThreads = 256;
constexpr int kMaxPairs = 0x7FFFFFFF - (1 << 16);  // (loops and tiles step past the end)

// Whether a list holds position i (by a warp); -1: neither it nor any later one.
__device__ __forceinline__ int listed(const int32_t* offsets, int E, int i) {
  int end = 0;
  bool in = false;
  for (int e = threadIdx.x & 31; e < E; e += 32) {
    const int lo = __ldg(offsets + e), hi = __ldg(offsets + e + 1);
    if (lo < hi) end = max(end, hi);
    in |= lo <= i && i < hi;
  }
  if (i >= __reduce_max_sync(fp8_impl::kFullMask, end)) return -1;
  return __any_sync(fp8_impl::kFullMask, in);
}

// One warp per list position: K bytes of codes in 16-byte pieces, and the row's scales.
// (Bound by the copies' bytes; a token's row is read topk times, from L2.)
// Offsets that ascend put the positions from the first to the last of them in lists, and no
// others; the lists that hold others than these are looked for. (Six CTAs an SM: the lookup would
// take 8 more registers and so one CTA, 75.8 us for 75.3 of a call of 1500 tokens x 16 of 896.)
__global__ void __launch_bounds__(kCopyThreads, 6) list_copy_kernel(const GemmArgs g, uint8_t* __restrict__ a,
                                                                    float* __restrict__ sa) {
  grid_launch_dependents();
  grid_wait();
  const int lane = threadIdx.x & 31, warps = gridDim.x * (kCopyThreads / 32);
  const int first = __ldg(g.offsets), last = __ldg(g.offsets + g.E);
  for (int i = (blockIdx.x * kCopyThreads + threadIdx.x) >> 5; i < g.M; i += warps) {
    if (i < first || i >= last) {
      const int in = listed(g.offsets, g.E, i);
      if (in < 0) break;
      if (in == 0) continue;
    }
    long long in, out;
    fp8_impl::pair_rows(g, i, &in, &out);
    if (in < 0) continue;  // (its product is not stored)
    const uint4* src = reinterpret_cast<const uint4*>(g.a + in * g.K);
    uint4* dst = reinterpret_cast<uint4*>(a + (long long)i * g.K);
    for (int c = lane; c < g.K / 16; c += 32 * 4) {
      uint4 v[4];
#pragma unroll
      for (int u = 0; u < 4; ++u)
        if (c + 32 * u < g.K / 16) v[u] = __ldg(src + c + 32 * u);
#pragma unroll
      for (int u = 0; u < 4; ++u)
        if (c + 32 * u < g.K / 16) dst[c + 32 * u] = v[u];
    }
    for (int b = lane; b < g.nbk; b += 32) sa[(long long)i * g.nbk + b] = __ldg(g.sa + in * g.nbk + b);
  }
}

int launch(GemmArgs& a, void* workspace, cudaStream_t stream) {
  if ((long long)a.E * a.N > 0x7FFFFFFFLL - 128 || a.a_rows > 0x7FFFFFFFLL) return MOE_ERR_CAPACITY;  // (TMA coordinates)
  a.nbk = (a.K - 1) / FP8_BLOCK + 1, a.nbn = (a.N - 1) / FP8_BLOCK + 1;
  DeviceInfo dev;
  int st = current_device(&dev);
  if (st != MOE_OK) return st;
  a.err = dev.error_word;
  long long rows = a.a_rows;
  const int bn = choose(a, dev.sm_count);
  bool named = a.offsets && a.in_rows != MOE_ROWS_LIST;
  if (a.offsets && copies(a.M, a.E, a.N, a.in_rows)) {
    uint8_t* copy = static_cast<uint8_t*>(workspace);
    float* scales = reinterpret_cast<float*>(copy + align256((size_t)a.M * a.K));
    const long long need = ((long long)a.M * 32 + kCopyThreads - 1) / kCopyThreads, most = 8LL * dev.sm_count;
    st = launch_pdl(list_copy_kernel, dim3((unsigned)(need < most ? need : most)), dim3(kCopyThreads), 0, stream, a, copy, scales);
    if (st != MOE_OK) return st;
    a.a = copy, a.sa = scales, rows = a.M, named = false;
  }
  return bn == 0 ? fp8_impl::launch_wide(a, rows, dev.sm_count, stream) : fp8_impl::launch_narrow(a, rows, named, bn, dev.sm_count, stream);
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
  return launch(g, nullptr, as_cuda(stream));
}

extern "C" size_t moe_expert_gemm_workspace(int n_pairs, int E, int N, int K, int in_rows) {
  if (n_pairs < 1 || E < 1 || N < 1 || K < 16 || !moe::copies(n_pairs, E, N, in_rows)) return 0;
  return moe::list_copy_bytes(n_pairs, K);
}

extern "C" int moe_expert_gemm(const uint8_t* a, const float* a_scales, int64_t a_rows, const uint8_t* w,
                               const float* w_scales, const int32_t* offsets, const int32_t* pairs, int n_pairs,
                               int topk, int in_rows, int out_rows, void* out, int out_dtype, int E, int N, int K,
                               void* workspace, size_t workspace_bytes, moe_stream_t stream) {
  using namespace moe;
  GemmArgs g = {};
  g.a = a, g.sa = a_scales, g.w = w, g.sw = w_scales, g.out = out, g.f32 = out_dtype == MOE_DTYPE_F32;
  g.M = n_pairs, g.N = N, g.K = K, g.E = E;
  g.offsets = offsets, g.pairs = pairs, g.a_rows = a_rows, g.topk = topk, g.in_rows = in_rows, g.out_rows = out_rows;
  if (E < 1 || topk < 1 || a_rows < 0 || (a_rows == 0 && n_pairs != 0)) return MOE_ERR_INVALID_ARGUMENT;
  if (in_rows != MOE_ROWS_TOKEN && in_rows != MOE_ROWS_LIST && in_rows != MOE_ROWS_PAIR) return MOE_ERR_INVALID_ARGUMENT;
  if (out_rows != MOE_ROWS_LIST && out_rows != MOE_ROWS_PAIR) return MOE_ERR_INVALID_ARGUMENT;
  const int st = check(g, out_dtype);
  if (st != MOE_OK || n_pairs == 0 || N == 0) return st;
  if (!offsets || !pairs) return MOE_ERR_INVALID_ARGUMENT;
  if (E > MOE_MAX_EXPERTS || n_pairs > kMaxPairs) return MOE_ERR_CAPACITY;
  if (!aligned(offsets, 4) || !aligned(pairs, 4) || !aligned(workspace, 16)) return MOE_ERR_ALIGNMENT;
  const size_t need = moe_expert_gemm_workspace(n_pairs, E, N, K, in_rows);
  if (need > 0 && (!workspace || workspace_bytes < need)) return MOE_ERR_WORKSPACE;
  return launch(g, workspace, as_cuda(stream));
}
