// Arguments and pieces shared by the tensor-core products of block-128 E4M3 codes.
#pragma once

#include <atomic>

#include "fp8_block.cuh"
#include "tcgen05.cuh"

namespace moe {
namespace fp8_impl {

constexpr int kMaxSmem = 227 * 1024;  // shared memory a CTA may have
constexpr int kSmSmem = 228 * 1024;   // ... and an SM, 1 KB of it reserved per CTA
constexpr int kStaticSmem = 1536;     // an upper bound on a kernel's static shared memory and its reserve
constexpr int kMaxRowTiles = 1 << 30;

struct GemmArgs {
  const uint8_t* a;
  const float* sa;
  const uint8_t* w;
  const float* sw;
  void* out;
  int f32, M, N, K;
  int nbk, nbn;  // blocks of 128 of K and N
  // grouped by expert (offsets != nullptr): M is the list's length
  const int32_t *offsets, *pairs;
  long long a_rows;
  int E, topk, in_rows, out_rows;
  uint32_t* err;
};

// The two kernels. g.a and g.sa hold `rows` rows, grouped in list order (in_rows and
// a_rows say which rows of the caller's they are, and so which pairs are in range).
// Few rows per weight tile: weights on the tensor core's 128 lanes, rows on its columns, bn
// of them a tile (16, 32, 64; dense also 128). named: g.a and g.sa are the caller's, their
// rows to be fetched as the pairs name them.
int launch_narrow(const GemmArgs& g, long long rows, bool named, int bn, int sm_count, cudaStream_t stream);
// CTAs that a dense narrow product of `tiles` tiles of bn (64 or 128) rows puts to work on each.
int narrow_splits(int bn, long long tiles, int nbk, int sm_count);
// Many: rows on the lanes, weights on the columns, two SMs per tile.
int launch_wide(const GemmArgs& g, long long rows, int sm_count, cudaStream_t stream);

// A kernel's shared-memory limit and carveout, set at its first launch on a device (two
// driver calls less on the later ones).
struct OncePerDevice {
  std::atomic<uint64_t> done{0};
  bool allow(const void* kernel, int bytes) {
    int dev = -1;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev > 63) return false;
    if (done.load(std::memory_order_acquire) >> dev & 1) return true;
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) != cudaSuccess ||
        prefer_max_shared(kernel) != MOE_OK)
      return false;
    done.fetch_or(1ull << dev, std::memory_order_release);
    return true;
  }
};

// A K-major byte matrix [rows, cols] for TMA: boxes of 128 columns x box_rows rows,
// 128-byte swizzle, zeros outside.
inline bool make_code_map(CUtensorMap* m, const void* ptr, long long rows, int cols, int box_rows) {
  auto fn = encode_fn();
  if (!fn) return false;
  cuuint64_t dims[2] = {(cuuint64_t)cols, (cuuint64_t)rows};
  cuuint64_t strides[1] = {(cuuint64_t)cols};
  cuuint32_t box[2] = {(cuuint32_t)FP8_BLOCK, (cuuint32_t)box_rows};
  cuuint32_t estr[2] = {1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(ptr), dims, strides, box, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// E4M3 x E4M3 -> FP32, both K-major, M = m, N = n.
__host__ __device__ constexpr uint32_t instr_desc_e4m3(int n, int m) {
  return (1u << 4) | ((uint32_t)(n >> 3) << 17) | ((uint32_t)(m >> 4) << 24);
}

__device__ __forceinline__ void mma_e4m3(uint32_t tmem_d, uint64_t adesc, uint64_t bdesc, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n}\n" ::"r"(tmem_d),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(acc));
}

__device__ __forceinline__ int clamp_offset(int v, int n) { return min(max(v, 0), n); }

// The row of a, and of out, of list position i with pair code p; both -1 (with the error
// bit) for a pair or a row out of range.
__device__ __forceinline__ void code_rows(const GemmArgs& g, int i, int p, long long* in, long long* out) {
  const long long r = g.in_rows == MOE_ROWS_TOKEN ? p / g.topk : (g.in_rows == MOE_ROWS_LIST ? i : p);
  const bool ok = p >= 0 && p < g.M && r < g.a_rows;
  if (!ok) set_error(g.err, MOE_DEVERR_ROW_INDEX);
  *in = ok ? r : -1;
  *out = ok ? (g.out_rows == MOE_ROWS_LIST ? i : p) : -1;
}
__device__ __forceinline__ void pair_rows(const GemmArgs& g, int i, long long* in, long long* out) {
  code_rows(g, i, __ldg(g.pairs + i), in, out);
}

// Exclusive prefix sum of the experts' tile counts, ceil(rows / tile) each, to
// table[0 .. E] (shared memory); by the whole CTA. Sums stop at kMaxRowTiles: lists that
// overlap (offsets that do not ascend) may add up to more tiles than there are rows.
__device__ __forceinline__ void tile_table(const GemmArgs& g, int tile, int* table, int* warp_sums) {
  const int nt = blockDim.x, per = (g.E + nt - 1) / nt, e0 = threadIdx.x * per, e1 = min(e0 + per, g.E);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  auto add = [](int a, int b) { return (int)min((uint32_t)a + (uint32_t)b, (uint32_t)kMaxRowTiles); };
  int n = 0;
  for (int e = e0; e < e1; ++e) {
    const int rows = clamp_offset(__ldg(g.offsets + e + 1), g.M) - clamp_offset(__ldg(g.offsets + e), g.M);
    const int c = rows > 0 ? (rows - 1) / tile + 1 : 0;
    table[e] = c;
    n = add(n, c);
  }
  int incl = n;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(kFullMask, incl, o);
    if (lane >= o) incl = add(incl, y);
  }
  if (lane == 31) warp_sums[warp] = incl;
  const int below = __shfl_up_sync(kFullMask, incl, 1);  // (not incl - n: the sums may be capped)
  __syncthreads();
  int base = lane > 0 ? below : 0;
  for (int w = 0; w < warp; ++w) base = add(base, warp_sums[w]);
  for (int e = e0; e < e1; ++e) {
    const int c = table[e];
    table[e] = base;
    base = add(base, c);
  }
  if (e0 < g.E && e1 == g.E) table[g.E] = base;
  __syncthreads();
}

// The expert of tile q: table[e] <= q < table[e + 1].
__device__ __forceinline__ int tile_expert(const int* table, int E, int q) {
  int lo = 0, hi = E;  // table[lo] <= q < table[hi]
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (table[mid] <= q)
      lo = mid;
    else
      hi = mid;
  }
  return lo;
}

}  // namespace fp8_impl
}  // namespace moe
