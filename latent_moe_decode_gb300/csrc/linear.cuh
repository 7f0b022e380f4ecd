// Arguments and pieces shared by the BF16 products with an epilogue.
#pragma once

#include <atomic>

#include "activation.cuh"
#include "narrow_shape.h"
#include "tcgen05.cuh"

namespace moe {
namespace linear_impl {

constexpr unsigned kFullMask = 0xFFFFFFFFu;
constexpr int kMaxCutBlocks = 128;    // of these one sum of the tensor core takes at most (8192 of K: cut off towards zero by 1e-5 of
                                      // the whole, 5e-5 where all terms have one sign; rounding to BF16 is off by up to 4e-3)

// An operand's element (r, k): rows of K values (K-major), or, transposed, K rows of values r.
struct Operand {
  const uint16_t* p;
  long long ld;      // elements between the rows that are stored
  bool transposed;
};

// What happens to the sums z[m, n] (+ bias): pre = z, out = act(z) + residual; gated:
// out = act(z[m, n]) * z[m, N + n].
struct Epilogue {
  const void* bias;
  const void* residual;
  void* out;
  uint16_t* pre;
  long long ldr, ldo, ldp;
  int bias_f32, residual_f32, out_f32, act;
};

// out[m, n] over M x N (gated: b has 2 N rows, the gate's and then the other's).
struct Product {
  Operand a, b;
  int M, N, K;
  Epilogue e;
};

// The products (one or two, gated: one) with rows of a on the tensor core's lanes and those of b on
// its columns, two SMs per tile: the columns of b's rows a tile, the pairs of SMs that work on
// each product, and when they are estimated to end (in ns).
struct WidePlan {
  int bn[2], pairs[2];
  double ns;
};
WidePlan plan_wide(const Product* products, int count, bool gated, const DeviceInfo& dev);
int launch_wide(const Product* products, int count, bool gated, const WidePlan& plan, const DeviceInfo& dev, cudaStream_t stream);

// One product with rows of b on the lanes and those of a (not transposed) on the columns, bn of
// them a tile, K split over a cluster: for few rows of a.
struct NarrowPlan {
  int bn, splits, per_sm;
  double ns;
};
int plan_narrow(const Product& product, bool gated, const DeviceInfo& dev, NarrowPlan* plan);
int launch_narrow(const Product& product, bool gated, const NarrowPlan& plan, const DeviceInfo& dev, cudaStream_t stream);

// dz = dout act'(pre) [T, n] (pre NULL: dout), rounded once to BF16 for the products, and the sum of
// its rows before that rounding in FP32; either may be left out (NULL).
int launch_dz(const uint16_t* dout, long long ldd, const uint16_t* pre, long long ldp, int act, int T, int N, uint16_t* dz,
              long long ldz, float* dbias, const DeviceInfo& dev, cudaStream_t stream);
// [dg | du] = [dout u act'(g) | dout act(g)] of pre = [g | u].
int launch_gated_dz(const uint16_t* dout, long long ldd, const uint16_t* pre, long long ldp, int act, int T, int F,
                    uint16_t* dz, long long ldz, const DeviceInfo& dev, cudaStream_t stream);

// A kernel's shared-memory limit and carveout, set at its first launch on a device.
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

// Boxes of 64 x box_rows elements (128-byte swizzle, zeros outside) of the matrix that is stored:
// [rows, K], or [K, rows] transposed.
inline bool make_map(CUtensorMap* m, const Operand& o, long long rows, int K, int box_rows) {
  auto fn = encode_fn();
  if (!fn) return false;
  const long long inner = o.transposed ? rows : K, outer = o.transposed ? K : rows;
  cuuint64_t dims[2] = {(cuuint64_t)inner, (cuuint64_t)outer};
  cuuint64_t strides[1] = {(cuuint64_t)o.ld * 2};
  cuuint32_t box[2] = {64u, (cuuint32_t)(o.transposed ? kBlockK : box_rows)};
  cuuint32_t estr[2] = {1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<uint16_t*>(o.p), dims, strides, box, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Descriptor of a stage's operand tile. K-major: rows of 64 values of K. Transposed: blocks of 64
// rows, each of kBlockK lines of those 64 values, 8 lines 1024 bytes apart from the next 8 and a
// block 64 * 128 bytes from the next.
__device__ __forceinline__ uint64_t operand_desc(uint32_t saddr, bool transposed) {
  uint64_t d = sw128_desc(saddr);
  if (transposed) d = (d & ~((uint64_t)0x3FFF << 16)) | (uint64_t)(64 * 128 >> 4) << 16;
  return d;
}
// Its step along K by 16 values (in units of 16 bytes).
__device__ __forceinline__ uint32_t operand_step(bool transposed) { return transposed ? 16 * 128 >> 4 : 32 >> 4; }

// BF16 x BF16 -> FP32.
__device__ __forceinline__ uint32_t instr_desc(int m, int n, bool a_transposed, bool b_transposed) {
  return (1u << 4) | (1u << 7) | (1u << 10) | ((uint32_t)a_transposed << 15) | ((uint32_t)b_transposed << 16) |
         ((uint32_t)(n >> 3) << 17) | ((uint32_t)(m >> 4) << 24);
}

__device__ __forceinline__ float load_as_f32(const void* p, long long i, int f32) {
  return f32 ? static_cast<const float*>(p)[i] : bf16_to_f32(static_cast<const uint16_t*>(p)[i]);
}

// 16 bytes to a shared::cluster address, arriving on `bar` of the same CTA.
__device__ __forceinline__ void send16(uint32_t addr, float a, float b, float c, float d, uint32_t bar) {
  asm volatile("st.async.weak.shared::cluster.mbarrier::complete_tx::bytes.v4.f32 [%0], {%1,%2,%3,%4}, [%5];" ::"r"(addr), "f"(a), "f"(b),
               "f"(c), "f"(d), "r"(bar)
               : "memory");
}
// (Relaxed: for what orders no memory of this thread's; a release waits for all its stores.)
__device__ __forceinline__ void cluster_arrive_relaxed() { asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }

constexpr int kMaxSplits = 8;

// Four values of the splits' partial sums, `stride` values apart, added in the order of the splits.
__device__ __forceinline__ void sum_partials(const float* p, int splits, int stride, float* s) {
  float4 v = *reinterpret_cast<const float4*>(p);
  s[0] = v.x, s[1] = v.y, s[2] = v.z, s[3] = v.w;
#pragma unroll
  for (int q = 1; q < kMaxSplits; ++q)
    if (q < splits) {
      v = *reinterpret_cast<const float4*>(p + q * stride);
      s[0] = __fadd_rn(s[0], v.x), s[1] = __fadd_rn(s[1], v.y), s[2] = __fadd_rn(s[2], v.z), s[3] = __fadd_rn(s[3], v.w);
    }
}

}  // namespace linear_impl
}  // namespace moe
