// BF16 rows (or silu(gate) * up of [gate | up] rows) to E4M3 codes with one FP32 scale
// per row and 128 columns.
//
// Per block: amax = max |v|, scale = amax / 448 (or the smallest power of two at or
// above it), q = E4M3(v * 448 / amax). Bound by HBM: 2 (swiglu: 4) bytes in and 1 + 1/32
// out per value.
//
// A block is 16 lanes with one 16-byte load each (two with swiglu), so nothing is read
// twice and nothing staged. A warp takes up to eight consecutive blocks of a row at a
// time, two per load instruction (512 contiguous bytes; 256 a store), all loads ahead of
// the arithmetic. The stream only hides some 20 instructions a value, so:
//   - the four maxima of a half-warp are reduced together, five exchanges instead of
//     sixteen, which leaves each on four lanes;
//   - those lanes divide for that block alone, and hand the multiplier back;
//   - silu is 2^x and 1/x of the special-function unit. Over all BF16 gates its error is at
//     most 0.83 x 2^-20 of the value to |gate| = 12 (rounding the exponent's argument alone can
//     make 0.7) and 3.4 x 2^-20 to 64, measured with the scale's division (tests; the bound
//     that follows from the operations is 1.45 x 2^-20 to 12). A code moves only beside a tie:
//     39 of 16.7 million, as of the plain form in FP32.
#include "fp8_block.cuh"

namespace moe {
namespace {

using namespace fp8_impl;

constexpr int kThreads = 128;
// CTAs an SM at most, three times those resident, so that their ends are not all one wave's
// (16320 x 1024 with swiglu 16.0 us, 16.7 with 14 and 16.5 with 8 of 256 threads; 40000 x 2048
// 70.6, 75.6 and 72.2).
constexpr int kCtasPerSm = 24;
constexpr int kUnroll = 4;          // load instructions of a warp in flight (of each half with swiglu)
constexpr int kRun = 2 * kUnroll;  // blocks of a row that a warp takes at a time

__device__ __forceinline__ float silu(float g) {
  float e, r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(__fmul_rn(g, -1.4426950408889634f)));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(__fadd_rn(1.f, e)));
  return __fmul_rn(g, r);
}

// units: rows times the runs of a row.
template <bool SWIGLU, bool POW2>
__global__ void __launch_bounds__(kThreads) quantize_kernel(const uint16_t* __restrict__ x, long long ldx, int cols,
                                                            int nb, int runs, int units, uint8_t* __restrict__ q,
                                                            float* __restrict__ scales) {
  const int lane = threadIdx.x & 31, warps = gridDim.x * (kThreads / 32);
  grid_launch_dependents();
  grid_wait();
  const uint64_t once = policy_evict_first();
  for (int u = (int)((blockIdx.x * kThreads + threadIdx.x) >> 5); u < units; u += warps) {
    const int row = u / runs, b0 = (u - row * runs) * kRun + (lane >> 4);  // this half-warp's first block
    const int col0 = b0 * FP8_BLOCK + 8 * (lane & 15);
    const uint16_t* p = x + (long long)row * ldx + col0;
    uint4 a[kUnroll], b[kUnroll];
#pragma unroll
    for (int i = 0; i < kUnroll; ++i) {
      const bool in = col0 + 2 * i * FP8_BLOCK < cols;
      a[i] = in ? ld_stream16(p + 2 * i * FP8_BLOCK, once) : make_uint4(0, 0, 0, 0);
      if (SWIGLU) b[i] = in ? ld_stream16(p + cols + 2 * i * FP8_BLOCK, once) : make_uint4(0, 0, 0, 0);
    }
    float v[kUnroll][8];
    uint32_t m[kUnroll];
#pragma unroll
    for (int i = 0; i < kUnroll; ++i) {
      bf16x8_to_f32(a[i], v[i]);
      if (SWIGLU) {
        float up[8];
        bf16x8_to_f32(b[i], up);
#pragma unroll
        for (int j = 0; j < 8; ++j) v[i][j] = __fmul_rn(silu(v[i][j]), up[j]);
      }
      m[i] = magnitude(v[i]);
    }
    // lanes with bits 3, 2 = i end with the maximum of load i's block
    static_assert(kUnroll == 4, "two exchange steps");
    const bool h = lane & 8, l = lane & 4;
    uint32_t k0 = max(h ? m[2] : m[0], __shfl_xor_sync(kFullMask, h ? m[0] : m[2], 8));
    uint32_t k1 = max(h ? m[3] : m[1], __shfl_xor_sync(kFullMask, h ? m[1] : m[3], 8));
    uint32_t k = max(l ? k1 : k0, __shfl_xor_sync(kFullMask, l ? k0 : k1, 4));
    k = max(k, __shfl_xor_sync(kFullMask, k, 2));
    k = max(k, __shfl_xor_sync(kFullMask, k, 1));
    const BlockScale s = block_scale<POW2>(k);
    const int mine = b0 + 2 * ((lane >> 2) & 3);  // that block
    if ((lane & 3) == 0 && mine < nb) scales[(long long)row * nb + mine] = s.scale;
#pragma unroll
    for (int i = 0; i < kUnroll; ++i) {
      BlockScale t;
      t.special = false;  // (a multiplier of NaN makes every code 0x7F)
      t.mult = __shfl_sync(kFullMask, s.special ? s.scale : s.mult, (lane & 16) + 4 * i);
      const int c = col0 + 2 * i * FP8_BLOCK;
      if (c < cols) *reinterpret_cast<uint2*>(q + (long long)row * cols + c) = encode8(v[i], t);
    }
  }
}

int quantize(const uint16_t* x, int64_t ldx, int rows, int cols, uint8_t* q, float* scales, int scale_rule, bool swiglu,
             cudaStream_t stream) {
  if (rows < 0 || cols < 8 || cols % 8 != 0 || cols > (1 << 29)) return MOE_ERR_INVALID_ARGUMENT;
  if (scale_rule != FP8_SCALE_AMAX && scale_rule != FP8_SCALE_POW2) return MOE_ERR_INVALID_ARGUMENT;
  if (ldx < (swiglu ? 2LL * cols : (long long)cols) || ldx % 8 != 0) return MOE_ERR_INVALID_ARGUMENT;
  if (rows == 0) return MOE_OK;
  if (!x || !q || !scales) return MOE_ERR_INVALID_ARGUMENT;
  const int nb = (cols + FP8_BLOCK - 1) / FP8_BLOCK;
  if ((long long)rows * nb >= (1LL << 31) - (1LL << 24)) return MOE_ERR_CAPACITY;  // (the loop's index passes the end)
  if (!aligned(x, 16) || !aligned(q, 8) || !aligned(scales, 4)) return MOE_ERR_ALIGNMENT;
  DeviceInfo dev;
  int st = current_device(&dev);
  if (st != MOE_OK) return st;
  const int runs = (nb + kRun - 1) / kRun, units = rows * runs;
  const long long need = ((long long)units + kThreads / 32 - 1) / (kThreads / 32);
  const long long most = (long long)kCtasPerSm * dev.sm_count;
  const bool p2 = scale_rule == FP8_SCALE_POW2;
  auto kern = swiglu ? (p2 ? quantize_kernel<true, true> : quantize_kernel<true, false>)
                     : (p2 ? quantize_kernel<false, true> : quantize_kernel<false, false>);
  return launch_pdl(kern, dim3((unsigned)(need < most ? need : most)), dim3(kThreads), 0, stream, x, (long long)ldx,
                    cols, nb, runs, units, q, scales);
}

}  // namespace
}  // namespace moe

extern "C" int fp8_block_quantize_rows(const uint16_t* x, int64_t ldx, int rows, int cols, uint8_t* q, float* scales,
                                       int scale_rule, moe_stream_t stream) {
  return moe::quantize(x, ldx, rows, cols, q, scales, scale_rule, false, moe::as_cuda(stream));
}

extern "C" int fp8_block_quantize_swiglu(const uint16_t* x, int64_t ldx, int rows, int cols, uint8_t* q, float* scales,
                                         int scale_rule, moe_stream_t stream) {
  return moe::quantize(x, ldx, rows, cols, q, scales, scale_rule, true, moe::as_cuda(stream));
}
