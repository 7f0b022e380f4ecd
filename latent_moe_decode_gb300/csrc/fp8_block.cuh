// E4M3 codes with one FP32 scale per block of 128 columns: the scale of a block and the
// codes of its values, shared by the quantisation kernels and the block norm. A block
// is held by 16 consecutive lanes, 8 consecutive values (as FP32) in each.
#pragma once

#include "common.cuh"

namespace moe {
namespace fp8_impl {

constexpr unsigned kFullMask = 0xFFFFFFFFu;
constexpr uint32_t kTiny = (uint32_t)(127 - 110) << 23;  // 2^-110: keeps 448 / amax finite
constexpr uint32_t kInf = 0x7F800000u;

struct BlockScale {
  float scale, mult;
  bool special;  // a NaN or an infinity in the block
};

// Scale of a block from the largest magnitude bits of its values (the integer order of
// FP32 magnitudes is their order, with infinity and then NaN on top). POW2: the smallest
// power of two with amax <= 448 * scale; 448 = 1.75 * 2^8, so it is 2^(floor(log2 amax)
// - 8), one more where the significand is above 1.75.
template <bool POW2>
__device__ __forceinline__ BlockScale block_scale(uint32_t m) {
  BlockScale s;
  s.special = m >= kInf;
  if (s.special) {
    s.scale = __uint_as_float(0x7FC00000u);
    s.mult = 0.f;
  } else if (m == 0u) {
    s.scale = s.mult = 1.f;
  } else {
    m = max(m, kTiny);
    if (POW2) {
      const int e = (int)(m >> 23) - 127 - 8 + ((m & 0x7FFFFFu) > 0x600000u ? 1 : 0);
      s.scale = __int_as_float((e + 127) << 23);
      s.mult = __int_as_float((127 - e) << 23);
    } else {
      const float amax = __uint_as_float(m);
      s.scale = __fdiv_rn(amax, 448.f);
      s.mult = __fdiv_rn(448.f, amax);
    }
  }
  return s;
}

// The same (amax / 448), the warp's lanes in step and a block's lanes agreeing on m: even lanes
// divide for the scale, odd lanes for the multiplier.
__device__ __forceinline__ BlockScale block_scale_shared(uint32_t m) {
  BlockScale s;
  s.special = m >= kInf;
  const bool odd = threadIdx.x & 1;
  const float used = __uint_as_float(s.special ? kTiny : max(m, kTiny));
  const float d = __fdiv_rn(odd ? 448.f : used, odd ? used : 448.f), o = __shfl_xor_sync(kFullMask, d, 1);
  s.scale = s.special ? __uint_as_float(0x7FC00000u) : m == 0u ? 1.f : odd ? o : d;
  s.mult = m == 0u ? 1.f : odd ? d : o;
  return s;
}

// Bits of the largest magnitude of 8 values, NaN above all.
__device__ __forceinline__ uint32_t magnitude(const float (&v)[8]) {
  float m = fabsf(v[0]);
#pragma unroll
  for (int i = 1; i < 8; ++i) asm("max.NaN.f32 %0, %0, %1;" : "+f"(m) : "f"(fabsf(v[i])));
  return __float_as_uint(m);
}

// The largest magnitude over the 16 lanes of a block.
__device__ __forceinline__ uint32_t block_max(uint32_t m) {
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(kFullMask, m, o));
  return m;
}

__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}

// Eight codes: E4M3(v * mult), round to nearest even, saturated at +-448.
__device__ __forceinline__ uint2 encode8(const float (&v)[8], const BlockScale& s) {
  if (s.special) return make_uint2(0x7F7F7F7Fu, 0x7F7F7F7Fu);
  uint32_t p[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) p[i] = e4m3x2(__fmul_rn(v[2 * i], s.mult), __fmul_rn(v[2 * i + 1], s.mult));
  return make_uint2(p[0] | (p[1] << 16), p[2] | (p[3] << 16));
}

__device__ __forceinline__ void bf16x8_to_f32(uint4 v, float (&f)[8]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = bf16_lo(w[i]);
    f[2 * i + 1] = bf16_hi(w[i]);
  }
}

}  // namespace fp8_impl
}  // namespace moe
