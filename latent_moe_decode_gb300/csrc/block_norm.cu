// The norm after a block, its gate and the residual's scale, and the norm before the
// next block, in one pass over the rows:
//   u = y / sqrt(mean(y^2) + eps) * post_weight
//   h = residual + alpha * (gate * u)
//   n = h / sqrt(mean(h^2) + eps) * next_weight      (and n's E4M3 codes)
//
// Bound by HBM: each row of y, residual and gate is read once and h, n and the codes
// written once. A CTA holds a row in registers (8 consecutive columns per 16-byte
// fragment, up to V fragments a thread), so both sums of squares -- each thread's columns
// in order, a shuffle tree, the warps in order -- and all outputs come from one load. 16
// consecutive lanes hold one block of 128 columns for the codes.
// A row's two sums leave the memory idle while one CTA's registers fill the SM, so with
// more rows than SMs the CTAs are persistent and rows arrive in a ring of shared-memory
// stages by bulk copies, the next rows on their way while one is normalised; the weights
// stay in registers. Few rows (one CTA each) are loaded directly: a copy's round trip
// through shared memory would only add to their latency.
#include "fp8_block.cuh"

namespace moe {
namespace {

using namespace fp8_impl;

// Threads of a CTA: one fragment each up to H = 8192, else four (more registers a thread).
template <int V>
constexpr int kMaxThreads = V == 1 ? 1024 : 512;
constexpr int kMaxH = 16384;

constexpr int kMaxStages = 4;

struct BlockNormArgs {
  const uint16_t* y;
  long long ldy;
  const void* residual;
  const uint16_t *post, *gate, *next;
  float alpha, eps, inv_h;  // inv_h: 1 / H
  int T, H, nb;
  int stages;  // of the ring (streamed)
  uint32_t* err;
  void* h;
  uint16_t* n;
  uint8_t* q;
  float* scales;
};

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = __fadd_rn(v, __shfl_xor_sync(kFullMask, v, o));
  return v;
}

// The CTA's sum of one value per thread, in a fixed order, for every thread: trees over a
// warp's lanes, then (in every warp) over the warps' sums.
__device__ __forceinline__ float cta_sum(float v, float* slots) {
  const int lane = threadIdx.x & 31;
  v = warp_sum(v);
  if (lane == 0) slots[threadIdx.x >> 5] = v;
  __syncthreads();
  return warp_sum(lane < (int)(blockDim.x >> 5) ? slots[lane] : 0.f);
}

template <int V, bool F32, int GATE, bool STREAM>
__global__ void __launch_bounds__(kMaxThreads<V>) block_norm_kernel(const BlockNormArgs a) {
  extern __shared__ __align__(128) uint8_t ring[];
  __shared__ float slots[2][kMaxThreads<V> / 32];
  __shared__ __align__(8) uint64_t bars[kMaxStages];
  const int nv = a.H / 8;  // fragments of a row
  // a stage: the row of y, of the residual, of a full gate
  const uint32_t y_bytes = 2u * a.H, r_bytes = (F32 ? 4u : 2u) * a.H, g_bytes = GATE == MOE_GATE_FULL ? 2u * a.H : 0u;
  const uint32_t stage_bytes = y_bytes + r_bytes + g_bytes;
  auto issue = [&](int i, long long row) {  // (one thread)
    const uint32_t dst = smem_u32(ring) + i * stage_bytes, bar = smem_u32(&bars[i]);
    const uint64_t once = policy_evict_first();
    mbar_expect_tx(bar, stage_bytes);
    bulk_g2s(dst, a.y + row * a.ldy, y_bytes, bar, once);
    bulk_g2s(dst + y_bytes, static_cast<const uint8_t*>(a.residual) + row * r_bytes, r_bytes, bar, once);
    if (GATE == MOE_GATE_FULL) bulk_g2s(dst + y_bytes + r_bytes, a.gate + row * a.H, g_bytes, bar, once);
  };
  if (STREAM && threadIdx.x == 0) {
    for (int i = 0; i < a.stages; ++i) mbar_init(smem_u32(&bars[i]), 1);
    mbar_fence_init();
  }
  if (STREAM) __syncthreads();
  grid_launch_dependents();
  grid_wait();
  const uint4 zero = make_uint4(0, 0, 0, 0);
  if (STREAM && threadIdx.x == 0)
    for (int i = 0; i < a.stages && blockIdx.x + (long long)i * gridDim.x < a.T; ++i)
      issue(i, blockIdx.x + (long long)i * gridDim.x);
  uint4 post[V], next[V], channel[V];
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int f = i * blockDim.x + threadIdx.x;
    post[i] = a.post && f < nv ? ld_nc16(a.post + 8 * f) : zero;
    next[i] = f < nv ? ld_nc16(a.next + 8 * f) : zero;
    if (GATE == MOE_GATE_CHANNEL) channel[i] = f < nv ? ld_nc16(a.gate + 8 * f) : zero;
  }
  int stage = 0;
  uint32_t lap = 0;
  for (long long row = blockIdx.x; row < a.T; row += gridDim.x) {
    const long long at = row * a.H;
    float y[V][8], r[V][8];
    uint4 g[V];
    if (STREAM) {
      if (!__syncthreads_and(mbar_wait(smem_u32(&bars[stage]), lap, a.err))) {
        // (a copy never landed: the error is set; those in flight are waited for, each with the same bound)
        for (int i = 1; i < a.stages && row + (long long)i * gridDim.x < a.T; ++i) {
          const int s = (stage + i) % a.stages;
          mbar_wait(smem_u32(&bars[s]), s < stage ? lap ^ 1u : lap, a.err);
        }
        return;
      }
    }
    const uint8_t* const st = ring + stage * stage_bytes;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int f = i * blockDim.x + threadIdx.x;
      const bool in = f < nv;
      // (the residual not by the read-only path: h may be written over it)
      const uint8_t* yp = STREAM ? st + 16 * f : reinterpret_cast<const uint8_t*>(a.y + row * a.ldy + 8 * f);
      const uint8_t* rp = STREAM ? st + y_bytes + (F32 ? 32 : 16) * f : static_cast<const uint8_t*>(a.residual) + row * r_bytes + (F32 ? 32 : 16) * f;
      bf16x8_to_f32(in ? *reinterpret_cast<const uint4*>(yp) : zero, y[i]);
      if (F32) {
        const float4 lo = in ? reinterpret_cast<const float4*>(rp)[0] : make_float4(0, 0, 0, 0);
        const float4 hi = in ? reinterpret_cast<const float4*>(rp)[1] : make_float4(0, 0, 0, 0);
        r[i][0] = lo.x, r[i][1] = lo.y, r[i][2] = lo.z, r[i][3] = lo.w;
        r[i][4] = hi.x, r[i][5] = hi.y, r[i][6] = hi.z, r[i][7] = hi.w;
      } else {
        bf16x8_to_f32(in ? *reinterpret_cast<const uint4*>(rp) : zero, r[i]);
      }
      if (GATE == MOE_GATE_FULL)
        g[i] = !in ? zero : STREAM ? *reinterpret_cast<const uint4*>(st + y_bytes + r_bytes + 16 * f) : ld_nc16(a.gate + at + 8 * f);
      if (GATE == MOE_GATE_CHANNEL) g[i] = channel[i];
    }
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < V; ++i)
#pragma unroll
      for (int j = 0; j < 8; ++j) ss = __fmaf_rn(y[i][j], y[i][j], ss);
    float root = 1.f;
    if (a.post)
      root = rsqrtf(__fmaf_rn(cta_sum(ss, slots[0]), a.inv_h, a.eps));
    else if (STREAM)
      __syncthreads();
    if (STREAM) {  // every thread has its fragments: the stage takes the row after the ring's
      const long long later = row + (long long)a.stages * gridDim.x;
      if (threadIdx.x == 0 && later < a.T) issue(stage, later);
      if (++stage == a.stages) stage = 0, lap ^= 1u;
    }
    const float tg = GATE == MOE_GATE_TOKEN ? bf16_to_f32(a.gate[row]) : 1.f;
    ss = 0.f;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int f = i * blockDim.x + threadIdx.x;
      float p[8], gv[8];
      bf16x8_to_f32(post[i], p);
      if (GATE == MOE_GATE_FULL || GATE == MOE_GATE_CHANNEL) bf16x8_to_f32(g[i], gv);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        float u = y[i][j];
        if (a.post) u = __fmul_rn(__fmul_rn(u, root), p[j]);
        if (GATE == MOE_GATE_TOKEN) u = __fmul_rn(u, tg);
        if (GATE == MOE_GATE_FULL || GATE == MOE_GATE_CHANNEL) u = __fmul_rn(u, gv[j]);
        r[i][j] = __fmaf_rn(a.alpha, u, r[i][j]);
        ss = __fmaf_rn(r[i][j], r[i][j], ss);
      }
      if (f < nv) {
        if (F32) {
          float4* o = reinterpret_cast<float4*>(static_cast<float*>(a.h) + at + 8 * f);
          o[0] = make_float4(r[i][0], r[i][1], r[i][2], r[i][3]);
          o[1] = make_float4(r[i][4], r[i][5], r[i][6], r[i][7]);
        } else {
          st16(static_cast<uint16_t*>(a.h) + at + 8 * f,
               make_uint4(pack_bf16x2(r[i][0], r[i][1]), pack_bf16x2(r[i][2], r[i][3]), pack_bf16x2(r[i][4], r[i][5]),
                          pack_bf16x2(r[i][6], r[i][7])));
        }
      }
    }
    root = rsqrtf(__fmaf_rn(cta_sum(ss, slots[1]), a.inv_h, a.eps));
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int f = i * blockDim.x + threadIdx.x;
      float w[8];
      bf16x8_to_f32(next[i], w);
#pragma unroll
      for (int j = 0; j < 8; ++j) w[j] = __fmul_rn(__fmul_rn(r[i][j], root), w[j]);  // n
      if (a.n && f < nv)
        st16(a.n + at + 8 * f, make_uint4(pack_bf16x2(w[0], w[1]), pack_bf16x2(w[2], w[3]), pack_bf16x2(w[4], w[5]), pack_bf16x2(w[6], w[7])));
      if (a.q) {
        // (Of n, not of h * weight, whose ratios are the same: its multipliers can overflow where n's
        // cannot, and it is not zero where a root of 0 makes n so. Lanes past the row's end hold 0, or
        // NaN where an infinite root makes the rest of their block infinite or NaN. 73.4 us at 4096 x
        // 7168, 72.9 with the codes of h * weight.)
        const BlockScale s = block_scale_shared(block_max(magnitude(w)));
        if (f < nv) {
          *reinterpret_cast<uint2*>(a.q + at + 8 * f) = encode8(w, s);
          if ((f & 15) == 0) a.scales[row * a.nb + (f >> 4)] = s.scale;
        }
      }
    }
  }
}

template <int V, bool F32, int GATE>
int launch(BlockNormArgs& a, int threads, int sm_count, cudaStream_t s) {
  const size_t stage = (size_t)a.H * (2 + (F32 ? 4 : 2) + (GATE == MOE_GATE_FULL ? 2 : 0));
  a.stages = (int)((size_t)(226 * 1024) / stage);
  if (a.stages > kMaxStages) a.stages = kMaxStages;
  // Streamed when there is a second row to be on its way
  if (a.T <= sm_count || a.stages < 2)
    return launch_pdl(block_norm_kernel<V, F32, GATE, false>, dim3((unsigned)a.T), dim3(threads), 0, s, a);
  auto kern = block_norm_kernel<V, F32, GATE, true>;
  const size_t smem = a.stages * stage;
  if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, 226 * 1024) != cudaSuccess) return MOE_ERR_CUDA;
  int per_sm = 1;
  while (per_sm < 4 && (per_sm + 1) * (smem + 2048) <= 228u * 1024 && (per_sm + 1) * threads <= 1024) ++per_sm;
  const long long most = (long long)per_sm * sm_count;
  return launch_pdl(kern, dim3((unsigned)(a.T < most ? a.T : most)), dim3(threads), smem, s, a);
}

template <int V, bool F32>
int launch_gate(int kind, BlockNormArgs& a, int threads, int sm_count, cudaStream_t s) {
  switch (kind) {
    case MOE_GATE_TOKEN: return launch<V, F32, MOE_GATE_TOKEN>(a, threads, sm_count, s);
    case MOE_GATE_CHANNEL: return launch<V, F32, MOE_GATE_CHANNEL>(a, threads, sm_count, s);
    case MOE_GATE_FULL: return launch<V, F32, MOE_GATE_FULL>(a, threads, sm_count, s);
    default: return launch<V, F32, MOE_GATE_NONE>(a, threads, sm_count, s);
  }
}

}  // namespace
}  // namespace moe

extern "C" int moe_block_norm(const uint16_t* y, int64_t ldy, const void* residual, int residual_dtype,
                              const uint16_t* post_weight, const uint16_t* gate, int gate_kind,
                              const uint16_t* next_weight, float alpha, float eps, int T, int H, void* h, uint16_t* n,
                              uint8_t* q, float* scales, moe_stream_t stream) {
  using namespace moe;
  if (T < 0 || H < 8 || H % 8 != 0 || ldy < H || ldy % 8 != 0 || !(eps >= 0.f)) return MOE_ERR_INVALID_ARGUMENT;
  if (residual_dtype != MOE_DTYPE_F32 && residual_dtype != MOE_DTYPE_BF16) return MOE_ERR_INVALID_ARGUMENT;
  if (gate_kind < MOE_GATE_NONE || gate_kind > MOE_GATE_FULL || (gate_kind != MOE_GATE_NONE) != (gate != nullptr))
    return MOE_ERR_INVALID_ARGUMENT;
  if ((q == nullptr) != (scales == nullptr)) return MOE_ERR_INVALID_ARGUMENT;
  if (H > kMaxH) return MOE_ERR_CAPACITY;
  if (T == 0) return MOE_OK;
  if (!y || !residual || !next_weight || !h) return MOE_ERR_INVALID_ARGUMENT;
  if (!aligned(y, 16) || !aligned(residual, 16) || !aligned(h, 16) || !aligned(next_weight, 16) ||
      !aligned(post_weight, 16) || !aligned(n, 16) || !aligned(q, 8) || !aligned(scales, 4) ||
      !aligned(gate, gate_kind == MOE_GATE_TOKEN ? 2 : 16))
    return MOE_ERR_ALIGNMENT;
  DeviceInfo dev;
  int st = current_device(&dev);
  if (st != MOE_OK) return st;
  BlockNormArgs a;
  a.y = y, a.ldy = ldy, a.residual = residual, a.post = post_weight, a.gate = gate, a.next = next_weight;
  a.alpha = alpha, a.eps = eps, a.inv_h = 1.f / (float)H, a.T = T, a.H = H, a.nb = (H + FP8_BLOCK - 1) / FP8_BLOCK;
  a.h = h, a.n = n, a.q = q, a.scales = scales, a.err = dev.error_word;
  const int nv = H / 8, v = nv <= kMaxThreads<1> ? 1 : 4;
  const int threads = ((nv + v - 1) / v + 31) / 32 * 32;
  const cudaStream_t s = as_cuda(stream);
  const bool f32 = residual_dtype == MOE_DTYPE_F32;
  const int sms = dev.sm_count;
  if (v == 1) return f32 ? launch_gate<1, true>(gate_kind, a, threads, sms, s) : launch_gate<1, false>(gate_kind, a, threads, sms, s);
  return f32 ? launch_gate<4, true>(gate_kind, a, threads, sms, s) : launch_gate<4, false>(gate_kind, a, threads, sms, s);
}
