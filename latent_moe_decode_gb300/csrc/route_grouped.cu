// Routing with softmax or sigmoid scores and groups of experts: scores, balance bias,
// the groups of largest value, the top-K experts in them, renormalised weights.
//
// One warp per token. The token's keys and scores are kept in shared memory; softmax
// takes the row's maximum and sum by lane strides and shuffle trees; a group's value is
// found by the warp, the kept groups by topk_group rounds over the groups' values, and
// the choice by K rounds of a warp argmax over (key descending, expert ascending).
#include "topk.cuh"

namespace moe {
namespace {

using topk_impl::kFull;
using topk_impl::order_key;
using topk_impl::spec_sigmoid;

constexpr int kWarps = 4;

struct GroupedArgs {
  const float *logits, *bias;
  int T, E, K, n_group, topk_group, renorm;
  float scale;
  int32_t* ids;
  float* weights;
  uint16_t* weights_bf16;
};

__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(kFull, v, o));
  return v;
}
__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = __fadd_rn(v, __shfl_xor_sync(kFull, v, o));
  return v;
}
__device__ __forceinline__ float number(float v) { return v != v ? -INFINITY : v; }

// exp(x - m) with the limits of a row whose maximum is infinite.
__device__ __forceinline__ float soft_exp(float x, float m) {
  if (x != x || m == -INFINITY) return 0.f;
  return x == m ? 1.f : expf(x - m);
}

template <bool SOFTMAX, bool TOP2>
__global__ void __launch_bounds__(32 * kWarps) route_kernel(const GroupedArgs a) {
  extern __shared__ float smem[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5;
  float* key = smem + (size_t)warp * (2 * a.E + MOE_MAX_GROUPS);
  float* score = key + a.E;
  float* value = score + a.E;
  grid_launch_dependents();
  grid_wait();
  const int t = blockIdx.x * warps + warp;
  if (t >= a.T) return;
  const float* x = a.logits + (size_t)t * a.E;
  float m = -INFINITY, sum = 0.f;
  if (SOFTMAX) {
    for (int e = lane; e < a.E; e += 32) m = fmaxf(m, x[e]);
    m = warp_max(m);
    for (int e = lane; e < a.E; e += 32) sum = __fadd_rn(sum, soft_exp(x[e], m));
    sum = warp_sum(sum);
  }
  for (int e = lane; e < a.E; e += 32) {
    const float xv = x[e];
    float s;
    if (SOFTMAX)
      s = sum > 0.f ? __fdiv_rn(soft_exp(xv, m), sum) : 0.f;
    else
      s = xv != xv ? 0.f : spec_sigmoid(xv);
    score[e] = s;
    key[e] = xv != xv ? -INFINITY : number(a.bias ? __fadd_rn(s, a.bias[e]) : s);
  }
  __syncwarp();
  if (a.n_group > 1 && a.topk_group < a.n_group) {
    const int size = a.E / a.n_group;
    for (int g = 0; g < a.n_group; ++g) {
      float b1 = -INFINITY, b2 = -INFINITY;  // the lane's two largest keys of the group
      for (int i = lane; i < size; i += 32) {
        const float k = key[g * size + i];
        b2 = fmaxf(b2, fminf(b1, k));
        b1 = fmaxf(b1, k);
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) {
        const float o1 = __shfl_xor_sync(kFull, b1, o), o2 = __shfl_xor_sync(kFull, b2, o);
        b2 = fmaxf(fminf(b1, o1), fmaxf(b2, o2));
        b1 = fmaxf(b1, o1);
      }
      if (lane == 0) value[g] = TOP2 && size > 1 ? number(__fadd_rn(b1, b2)) : b1;
    }
    __syncwarp();
    // a group is dropped when at least topk_group groups order before it
    for (int g = 0; g < a.n_group; ++g) {
      const uint32_t kg = order_key(value[g]);
      int before = 0;
      for (int o = 0; o < a.n_group; ++o) {
        const uint32_t ko = order_key(value[o]);
        before += ko > kg || (ko == kg && o < g);
      }
      if (before >= a.topk_group)
        for (int i = lane; i < size; i += 32) key[g * size + i] = __uint_as_float(0x7FC00000u);  // (NaN: not kept)
    }
    __syncwarp();
  }
  int my_id = 0;
  float my_s = 0.f;
  for (int k = 0; k < a.K; ++k) {
    uint32_t best = 0;
    int at = 0x7FFFFFFF;
    for (int e = lane; e < a.E; e += 32) {
      const float kv = key[e];
      const uint32_t o = kv != kv ? 0u : order_key(kv);
      if (o > best) best = o, at = e;
    }
    const uint32_t top = __reduce_max_sync(kFull, best);
    const int win = (int)__reduce_min_sync(kFull, best == top ? (uint32_t)at : 0x7FFFFFFFu);
    if (lane == k) my_id = win, my_s = score[win];
    __syncwarp();
    if (lane == 0) key[win] = __uint_as_float(0x7FC00000u);
    __syncwarp();
  }
  float S = 0.f;
  for (int k = 0; k < a.K; ++k) S = __fadd_rn(S, __shfl_sync(kFull, my_s, k));
  if (lane < a.K) {
    float w = a.renorm ? (S == 0.f ? 0.f : __fdiv_rn(my_s, S)) : my_s;
    if (a.scale != 1.f) w = __fmul_rn(w, a.scale);
    const size_t o = (size_t)t * a.K + lane;
    a.ids[o] = my_id;
    if (a.weights) a.weights[o] = w;
    if (a.weights_bf16) a.weights_bf16[o] = f32_to_bf16(w);
  }
}

}  // namespace
}  // namespace moe

extern "C" int moe_topk_route_grouped(const float* logits, const float* bias, int T, int E, int K, int scoring,
                                      int n_group, int topk_group, int group_rule, int renormalize, float scale,
                                      int32_t* ids, float* weights, uint16_t* weights_bf16, moe_stream_t stream) {
  using namespace moe;
  if (T < 0 || E < 1 || K < 1 || n_group < 1 || topk_group < 1) return MOE_ERR_INVALID_ARGUMENT;
  if (scoring != MOE_SCORE_SIGMOID && scoring != MOE_SCORE_SOFTMAX) return MOE_ERR_INVALID_ARGUMENT;
  if (group_rule != MOE_GROUP_MAX && group_rule != MOE_GROUP_TOP2) return MOE_ERR_INVALID_ARGUMENT;
  if (E % n_group != 0 || topk_group > n_group || (long long)K > (long long)topk_group * (E / n_group))
    return MOE_ERR_INVALID_ARGUMENT;
  if (E > MOE_MAX_EXPERTS || K > MOE_MAX_TOPK || n_group > MOE_MAX_GROUPS) return MOE_ERR_CAPACITY;
  if (T == 0) return MOE_OK;
  if (!logits || !ids) return MOE_ERR_INVALID_ARGUMENT;
  if (!aligned(logits, 4) || !aligned(bias, 4) || !aligned(ids, 4) || !aligned(weights, 4) || !aligned(weights_bf16, 2))
    return MOE_ERR_ALIGNMENT;
  DeviceInfo dev;
  int st = current_device(&dev);
  if (st != MOE_OK) return st;
  const GroupedArgs a{logits, bias, T, E, K, n_group, topk_group, renormalize, scale, ids, weights, weights_bf16};
  const int warps = E <= 1024 ? kWarps : 1;
  const size_t smem = (size_t)warps * (2 * E + MOE_MAX_GROUPS) * sizeof(float);  // at most 34 KB
  const bool soft = scoring == MOE_SCORE_SOFTMAX, two = group_rule == MOE_GROUP_TOP2;
  auto kern = soft ? (two ? route_kernel<true, true> : route_kernel<true, false>)
                   : (two ? route_kernel<false, true> : route_kernel<false, false>);
  return launch_pdl(kern, dim3((T + warps - 1) / warps), dim3(32 * warps), smem, as_cuda(stream), a);
}
