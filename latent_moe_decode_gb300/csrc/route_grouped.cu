// Routing with softmax or sigmoid scores and groups of experts: scores, balance bias,
// the groups of largest value, the top-K experts in them, renormalised weights.
//
// A token is 4 E bytes of logits and a few hundred dependent operations, so a call is
// bound by latency (one token) and by issue (thousands): one warp per token, no step that
// takes the warp once per choice.
//   - Keys are FP32 values mapped to integers of the same order (0: not to be chosen), so
//     that NaN, infinities and dropped experts need no branches.
//   - Groups: the warp's lanes divide into 32 / n_group lanes per group, scan the keys in
//     shared memory in a skewed order (no bank conflicts), merge their two largest by
//     shuffles, and a group is kept when fewer than topk_group order before it.
//   - Choice: the K-th largest distinct value of the 32 lane maxima bounds the K-th largest
//     key from below (K lanes hold a key at least that large). The experts at or above it, about
//     K to 2 K, are compacted and ranked against each other by shuffles; more than 64 of
//     them (heavy ties) take K rounds of a warp argmax instead.
//   - Sigmoid scores without groups: keys from the hardware's approximate tanh, whose error
//     (measured over all inputs, see topk.cuh) widens the bound; exact keys for the
//     candidates alone.
//   - Softmax without a bias and with groups by their maximum chooses by the logits, the
//     order of the scores before their rounding (logit_key); its weights need the row's sum only
//     when they are not renormalised (e / S over the sum of e / S).
// More than 1024 experts, or 32 groups, take a plainer body: the row in shared memory,
// rounds over it for groups and choices.
#include "topk.cuh"

namespace moe {
namespace {

using topk_impl::kFull;
using topk_impl::order_key;
using topk_impl::rank_key;
using topk_impl::spec_sigmoid;

constexpr int kWarps = 4;

struct GroupedArgs {
  const float *logits, *bias;
  int T, E, K, n_group, topk_group, renorm;
  float scale;
  int32_t* ids;
  float* weights;
  uint16_t* weights_bf16;
  int softmax, top2;
  uint32_t by_size;  // ceil(2^32 / group size): e / size as a high product (groups of two or more)
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

// Softmax's key by logit, m the row's maximum: where that is infinite every other number scores 0,
// and ties; NaN lies below all (order_key).
__device__ __forceinline__ uint32_t logit_key(float x, float m) {
  return order_key(m == INFINITY && x < m ? 0.f : x);
}

// The weights of slots 0 .. K - 1 (lane k: slot k's expert and score).
__device__ __forceinline__ void write_weights(const GroupedArgs& a, int t, int id, float s) {
  const int lane = threadIdx.x & 31;
  float S = 0.f;
  if (a.renorm)
    for (int k = 0; k < a.K; ++k) S = __fadd_rn(S, __shfl_sync(kFull, s, k));
  if (lane < a.K) {
    float w = a.renorm ? (S == 0.f ? 0.f : __fdiv_rn(s, S)) : s;
    if (a.scale != 1.f) w = __fmul_rn(w, a.scale);
    const size_t o = (size_t)t * a.K + lane;
    a.ids[o] = id;
    if (a.weights) a.weights[o] = w;
    if (a.weights_bf16) a.weights_bf16[o] = f32_to_bf16(w);
  }
}

// Two largest keys of two pairs of them.
__device__ __forceinline__ void merge2(uint32_t& a1, uint32_t& a2, uint32_t b1, uint32_t b2) {
  a2 = max(min(a1, b1), max(a2, b2));
  a1 = max(a1, b1);
}

constexpr int kMaxE = 1024;  // experts of the register body
constexpr int kList = 64;    // candidates it ranks

struct RouteScratch {
  unsigned long long list[kList];  // candidates: (key, ~expert)
  int id[MOE_MAX_TOPK];            // the choice
  float s[MOE_MAX_TOPK];
};

// NJ experts a lane; VEC: expert 128 j + 4 lane + i in element 4 j + i (16-byte accesses, no
// group ends inside one), else expert 32 j + lane in element j. xs, keys: the token's logits
// and keys (the bias, until they are made) in shared memory. Scores are made four a lane at a
// time in a loop that is not unrolled: unrolled, its thousands of instructions, run once
// a call, took longer to fetch than to execute (11 tokens x 672 experts 9.0 us).
template <int NJ, bool VEC, bool GROUPS>
__device__ __forceinline__ void route_token(const GroupedArgs& a, int t, RouteScratch& ws, float* xs, uint32_t* keys) {
  const int lane = threadIdx.x & 31, E = a.E, K = a.K;
  auto expert = [&](int j) { return VEC ? 128 * (j >> 2) + 4 * lane + (j & 3) : 32 * j + lane; };
  const float* row = a.logits + (size_t)t * E;
  const bool by_logit = a.softmax && !a.bias && !(GROUPS && a.top2);
  const bool rough = !GROUPS && !a.softmax;  // approximate keys find the candidates
  const bool direct = !GROUPS && by_logit;
  uint32_t key[NJ];
  float m = -INFINITY;
  {
    float x[NJ], b[NJ];
#pragma unroll
    for (int j = 0; j < NJ; j += VEC ? 4 : 1) {
      const bool in = expert(j) < E;
      if constexpr (VEC) {
        const float4 v = in ? __ldg(reinterpret_cast<const float4*>(row + expert(j))) : make_float4(0, 0, 0, 0);
        const float4 w = in && a.bias ? __ldg(reinterpret_cast<const float4*>(a.bias + expert(j))) : make_float4(0, 0, 0, 0);
        x[j] = v.x, x[j + 1] = v.y, x[j + 2] = v.z, x[j + 3] = v.w;
        b[j] = w.x, b[j + 1] = w.y, b[j + 2] = w.z, b[j + 3] = w.w;
      } else {
        x[j] = in ? __ldg(row + expert(j)) : 0.f;
        b[j] = in && a.bias ? __ldg(a.bias + expert(j)) : 0.f;
      }
    }
#pragma unroll
    for (int j = 0; j < NJ; j += VEC ? 4 : 1) {
      if constexpr (VEC) {
        *reinterpret_cast<float4*>(xs + expert(j)) = make_float4(x[j], x[j + 1], x[j + 2], x[j + 3]);
        *reinterpret_cast<float4*>(keys + expert(j)) = make_float4(b[j], b[j + 1], b[j + 2], b[j + 3]);
      } else {
        xs[expert(j)] = x[j];
        keys[expert(j)] = __float_as_uint(b[j]);
      }
#pragma unroll
      for (int i = 0; i < (VEC ? 4 : 1); ++i)
        if (expert(j + i) < E) m = fmaxf(m, x[j + i]);  // (ignores NaN)
    }
    if (rough) {
#pragma unroll
      for (int j = 0; j < NJ; ++j)
        key[j] = expert(j) < E ? order_key(__fadd_rn(topk_impl::approx_sigmoid(x[j]), b[j])) : 0u;
    } else if (direct) {
#pragma unroll
      for (int j = 0; j < NJ; ++j) key[j] = expert(j) < E ? order_key(number(x[j])) : 0u;
    }
  }
  // (a lane reads back what it wrote until the next warp barrier)
  float inv = 1.f;
  const bool summed = a.softmax && (!by_logit || !a.renorm);  // xs then holds exp(x - max), NaN a NaN
  if (a.softmax) {
    m = warp_max(m);
    if (summed) {
      float sum = 0.f;
#pragma unroll 1
      for (int j0 = 0; j0 < NJ; j0 += 4)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int e = expert(j0 + i);
          const float v = xs[e], x = soft_exp(v, m);
          if (e < E) sum = __fadd_rn(sum, x);
          if (!by_logit) xs[e] = v != v ? v : x;
        }
      sum = warp_sum(sum);
      inv = sum > 0.f ? __fdiv_rn(1.f, sum) : 0.f;  // (two roundings a score, not a division)
    }
  }
  auto score = [&](float v) {  // of what xs holds
    if (a.softmax) return __fmul_rn(by_logit ? soft_exp(v, m) : v != v ? 0.f : v, inv);
    return v != v ? 0.f : spec_sigmoid(v);
  };
  auto exact_key = [&](float v, float bias) {
    if (by_logit) return logit_key(v, m);
    const float c = a.bias ? __fadd_rn(score(v), bias) : score(v);
    return order_key(v != v ? -INFINITY : number(c));
  };
  // 1) exact keys of all experts
  auto exact_keys = [&] {
#pragma unroll 1
    for (int j0 = 0; j0 < NJ; j0 += 4) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int e = expert(j0 + i);
        keys[e] = e < E ? exact_key(xs[e], __uint_as_float(keys[e])) : 0u;
      }
    }
#pragma unroll
    for (int j = 0; j < NJ; j += VEC ? 4 : 1) {
      if constexpr (VEC) {
        const uint4 k = *reinterpret_cast<const uint4*>(keys + expert(j));
        key[j] = k.x, key[j + 1] = k.y, key[j + 2] = k.z, key[j + 3] = k.w;
      } else {
        key[j] = keys[expert(j)];
      }
    }
  };
  // (Direct keys tell neither NaN from -infinity, see `mixed`, nor what ties beside +infinity: a NaN
  // check in their unrolled code would cost every call 0.4 us)
  if (!rough && (!direct || m == INFINITY)) exact_keys();
  // 2) groups: L lanes each (of a power of two), the two largest keys of a group in each
  if constexpr (GROUPS) {
    __syncwarp();
    const int size = E / a.n_group, L = 1 << (31 - __clz(32 / a.n_group)), g = lane / L, r = lane - g * L;
    const int steps = (size + L - 1) / L;
    uint32_t k1 = 0, k2 = 0;
    if (g < a.n_group) {
      int c = g % steps;  // (each group starts elsewhere: lanes on different banks)
      for (int i = 0; i < steps; ++i) {
        const int at = c * L + r;
        if (at < size) merge2(k1, k2, keys[g * size + at], 0u);
        if (++c == steps) c = 0;
      }
    }
    for (int o = L >> 1; o > 0; o >>= 1) {
      const uint32_t o1 = __shfl_xor_sync(kFull, k1, o), o2 = __shfl_xor_sync(kFull, k2, o);
      merge2(k1, k2, o1, o2);
    }
    if (a.top2 && size > 1 && g < a.n_group)
      k1 = order_key(number(__fadd_rn(topk_impl::key_value(k1), topk_impl::key_value(k2))));
    int before = 0;  // groups that order before this one
    for (int o = 0; o < a.n_group; ++o) {
      const uint32_t ko = __shfl_sync(kFull, k1, o * L);
      before += ko > k1 || (ko == k1 && o < g);
    }
    const uint32_t kept = __ballot_sync(kFull, before < a.topk_group);  // bit g L: group g is kept
#pragma unroll
    for (int j = 0; j < NJ; j += VEC ? 4 : 1) {
      const bool in = kept >> min(__umulhi((uint32_t)expert(j), a.by_size) * (uint32_t)L, 31u) & 1u;  // (past E: whatever)
#pragma unroll
      for (int i = 0; i < (VEC ? 4 : 1); ++i)
        if (!in) key[j + i] = 0u;
    }
  }
  // 3) bound: the K-th largest distinct one of the lanes' maxima
  uint32_t v = 0, bound = 0;
#pragma unroll
  for (int j = 0; j < NJ; ++j) v = max(v, key[j]);
  for (int k = 0; k < K; ++k) {
    bound = __reduce_max_sync(kFull, v);
    v = v == bound ? 0u : v;
  }
  const bool mixed = direct && bound <= order_key(-INFINITY);  // -infinity or NaN may be chosen: exact keys tell them apart
  // (K experts have an approximate key of at least it: the exact K-th largest is within the
  // approximation's error of it, and every expert chosen within twice that)
  bound = rough ? topk_impl::candidate_threshold(bound) : max(bound, 1u);
  // 4) candidates, compacted
  int mine = 0;
#pragma unroll
  for (int j = 0; j < NJ; ++j) mine += key[j] >= bound;
  int incl = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(kFull, incl, o);
    if (lane >= o) incl += y;
  }
  const int total = __shfl_sync(kFull, incl, 31);
  if (total <= kList) {
    int pos = incl - mine;
#pragma unroll
    for (int j = 0; j < NJ; ++j) {
      if (key[j] >= bound) {
        ws.list[pos] = rank_key(key[j], expert(j));
        ++pos;
      }
    }
    __syncwarp();
    if (rough || mixed) {  // the candidates' exact keys
      for (int i = lane; i < total; i += 32) {
        const int e = (int)(0xFFFFFFFFu - (uint32_t)ws.list[i]);
        ws.list[i] = rank_key(exact_key(xs[e], __uint_as_float(keys[e])), e);
      }
      __syncwarp();
    }
    // 5) a candidate's slot: how many order before it (lane i: candidates i and i + 32)
    auto place = [&](int i) {
      const unsigned long long c = i < total ? ws.list[i] : 0;
      int r = 0;
#pragma unroll 4
      for (int o = 0; o < total; ++o) r += ws.list[o] > c;
      if (i < total && r < K) {
        const int e = (int)(0xFFFFFFFFu - (uint32_t)c);
        ws.id[r] = e;
        ws.s[r] = score(xs[e]);
      }
    };
    place(lane);
    if (total > 32) place(lane + 32);
  } else {
    if (rough || mixed) exact_keys();
    __syncwarp();
#pragma unroll 1
    for (int k = 0; k < K; ++k) {
      uint32_t best = 0;
      int at = 0x7FFFFFFF;
#pragma unroll
      for (int j = 0; j < NJ; ++j)
        if (key[j] > best) best = key[j], at = expert(j);  // (ascending: the first maximum wins)
      const uint32_t top = __reduce_max_sync(kFull, best);
      const int win = (int)__reduce_min_sync(kFull, best == top ? (uint32_t)at : 0x7FFFFFFFu);
      if (at == win) {
        ws.id[k] = win;
        ws.s[k] = score(xs[win]);
      }
#pragma unroll
      for (int j = 0; j < NJ; ++j)
        if (expert(j) == win) key[j] = 0u;
    }
  }
  __syncwarp();
  write_weights(a, t, lane < K ? ws.id[lane] : 0, lane < K ? ws.s[lane] : 0.f);
}

template <int NJ, bool VEC, bool GROUPS>
__global__ void __launch_bounds__(32 * kWarps) route_kernel(const GroupedArgs a) {
  __shared__ RouteScratch ws[kWarps];
  __shared__ __align__(16) float xs[kWarps * NJ * 32];
  __shared__ __align__(16) uint32_t keys[kWarps * NJ * 32];
  const int warp = threadIdx.x >> 5, t = blockIdx.x * kWarps + warp;
  grid_launch_dependents();
  if (t < a.T && (threadIdx.x & 31) == 0 && VEC) prefetch_l2(a.logits + (size_t)t * a.E, (uint32_t)a.E * 4u);  // (a hint)
  grid_wait();
  if (t < a.T) route_token<NJ, VEC, GROUPS>(a, t, ws[warp], xs + warp * NJ * 32, keys + warp * NJ * 32);
}

template <bool SOFTMAX, bool TOP2>
__global__ void __launch_bounds__(32 * kWarps) route_any_kernel(const GroupedArgs a) {
  extern __shared__ float smem[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5;
  float* score = smem + (size_t)warp * (2 * a.E + MOE_MAX_GROUPS);
  uint32_t* key = reinterpret_cast<uint32_t*>(score + a.E);  // (0: not to be chosen)
  uint32_t* value = key + a.E;
  grid_launch_dependents();
  grid_wait();
  const int t = blockIdx.x * warps + warp;
  if (t >= a.T) return;
  const float* x = a.logits + (size_t)t * a.E;
  const int size = a.E / a.n_group;
  const bool grouped = a.n_group > 1 && a.topk_group < a.n_group, by_logit = SOFTMAX && !a.bias && !(TOP2 && grouped && size > 1);
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
    key[e] = by_logit ? logit_key(xv, m) : order_key(xv != xv ? -INFINITY : number(a.bias ? __fadd_rn(s, a.bias[e]) : s));
  }
  __syncwarp();
  if (grouped) {
    for (int g = 0; g < a.n_group; ++g) {
      uint32_t b1 = 0, b2 = 0;  // the lane's two largest keys of the group
      for (int i = lane; i < size; i += 32) merge2(b1, b2, key[g * size + i], 0u);
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) {
        const uint32_t o1 = __shfl_xor_sync(kFull, b1, o), o2 = __shfl_xor_sync(kFull, b2, o);
        merge2(b1, b2, o1, o2);
      }
      if (lane == 0)
        value[g] = TOP2 && size > 1 ? order_key(number(__fadd_rn(topk_impl::key_value(b1), topk_impl::key_value(b2)))) : b1;
    }
    __syncwarp();
    // a group is dropped when at least topk_group groups order before it
    for (int g = 0; g < a.n_group; ++g) {
      int before = 0;
      for (int o = 0; o < a.n_group; ++o) before += value[o] > value[g] || (value[o] == value[g] && o < g);
      if (before >= a.topk_group)
        for (int i = lane; i < size; i += 32) key[g * size + i] = 0u;
    }
    __syncwarp();
  }
  int my_id = 0;
  float my_s = 0.f;
  for (int k = 0; k < a.K; ++k) {
    uint32_t best = 0;
    int at = 0x7FFFFFFF;
    for (int e = lane; e < a.E; e += 32) {
      const uint32_t o = key[e];
      if (o > best) best = o, at = e;
    }
    const uint32_t top = __reduce_max_sync(kFull, best);
    const int win = (int)__reduce_min_sync(kFull, best == top ? (uint32_t)at : 0x7FFFFFFFu);
    if (lane == k) my_id = win, my_s = score[win];
    __syncwarp();
    if (lane == 0) key[win] = 0u;
    __syncwarp();
  }
  write_weights(a, t, my_id, my_s);
}

// Dynamic shared memory (never touched) that keeps an SM from taking more than one wave's
// share of `blocks` CTAs: calls in a row place a call's CTAs while earlier ones still hold
// some SMs, and the fullest SM sets the call's time (4096 tokens x 256 experts: 9.1 us a
// call without, 7.7 with). fixed: a CTA's own shared memory.
size_t one_wave_pad(long long blocks, size_t fixed, const DeviceInfo& dev) {
  const long long cap = (blocks + dev.sm_count - 1) / dev.sm_count;
  if (cap < 2 || cap >= 8) return 0;
  const long long pad = (dev.smem_per_sm / cap - (long long)fixed - dev.smem_reserved) / 1024 * 1024 - 1024;
  return pad > 0 && pad + (long long)fixed <= 48 * 1024 ? (size_t)pad : 0;
}

template <int NJ, bool VEC, bool GROUPS>
int launch_registers(const GroupedArgs& a, const DeviceInfo& dev, cudaStream_t s) {
  const unsigned blocks = (unsigned)((a.T - 1) / kWarps + 1);
  const size_t fixed = kWarps * (sizeof(RouteScratch) + 2 * NJ * 32 * sizeof(uint32_t));
  return launch_pdl(route_kernel<NJ, VEC, GROUPS>, dim3(blocks), dim3(32 * kWarps), one_wave_pad(blocks, fixed, dev), s, a);
}

template <bool VEC, bool GROUPS>
int launch_nj(const GroupedArgs& a, const DeviceInfo& dev, cudaStream_t s) {
  if (a.E <= 128) return launch_registers<4, VEC, GROUPS>(a, dev, s);
  if (a.E <= 256) return launch_registers<8, VEC, GROUPS>(a, dev, s);
  if (a.E <= 512) return launch_registers<16, VEC, GROUPS>(a, dev, s);
  if (a.E <= 896) return launch_registers<28, VEC, GROUPS>(a, dev, s);
  return launch_registers<32, VEC, GROUPS>(a, dev, s);
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
  const int size = E / n_group;
  GroupedArgs a{logits, bias, T, E, K, n_group, topk_group, renormalize, scale, ids, weights, weights_bf16};
  a.softmax = scoring == MOE_SCORE_SOFTMAX, a.top2 = group_rule == MOE_GROUP_TOP2;
  a.by_size = size > 1 ? (uint32_t)(((1ull << 32) + size - 1) / size) : 0;
  const bool grouped = n_group > 1 && topk_group < n_group;
  if (E <= kMaxE && (!grouped || (n_group <= 32 && size > 1))) {
    const bool vec = E % 4 == 0 && aligned(logits, 16) && (!grouped || size % 4 == 0);
    const cudaStream_t st = as_cuda(stream);
    if (grouped) return vec ? launch_nj<true, true>(a, dev, st) : launch_nj<false, true>(a, dev, st);
    return vec ? launch_nj<true, false>(a, dev, st) : launch_nj<false, false>(a, dev, st);
  }
  const int warps = E <= kMaxE ? kWarps : 1;
  const size_t smem = (size_t)warps * (2 * E + MOE_MAX_GROUPS) * sizeof(float);  // at most 34 KB
  auto kern = a.softmax ? (a.top2 ? route_any_kernel<true, true> : route_any_kernel<true, false>)
                        : (a.top2 ? route_any_kernel<false, true> : route_any_kernel<false, false>);
  return launch_pdl(kern, dim3((T - 1) / warps + 1), dim3(32 * warps), smem, as_cuda(stream), a);
}
