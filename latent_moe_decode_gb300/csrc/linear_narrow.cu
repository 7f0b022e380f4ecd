// BF16 product with an epilogue for few rows of a: rows of b (weights) on the tensor core's 128
// lanes, those of a on its columns.
//   D^T[n, m] = sum_k b[n, k] a[m, k]
//
// Bound by the stream of b from HBM, so the tiles are small enough to put every SM to work: 128
// rows of b x bn of a, K split over a cluster of S CTAs, one or two CTAs an SM. (Asking L2 for a
// CTA's share of b before it waits for the preceding kernel made calls longer: that kernel's end
// was not reported before these requests had been served.)
// Gated, a tile holds 64 rows of the gate and the same 64 of the other half.
//   - warp 8: TMA producer, warp 9: MMA issuer. A stage is 64 of K of both operands;
//   - the K of a CTA is taken in `runs` contiguous parts, each with TMEM columns of its own: the
//     tensor core cuts its running sum off towards zero at every step, which shorter sums, added
//     with rounding to nearest, keep to some 4e-7 of the whole;
//   - warps 0-7 add the runs and send the partial sums from their registers to the CTA of the
//     cluster that adds them up, in rank order, and finishes them: sixteen rows of a at one row of
//     b a thread (four took 450 cycles a turn, too, mostly branches). The partials arrive on a
//     barrier of their own; where they take the stages' place a cluster barrier comes first.
//     (Loads of the others' partials, between two cluster barriers, took 2 to 5 us; bulk copies,
//     which have to be left in shared memory first, no less.)
#include "linear.cuh"

namespace moe {
namespace linear_impl {
namespace {

constexpr int kEpiWarps = 8;
constexpr int kWarps = kEpiWarps + 2;
constexpr int kThreads = 32 * kWarps;
constexpr int kMaxExactRun = 12;  // blocks of K of a run of an FP32 result, in any case (16 are off by 1e-6 of the whole)

struct NarrowArgs {
  Epilogue e;
  int M, N, nbk;
  int bn, splits, stages, runs, tmem_cols;
  int apart;           // the partials have a place of their own beside the stages
  int row_tiles;       // of a
  int b_transposed;
};

__device__ __forceinline__ void mma(uint32_t tmem_d, uint64_t adesc, uint64_t bdesc, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}\n" ::"r"(tmem_d),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(acc));
}

template <int W>
struct Width {
  static constexpr int value = W;
};

// Column n of `rows` (up to 16) rows from `row` on: the residual, and the epilogue. A warp's lanes hold
// consecutive columns.
__device__ __forceinline__ void fetch_residual(const NarrowArgs& g, long long row, int n, int rows, float (&r)[16]) {
  const Epilogue& e = g.e;
  if (!e.residual) return;
  // (the loads of a type together: a choice for each would wait for each)
  if (e.residual_f32) {
    const float* at = static_cast<const float*>(e.residual) + row * e.ldr + n;
#pragma unroll
    for (int j = 0; j < 16; ++j, at += e.ldr) r[j] = j < rows ? *at : 0.f;
  } else {
    const uint16_t* at = static_cast<const uint16_t*>(e.residual) + row * e.ldr + n;
    uint16_t u[16];
#pragma unroll
    for (int j = 0; j < 16; ++j, at += e.ldr) u[j] = j < rows ? *at : (uint16_t)0;
#pragma unroll
    for (int j = 0; j < 16; ++j) r[j] = bf16_to_f32(u[j]);
  }
}
__device__ __forceinline__ void store_column(void* p, long long ld, int f32, long long row, int n, int rows, const float (&v)[16]) {
  if (f32) {
    float* at = static_cast<float*>(p) + row * ld + n;
#pragma unroll
    for (int j = 0; j < 16; ++j, at += ld)
      if (j < rows) *at = v[j];
  } else {
    uint16_t* at = static_cast<uint16_t*>(p) + row * ld + n;
#pragma unroll
    for (int j = 0; j < 16; ++j, at += ld)
      if (j < rows) *at = f32_to_bf16(v[j]);
  }
}
template <bool GATED>
__device__ __forceinline__ void finish_rows(const NarrowArgs& g, long long row, int n, int rows, float (&z)[16], const float (&u)[16],
                                            const float (&r)[16]) {
  const Epilogue& e = g.e;
  if (GATED) {
    if (e.pre) {
      store_column(e.pre, e.ldp, 0, row, n, rows, z);
      store_column(e.pre, e.ldp, 0, row, g.N + n, rows, u);
    }
    act_impl::apply<true>(e.act, z);
#pragma unroll
    for (int j = 0; j < 16; ++j) z[j] = __fmul_rn(z[j], u[j]);
    store_column(e.out, e.ldo, 0, row, n, rows, z);
    return;
  }
  const float bias = e.bias ? load_as_f32(e.bias, n, e.bias_f32) : 0.f;
#pragma unroll
  for (int j = 0; j < 16; ++j) z[j] = __fadd_rn(z[j], bias);
  if (e.pre) store_column(e.pre, e.ldp, 0, row, n, rows, z);
  if (e.out_f32)
    act_impl::apply<false>(e.act, z);
  else
    act_impl::apply<true>(e.act, z);
  if (e.residual) {
#pragma unroll
    for (int j = 0; j < 16; ++j) z[j] = __fadd_rn(z[j], r[j]);
  }
  store_column(e.out, e.ldo, e.out_f32, row, n, rows, z);
}

template <bool GATED>
__global__ void __launch_bounds__(kThreads, 2)
    linear_narrow_kernel(const __grid_constant__ CUtensorMap tm_a, const __grid_constant__ CUtensorMap tm_b,
                         const __grid_constant__ NarrowArgs g, uint32_t* err) {
  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(8) uint64_t bars[2 * kNarrowStages + 2];
  __shared__ uint32_t tmem_slot;
  const int warp = __shfl_sync(kFullMask, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;  // (warp: uniform)
  const uint32_t raw = smem_u32(smem_raw), base = (raw + 1023u) & ~1023u;
  // the partial sums that this CTA adds up: beside the stages, or in their place once they are consumed
  const uint32_t partials = base + (uint32_t)(g.apart ? g.stages * (kBBytes + g.bn * kBlockK * 2) : 0);
  float* const sums = reinterpret_cast<float*>(smem_raw + (partials - raw));
  auto full = [&](int i) { return smem_u32(&bars[i]); };
  auto empty = [&](int i) { return smem_u32(&bars[kNarrowStages + i]); };
  const uint32_t done = smem_u32(&bars[2 * kNarrowStages]), came = done + 8;  // the products; the partials for this CTA
  const int S = g.splits, stages = g.stages;

  if (threadIdx.x == 0) {
    for (int i = 0; i < stages; ++i) {
      mbar_init(full(i), 1);
      mbar_init(empty(i), 1);
    }
    mbar_init(done, 1);
    mbar_init(came, 1);
    mbar_fence_init();
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&tm_a)) : "memory");
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&tm_b)) : "memory");
  }
  if (warp == kEpiWarps + 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&tmem_slot)), "r"(g.tmem_cols));
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  }
  tcgen05_before_sync();
  __syncthreads();
  tcgen05_after_sync();
  const uint32_t tmem = tmem_slot;
  if (g.apart) cluster_arrive_relaxed();  // (this CTA has started)

  constexpr int kOutCols = GATED ? kLanes / 2 : kLanes;  // columns of out a tile
  const int rank = blockIdx.x % S, tile = blockIdx.x / S;
  const int m0 = tile % g.row_tiles * g.bn, n0 = tile / g.row_tiles * kOutCols, cnt = min(g.bn, g.M - m0);
  const int kb0 = (int)((long long)rank * g.nbk / S), kb1 = (int)((long long)(rank + 1) * g.nbk / S);
  const int run = (kb1 - kb0 - 1) / g.runs + 1;  // blocks
  const uint32_t stage_bytes = kBBytes + (uint32_t)g.bn * kBlockK * 2;

  grid_wait();
  grid_launch_dependents();

  if (warp == kEpiWarps) {  // TMA producer
    Ring st;
    bool ok = true;
    for (int kb = kb0; kb < kb1; ++kb) {
      ok = __all_sync(kFullMask, mbar_wait_asleep(empty(st.slot), st.lap ^ 1u, err));
      if (!ok) break;
      const uint32_t dst = base + st.slot * stage_bytes, bar = full(st.slot);
      const int k0 = kb * kBlockK;
      if (elect_one()) {
        mbar_expect_tx(bar, stage_bytes);
        if (GATED) {
          tma_load_2d(dst, &tm_b, k0, n0, bar);
          tma_load_2d(dst + kBBytes / 2, &tm_b, k0, g.N + n0, bar);
        } else if (g.b_transposed) {
          tma_load_2d(dst, &tm_b, n0, k0, bar);
          tma_load_2d(dst + kBBytes / 2, &tm_b, n0 + 64, k0, bar);
        } else {
          tma_load_2d(dst, &tm_b, k0, n0, bar);
        }
        tma_load_2d(dst + kBBytes, &tm_a, k0, m0, bar);
      }
      __syncwarp();
      st.next((uint32_t)stages);
    }
    // The CTA may not exit with arrivals on its barriers to come: those of the last commits, which
    // are after the copies; without them (the issuer gave up) the copies in flight.
    const int issued = kb1 - kb0, first = issued > stages ? issued - stages : 0;
    for (int i = first; i < issued && ok; ++i)
      ok = __all_sync(kFullMask, mbar_wait_asleep(empty(i % stages), (uint32_t)(i / stages) & 1u, err));
    for (int i = first; i < issued && !ok; ++i) mbar_wait_asleep(full(i % stages), (uint32_t)(i / stages) & 1u, err);
  } else if (warp == kEpiWarps + 1) {  // MMA issuer
    // (the whole warp walks the loop, so that descriptors stay in uniform registers)
    const uint32_t idesc = instr_desc(kLanes, g.bn, g.b_transposed, false);
    const uint64_t b0 = operand_desc(base, g.b_transposed), a0 = operand_desc(base + kBBytes, false);
    const uint32_t bs = operand_step(g.b_transposed), as = operand_step(false);
    Ring st;
    int left = run;
    uint32_t d = tmem;
    for (int kb = kb0; kb < kb1; ++kb) {
      if (!__all_sync(kFullMask, mbar_wait_asleep(full(st.slot), st.lap, err))) break;
      tcgen05_after_sync();
      const uint64_t at = (uint64_t)(st.slot * (stage_bytes >> 4));
      if (elect_one()) {
#pragma unroll
        for (uint32_t k = 0; k < 4; ++k) mma(d, b0 + at + k * bs, a0 + at + k * as, idesc, left < run || k > 0 ? 1u : 0u);
        mma_commit(empty(st.slot));
        if (kb + 1 == kb1) mma_commit(done);
      }
      __syncwarp();
      st.next((uint32_t)stages);
      if (--left == 0) left = run, d += g.bn;
    }
  }
  __syncwarp();

  // The partials, four columns of a lane together, to the rank that sums them: [split][columns / 4][lane][4].
  const int quads = (cnt + 3) / 4, share = (quads - 1) / S + 1;  // groups of four columns; those of a rank
  const int first = rank * share, have = min(share, quads - first);  // this rank's (none: <= 0)
  const bool adds = (GATED || S > 1) && have > 0;
  if (threadIdx.x == 0 && adds && S > 1) mbar_expect_tx(came, (uint32_t)(S * have * kLanes) * 16);
  bool ok = true;
  if (warp < kEpiWarps) {
    ok = __all_sync(kFullMask, mbar_wait_asleep(done, 0u, err));
    tcgen05_after_sync();
  }
  if (!g.apart) cluster_arrive_relaxed();  // this CTA's stages are consumed
  bool free = false;                        // (those of the others are)
  if (warp < kEpiWarps && ok) {
    const uint32_t tl = tmem + ((uint32_t)((warp & 3) * 32) << 16);
    const int runs = (kb1 - kb0 - 1) / run + 1;  // those that there are
    auto send = [&](int c, auto width) {  // columns c .. c + width - 1
      constexpr int W = decltype(width)::value;
      const int n = n0 + 32 * (warp & 3) + lane;
      float z[W], res[W / 16][16] = {};
      if (!GATED && S == 1 && n < g.N) {
#pragma unroll
        for (int h = 0; h < W; h += 16) fetch_residual(g, m0 + c + h, n, cnt - c - h, res[h / 16]);
      }
      __syncwarp();  // (lanes beyond N had nothing to fetch; what follows is one instruction of the whole warp)
      for (int r = 0; r < runs; ++r) {
        uint32_t v[W];
        if constexpr (W == 16)
          tmem_ld16(tl + r * g.bn + c, v);
        else
          tmem_ld32(tl + r * g.bn + c, v);
        tmem_wait_ld();
        tmem_loaded(v);
#pragma unroll
        for (int j = 0; j < W; ++j) z[j] = r == 0 ? __uint_as_float(v[j]) : __fadd_rn(z[j], __uint_as_float(v[j]));
      }
      if (!GATED && S == 1) {  // (nothing to add)
#pragma unroll
        for (int h = 0; h < W; h += 16) {
          float zh[16];
#pragma unroll
          for (int j = 0; j < 16; ++j) zh[j] = z[h + j];
          if (n < g.N && c + h < cnt) finish_rows<GATED>(g, m0 + c + h, n, cnt - c - h, zh, zh, res[h / 16]);
        }
        __syncwarp();
        return;
      }
      if (!free) cluster_wait(), free = true;
      if (S == 1) {  // (gated; not sent: the launch is of no cluster, in which st.async is an illegal instruction)
#pragma unroll
        for (int j = 0; j < W / 4; ++j)
          if (c / 4 + j < quads)
            *reinterpret_cast<float4*>(sums + ((c / 4 + j) * kLanes + 32 * (warp & 3) + lane) * 4) =
                make_float4(z[4 * j], z[4 * j + 1], z[4 * j + 2], z[4 * j + 3]);
        return;
      }
      int owner = c / 4 / share, at = c / 4 - owner * share;
#pragma unroll
      for (int j = 0; j < W / 4; ++j) {
        if (c / 4 + j < quads)
          send16(map_rank(partials, owner) + (uint32_t)((rank * share + at) * kLanes + 32 * (warp & 3) + lane) * 16, z[4 * j], z[4 * j + 1],
                 z[4 * j + 2], z[4 * j + 3], map_rank(came, owner));
        if (++at == share) at = 0, ++owner;
      }
    };
    if (cnt <= 32) {
      if (16 * (warp >> 2) < cnt) send(16 * (warp >> 2), Width<16>());
    } else {
      int c = 32 * (warp >> 2);
      for (; c + 32 <= g.bn && c < cnt; c += 64) send(c, Width<32>());
      if (c < cnt) send(c, Width<16>());
    }
    tcgen05_before_sync();
  }
  __syncwarp();
  if (!free) cluster_wait();
  __syncwarp();
  if (adds) {
    // Sixteen columns (gated: of lanes n and 64 + n) a thread; the first residual while the partials are on their way.
    const int items = (have + 3) / 4 * kOutCols;
    auto place = [&](int it, int* c, int* n) {
      *c = 4 * first + it / kOutCols * 16;
      *n = n0 + it % kOutCols;
    };
    int c, n;
    float r[16] = {};
    place(threadIdx.x, &c, &n);
    if (!GATED && (int)threadIdx.x < items && n < g.N) fetch_residual(g, m0 + c, n, min(cnt, 4 * (first + have)) - c, r);
    __syncwarp();
    if (S > 1)
      mbar_wait_asleep(came, 0u, err);
    else
      __syncthreads();
    for (int it = threadIdx.x; it < items; it += kThreads) {
      place(it, &c, &n);
      const int rows = min(cnt, 4 * (first + have)) - c;
      if (n >= g.N) continue;
      if (!GATED && it >= kThreads) fetch_residual(g, m0 + c, n, rows, r);
      float z[16], u[16];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if (4 * j >= rows) break;
        const float* at = sums + ((it / kOutCols * 4 + j) * kLanes + it % kOutCols) * 4;
        sum_partials(at, S, share * kLanes * 4, z + 4 * j);
        if (GATED) sum_partials(at + kLanes / 2 * 4, S, share * kLanes * 4, u + 4 * j);
      }
      finish_rows<GATED>(g, m0 + c, n, rows, z, u, r);
    }
  }
  __syncwarp();
  cluster_arrive_relaxed();
  cluster_wait();  // no CTA leaves before the partials for it have come
  tcgen05_after_sync();
  if (warp == kEpiWarps + 1)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(g.tmem_cols));
}

// Clusters of `splits` whole-SM CTAs that are resident at once, looked up once a device; -1 where that fails.
int max_clusters(int splits, const DeviceInfo& dev) {
  static PerDevice<kMaxSplits + 1> known;
  return known.get(dev.device, splits, [&] {
    return resident_clusters(reinterpret_cast<const void*>(linear_narrow_kernel<false>), splits, kThreads, room(1) + 1024, kMaxSmem - kStaticSmem);
  });
}

}  // namespace

// Equal tiles of the rows of a, in sixteens, K split over clusters that are all resident; two CTAs
// an SM only where there are more of them than SMs (fewer would not be dealt out evenly). The estimate: 3.1
// to 3.3 us of launch, first loads and end; the stages' way into an SM at 109 bytes a ns for one
// CTA, 144 for two; all bytes at 10 TB/s (the weights partly in L2) where two CTAs an SM ask for them, 6.2
// where one does; the partials, 23 ns a column (none to send: 7). Fitted to 1950 points, T 1 to 1500,
// N 256 to 7168, K 512 to 7168, tiles of 16 to 256 rows, 1 to 8 splits: 8 % off (rms); the tile and split it
// chooses are 2.5 % slower than the best of them on average, 14 % at most. (Without bias or activation, which it does not count.)
int plan_narrow(const Product& s, bool gated, const DeviceInfo& dev, NarrowPlan* plan) {
  NarrowPlan best = {0, 0, 0, 1e30};
  const int nbk = (s.K - 1) / kBlockK + 1;
  const long long lane_tiles = (s.N - 1) / (gated ? kLanes / 2 : kLanes) + 1;
  const double hbm = 2e-3 / 6.7756 * ((double)(gated ? 2 : 1) * s.N * s.K + (double)s.M * (s.K + s.N));
  const int extra = s.e.residual ? 3 : 0;  // (its loads, a thread's sixteen at a time)
  int last = 0;
  for (int most : {256, 192, 128, 96, 64, 48, 32, 16}) {
    const int row_tiles = (s.M - 1) / most + 1, bn = ((s.M - 1) / row_tiles + 1 + 15) / 16 * 16, stage = narrow_stage_bytes(bn);
    if (bn == last) continue;
    last = bn;
    const long long tiles = ((s.M - 1) / bn + 1) * lane_tiles;
    for (int splits = 1; splits <= kMaxSplits && splits <= nbk; ++splits) {
      if (splits > 1 && tiles * splits > 2LL * dev.sm_count) break;
      const double feed = (double)((nbk - 1) / splits + 1) * stage;
      const long long ctas = tiles * splits;
      for (int per_sm = 1; per_sm <= 2; ++per_sm) {
        if (per_sm == 2 && ctas <= dev.sm_count) continue;
        if ((nbk - 1) / splits + 1 > (s.e.out_f32 ? kMaxExactRun : kMaxCutBlocks) * (512 / per_sm / bn)) continue;
        if (bn > 512 / per_sm || partial_bytes(bn, splits) > room(per_sm)) continue;
        if (splits > 1) {
          const int clusters = max_clusters(splits, dev);
          if (clusters < 0) return MOE_ERR_CUDA;
          if (tiles > (long long)per_sm * clusters) continue;
        }
        if (ctas > (long long)dev.sm_count * per_sm) continue;  // (more than one wave is the wide kernel's)
        const double here = per_sm == 2 && ctas > dev.sm_count ? 2.0 : 1.0;
        const double body = here * feed / (per_sm == 2 ? 143.6 : 108.9);
        const double stream = hbm * (1.517 - 0.845 * (ctas < 2LL * dev.sm_count ? ctas / (2.0 * dev.sm_count) : 1.0));
        const double tail = splits > 1 ? here * bn * 23 - 240 : here * bn * (7.3 + extra);
        const double ns = 3320 + (body > stream ? body : stream) + tail;
        if (ns < best.ns) best = {bn, splits, per_sm, ns};
      }
    }
  }
  *plan = best;
  return MOE_OK;
}

namespace {

template <bool GATED>
int launch(const Product& s, const NarrowPlan& plan, const DeviceInfo& dev, cudaStream_t stream) {
  NarrowArgs g = {};
  g.e = s.e, g.M = s.M, g.N = s.N, g.nbk = (s.K - 1) / kBlockK + 1, g.b_transposed = s.b.transposed;
  g.bn = plan.bn, g.splits = plan.splits;
  g.row_tiles = (s.M - 1) / g.bn + 1;
  const int cols = GATED ? kLanes / 2 : kLanes;
  const long long tiles = (long long)g.row_tiles * ((s.N - 1) / cols + 1);
  if (tiles >= (1LL << 31) - (1 << 16)) return MOE_ERR_CAPACITY;
  const NarrowShape shape = narrow_shape(plan.bn, plan.splits, plan.per_sm, g.nbk);
  g.stages = shape.stages, g.runs = shape.runs, g.tmem_cols = shape.tmem_cols, g.apart = shape.apart;
  CUtensorMap tm_a, tm_b;
  if (!make_map(&tm_a, s.a, s.M, s.K, g.bn)) return MOE_ERR_CUDA;
  if (!make_map(&tm_b, s.b, GATED ? 2LL * s.N : s.N, s.K, GATED ? kLanes / 2 : kLanes)) return MOE_ERR_CUDA;
  auto kern = linear_narrow_kernel<GATED>;
  static OncePerDevice once;
  if (!once.allow(reinterpret_cast<const void*>(kern), kMaxSmem - kStaticSmem)) return MOE_ERR_CUDA;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(tiles * g.splits));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = shape.smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = (unsigned)g.splits, attr[1].val.clusterDim.y = 1, attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = g.splits > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kern, tm_a, tm_b, g, dev.error_word) == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

}  // namespace

int launch_narrow(const Product& product, bool gated, const NarrowPlan& plan, const DeviceInfo& dev, cudaStream_t stream) {
  return gated ? launch<true>(product, plan, dev, stream) : launch<false>(product, plan, dev, stream);
}

}  // namespace linear_impl
}  // namespace moe
