// Block-128 E4M3 product for few rows per weight tile (decode batches, experts with a
// handful of rows): weights on the tensor core's lanes, rows on its columns.
//   D^T[n, c] = sum over blocks b of sw[n / 128, b] sa[c, b] sum_{k in b} w[n, k] a[c, k]
//
// Bound by the weights' stream from HBM. A tile is 128 weight rows x BN rows of a; a
// stage of the pipeline is one block of 128 columns of both: exactly the span of one
// scale, one 128-byte swizzle row, and four K = 32 MMAs. Each stage's sum goes to its own
// TMEM slot (the accumulator starts anew), and the epilogue warps fold it into FP32
// registers with the block's scales while the next stages multiply:
//   - warps 0-3: epilogue, one weight row (TMEM lane) per thread, BN accumulators each; a
//     lane fetches the scales of its columns one block ahead, times the weights' scale,
//     and hands them to its warp through shared memory (read back four columns a load);
//   - warp 4: TMA producer (weights one box, rows one box, or four rows per gather4 when
//     the rows are those of an expert's list);
//   - warp 5: MMA issuer.
// Dense: tiles with fewer than two per SM split K over a cluster of S CTAs, whose scaled
// partials are summed in rank order through distributed shared memory. Grouped: a
// persistent grid walks the tiles (expert, weight tile, row tile), found in a table of
// tile counts that every CTA builds from the offsets.
#include "fp8_gemm.cuh"

namespace moe {
namespace fp8_impl {
namespace {

constexpr int kThreads = 192;
constexpr int kWBytes = 128 * FP8_BLOCK;  // the weights of a stage
constexpr int kMaxStages = 12;
constexpr int kMaxSplits = 8;

template <int BN>
struct Narrow {
  static constexpr int kStageBytes = kWBytes + BN * FP8_BLOCK;
  static constexpr int kSlots = BN <= 32 ? 4 : 2;    // TMEM accumulators in flight
  static constexpr int kTmemCols = kSlots * BN;      // 64 .. 256
  static constexpr int kScaleBytes = 4 * 2 * BN * 4;  // [warp][parity][column]
};

struct Tile {
  int e, n0, pos, cnt;  // expert, first weight row, first list position (or row), rows
};

template <int BN, bool GROUPED>
__device__ __forceinline__ Tile tile_at(const GemmArgs& g, const int* table, int t) {
  Tile r;
  if constexpr (GROUPED) {
    // row tiles of one weight tile are neighbours: they meet its weights in L2
    r.e = tile_expert(table, g.E, t / g.nbn);
    const int c = table[r.e + 1] - table[r.e], local = t - table[r.e] * g.nbn;
    const int lo = clamp_offset(__ldg(g.offsets + r.e), g.M), hi = clamp_offset(__ldg(g.offsets + r.e + 1), g.M);
    r.n0 = local / c * 128;
    r.pos = lo + local % c * BN;
    r.cnt = min(BN, hi - r.pos);
  } else {
    const int mt = (g.M + BN - 1) / BN;
    r.e = 0;
    r.n0 = t / mt * 128;
    r.pos = t % mt * BN;
    r.cnt = min(BN, g.M - r.pos);
  }
  return r;
}

__device__ __forceinline__ void store(const GemmArgs& g, long long row, int n, float v) {
  if (g.f32)
    static_cast<float*>(g.out)[row * g.N + n] = v;
  else
    static_cast<uint16_t*>(g.out)[row * g.N + n] = f32_to_bf16(v);
}

template <int BN, bool GROUPED>
__global__ void __launch_bounds__(kThreads)
    narrow_kernel(const __grid_constant__ CUtensorMap tm_w, const __grid_constant__ CUtensorMap tm_a, const GemmArgs g,
                  int stages, int S, int max_row_tiles) {
  using C = Narrow<BN>;
  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(8) uint64_t bars[2 * kMaxStages + 2 * C::kSlots];
  __shared__ uint32_t tmem_slot;
  __shared__ int warp_sums[kThreads / 32];
  __shared__ int4 row_mem[GROUPED ? BN / 4 : 1];  // the rows of a tile, four per gather
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t raw = smem_u32(smem_raw), base = (raw + 1023u) & ~1023u;
  uint8_t* const mem = smem_raw + (base - raw);
  float* const scale_mem = reinterpret_cast<float*>(mem + stages * C::kStageBytes);
  int* const table = reinterpret_cast<int*>(mem + stages * C::kStageBytes + C::kScaleBytes);
  auto full = [&](int i) { return smem_u32(&bars[i]); };
  auto empty = [&](int i) { return smem_u32(&bars[kMaxStages + i]); };
  auto tfull = [&](int i) { return smem_u32(&bars[2 * kMaxStages + i]); };
  auto tempty = [&](int i) { return smem_u32(&bars[2 * kMaxStages + C::kSlots + i]); };

  if (threadIdx.x == 0) {
    for (int i = 0; i < stages; ++i) {
      mbar_init(full(i), 1);
      mbar_init(empty(i), 1);
    }
    for (int i = 0; i < C::kSlots; ++i) {
      mbar_init(tfull(i), 1);
      mbar_init(tempty(i), 4);  // one arrival per epilogue warp
    }
    mbar_fence_init();
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&tm_w)) : "memory");
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&tm_a)) : "memory");
  }
  if (warp == 5) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&tmem_slot)),
                 "r"(C::kTmemCols));
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  }
  tcgen05_before_sync();
  __syncthreads();
  tcgen05_after_sync();
  const uint32_t tmem = tmem_slot;
  grid_wait();
  grid_launch_dependents();
  int tiles;
  if constexpr (GROUPED) {
    tile_table(g, BN, table, warp_sums);
    tiles = min(table[g.E], max_row_tiles) * g.nbn;
  } else {
    tiles = g.nbn * ((g.M + BN - 1) / BN);
  }
  const int rank = blockIdx.x % S, t0 = blockIdx.x / S, step = gridDim.x / S;
  const int kb0 = (int)((long long)rank * g.nbk / S), kb1 = (int)((long long)(rank + 1) * g.nbk / S);

  if (warp == 4) {  // TMA producer
    Ring st;
    int issued = 0;
    bool ok = true;
    for (int t = t0; t < tiles && ok; t += step) {
      const Tile ti = tile_at<BN, GROUPED>(g, table, t);
      if constexpr (GROUPED) {
        int r[4];  // rows 4 lane .. 4 lane + 3 of the tile (row 0 for those past its end)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int c = 4 * lane + i;
          long long in = -1, out;
          if (c < ti.cnt) pair_rows(g, ti.pos + c, &in, &out);
          r[i] = in < 0 ? 0 : (int)in;
        }
        if (lane < BN / 4) row_mem[lane] = make_int4(r[0], r[1], r[2], r[3]);
        __syncwarp();
      }
      const int wrow = ti.e * g.N + ti.n0;
      for (int kb = kb0; kb < kb1; ++kb) {
        ok = __all_sync(kFullMask, mbar_wait_asleep(empty(st.slot), st.lap ^ 1u, g.err));
        if (!ok) break;
        const uint32_t dst = base + st.slot * C::kStageBytes, bar = full(st.slot);
        if (elect_one()) {
          mbar_expect_tx(bar, C::kStageBytes);
          tma_load_2d(dst, &tm_w, kb * FP8_BLOCK, wrow, bar);
          if constexpr (GROUPED) {  // (by one thread: per lane the instruction is issued lane after lane)
#pragma unroll 8
            for (int j = 0; j < BN / 4; ++j) {
              const int4 r = row_mem[j];
              tma_gather4(dst + kWBytes + j * 4 * FP8_BLOCK, &tm_a, kb * FP8_BLOCK, r.x, r.y, r.z, r.w, bar);
            }
          } else {
            tma_load_2d(dst + kWBytes, &tm_a, kb * FP8_BLOCK, ti.pos, bar);
          }
        }
        __syncwarp();
        st.next(stages);
        ++issued;
      }
    }
    // the copies still in flight land before the CTA may exit
    for (int i = issued > stages ? issued - stages : 0; i < issued; ++i)
      mbar_wait_asleep(full(i % stages), (uint32_t)(i / stages) & 1u, g.err);
  } else if (warp == 5) {  // MMA issuer
    // (the whole warp walks the loop, so that descriptors stay in uniform registers)
    constexpr uint32_t idesc = instr_desc_e4m3(BN, 128);
    const uint64_t weights0 = sw128_desc(base), rows0 = sw128_desc(base + kWBytes);
    Ring st, sl;
    bool ok = true;
    for (int t = t0; t < tiles && ok; t += step) {
      for (int kb = kb0; kb < kb1; ++kb) {
        ok = __all_sync(kFullMask, mbar_wait_asleep(tempty(sl.slot), sl.lap ^ 1u, g.err) && mbar_wait_asleep(full(st.slot), st.lap, g.err));
        if (!ok) break;
        tcgen05_after_sync();
        const uint64_t at = (uint64_t)(st.slot * (C::kStageBytes >> 4));
        if (elect_one()) {
#pragma unroll
          for (int k = 0; k < 4; ++k)
            mma_e4m3(tmem + sl.slot * BN, weights0 + at + 2 * k, rows0 + at + 2 * k, idesc, k > 0 ? 1u : 0u);
          mma_commit(empty(st.slot));
          mma_commit(tfull(sl.slot));
        }
        __syncwarp();
        st.next(stages);
        sl.next(C::kSlots);
      }
    }
    __syncwarp();
  } else {  // epilogue
    constexpr int CL = (BN + 31) / 32;  // columns whose scales a lane fetches
    constexpr int P = BN < 32 ? BN : 32;  // columns per TMEM load
    float* const sc = scale_mem + warp * 2 * BN;
    const uint32_t tl = tmem + ((uint32_t)(warp * 32) << 16);
    Ring sl;
    int parity = 0;  // of the warp's scale buffers
    bool ok = true;
    for (int t = t0; t < tiles && ok; t += step) {
      const Tile ti = tile_at<BN, GROUPED>(g, table, t);
      const float* sap[CL];
      long long out_row[CL];
#pragma unroll
      for (int i = 0; i < CL; ++i) {
        const int c = lane + 32 * i;
        long long in = -1, out = -1;
        if (c < ti.cnt) {
          if constexpr (GROUPED)
            pair_rows(g, ti.pos + c, &in, &out);
          else
            in = out = ti.pos + c;
        }
        sap[i] = in < 0 ? nullptr : g.sa + in * g.nbk;
        out_row[i] = out;
      }
      const float* swp = g.sw + ((long long)ti.e * g.nbn + ti.n0 / FP8_BLOCK) * g.nbk;
      uint64_t acc[BN / 2];
#pragma unroll
      for (int i = 0; i < BN / 2; ++i) acc[i] = 0;
      float s[CL], b = 0.f;
      auto fetch = [&](int kb) {
        b = __ldg(swp + kb);
#pragma unroll
        for (int i = 0; i < CL; ++i) s[i] = sap[i] ? __ldg(sap[i] + kb) : 0.f;
      };
      fetch(kb0);
      for (int kb = kb0; kb < kb1; ++kb) {
        float* const buf = sc + parity * BN;  // (the other parity may still be read by slower lanes)
#pragma unroll
        for (int i = 0; i < CL; ++i)
          if (lane + 32 * i < BN) buf[lane + 32 * i] = __fmul_rn(s[i], b);
        if (kb + 1 < kb1) fetch(kb + 1);
        __syncwarp();
        ok = __all_sync(kFullMask, mbar_wait_asleep(tfull(sl.slot), sl.lap, g.err));
        if (!ok) break;
        tcgen05_after_sync();
#pragma unroll
        for (int p = 0; p < BN / P; ++p) {
          uint32_t v[P];
          if constexpr (P == 16)
            tmem_ld16(tl + sl.slot * BN, v);
          else
            tmem_ld32(tl + sl.slot * BN + p * P, v);
          tmem_wait_ld();
          tmem_loaded(v);
          if (p == BN / P - 1) {  // the slot is read
            tcgen05_before_sync();
            __syncwarp();
            if (lane == 0) mbar_arrive(tempty(sl.slot));
          }
#pragma unroll
          for (int i = 0; i < P / 4; ++i) {
            const ulonglong2 f = *reinterpret_cast<const ulonglong2*>(buf + p * P + 4 * i);
            uint64_t* a = acc + (p * P) / 2 + 2 * i;
            a[0] = fma2(pack2(v[4 * i], v[4 * i + 1]), f.x, a[0]);
            a[1] = fma2(pack2(v[4 * i + 2], v[4 * i + 3]), f.y, a[1]);
          }
        }
        parity ^= 1;
        sl.next(C::kSlots);
      }
      if (!ok) break;
      const int n = ti.n0 + threadIdx.x;  // this thread's weight row
      if (S == 1) {
#pragma unroll
        for (int c = 0; c < BN; c += 2) {
          float v[2];
          unpack2(acc[c / 2], &v[0], &v[1]);
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const long long row = __shfl_sync(kFullMask, out_row[(c + i) / 32], (c + i) & 31);
            if (row >= 0 && n < g.N) store(g, row, n, v[i]);
          }
        }
      } else {  // partial columns for the cluster's sum (the stages are all consumed)
        float* part = reinterpret_cast<float*>(mem);
#pragma unroll
        for (int c = 0; c < BN; c += 2) {
          float v[2];
          unpack2(acc[c / 2], &v[0], &v[1]);
          part[c * 128 + threadIdx.x] = v[0];
          part[(c + 1) * 128 + threadIdx.x] = v[1];
        }
      }
    }
  }
  if (S > 1) {  // (one tile per cluster; dense)
    __syncwarp();
    cluster_sync();  // every split's partial is written and visible
    if (warp < 4) {
      const Tile ti = tile_at<BN, GROUPED>(g, table, t0);
      const int n = ti.n0 + threadIdx.x;
      uint32_t peer[kMaxSplits];
#pragma unroll
      for (int q = 0; q < kMaxSplits; ++q) peer[q] = map_rank(base, q < S ? q : 0) + 4u * threadIdx.x;
      for (int c = rank; c < ti.cnt; c += S) {
        float sum = 0.f;
#pragma unroll
        for (int q = 0; q < kMaxSplits; ++q) {
          if (q < S) {
            float v;
            asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(peer[q] + 512u * c) : "memory");
            sum = __fadd_rn(sum, v);
          }
        }
        if (n < g.N) store(g, ti.pos + c, n, sum);
      }
    }
    cluster_sync();  // no CTA leaves while its partial may be read
  }
  tcgen05_before_sync();
  __syncthreads();
  if (warp == 5) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(C::kTmemCols));
}

template <int BN, bool GROUPED>
int launch(const GemmArgs& g, int sm_count, cudaStream_t stream) {
  using C = Narrow<BN>;
  CUtensorMap tm_w, tm_a;
  if (!make_code_map(&tm_w, g.w, (long long)g.E * g.N, g.K, 128)) return MOE_ERR_CUDA;
  if (!make_code_map(&tm_a, g.a, g.a_rows, g.K, GROUPED ? 1 : BN)) return MOE_ERR_CUDA;
  auto kern = narrow_kernel<BN, GROUPED>;
  const size_t extra = 1024 + C::kScaleBytes + (GROUPED ? (g.E + 1) * 4 : 0);
  // row tiles (grouped: at most, of ascending offsets)
  const long long rows = GROUPED ? (long long)g.M / BN + (g.E < g.M ? g.E : g.M) : ((long long)g.M + BN - 1) / BN;
  const long long tiles = rows * g.nbn;
  if (tiles >= (1LL << 31) - (1 << 16) || rows >= kMaxRowTiles) return MOE_ERR_CAPACITY;
  int S = 1, stages = (int)((kMaxSmem - kStaticSmem - extra) / C::kStageBytes);
  if (stages > kMaxStages) stages = kMaxStages;
  // A CTA takes at least its TMEM columns' share of an SM's shared memory, so that the CTAs
  // an SM holds never ask for more than its 512 columns: tcgen05.alloc would make one
  // wait for another, in a ring of waits where clusters meet at barriers.
  const size_t least = (size_t)C::kTmemCols * (kSmSmem / 512);
  if (!GROUPED) {
    // the most splits whose CTAs are all resident at once, two per SM while they fit
    for (int s = kMaxSplits; s >= 2; --s) {
      const int kbs = (g.nbk + s - 1) / s, st = kbs < kMaxStages ? kbs : kMaxStages;
      size_t bytes = extra + (size_t)st * C::kStageBytes;
      bytes = bytes < least ? least : bytes;
      const int per_sm = 2 * (bytes + kStaticSmem) <= kSmSmem ? 2 : 1;
      if (s <= g.nbk && bytes + kStaticSmem <= (size_t)kMaxSmem && (size_t)st * C::kStageBytes >= (size_t)BN * 512 &&
          tiles * s <= (long long)per_sm * sm_count) {
        S = s, stages = st;
        break;
      }
    }
  }
  size_t smem = extra + (size_t)stages * C::kStageBytes;
  if (smem < least) smem = least;
  const void* f = reinterpret_cast<const void*>(kern);
  if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxSmem - kStaticSmem) != cudaSuccess ||
      prefer_max_shared(f) != MOE_OK)
    return MOE_ERR_CUDA;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(S > 1 ? tiles * S : (tiles < sm_count ? tiles : sm_count)));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = S, attr[1].val.clusterDim.y = 1, attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = S > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kern, tm_w, tm_a, g, stages, S, (int)rows) == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

template <bool GROUPED>
int launch_bn(int bn, const GemmArgs& g, int sm_count, cudaStream_t stream) {
  switch (bn) {
    case 16: return launch<16, GROUPED>(g, sm_count, stream);
    case 32: return launch<32, GROUPED>(g, sm_count, stream);
    case 64: return launch<64, GROUPED>(g, sm_count, stream);
    default: return launch<128, GROUPED>(g, sm_count, stream);
  }
}

}  // namespace

int launch_narrow(const GemmArgs& g, int sm_count, cudaStream_t stream) {
  // dense: the narrowest tile that holds every row; grouped: that holds an expert of average load and half
  const long long want = g.offsets ? (3LL * g.M / 2 + g.E - 1) / g.E : g.M;
  int bn = 16;
  while (bn < 128 && bn < want) bn *= 2;
  return g.offsets ? launch_bn<true>(bn, g, sm_count, stream) : launch_bn<false>(bn, g, sm_count, stream);
}

}  // namespace fp8_impl
}  // namespace moe
