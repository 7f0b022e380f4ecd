// Block-128 E4M3 product for few rows per weight tile (decode batches, experts with a
// handful of rows): weights on the tensor core's lanes, rows on its columns.
//   D^T[n, c] = sum over blocks b of sw[n / 128, b] sa[c, b] sum_{k in b} w[n, k] a[c, k]
//
// Bound by the weights' stream from HBM. A tile is 128 weight rows x BN rows of a; a
// stage of the pipeline is one block of 128 columns of both: exactly the span of one
// scale, one 128-byte swizzle row, and four K = 32 MMAs. Each stage's sum goes to its own
// TMEM slot (the accumulator starts anew), and the epilogue warps fold it into FP32
// registers with the block's scales while the next stages multiply:
//   - NG groups of 4 CG epilogue warps, one weight row (TMEM lane) and BN / CG columns per
//     thread; with two groups they take a persistent CTA's tiles in turn, each with TMEM
//     slots of its own, so one tile's output and the next tile's first blocks overlap;
//   - a TMA producer warp (a box of weights and one of rows a stage) and an MMA issuer warp;
//     rows that an expert's list names one by one are copied by a warp of their own;
//   - a scale warp: the columns' scales of a block, times the weights' scale, to shared
//     memory beside the block's TMEM slot (one barrier tells the epilogue of both).
// Dense: tiles with fewer than two per SM split K over a cluster of S CTAs, whose scaled
// partials are summed in rank order through distributed shared memory. Grouped: a
// persistent grid walks the tiles (expert, weight tile, row tile), found in a table of
// tile counts that every CTA builds from the offsets. (TMA's gather4 for the named rows
// took 72 cycles for four, so that at 32 rows a tile the copies and not HBM set the pace:
// 885 us for 1020 tokens x 16 of 896 experts against 505.)
#include "fp8_gemm.cuh"

namespace moe {
namespace fp8_impl {
namespace {

constexpr int kWBytes = 128 * FP8_BLOCK;  // the weights of a stage
constexpr int kMaxStages = 12;
constexpr int kMaxSplits = 8;

// Where the rows of a tile come from: consecutive rows of a; consecutive positions of an
// expert's list, rows in list order; or the rows that the list's pairs name.
enum Rows { kDense, kListed, kNamed };

template <int BN, Rows ROWS, int NG, int CG>
struct Narrow {
  static constexpr int kEpiWarps = 4 * NG * CG;
  static constexpr int kThreads = 32 * (kEpiWarps + (ROWS == kNamed ? 4 : 3));
  static constexpr int kStageBytes = kWBytes + BN * FP8_BLOCK;
  static constexpr int kSlots = NG * BN <= 64 ? 4 : 2;  // TMEM accumulators of a group
  static constexpr int kTmemCols = NG * kSlots * BN;    // 64 .. 256
  static constexpr int kPerSm = NG == 1 && BN <= 64 ? 2 : 1;  // CTAs an SM holds
  static constexpr int kScaleBytes = NG * kSlots * BN * 4;
};

struct Tile {
  int e, n0, pos, cnt;  // expert, first weight row, first list position (or row), rows
};

// Grouped: table[0 .. E] the experts' first tiles, table[E + 1 ..] their first positions.
template <int BN, Rows ROWS>
__device__ __forceinline__ Tile tile_at(const GemmArgs& g, const int* table, int t) {
  Tile r;
  if constexpr (ROWS != kDense) {
    // row tiles of one weight tile are neighbours: they meet its weights in L2
    r.e = tile_expert(table, g.E, t / g.nbn);
    const int c = table[r.e + 1] - table[r.e], local = t - table[r.e] * g.nbn;
    const int lo = table[g.E + 1 + r.e], hi = table[g.E + 2 + r.e];
    r.n0 = local / c * 128;
    r.pos = lo + local % c * BN;
    r.cnt = min(BN, hi - r.pos);
  } else {
    const int mt = (g.M - 1) / BN + 1;
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

template <int BN, Rows ROWS, int NG, int CG>
__global__ void __launch_bounds__(Narrow<BN, ROWS, NG, CG>::kThreads, Narrow<BN, ROWS, NG, CG>::kPerSm)
    narrow_kernel(const __grid_constant__ CUtensorMap tm_w, const __grid_constant__ CUtensorMap tm_a, const GemmArgs g,
                  long long a_rows, int stages, int S, int max_row_tiles) {
  using C = Narrow<BN, ROWS, NG, CG>;
  constexpr bool GROUPED = ROWS != kDense;
  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(8) uint64_t bars[2 * kMaxStages + 3 * NG * C::kSlots];
  __shared__ uint32_t tmem_slot;
  __shared__ int warp_sums[C::kThreads / 32];
  const int warp = __shfl_sync(kFullMask, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;  // (warp: uniform)
  const uint32_t raw = smem_u32(smem_raw), base = (raw + 1023u) & ~1023u;
  uint8_t* const mem = smem_raw + (base - raw);
  float* const scale_mem = reinterpret_cast<float*>(mem + stages * C::kStageBytes);  // [group][slot][column]
  int* const table = reinterpret_cast<int*>(mem + stages * C::kStageBytes + C::kScaleBytes);
  auto full = [&](int i) { return smem_u32(&bars[i]); };
  auto empty = [&](int i) { return smem_u32(&bars[kMaxStages + i]); };
  // (group * kSlots + slot): sums and scales are there; the sums are read; the scales are read
  auto tfull = [&](int i) { return smem_u32(&bars[2 * kMaxStages + i]); };
  auto tempty = [&](int i) { return smem_u32(&bars[2 * kMaxStages + NG * C::kSlots + i]); };
  auto sempty = [&](int i) { return smem_u32(&bars[2 * kMaxStages + 2 * NG * C::kSlots + i]); };

  if (threadIdx.x == 0) {
    for (int i = 0; i < stages; ++i) {
      mbar_init(full(i), ROWS == kNamed ? 33 : 1);  // the boxes' bytes; each lane's share of the named rows
      mbar_init(empty(i), 1);
    }
    for (int i = 0; i < NG * C::kSlots; ++i) {
      mbar_init(tfull(i), 2);   // the MMA's commit and the scale warp
      mbar_init(tempty(i), 4 * CG);  // one arrival per epilogue warp of the group
      mbar_init(sempty(i), 4 * CG);
    }
    mbar_fence_init();
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&tm_w)) : "memory");
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&tm_a)) : "memory");
  }
  if (warp == C::kEpiWarps + 1) {
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
    for (int e = threadIdx.x; e <= g.E; e += C::kThreads) table[g.E + 1 + e] = clamp_offset(__ldg(g.offsets + e), g.M);
    tile_table(g, BN, table, warp_sums);
    tiles = min(table[g.E], max_row_tiles) * g.nbn;
  } else {
    tiles = g.nbn * ((g.M - 1) / BN + 1);
  }
  const int rank = blockIdx.x % S, t0 = blockIdx.x / S, step = gridDim.x / S;
  const int kb0 = (int)((long long)rank * g.nbk / S), kb1 = (int)((long long)(rank + 1) * g.nbk / S);
  // A group's blocks are numbered on through its tiles: block i goes to slot i % kSlots.
  constexpr uint32_t kMask = C::kSlots - 1;
  auto lap = [](uint32_t i) { return (i / C::kSlots) & 1u; };

  if (warp == C::kEpiWarps) {  // TMA producer
    Ring st;
    int issued = 0;
    bool ok = true;
    for (int t = t0; t < tiles && ok; t += step) {
      const Tile ti = tile_at<BN, ROWS>(g, table, t);
      const int wrow = ti.e * g.N + ti.n0;
      for (int kb = kb0; kb < kb1; ++kb) {
        ok = __all_sync(kFullMask, mbar_wait_asleep(empty(st.slot), st.lap ^ 1u, g.err));
        if (!ok) break;
        const uint32_t dst = base + st.slot * C::kStageBytes, bar = full(st.slot);
        if (elect_one()) {
          mbar_expect_tx(bar, ROWS == kNamed ? kWBytes : C::kStageBytes);
          tma_load_2d(dst, &tm_w, kb * FP8_BLOCK, wrow, bar);
          if (ROWS != kNamed) tma_load_2d(dst + kWBytes, &tm_a, kb * FP8_BLOCK, ti.pos, bar);
        }
        __syncwarp();
        st.next(stages);
        ++issued;
      }
    }
    // The CTA may not exit with arrivals on its barriers to come: the issuer's last commits, which are
    // after the copies; without them (it gave up) the copies in flight.
    const int first = issued > stages ? issued - stages : 0;
    for (int i = first; i < issued && ok; ++i)
      ok = __all_sync(kFullMask, mbar_wait_asleep(empty(i % stages), (uint32_t)(i / stages) & 1u, g.err));
    for (int i = first; i < issued && !ok; ++i) mbar_wait_asleep(full(i % stages), (uint32_t)(i / stages) & 1u, g.err);
  } else if (warp == C::kEpiWarps + 1) {  // MMA issuer
    // (the whole warp walks the loop, so that descriptors stay in uniform registers)
    constexpr uint32_t idesc = instr_desc_e4m3(BN, 128);
    const uint64_t weights0 = sw128_desc(base), rows0 = sw128_desc(base + kWBytes);
    Ring st;
    uint32_t at0 = 0, at1 = 0;  // the groups' next blocks
    int grp = 0;
    bool ok = true;
    for (int t = t0; t < tiles && ok; t += step) {
      uint32_t i = grp ? at1 : at0;
      for (int kb = kb0; kb < kb1; ++kb, ++i) {
        const int sl = grp * C::kSlots + (int)(i & kMask);
        ok = __all_sync(kFullMask, mbar_wait_asleep(tempty(sl), lap(i) ^ 1u, g.err) && mbar_wait_asleep(full(st.slot), st.lap, g.err));
        if (!ok) break;
        // (the named rows were not written by the proxy that reads them)
        if (ROWS == kNamed) asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        tcgen05_after_sync();
        const uint64_t at = (uint64_t)(st.slot * (C::kStageBytes >> 4));
        if (elect_one()) {
#pragma unroll
          for (int k = 0; k < 4; ++k)
            mma_e4m3(tmem + sl * BN, weights0 + at + 2 * k, rows0 + at + 2 * k, idesc, k > 0 ? 1u : 0u);
          mma_commit(empty(st.slot));
          mma_commit(tfull(sl));
        }
        __syncwarp();
        st.next(stages);
      }
      if (grp) at1 = i; else at0 = i;
      if (NG == 2) grp ^= 1;
    }
    __syncwarp();
  } else if (warp == C::kEpiWarps + 2) {  // scales
    constexpr int CL = (BN + 31) / 32;  // columns of a lane: lane, lane + 32, ...
    uint32_t at0 = 0, at1 = 0;
    int grp = 0;
    bool ok = true;
    int code[CL] = {};  // pair codes of the tile's columns: those of the next tile are looked up under the present one
    auto look = [&](const Tile& ti) {
#pragma unroll
      for (int i = 0; i < CL; ++i) code[i] = lane + 32 * i < ti.cnt ? __ldg(g.pairs + ti.pos + lane + 32 * i) : 0;
    };
    Tile ti = {0, 0, 0, 0};
    if (t0 < tiles) {
      ti = tile_at<BN, ROWS>(g, table, t0);
      if (ROWS == kNamed) look(ti);
    }
    for (int t = t0; t < tiles && ok; t += step) {
      const float* sap[CL];
#pragma unroll
      for (int i = 0; i < CL; ++i) {
        const int c = lane + 32 * i;
        long long in = ti.pos + c, out;
        if (c >= ti.cnt)
          in = -1;
        else if (ROWS == kNamed)
          code_rows(g, ti.pos + c, code[i], &in, &out);
        sap[i] = in >= 0 && in < a_rows ? g.sa + in * g.nbk : nullptr;
      }
      const float* swp = g.sw + ((long long)ti.e * g.nbn + ti.n0 / FP8_BLOCK) * g.nbk;
      if (t + step < tiles) {
        ti = tile_at<BN, ROWS>(g, table, t + step);
        if (ROWS == kNamed) look(ti);
      }
      float s[CL], b = 0.f;
      auto fetch = [&](int kb) {
        b = __ldg(swp + kb);
#pragma unroll
        for (int i = 0; i < CL; ++i) s[i] = sap[i] ? __ldg(sap[i] + kb) : 0.f;
      };
      fetch(kb0);
      uint32_t i = grp ? at1 : at0;
      for (int kb = kb0; kb < kb1; ++kb, ++i) {
        const int sl = grp * C::kSlots + (int)(i & kMask);
        ok = __all_sync(kFullMask, mbar_wait_asleep(sempty(sl), lap(i) ^ 1u, g.err));
        if (!ok) break;
#pragma unroll
        for (int j = 0; j < CL; ++j)
          if (lane + 32 * j < BN) scale_mem[sl * BN + lane + 32 * j] = __fmul_rn(s[j], b);
        __syncwarp();
        if (lane == 0) mbar_arrive(tfull(sl));
        if (kb + 1 < kb1) fetch(kb + 1);
      }
      if (grp) at1 = i; else at0 = i;
      if (NG == 2) grp ^= 1;
    }
  } else if (ROWS == kNamed && warp == C::kEpiWarps + 3) {  // named rows
    // A lane copies 16 bytes of rows lane / 8 + 4 j: a row's 128 bytes by eight lanes, to the
    // places that the 128-byte swizzle gives them. The copies themselves arrive on the
    // stage's barrier, so as many stages are on their way as there are.
    constexpr int R = BN / 4;
    const int chunk = lane & 7, row0 = lane >> 3;
    Ring st;
    bool ok = true;
    int code[R] = {};
    auto look = [&](const Tile& ti) {
#pragma unroll
      for (int j = 0; j < R; ++j) code[j] = row0 + 4 * j < ti.cnt ? __ldg(g.pairs + ti.pos + row0 + 4 * j) : 0;
    };
    Tile ti = {0, 0, 0, 0};
    if (t0 < tiles) {
      ti = tile_at<BN, ROWS>(g, table, t0);
      look(ti);
    }
    for (int t = t0; t < tiles && ok; t += step) {
      const uint8_t* src[R];
#pragma unroll
      for (int j = 0; j < R; ++j) {
        const int c = row0 + 4 * j;
        long long in = -1, out;
        if (c < ti.cnt) code_rows(g, ti.pos + c, code[j], &in, &out);
        src[j] = in < 0 ? nullptr : g.a + in * g.K + 16 * chunk;
      }
      if (t + step < tiles) {
        ti = tile_at<BN, ROWS>(g, table, t + step);
        look(ti);
      }
      for (int kb = kb0; kb < kb1; ++kb) {
        ok = __all_sync(kFullMask, mbar_wait_asleep(empty(st.slot), st.lap ^ 1u, g.err));
        if (!ok) break;
        const uint32_t dst = base + st.slot * C::kStageBytes + kWBytes + row0 * FP8_BLOCK;
        const bool in_k = kb * FP8_BLOCK + 16 * chunk < g.K;
#pragma unroll
        for (int j = 0; j < R; ++j) {
          const int row = row0 + 4 * j;
          const bool in = src[j] != nullptr && in_k;
          asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst + 4 * FP8_BLOCK * j + 16 * (chunk ^ (row & 7))),
                       "l"(in ? src[j] + (size_t)kb * FP8_BLOCK : g.a), "r"(in ? 16 : 0)
                       : "memory");
        }
        asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(full(st.slot)) : "memory");
        st.next(stages);
      }
    }
    asm volatile("cp.async.wait_all;" ::: "memory");  // (a CTA that gave up leaves none behind)
  } else {  // epilogue
    constexpr int CW = BN / CG;           // columns of a thread
    constexpr int CL = (CW + 31) / 32;
    constexpr int P = CW < 32 ? CW : 32;  // columns per TMEM load
    const int grp = (warp >> 2) / CG, c0 = (warp >> 2) % CG * CW;  // its group, its first column
    const int row = threadIdx.x & 127;                             // its weight row of a tile
    const uint32_t tl = tmem + ((uint32_t)((warp & 3) * 32) << 16) + c0;
    uint32_t i = 0;
    bool ok = true;
    for (int t = t0 + grp * step; t < tiles && ok; t += NG * step) {
      const Tile ti = tile_at<BN, ROWS>(g, table, t);
      int code[CL];  // (used only at the tile's end)
#pragma unroll
      for (int j = 0; j < CL; ++j)
        code[j] = GROUPED && c0 + lane + 32 * j < ti.cnt ? __ldg(g.pairs + ti.pos + c0 + lane + 32 * j) : 0;
      float acc[CW];
#pragma unroll
      for (int j = 0; j < CW; ++j) acc[j] = 0.f;
      for (int kb = kb0; kb < kb1; ++kb, ++i) {
        const int sl = grp * C::kSlots + (int)(i & kMask);
        ok = __all_sync(kFullMask, mbar_wait_asleep(tfull(sl), lap(i), g.err));
        if (!ok) break;
        tcgen05_after_sync();
        const float4* const sc = reinterpret_cast<const float4*>(scale_mem + sl * BN + c0);
#pragma unroll
        for (int p = 0; p < CW / P; ++p) {
          uint32_t v[P];
          if constexpr (P == 16)
            tmem_ld16(tl + sl * BN, v);
          else
            tmem_ld32(tl + sl * BN + p * P, v);
          tmem_wait_ld();
          tmem_loaded(v);
          if (p == CW / P - 1) {  // the sums are read
            tcgen05_before_sync();
            __syncwarp();
            if (lane == 0) mbar_arrive(tempty(sl));
          }
#pragma unroll
          for (int j = 0; j < P / 4; ++j) {
            const float4 f = sc[p * (P / 4) + j];
            float* const a = acc + p * P + 4 * j;
            a[0] = __fmaf_rn(__uint_as_float(v[4 * j]), f.x, a[0]);
            a[1] = __fmaf_rn(__uint_as_float(v[4 * j + 1]), f.y, a[1]);
            a[2] = __fmaf_rn(__uint_as_float(v[4 * j + 2]), f.z, a[2]);
            a[3] = __fmaf_rn(__uint_as_float(v[4 * j + 3]), f.w, a[3]);
          }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(sempty(sl));
      }
      if (!ok) break;
      const int n = ti.n0 + row;  // this thread's weight row
      if (S == 1) {
        long long out_row[CL];
#pragma unroll
        for (int j = 0; j < CL; ++j) {
          const int c = c0 + lane + 32 * j;
          long long in, out = -1;
          if (c < ti.cnt && lane + 32 * j < CW) {
            if constexpr (GROUPED)
              code_rows(g, ti.pos + c, code[j], &in, &out);
            else
              out = ti.pos + c;
          }
          out_row[j] = out;
        }
#pragma unroll
        for (int c = 0; c < CW; ++c) {
          const long long r = __shfl_sync(kFullMask, out_row[c / 32], c & 31);
          if (r >= 0 && n < g.N) store(g, r, n, acc[c]);
        }
      } else {  // partial columns for the cluster's sum (the stages are all consumed)
        float* part = reinterpret_cast<float*>(mem);
#pragma unroll
        for (int c = 0; c < CW; ++c) part[(c0 + c) * 128 + row] = acc[c];
      }
    }
  }
  if (S > 1) {  // (one tile per cluster; dense)
    __syncwarp();
    cluster_sync();  // every split's partial is written and visible
    if (warp < C::kEpiWarps) {
      const Tile ti = tile_at<BN, ROWS>(g, table, t0);
      const int row = threadIdx.x & 127, n = ti.n0 + row;
      uint32_t peer[kMaxSplits];
#pragma unroll
      for (int q = 0; q < kMaxSplits; ++q) peer[q] = map_rank(base, q < S ? q : 0) + 4u * row;
      for (int c = rank + S * (warp >> 2); c < ti.cnt; c += S * NG * CG) {
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
  if (warp == C::kEpiWarps + 1)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(C::kTmemCols));
}

template <int BN, Rows ROWS, int NG, int CG>
int launch(const GemmArgs& g, long long a_rows, int S, int stages, size_t smem, long long rows, int sm_count, cudaStream_t stream) {
  CUtensorMap tm_w, tm_a;
  if (!make_code_map(&tm_w, g.w, (long long)g.E * g.N, g.K, 128)) return MOE_ERR_CUDA;
  if (!make_code_map(&tm_a, g.a, a_rows, g.K, BN)) return MOE_ERR_CUDA;
  auto kern = narrow_kernel<BN, ROWS, NG, CG>;
  static OncePerDevice once;
  if (!once.allow(reinterpret_cast<const void*>(kern), kMaxSmem - kStaticSmem)) return MOE_ERR_CUDA;
  const long long tiles = rows * g.nbn;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(NG == 1 ? tiles * S : (tiles < sm_count ? tiles : sm_count)));
  cfg.blockDim = dim3(Narrow<BN, ROWS, NG, CG>::kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = S, attr[1].val.clusterDim.y = 1, attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = S > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kern, tm_w, tm_a, g, a_rows, stages, S, (int)rows) == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

// The dense form whose CTAs share a tile: BN / 32 epilogue groups of 32 columns (more
// accumulators a thread would leave no room for a second CTA), and the stages and shared
// memory it takes at most.
template <int BN>
struct Split {
  static constexpr int kParts = BN <= 32 ? 1 : BN / 32;
  using C = Narrow<BN, kDense, 1, kParts>;
  static constexpr int kShare = C::kPerSm > 1 ? kSmSmem / C::kPerSm : kMaxSmem;
  static constexpr int kMost = (kShare - kStaticSmem - 1024 - C::kScaleBytes) / C::kStageBytes < kMaxStages
                                   ? (kShare - kStaticSmem - 1024 - C::kScaleBytes) / C::kStageBytes
                                   : kMaxStages;
  static_assert((size_t)kMost * C::kStageBytes >= (size_t)BN * 512, "the stages hold a partial tile");
};

// Clusters of s such CTAs that are resident at once (clusters stay within a GPC, so whole-SM
// CTAs leave some of its SMs over); looked up once.
template <int BN>
int max_clusters(int s) {
  static std::atomic<int> known[kMaxSplits + 1];
  int n = known[s].load(std::memory_order_relaxed);
  if (n != 0) return n;
  using P = Split<BN>;
  auto kern = narrow_kernel<BN, kDense, 1, P::kParts>;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(s * 64);
  cfg.blockDim = dim3(P::C::kThreads);
  cfg.dynamicSmemBytes = P::kShare - kStaticSmem;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = s, attr[0].val.clusterDim.y = 1, attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxSmem - kStaticSmem) != cudaSuccess ||
      cudaOccupancyMaxActiveClusters(&n, kern, &cfg) != cudaSuccess) {
    cudaGetLastError();
    n = 0;
  }
  if (n <= 0) n = -1;
  known[s].store(n, std::memory_order_relaxed);
  return n;
}

// The CTAs of a tile: the most whose clusters are all resident at once where a CTA takes an
// SM; where two share one, as many as there are places (a few clusters then wait for a
// place: 1 x 7168 x 3584 took 6.0 us so and 6.5 with one CTA less a tile, 32 rows 7.4 and 9.3).
template <int BN>
int splits(long long tiles, int nbk, int sm_count) {
  using C = typename Split<BN>::C;
  for (int s = kMaxSplits; s >= 2; --s)
    if (s <= nbk && (C::kPerSm > 1 ? tiles * s <= (long long)C::kPerSm * sm_count : tiles <= max_clusters<BN>(s))) return s;
  return 1;
}

template <int BN, Rows ROWS>
int plan(const GemmArgs& g, long long a_rows, int sm_count, cudaStream_t stream) {
  constexpr int kGroups = 2;
  constexpr bool GROUPED = ROWS != kDense;
  using One = typename Split<BN>::C;
  using Many = Narrow<BN, ROWS, kGroups, 1>;
  // row tiles (grouped: at most, of ascending offsets)
  const long long rows = GROUPED ? (long long)g.M / BN + (g.E < g.M ? g.E : g.M) : ((long long)g.M + BN - 1) / BN;
  const long long tiles = rows * g.nbn;
  if (tiles >= (1LL << 31) - (1 << 16) || rows >= kMaxRowTiles) return MOE_ERR_CAPACITY;
  // A CTA takes at least its TMEM columns' share of an SM's shared memory, so that the CTAs
  // an SM holds never ask for more than its 512 columns: tcgen05.alloc would make one
  // wait for another, in a ring of waits where clusters meet at barriers.
  auto shared = [&](size_t extra, int stages, int stage_bytes, int cols) {
    const size_t need = 1024 + extra + (size_t)stages * stage_bytes, least = (size_t)cols * (kSmSmem / 512) - kStaticSmem;
    return need < least ? least : need;
  };
  if constexpr (!GROUPED) {
    // Split K while there are SMs without work: into the most parts whose CTAs are resident
    // at once (a part's blocks need not all have a stage).
    const int s = splits<BN>(tiles, g.nbk, sm_count);
    if (s > 1 || BN > 64) {
      const int kbs = (g.nbk + s - 1) / s;
      int st = kbs < Split<BN>::kMost ? kbs : Split<BN>::kMost;
      while ((size_t)st * One::kStageBytes < (size_t)BN * 512) ++st;
      return launch<BN, kDense, 1, Split<BN>::kParts>(g, a_rows, s, st, shared(One::kScaleBytes, st, One::kStageBytes, One::kTmemCols),
                                          rows, sm_count, stream);
    }
  }
  if constexpr (BN <= 64) {
    const size_t extra = Many::kScaleBytes + (GROUPED ? 2 * (g.E + 1) * 4 : 0);
    int stages = (int)((kMaxSmem - kStaticSmem - 1024 - extra) / Many::kStageBytes);
    if (stages > kMaxStages) stages = kMaxStages;
    return launch<BN, ROWS, kGroups, 1>(g, a_rows, 1, stages, shared(extra, stages, Many::kStageBytes, Many::kTmemCols),
                                           rows, sm_count, stream);
  }
  return MOE_ERR_INVALID_ARGUMENT;  // (not reached)
}

template <Rows ROWS>
int launch_bn(int bn, const GemmArgs& g, long long a_rows, int sm_count, cudaStream_t stream) {
  switch (bn) {
    case 16: return plan<16, ROWS>(g, a_rows, sm_count, stream);
    case 32: return plan<32, ROWS>(g, a_rows, sm_count, stream);
    case 64:
      if constexpr (ROWS != kNamed) return plan<64, ROWS>(g, a_rows, sm_count, stream);  // (lists this long are copied)
      return MOE_ERR_INVALID_ARGUMENT;
    default:
      if constexpr (ROWS == kDense) return plan<128, kDense>(g, a_rows, sm_count, stream);
      return MOE_ERR_INVALID_ARGUMENT;
  }
}

}  // namespace

int narrow_splits(int bn, long long tiles, int nbk, int sm_count) {
  return bn > 64 ? splits<128>(tiles, nbk, sm_count) : splits<64>(tiles, nbk, sm_count);
}

int launch_narrow(const GemmArgs& g, long long rows, bool named, int bn, int sm_count, cudaStream_t stream) {
  if (!g.offsets) return launch_bn<kDense>(bn, g, rows, sm_count, stream);
  return named ? launch_bn<kNamed>(bn, g, rows, sm_count, stream) : launch_bn<kListed>(bn, g, rows, sm_count, stream);
}

}  // namespace fp8_impl
}  // namespace moe
