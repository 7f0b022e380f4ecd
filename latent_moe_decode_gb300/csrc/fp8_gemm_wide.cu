// Block-128 E4M3 product for many rows per weight tile (prompts, experts with hundreds of
// rows): rows on the tensor core's lanes, weights on its columns, two SMs per tile.
//
// Bound by the tensor cores. A pair of CTAs (cta_group::2, M = 256) works on 256 rows of
// a (128 lanes of each CTA) and 256 weight rows (128 staged by each), so an SM stages 32
// KB per block of 128 columns for 512 cycles of multiplication: half of what two single
// CTAs would draw from L2 for the same work. The columns are multiplied in two halves of
// 128, each with two TMEM slots of its own: one half's sums are read while the other
// half multiplies. With the rows on the lanes a thread's scale is one number for a half:
//   - warps 0-15: epilogue. Warp w reads lanes 32 (w % 4).. and columns 64 (w / 4).. and
//     folds each block's sums, times its scale, into 64 FP32 registers a thread;
//   - warp 16: TMA producer;
//   - warps 17 and 18: MMA issuers, one for each half of the columns (in the pair's even
//     CTA, for both): among the epilogue warps one warp's issue loop took longer than the
//     multiplication it issues;
//   - warp 19: scales. It walks the rows' scales and leaves the products sa sw of a block
//     in shared memory beside each half's TMEM slot (one barrier tells the epilogue of
//     both), so that the row-major scales are fetched once per CTA and not per warp.
// A persistent grid of pairs walks the tiles, row tiles of the same weights side by side.
// Grouped, the rows of an expert's list are read as one box, so they have to lie in list
// order: the caller copies rows that do not (MOE_ROWS_TOKEN, MOE_ROWS_PAIR) there first.
// (TMA's gather4, which could fetch them from where they are, moved 128 rows x 128 bytes
// in 2300 cycles, against 900 for a whole block with the copies: 4096 tokens x 8 of 64
// experts took 1166 us with it.)
#include "fp8_gemm.cuh"

namespace moe {
namespace fp8_impl {
namespace {

constexpr int kEpiWarps = 16;
constexpr int kThreads = 32 * (kEpiWarps + 4);
// Registers a thread: 96 at launch (65536 / 640, in eights); four warpgroups of epilogue
// and one of the rest then share the same total, 4 * 112 + 32 = 5 * 96.
constexpr int kEpiRegs = 112, kAuxRegs = 32;
constexpr int kRows = 256, kCols = 256;       // a pair's tile
constexpr int kHalf = 128 * FP8_BLOCK;        // bytes of one CTA's rows, or weights, of a stage
constexpr int kStageBytes = 2 * kHalf;
constexpr int kStages = 5;
constexpr int kSlots = 2;                     // TMEM accumulators of each half of the columns: all 512 columns
constexpr int kScaleBytes = kSlots * 2 * 128 * 4;
constexpr int kPadCols = 16;                  // columns of a warp's pad, 32 rows of it
constexpr int kPadBytes = kEpiWarps * 32 * (kPadCols + 1) * 4;

struct Tile {
  int e, n0, pos, cnt;  // expert, first weight row, this CTA's first row and its rows (may be <= 0)
};

template <bool GROUPED>
__device__ __forceinline__ Tile tile_at(const GemmArgs& g, const int* table, int t, int half) {
  Tile r;
  const int nt = (g.nbn + 1) / 2;
  if constexpr (GROUPED) {
    r.e = tile_expert(table, g.E, t / nt);
    const int c = table[r.e + 1] - table[r.e], local = t - table[r.e] * nt;
    const int lo = clamp_offset(__ldg(g.offsets + r.e), g.M), hi = clamp_offset(__ldg(g.offsets + r.e + 1), g.M);
    r.n0 = local / c * kCols;
    r.pos = lo + local % c * kRows + half * 128;
    r.cnt = min(128, hi - r.pos);
  } else {
    const int mt = (g.M - 1) / kRows + 1;
    r.e = 0;
    r.n0 = t / mt * kCols;
    r.pos = t % mt * kRows + half * 128;
    r.cnt = min(128, g.M - r.pos);
  }
  return r;
}

__device__ __forceinline__ void mma_e4m3_pair(uint32_t tmem_d, uint64_t adesc, uint64_t bdesc, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %2, %3, p;\n}\n" ::"r"(tmem_d),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(acc));
}

// Arrive on a barrier of the cluster (a shared::cluster address). Relaxed: what it reports is a
// TMEM read, ordered by the tcgen05 fence; a release at cluster scope costs a memory barrier.
__device__ __forceinline__ void mbar_arrive_cluster(uint32_t bar) {
  asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}

__device__ __forceinline__ void st32(void* p, const uint32_t (&v)[8]) {
  asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]),
               "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
               : "memory");
}

// Four lanes' four 32-byte pieces, transposed: lane j of the four ends with piece j of each.
__device__ __forceinline__ void transpose4(uint32_t (&u)[4][8]) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int step = 1; step <= 2; step <<= 1) {
    const bool up = lane & step;
#pragma unroll
    for (int a = 0; a < 4; ++a) {
      if (a & step) continue;
#pragma unroll
      for (int w = 0; w < 8; ++w) {
        const uint32_t got = __shfl_xor_sync(kFullMask, up ? u[a][w] : u[a + step][w], step);
        (up ? u[a][w] : u[a + step][w]) = got;
      }
    }
  }
}

// The warp's 64 columns from n on of its 32 rows (`row` this lane's, -1: none). Where rows
// start at multiples of 32 or 16 bytes (vec) four lanes exchange their pieces first, so that
// a store covers 128 contiguous bytes of eight rows and not 32 of all 32 (those took an eighth
// of the time of 4096 x 7168 x 3584); else by way of the warp's pad in shared memory, 16
// columns of two rows a store (one value of 32 rows a store took 45 us for 500 x 1000 x 3008).
__device__ __forceinline__ void store_rows(const GemmArgs& g, long long row, int n, const float (&acc)[64], int vec,
                                           float (*pad)[kPadCols + 1]) {
  const int lane = threadIdx.x & 31;
  if (vec) {
    uint32_t u[4][8];
    auto store4 = [&](int size, int at) {  // bytes a value; first column
      transpose4(u);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const long long r = __shfl_sync(kFullMask, row, (lane & ~3) + i);
        const int c = at + 32 / size * (lane & 3);
        uint8_t* const to = static_cast<uint8_t*>(g.out) + (r * g.N + c) * size;
        if (r < 0) continue;
        if (vec == 32 && at + 128 / size <= g.N) {
          st32(to, u[i]);
        } else {
          if (c < g.N) *reinterpret_cast<uint4*>(to) = make_uint4(u[i][0], u[i][1], u[i][2], u[i][3]);
          if (c + 16 / size < g.N) *reinterpret_cast<uint4*>(to + 16) = make_uint4(u[i][4], u[i][5], u[i][6], u[i][7]);
        }
      }
    };
    if (g.f32) {
#pragma unroll
      for (int half = 0; half < 2; ++half) {
#pragma unroll
        for (int i = 0; i < 32; ++i) u[i >> 3][i & 7] = __float_as_uint(acc[32 * half + i]);
        store4(4, n + 32 * half);
      }
    } else {
#pragma unroll
      for (int i = 0; i < 32; ++i) u[i >> 3][i & 7] = pack_bf16x2(acc[2 * i], acc[2 * i + 1]);
      store4(2, n);
    }
  } else {
#pragma unroll
    for (int c0 = 0; c0 < 64; c0 += kPadCols) {
      __syncwarp();
#pragma unroll
      for (int i = 0; i < kPadCols; ++i) pad[lane][i] = acc[c0 + i];
      __syncwarp();
      const int c = n + c0 + lane % kPadCols;
#pragma unroll 4
      for (int i = 0; i < kPadCols; ++i) {
        const int l = 2 * i + lane / kPadCols;  // the lane whose row this is
        const long long r = __shfl_sync(kFullMask, row, l);
        const float v = pad[l][lane % kPadCols];
        if (r < 0 || c >= g.N) continue;
        if (g.f32)
          static_cast<float*>(g.out)[r * g.N + c] = v;
        else
          static_cast<uint16_t*>(g.out)[r * g.N + c] = f32_to_bf16(v);
      }
    }
  }
}

template <bool GROUPED>
__global__ void __launch_bounds__(kThreads, 1) __cluster_dims__(2, 1, 1)
    wide_kernel(const __grid_constant__ CUtensorMap tm_w, const __grid_constant__ CUtensorMap tm_a, const GemmArgs g,
                long long rows, int max_row_tiles, int vec) {
  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(8) uint64_t bars[2 * kStages + 6 * kSlots];
  __shared__ uint32_t tmem_slot;
  __shared__ int warp_sums[kThreads / 32];
  const int warp = __shfl_sync(kFullMask, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;  // (warp: uniform)
  const int half = (int)cluster_rank();  // 0: the pair's leader
  const uint32_t raw = smem_u32(smem_raw), base = (raw + 1023u) & ~1023u;
  uint8_t* const mem = smem_raw + (base - raw);
  float* const scale_mem = reinterpret_cast<float*>(mem + kStages * kStageBytes);  // [slot][weight block][row]
  auto* const pads = reinterpret_cast<float(*)[32][kPadCols + 1]>(mem + kStages * kStageBytes + kScaleBytes);  // [warp]
  int* const table = reinterpret_cast<int*>(mem + kStages * kStageBytes + kScaleBytes + kPadBytes);
  auto full = [&](int i) { return smem_u32(&bars[i]); };  // (the leader's: both CTAs' bytes)
  auto empty = [&](int i) { return smem_u32(&bars[kStages + i]); };
  // (slot, column half): sums and scales are there; they are read, as the issuer (the
  // leader's barrier: both CTAs' warps) and as the scale warp sees it
  auto tfull = [&](int i, int h) { return smem_u32(&bars[2 * kStages + 2 * i + h]); };
  auto tempty = [&](int i, int h) { return smem_u32(&bars[2 * kStages + 2 * kSlots + 2 * i + h]); };
  auto sempty = [&](int i, int h) { return smem_u32(&bars[2 * kStages + 4 * kSlots + 2 * i + h]); };

  if (threadIdx.x == 0) {
    for (int i = 0; i < kStages; ++i) {
      mbar_init(full(i), 1);
      mbar_init(empty(i), 2);  // both issuers
    }
    for (int i = 0; i < 2 * kSlots; ++i) {
      mbar_init(tfull(i >> 1, i & 1), 2);           // the MMA's commit and the scale warp
      mbar_init(tempty(i >> 1, i & 1), kEpiWarps);  // half the epilogue warps of each CTA
      mbar_init(sempty(i >> 1, i & 1), kEpiWarps / 2);
    }
    mbar_fence_init();
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&tm_w)) : "memory");
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&tm_a)) : "memory");
  }
  if (warp == kEpiWarps + 1) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&tmem_slot)),
                 "r"(kSlots * kCols));
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;");
  }
  tcgen05_before_sync();
  cluster_sync();  // the peer's barriers are initialised before anything may arrive on them
  tcgen05_after_sync();
  const uint32_t tmem = tmem_slot;
  grid_wait();
  grid_launch_dependents();
  const int nt = (g.nbn + 1) / 2;
  int tiles;
  if constexpr (GROUPED) {
    tile_table(g, kRows, table, warp_sums);
    tiles = min(table[g.E], max_row_tiles) * nt;
  } else {
    tiles = ((g.M - 1) / kRows + 1) * nt;
  }
  const int t0 = blockIdx.x >> 1, step = gridDim.x >> 1;

  if (warp >= kEpiWarps) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kAuxRegs));
    if (warp == kEpiWarps) {  // TMA producer
      Ring st;
      int issued = 0;
      const uint32_t lead = map_rank(full(0), 0);
      bool ok = true;
      for (int t = t0; t < tiles && ok; t += step) {
        const Tile ti = tile_at<GROUPED>(g, table, t, half);
        const int wrow = ti.e * g.N + ti.n0 + half * 64;
        for (int kb = 0; kb < g.nbk; ++kb) {
          ok = __all_sync(kFullMask, mbar_wait_asleep(empty(st.slot), st.lap ^ 1u, g.err));
          if (!ok) break;
          const uint32_t dst = base + st.slot * kStageBytes, bar = lead + 8 * st.slot;
          if (elect_one()) {
            if (half == 0) mbar_expect_tx(full(st.slot), 2 * kStageBytes);
            tma_load_2d_pair(dst + kHalf, &tm_w, kb * FP8_BLOCK, wrow, bar);
            tma_load_2d_pair(dst + kHalf + kHalf / 2, &tm_w, kb * FP8_BLOCK, wrow + 128, bar);
            tma_load_2d_pair(dst, &tm_a, kb * FP8_BLOCK, ti.pos, bar);
          }
          __syncwarp();
          st.next(kStages);
          ++issued;
        }
      }
      // Neither CTA may exit with arrivals on its barriers to come: the issuers' last commits, which
      // are after the copies; without them (an issuer gave up) the pair's copies in flight.
      const int first = issued > kStages ? issued - kStages : 0;
      for (int i = first; i < issued && ok; ++i)
        ok = __all_sync(kFullMask, mbar_wait_asleep(empty(i % kStages), (uint32_t)(i / kStages) & 1u, g.err));
      if (half == 0 && !ok)
        for (int i = first; i < issued; ++i) mbar_wait_asleep(full(i % kStages), (uint32_t)(i / kStages) & 1u, g.err);
    } else if (warp == kEpiWarps + 1 || warp == kEpiWarps + 2) {  // MMA issuers
      // (the whole warp walks the loop, so that descriptors stay in uniform registers)
      if (half == 0) {
        constexpr uint32_t idesc = instr_desc_e4m3(kCols / 2, kRows);
        const int h = warp - kEpiWarps - 1;
        const uint64_t rows0 = sw128_desc(base), weights0 = sw128_desc(base + kHalf + h * (kHalf / 2));
        Ring st;
        uint32_t laps = 0;  // bit i: the lap of TMEM slot i (a tile's blocks take the slots in turn from 0)
        bool ok = true;
        for (int t = t0; t < tiles && ok; t += step) {
          for (int kb = 0; kb < g.nbk; ++kb) {
            const int sl = kb & 1;
            const uint32_t at = st.slot * (kStageBytes >> 4), d = tmem + sl * kCols + h * (kCols / 2);
            const uint64_t rd = rows0 + at, wd = weights0 + at;
            const uint32_t done = tfull(sl, h), used = empty(st.slot);
            ok = __all_sync(kFullMask, mbar_wait_asleep(full(st.slot), st.lap, g.err) &&
                                           mbar_wait_asleep(tempty(sl, h), ((laps >> sl) & 1u) ^ 1u, g.err));
            if (!ok) break;
            tcgen05_after_sync();
            if (elect_one()) {
#pragma unroll
              for (int k = 0; k < 4; ++k) mma_e4m3_pair(d, rd + 2 * k, wd + 2 * k, idesc, k > 0 ? 1u : 0u);
              mma_commit_pair(done, (uint16_t)3);
              mma_commit_pair(used, (uint16_t)3);
            }
            __syncwarp();
            st.next(kStages);
            laps ^= 1u << sl;
          }
        }
      }
      __syncwarp();
    } else if (warp == kEpiWarps + 3) {  // scales
      uint32_t laps = 0;
      bool ok = true;
      for (int t = t0; t < tiles && ok; t += step) {
        const Tile ti = tile_at<GROUPED>(g, table, t, half);
        // rows 4 lane .. 4 lane + 3 of the tile, those of them that there are
        const float* sa = g.sa + ((long long)ti.pos + 4 * lane) * g.nbk;
        const int n = (int)min((long long)ti.cnt, rows - ti.pos) - 4 * lane;
        const int wb = ti.n0 / FP8_BLOCK;
        const float* sw0 = g.sw + ((long long)ti.e * g.nbn + wb) * g.nbk;
        const int next = wb + 1 < g.nbn ? g.nbk : 0;  // to the second half's scales
        float s[4], b0 = 0.f, b1 = 0.f;
        auto fetch = [&](int kb) {
          b0 = __ldg(sw0 + kb);
          b1 = __ldg(sw0 + next + kb);
#pragma unroll
          for (int i = 0; i < 4; ++i) s[i] = i < n ? __ldg(sa + (long long)i * g.nbk + kb) : 0.f;
        };
        fetch(0);
        for (int kb = 0; kb < g.nbk; ++kb) {
          const int sl = kb & 1;
          const uint32_t lap = ((laps >> sl) & 1u) ^ 1u;
          ok = __all_sync(kFullMask, mbar_wait_asleep(sempty(sl, 0), lap, g.err) && mbar_wait_asleep(sempty(sl, 1), lap, g.err));
          if (!ok) break;
          float4* d = reinterpret_cast<float4*>(scale_mem + sl * 256) + lane;
          d[0] = make_float4(__fmul_rn(s[0], b0), __fmul_rn(s[1], b0), __fmul_rn(s[2], b0), __fmul_rn(s[3], b0));
          d[32] = make_float4(__fmul_rn(s[0], b1), __fmul_rn(s[1], b1), __fmul_rn(s[2], b1), __fmul_rn(s[3], b1));
          __syncwarp();
          if (lane < 2) mbar_arrive(tfull(sl, lane));
          if (kb + 1 < g.nbk) fetch(kb + 1);
          laps ^= 1u << sl;
        }
      }
    }
  } else {  // epilogue
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kEpiRegs));
    const int q = warp & 3, cg = warp >> 2, h = cg >> 1, row = q * 32 + lane;  // half h of the columns
    const uint32_t tl = tmem + ((uint32_t)(q * 32) << 16) + cg * 64;
    const float* const sc = scale_mem + h * 128 + row;
    const uint32_t lead = map_rank(tempty(0, h), 0);  // the leader's; the next slot's is 16 bytes on
    uint32_t laps = 0;
    bool ok = true;
    for (int t = t0; t < tiles && ok; t += step) {
      float acc[64];
#pragma unroll
      for (int i = 0; i < 64; ++i) acc[i] = 0.f;
      auto fold = [&](const int sl) {  // one block's sums, from slot sl
        ok = __all_sync(kFullMask, mbar_wait_asleep(tfull(sl, h), (laps >> sl) & 1u, g.err));
        laps ^= 1u << sl;
        tcgen05_after_sync();
        const float sv = sc[sl * 256];
#pragma unroll
        for (int p = 0; p < 2; ++p) {
          uint32_t v[32];
          tmem_ld32(tl + sl * kCols + 32 * p, v);
          tmem_wait_ld();
          tmem_loaded(v);
          if (p == 1) {  // the slot is read
            tcgen05_before_sync();
            __syncwarp();
            if (lane == 0) {
              mbar_arrive_cluster(lead + 16 * sl);
              mbar_arrive(sempty(sl, h));
            }
          }
          // (FFMA and not the packed form, whose operand pairs cost two moves each here)
#pragma unroll
          for (int i = 0; i < 32; ++i) acc[32 * p + i] = __fmaf_rn(__uint_as_float(v[i]), sv, acc[32 * p + i]);
        }
      };
      // where the tile goes is looked up between two blocks, which have time to spare; at the
      // tile's end the multiplication would wait for it (5 us of 77 at 4096 x 7168 x 3584)
      long long out = -1;
      int n = 0;
      for (int kb = 0; kb < g.nbk && ok; kb += 2) {
        fold(0);
        if (kb == 0) {
          const Tile ti = tile_at<GROUPED>(g, table, t, half);
          n = ti.n0 + cg * 64;
          if (row < ti.cnt) {
            long long in;
            out = ti.pos + row;
            if constexpr (GROUPED) pair_rows(g, ti.pos + row, &in, &out);
          }
          __syncwarp();
        }
        if (kb + 1 < g.nbk && ok) fold(1);
      }
      if (!ok) break;
      if (n < g.N) store_rows(g, out, n, acc, vec, pads[warp]);
      __syncwarp();
    }
  }
  tcgen05_before_sync();
  __syncwarp();
  cluster_sync();  // neither CTA leaves while the other may still touch its shared memory
  if (warp == kEpiWarps + 1)
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kSlots * kCols));
}

template <bool GROUPED>
int launch(const GemmArgs& g, long long a_rows, int sm_count, cudaStream_t stream) {
  CUtensorMap tm_w, tm_a;
  if (!make_code_map(&tm_w, g.w, (long long)g.E * g.N, g.K, 64)) return MOE_ERR_CUDA;
  if (!make_code_map(&tm_a, g.a, a_rows, g.K, 128)) return MOE_ERR_CUDA;
  auto kern = wide_kernel<GROUPED>;
  const long long rows = GROUPED ? (long long)g.M / kRows + (g.E < g.M ? g.E : g.M) : ((long long)g.M - 1) / kRows + 1;
  const long long tiles = rows * ((g.nbn + 1) / 2);
  if (tiles >= (1LL << 31) - (1 << 16) || rows >= kMaxRowTiles) return MOE_ERR_CAPACITY;
  static_assert(1024 + kStages * kStageBytes + kScaleBytes + kPadBytes + (MOE_MAX_EXPERTS + 1) * 4 + kStaticSmem <= kMaxSmem, "");
  // All the shared memory a CTA may have: the pair holds both SMs' TMEM whole, so nothing
  // that allocates TMEM may share them.
  const size_t smem = kMaxSmem - kStaticSmem;
  static OncePerDevice once;
  if (!once.allow(reinterpret_cast<const void*>(kern), (int)smem)) return MOE_ERR_CUDA;
  const size_t esize = g.f32 ? 4 : 2;
  const size_t row_bytes = g.N * esize;
  const int vec = aligned(g.out, 32) && row_bytes % 32 == 0 ? 32 : aligned(g.out, 16) && row_bytes % 16 == 0 ? 16 : 0;
  const int pairs = sm_count / 2;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(2u * (unsigned)(tiles < pairs ? tiles : pairs));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, tm_w, tm_a, g, a_rows, (int)rows, vec) == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

}  // namespace

int launch_wide(const GemmArgs& g, long long rows, int sm_count, cudaStream_t stream) {
  return g.offsets ? launch<true>(g, rows, sm_count, stream) : launch<false>(g, rows, sm_count, stream);
}

}  // namespace fp8_impl
}  // namespace moe
