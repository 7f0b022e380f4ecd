// BF16 product with an epilogue for many rows: rows of a on the tensor core's lanes, rows of b
// on its columns, two SMs per tile.
//
// Bound by the tensor cores. A pair of CTAs (cta_group::2, M = 256) works on 256 rows of a
// (128 lanes of each CTA) and bn <= 256 rows of b (half of them staged by each): for 512 cycles
// of multiplication an SM stages 32 KB, half of what two single CTAs would draw from L2.
// Gated, the leader stages bn / 2 rows of the gate and its peer the same rows of the other
// half, so that a thread finds both values of a column in its own TMEM lane.
//   - warps 0-7: epilogue. Warp w reads lanes 32 (w % 4).., every second chunk of columns;
//   - warp 8: TMA producer; warp 9: MMA issuer (in the pair's leader, for both).
// Two accumulators in TMEM: a tile's epilogue runs under the next tile's multiplication.
// A persistent grid of pairs walks the tiles of one or two products.
// FP32 results: the tensor core cuts its running sum off after every 16 values of K, always
// towards zero, which adds up to some 2e-8 of the sum a step (9e-6 at K = 7184), to 1e-7 where all terms
// have one sign. There a tile's sums are taken in runs of kRun blocks, the runs added in registers with
// rounding to nearest (4e-7). The registers are read from TMEM under the next run's multiplication.
// So are the sums of BF16 results over more than kWhole blocks (weights' gradients over many rows: one
// run of 2^20 terms of one sign was 6.6e-3 too small, more than the rounding to BF16).
#include "linear.cuh"

namespace moe {
namespace linear_impl {
namespace {

constexpr int kEpiWarps = 8;
constexpr int kThreads = 32 * (kEpiWarps + 2);
constexpr int kRows = 256;                 // a pair's tile
constexpr int kMaxCols = 256;
constexpr int kHalf = 128 * kBlockK * 2;   // bytes of one CTA's rows of a, or of b, of a stage
constexpr int kMaxStages = 10;
constexpr int kRun = 8;                    // blocks of K that an FP32 result's sums take in one go
constexpr int kWhole = kMaxCutBlocks;       // that a BF16 result's sums take whole
constexpr int kPadBytes = 32 * 32 * 4;      // of an epilogue warp

struct Part {  // of the launch: one product
  Epilogue e;
  int M, N, nbk;       // nbk: blocks of kBlockK of K
  int run, run0;       // of them in one accumulator; in a tile's first two
  int early;           // the residual is what the sums start from
  int row_tiles, tiles;
  int pairs;           // of CTAs that work on it
  int bn;              // b's rows a tile
  int a_transposed, b_transposed;
  int boxes;           // out and pre go out in boxes of 32 rows (TMA)
  int wide;            // rows of out, residual and pre start at multiples of so many bytes (0, 16, 32)
};
struct Parts {
  Part p[2];
  int stages, stage_bytes;
};
struct Maps {
  CUtensorMap m[4];    // a, b of each product
  CUtensorMap out[2];  // of each
  CUtensorMap pre;     // of the first
};

__device__ __forceinline__ void mma_pair(uint32_t tmem_d, uint64_t adesc, uint64_t bdesc, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n}\n" ::"r"(tmem_d),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(acc));
}

// Arrive on a barrier of the cluster (a shared::cluster address). Relaxed: what it reports is a
// TMEM read, ordered by the tcgen05 fence.
__device__ __forceinline__ void mbar_arrive_cluster(uint32_t bar) {
  asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}

__device__ __forceinline__ void st32(void* p, const uint32_t* v) {
  asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]),
               "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
               : "memory");
}
__device__ __forceinline__ void ld32(const void* p, uint32_t* v) {
  asm volatile("ld.global.v8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
               : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7])
               : "l"(p)
               : "memory");
}

// The copies from this thread's boxes have been read from shared memory.
__device__ __forceinline__ void bulk_wait_read_all() { asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory"); }

// Where a chunk of a warp's 32 rows lies: lane l's row is row0 + l, its columns n .. n + C - 1; out has
// M rows and N columns. wide: all columns exist, and the bytes that a store may take, 16 or 32.
struct Chunk {
  int row0, M, n, N, wide;
};

// A lane's C (16 or 32) values of its row of a matrix, as FP32; and back. Each lane loads and stores
// its own row in pieces of 16 or 32 bytes; where rows are not so aligned the values pass through
// the warp's pad in shared memory, C columns of 32 / C rows a load or store, a value's place in
// its row of the pad turned by the row's number, against bank conflicts. (All lanes take part.)
template <int C, bool F32>
__device__ __forceinline__ void load_wide(const void* p, long long ld, const Chunk& k, float (&v)[C]) {
  const int row = k.row0 + (threadIdx.x & 31);
  if (row >= k.M) return;
  constexpr int kWords = F32 ? C : C / 2;
  const uint8_t* const at = static_cast<const uint8_t*>(p) + ((long long)row * ld + k.n) * (F32 ? 4 : 2);
  uint32_t u[kWords];
#pragma unroll
  for (int j = 0; j < kWords; j += 8) {
    if (k.wide == 32) {
      ld32(at + 4 * j, u + j);
    } else {
      const uint4 q0 = *reinterpret_cast<const uint4*>(at + 4 * j), q1 = *reinterpret_cast<const uint4*>(at + 4 * j + 16);
      u[j] = q0.x, u[j + 1] = q0.y, u[j + 2] = q0.z, u[j + 3] = q0.w;
      u[j + 4] = q1.x, u[j + 5] = q1.y, u[j + 6] = q1.z, u[j + 7] = q1.w;
    }
  }
  if constexpr (F32) {
#pragma unroll
    for (int j = 0; j < C; ++j) v[j] = __uint_as_float(u[j]);
  } else {
#pragma unroll
    for (int j = 0; j < C / 2; ++j) v[2 * j] = bf16_lo(u[j]), v[2 * j + 1] = bf16_hi(u[j]);
  }
}
template <int C>
__device__ __forceinline__ void load_rows(const void* p, long long ld, const Chunk& k, int f32, float (&v)[C], float* pad) {
  const int lane = threadIdx.x & 31;
  if (k.wide) {
    if (f32)
      load_wide<C, true>(p, ld, k, v);
    else
      load_wide<C, false>(p, ld, k, v);
  } else {
    const int c = lane % C, r0 = lane / C;
    if (lane == 0) bulk_wait_read_all();  // (the pad may still be read)
    __syncwarp();
#pragma unroll 8
    for (int r = r0; r < 32; r += 32 / C) {
      const long long row = k.row0 + r;
      pad[r * C + (c ^ (r & (C - 1)))] = row < k.M && k.n + c < k.N ? load_as_f32(p, row * ld + k.n + c, f32) : 0.f;
    }
    __syncwarp();
#pragma unroll
    for (int j = 0; j < C; ++j) v[j] = pad[lane * C + (j ^ (lane & (C - 1)))];
  }
}
template <int C, bool F32>
__device__ __forceinline__ void store_wide(void* p, long long ld, const Chunk& k, const float (&v)[C]) {
  const int row = k.row0 + (threadIdx.x & 31);
  if (row >= k.M) return;
  constexpr int kWords = F32 ? C : C / 2;
  uint8_t* const at = static_cast<uint8_t*>(p) + ((long long)row * ld + k.n) * (F32 ? 4 : 2);
#pragma unroll
  for (int j = 0; j < kWords; j += 8) {
    uint32_t u[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if constexpr (F32)
        u[i] = __float_as_uint(v[j + i]);
      else
        u[i] = pack_bf16x2(v[2 * (j + i)], v[2 * (j + i) + 1]);
    }
    if (k.wide == 32) {
      st32(at + 4 * j, u);
    } else {
      st16(at + 4 * j, make_uint4(u[0], u[1], u[2], u[3]));
      st16(at + 4 * j + 16, make_uint4(u[4], u[5], u[6], u[7]));
    }
  }
}
template <int C>
__device__ __forceinline__ void store_rows(void* p, long long ld, const Chunk& k, int f32, const float (&v)[C], float* pad) {
  const int lane = threadIdx.x & 31;
  if (k.wide) {
    if (f32)
      store_wide<C, true>(p, ld, k, v);
    else
      store_wide<C, false>(p, ld, k, v);
  } else {
    const int c = lane % C, r0 = lane / C;
    if (lane == 0) bulk_wait_read_all();  // (the pad may still be read)
    __syncwarp();
#pragma unroll
    for (int j = 0; j < C; ++j) pad[lane * C + (j ^ (lane & (C - 1)))] = v[j];
    __syncwarp();
#pragma unroll 8
    for (int r = r0; r < 32; r += 32 / C) {
      const long long row = k.row0 + r;
      const float w = pad[r * C + (c ^ (r & (C - 1)))];
      if (row < k.M && k.n + c < k.N) {
        if (f32)
          static_cast<float*>(p)[row * ld + k.n + c] = w;
        else
          static_cast<uint16_t*>(p)[row * ld + k.n + c] = f32_to_bf16(w);
      }
    }
  }
}

// The same stores by TMA: 64 bytes of each row (32 BF16 columns, 16 of FP32) in one of the pad's halves, in 16-byte
// pieces turned as the 64-byte swizzle has them, while the copy from the other half is read. TMA
// leaves out what lies beyond the matrix (whose rows are whole pieces). (A store instruction of 32 bytes of 32 rows takes the
// SM some 110 cycles: a tile of 256 x 256 in BF16 3.8 us, gradients of weights over few rows
// bound by it.)
struct Boxes {
  float* pad;
  uint32_t half;
  float* row;  // 16 values of the bias
};
template <int C, bool F32>
__device__ __forceinline__ void store_box(const CUtensorMap* map, int row0, int n, const float (&v)[C], Boxes& b) {
  static_assert(C * (F32 ? 4 : 2) == 64, "");
  const int lane = threadIdx.x & 31;
  float4* const to = reinterpret_cast<float4*>(b.pad + 512 * b.half) + 4 * lane;
  if (lane == 0) asm volatile("cp.async.bulk.wait_group.read 1;" ::: "memory");
  __syncwarp();
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float4 q;
    if constexpr (F32)
      q = make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
    else
      q = make_float4(__uint_as_float(pack_bf16x2(v[8 * i], v[8 * i + 1])), __uint_as_float(pack_bf16x2(v[8 * i + 2], v[8 * i + 3])),
                      __uint_as_float(pack_bf16x2(v[8 * i + 4], v[8 * i + 5])), __uint_as_float(pack_bf16x2(v[8 * i + 6], v[8 * i + 7])));
    to[i ^ ((lane >> 1) & 3)] = q;
  }
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  __syncwarp();
  if (lane == 0) {
    asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.bulk_group [%0, {%1, %2}], [%3];" ::"l"(reinterpret_cast<uint64_t>(map)), "r"(n),
                 "r"(row0), "r"(smem_u32(b.pad + 512 * b.half))
                 : "memory");
    asm volatile("cp.async.bulk.commit_group;" ::: "memory");
  }
  b.half ^= 1u;
}

// z + bias, of which lane l holds column l of 32; z's C columns start at 16 h of them. Through shared memory,
// 16 at a time. (FP32 results' sums start from it. 4096 x 7168 x 512, us: FP32 42, BF16 32 to 38; loaded in the epilogue
// and handed round by 32 shuffles 49 and 33, asked for a tile ahead no less; without a bias 32 and 23 to 26.)
template <int C>
__device__ __forceinline__ void add_bias(float (&z)[C], float bias, int h, float* row) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int i = 0; i < C; i += 16, ++h) {
    __syncwarp();
    if (lane >> 4 == h) row[lane & 15] = bias;
    __syncwarp();
#pragma unroll
    for (int j = 0; j < 16; j += 4) {
      const float4 q = *reinterpret_cast<const float4*>(row + j);
      z[i + j] = __fadd_rn(z[i + j], q.x), z[i + j + 1] = __fadd_rn(z[i + j + 1], q.y);
      z[i + j + 2] = __fadd_rn(z[i + j + 2], q.z), z[i + j + 3] = __fadd_rn(z[i + j + 3], q.w);
    }
  }
}

// The epilogue of C columns of a warp's 32 rows, but for the bias.
template <bool F32, int C>
__device__ __forceinline__ void finish(const Part& p, const Chunk& k, float (&z)[C], Boxes& b, const CUtensorMap* out, const CUtensorMap* pre) {
  const Epilogue& e = p.e;
  if (e.pre) {
    if constexpr (!F32) {
      if (p.boxes)
        store_box<C, false>(pre, k.row0, k.n, z, b);
      else
        store_rows(e.pre, e.ldp, k, 0, z, b.pad);
    } else {
      store_rows(e.pre, e.ldp, k, 0, z, b.pad);
    }
  }
  act_impl::apply<!F32>(e.act, z);
  if (e.residual && !p.early) {
    float r[C];
    load_rows(e.residual, e.ldr, k, e.residual_f32, r, b.pad);
#pragma unroll
    for (int i = 0; i < C; ++i) z[i] = __fadd_rn(z[i], r[i]);
  }
  if (p.boxes)
    store_box<C, F32>(out, k.row0, k.n, z, b);
  else
    store_rows(e.out, e.ldo, k, F32 && e.out_f32, z, b.pad);
}

// The same for C columns of the gate g and of the other half u.
template <int C>
__device__ __forceinline__ void finish_gated(const Part& p, const Chunk& k, float (&g)[C], float (&u)[C], float* pad) {
  const Epilogue& e = p.e;
  if (e.pre) {
    store_rows(e.pre, e.ldp, k, 0, g, pad);
    store_rows(e.pre + p.N, e.ldp, k, 0, u, pad);
  }
  act_impl::apply<true>(e.act, g);
#pragma unroll
  for (int i = 0; i < C; ++i) g[i] = __fmul_rn(g[i], u[i]);
  store_rows(e.out, e.ldo, k, 0, g, pad);
}

// What a kernel computes: BF16 products, products whose sums are taken in runs (FP32 results among them),
// gated pairs, gated pairs in runs.
enum Kind { kBf16, kF32, kGated, kGatedRuns };
constexpr bool is_gated(Kind kind) { return kind == kGated || kind == kGatedRuns; }

struct Tile {
  int m0, n0;  // this CTA's first row of a, the tile's first column of out
};

template <Kind KIND>
__device__ __forceinline__ Tile tile_at(const Part& p, int t, int half) {
  return {t % p.row_tiles * kRows + half * 128, t / p.row_tiles * (is_gated(KIND) ? p.bn / 2 : p.bn)};
}

// The block after the run that starts with k0.
__device__ __forceinline__ int run_end(const Part& p, int k0) { return min(k0 + (k0 < 2 * p.run0 ? p.run0 : p.run), p.nbk); }

template <Kind KIND>
__global__ void __launch_bounds__(kThreads, 1) __cluster_dims__(2, 1, 1)
    linear_wide_kernel(const __grid_constant__ Maps maps, const __grid_constant__ Parts g, uint32_t* err) {
  constexpr bool GATED = is_gated(KIND);
  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(8) uint64_t bars[2 * kMaxStages + 4];
  __shared__ uint32_t tmem_slot;
  const int warp = __shfl_sync(kFullMask, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;  // (warp: uniform)
  const int half = (int)cluster_rank();  // 0: the pair's leader
  const uint32_t raw = smem_u32(smem_raw), base = (raw + 1023u) & ~1023u;
  uint8_t* const mem = smem_raw + (base - raw);
  const uint32_t stages = (uint32_t)g.stages, stage_bytes = (uint32_t)g.stage_bytes;
  auto full = [&](int i) { return smem_u32(&bars[i]); };  // (the leader's: both CTAs' bytes)
  auto empty = [&](int i) { return smem_u32(&bars[kMaxStages + i]); };
  auto tfull = [&](int i) { return smem_u32(&bars[2 * kMaxStages + i]); };
  auto tempty = [&](int i) { return smem_u32(&bars[2 * kMaxStages + 2 + i]); };  // (the leader's: both CTAs' warps)

  if (threadIdx.x == 0) {
    for (int i = 0; i < (int)stages; ++i) {
      mbar_init(full(i), 1);
      mbar_init(empty(i), 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(tfull(i), 1);
      mbar_init(tempty(i), 2 * kEpiWarps);
    }
    mbar_fence_init();
  }
  if (warp == kEpiWarps + 1) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&tmem_slot)),
                 "r"(2 * kMaxCols));
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;");
  }
  tcgen05_before_sync();
  cluster_sync();  // the peer's barriers are initialised before anything may arrive on them
  tcgen05_after_sync();
  const uint32_t tmem = tmem_slot;
  grid_wait();
  grid_launch_dependents();
  // This pair's product and its tiles: t0, t0 + step, ..
  const int pair = blockIdx.x >> 1, second = pair >= g.p[0].pairs;
  const Part& p = g.p[second];
  const int t0 = pair - (second ? g.p[0].pairs : 0), step = p.pairs;

  if (warp == kEpiWarps) {  // TMA producer
    Ring st;
    int issued = 0;
    const uint32_t lead = map_rank(full(0), 0);
    const CUtensorMap *ma = &maps.m[2 * second], *mb = ma + 1;
    const int rows_b = p.bn / 2;  // this CTA's
    const uint32_t bytes = 2u * (kHalf + (uint32_t)(p.b_transposed ? (rows_b + 63) / 64 * 64 : rows_b) * 128);
    bool ok = true;
    for (int t = t0; t < p.tiles && ok; t += step) {
      const Tile ti = tile_at<KIND>(p, t, half);
      const int b0 = GATED ? ti.n0 + half * p.N : ti.n0 + half * rows_b;
      for (int kb = 0; kb < p.nbk; ++kb) {
        ok = __all_sync(kFullMask, mbar_wait_asleep(empty(st.slot), st.lap ^ 1u, err));
        if (!ok) break;
        const uint32_t dst = base + st.slot * stage_bytes, bar = lead + 8 * st.slot;
        const int k0 = kb * kBlockK;
        if (elect_one()) {
          if (half == 0) mbar_expect_tx(full(st.slot), bytes);
          if (p.a_transposed) {
            tma_load_2d_pair(dst, ma, ti.m0, k0, bar);
            tma_load_2d_pair(dst + kHalf / 2, ma, ti.m0 + 64, k0, bar);
          } else {
            tma_load_2d_pair(dst, ma, k0, ti.m0, bar);
          }
          if (p.b_transposed) {
            for (int r = 0; r < rows_b; r += 64) tma_load_2d_pair(dst + kHalf + r * 128, mb, b0 + r, k0, bar);
          } else {
            tma_load_2d_pair(dst + kHalf, mb, k0, b0, bar);
          }
        }
        __syncwarp();
        st.next(stages);
        ++issued;
      }
    }
    // Neither CTA may exit with arrivals on its barriers to come: the issuer's last commits, which
    // are after the copies; without them (it gave up) the pair's copies in flight.
    const int n = (int)stages, first = issued > n ? issued - n : 0;
    for (int i = first; i < issued && ok; ++i)
      ok = __all_sync(kFullMask, mbar_wait_asleep(empty(i % n), (uint32_t)(i / n) & 1u, err));
    if (half == 0 && !ok)
      for (int i = first; i < issued; ++i) mbar_wait_asleep(full(i % n), (uint32_t)(i / n) & 1u, err);
  } else if (warp == kEpiWarps + 1) {  // MMA issuer
    // (the whole warp walks the loop, so that descriptors stay in uniform registers)
    if (half == 0) {
      const uint32_t idesc = instr_desc(kRows, p.bn, p.a_transposed, p.b_transposed);
      const uint64_t a0 = operand_desc(base, p.a_transposed), b0 = operand_desc(base + kHalf, p.b_transposed);
      const uint32_t as = operand_step(p.a_transposed), bs = operand_step(p.b_transposed);
      Ring st;
      uint32_t i = 0;  // this pair's runs: accumulator i & 1, its lap i >> 1
      bool ok = true;
      for (int t = t0; t < p.tiles && ok; t += step) {
        for (int k0 = 0, k1; k0 < p.nbk && ok; k0 = k1, ++i) {
          const uint32_t d = tmem + (i & 1u) * kMaxCols;
          k1 = run_end(p, k0);
          ok = __all_sync(kFullMask, mbar_wait_asleep(tempty(i & 1u), ((i >> 1) & 1u) ^ 1u, err));
          for (int kb = k0; kb < k1 && ok; ++kb) {
            ok = __all_sync(kFullMask, mbar_wait_asleep(full(st.slot), st.lap, err));
            if (!ok) break;
            tcgen05_after_sync();
            const uint32_t at = st.slot * (stage_bytes >> 4);
            if (elect_one()) {
#pragma unroll
              for (uint32_t k = 0; k < 4; ++k) mma_pair(d, a0 + at + k * as, b0 + at + k * bs, idesc, kb > k0 || k > 0 ? 1u : 0u);
              mma_commit_pair(empty(st.slot), (uint16_t)3);
              if (kb + 1 == k1) mma_commit_pair(tfull(i & 1u), (uint16_t)3);
            }
            __syncwarp();
            st.next(stages);
          }
        }
      }
    }
    __syncwarp();
  } else {  // epilogue
    const int q = warp & 3, cg = warp >> 2;
    uint8_t* const pads = mem + stages * stage_bytes;
    Boxes box = {reinterpret_cast<float*>(pads + warp * kPadBytes), 0u, reinterpret_cast<float*>(pads + kEpiWarps * kPadBytes + warp * 64)};
    const CUtensorMap *const to_out = &maps.out[second], *const to_pre = &maps.pre;
    const uint32_t lead = map_rank(tempty(0), 0);
    uint32_t i = 0;
    bool ok = true;
    auto filled = [&] {
      ok = __all_sync(kFullMask, mbar_wait_asleep(tfull(i & 1u), (i >> 1) & 1u, err));
      tcgen05_after_sync();
      return ok;
    };
    auto release = [&] {  // the accumulator is read
      tcgen05_before_sync();
      __syncwarp();
      if (lane == 0) mbar_arrive_cluster(lead + 8 * (i & 1u));
      ++i;
    };
    for (int t = t0; t < p.tiles && ok; t += step) {
      const Tile ti = tile_at<KIND>(p, t, half);
      const uint32_t tl = tmem + ((uint32_t)(q * 32) << 16);
      const int row0 = ti.m0 + 32 * q;
      // the columns that out has, of rows that it has
      const int cols = row0 < p.M ? min(GATED ? p.bn / 2 : p.bn, p.N - ti.n0) : 0;
      // The bias of this warp's columns, lane l's of each 32.
      constexpr int kChunks = kMaxCols / 64;
      float bias[kChunks] = {};
      if (!GATED && p.e.bias) {
#pragma unroll
        for (int j = 0; j < kChunks; ++j) {
          const int n = ti.n0 + 64 * j + 32 * cg + lane;
          if (n < p.N) bias[j] = load_as_f32(p.e.bias, n, p.e.bias_f32);
        }
      }
      auto chunk = [&](int c, int C) { return Chunk{row0, p.M, ti.n0 + c, p.N, ti.n0 + c + C <= p.N ? p.wide : 0}; };
      if constexpr (KIND == kF32) {
        // Pieces of 16 columns, of every second 32: the j-th starts at piece(j).
        constexpr int kPieces = kMaxCols / 32;
        auto piece = [&](int j) { return 32 * (j & ~1) + 32 * cg + 16 * (j & 1); };
        float acc[16 * kPieces];
#pragma unroll
        for (int j = 0; j < 16 * kPieces; ++j) acc[j] = 0.f;
        if (p.early) {
#pragma unroll
          for (int j = 0; j < kPieces; ++j) {
            if (piece(j) >= cols) break;
            auto& v = reinterpret_cast<float(&)[16]>(acc[16 * j]);
            if (p.e.residual_f32)
              load_wide<16, true>(p.e.residual, p.e.ldr, chunk(piece(j), 16), v);
            else
              load_wide<16, false>(p.e.residual, p.e.ldr, chunk(piece(j), 16), v);
          }
        }
        __syncwarp();
        if (p.e.bias) {  // (where the sums start, too)
#pragma unroll
          for (int j = 0; j < kPieces; ++j) {
            if (piece(j) >= cols) break;
            add_bias(reinterpret_cast<float(&)[16]>(acc[16 * j]), bias[j / 2], j & 1, box.row);
          }
        }
        for (int k0 = 0; k0 < p.nbk; k0 = run_end(p, k0)) {
          if (!filled()) break;
#pragma unroll
          for (int j = 0; j < kPieces; ++j) {
            if (piece(j) >= cols) break;
            uint32_t v[16];
            tmem_ld16(tl + (i & 1u) * kMaxCols + piece(j), v);
            tmem_wait_ld();
            tmem_loaded(v);
#pragma unroll
            for (int l = 0; l < 16; ++l) acc[16 * j + l] = __fadd_rn(acc[16 * j + l], __uint_as_float(v[l]));
          }
          release();
        }
        if (!ok) break;
#pragma unroll 1
        for (int j = 0; j < kPieces; ++j) {
          if (piece(j) >= cols) break;
          float z[16];
#pragma unroll
          for (int l = 0; l < 16; ++l) z[l] = acc[l];
          finish<true>(p, chunk(piece(j), 16), z, box, to_out, to_pre);
          __syncwarp();
#pragma unroll
          for (int l = 0; l < 16 * (kPieces - 1); ++l) acc[l] = acc[l + 16];
        }
      } else if constexpr (KIND == kGatedRuns) {
        // Pieces of 16 columns of both halves, every second one: the j-th starts at piece(j).
        constexpr int kPieces = kMaxCols / 64;
        auto piece = [&](int j) { return 32 * j + 16 * cg; };
        float acc[32 * kPieces];
#pragma unroll
        for (int j = 0; j < 32 * kPieces; ++j) acc[j] = 0.f;
        for (int k0 = 0; k0 < p.nbk; k0 = run_end(p, k0)) {
          if (!filled()) break;
#pragma unroll
          for (int j = 0; j < 2 * kPieces; ++j) {
            if (piece(j / 2) >= cols) break;
            uint32_t v[16];
            tmem_ld16(tl + (i & 1u) * kMaxCols + (j & 1 ? p.bn / 2 : 0) + piece(j / 2), v);
            tmem_wait_ld();
            tmem_loaded(v);
#pragma unroll
            for (int l = 0; l < 16; ++l) acc[16 * j + l] = __fadd_rn(acc[16 * j + l], __uint_as_float(v[l]));
          }
          release();
        }
        if (!ok) break;
#pragma unroll 1
        for (int j = 0; j < kPieces; ++j) {
          if (piece(j) >= cols) break;
          float a[16], b[16];
#pragma unroll
          for (int l = 0; l < 16; ++l) a[l] = acc[l], b[l] = acc[16 + l];
          finish_gated(p, chunk(piece(j), 16), a, b, box.pad);
          __syncwarp();
#pragma unroll
          for (int l = 0; l < 32 * (kPieces - 1); ++l) acc[l] = acc[l + 32];
        }
      } else {
        if (!filled()) break;
        const uint32_t ta = tl + (i & 1u) * kMaxCols;
        constexpr int kStep = GATED ? 16 : 32;
        for (int c = kStep * cg; c < cols; c += 2 * kStep) {
          if constexpr (GATED) {
            uint32_t v[16], w[16];
            tmem_ld16(ta + c, v);
            tmem_ld16(ta + p.bn / 2 + c, w);
            tmem_wait_ld();
            tmem_loaded(v);
            tmem_loaded(w);
            float a[16], b[16];
#pragma unroll
            for (int j = 0; j < 16; ++j) a[j] = __uint_as_float(v[j]), b[j] = __uint_as_float(w[j]);
            finish_gated(p, chunk(c, 16), a, b, box.pad);
          } else {
            uint32_t v[32];
            tmem_ld32(ta + c, v);
            tmem_wait_ld();
            tmem_loaded(v);
            float z[32];
#pragma unroll
            for (int j = 0; j < 32; ++j) z[j] = __uint_as_float(v[j]);
            if (p.e.bias) {
              add_bias(z, bias[0], 0, box.row);
#pragma unroll
              for (int j = 0; j + 1 < kChunks; ++j) bias[j] = bias[j + 1];
            }
            finish<false>(p, chunk(c, 32), z, box, to_out, to_pre);
          }
          __syncwarp();
        }
        release();
      }
    }
    if (lane == 0) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");  // (the stores by TMA are done)
    __syncwarp();
  }
  tcgen05_before_sync();
  __syncwarp();
  cluster_sync();  // neither CTA leaves while the other may still touch its shared memory
  if (warp == kEpiWarps + 1)
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(2 * kMaxCols));
}

// Whether a matrix's rows start at multiples of `bytes`.
bool starts(const void* p, long long ld, int size, int bytes) { return !p || (aligned(p, bytes) && ld * size % bytes == 0); }

constexpr int kSmem = kMaxSmem - kStaticSmem;  // all that a CTA may have: the pair holds both SMs' TMEM
                                              // whole, so nothing that allocates TMEM may share them
constexpr int kStageRoom = kSmem - 1024 - kEpiWarps * (kPadBytes + 64);

int stage_bytes(int bn, bool b_transposed) { return kHalf + (b_transposed ? (bn / 2 + 63) / 64 * 64 : bn / 2) * 128; }

// Boxes of 32 rows x 64 bytes of a result [rows, cols] (64-byte swizzle).
bool make_out_map(CUtensorMap* m, const void* p, long long ld, int rows, int cols, bool f32) {
  auto fn = encode_fn();
  if (!fn) return false;
  cuuint64_t dims[2] = {(cuuint64_t)cols, (cuuint64_t)rows};
  cuuint64_t strides[1] = {(cuuint64_t)ld * (f32 ? 4 : 2)};
  cuuint32_t box[2] = {f32 ? 16u : 32u, 32u};
  cuuint32_t estr[2] = {1, 1};
  return fn(m, f32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(p), dims, strides, box, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_64B, CU_TENSOR_MAP_L2_PROMOTION_NONE, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) ==
         CUDA_SUCCESS;
}

template <Kind KIND>
int launch(const Product* products, int count, const WidePlan& plan, cudaStream_t stream, uint32_t* err) {
  constexpr bool GATED = is_gated(KIND);
  Parts parts = {};
  Maps maps = {};
  int pairs = 0;
  for (int i = 0; i < count; ++i) {
    const Product& s = products[i];
    Part& p = parts.p[i];
    p.e = s.e, p.M = s.M, p.N = s.N, p.nbk = (s.K - 1) / kBlockK + 1;
    p.run = s.e.out_f32 ? kRun : p.nbk > kWhole ? 2 * kRun : p.nbk;
    p.run0 = s.e.out_f32 && p.nbk >= 7 * kRun ? 2 * kRun : p.run;
    p.a_transposed = s.a.transposed, p.b_transposed = s.b.transposed;
    p.bn = plan.bn[i], p.pairs = plan.pairs[i];
    pairs += p.pairs;
    p.row_tiles = (s.M - 1) / kRows + 1;
    p.tiles = p.row_tiles * ((s.N - 1) / (GATED ? p.bn / 2 : p.bn) + 1);
    const Epilogue& e = s.e;
    for (int bytes = 32; bytes >= 16 && !p.wide; bytes /= 2)
      if (starts(e.out, e.ldo, e.out_f32 ? 4 : 2, bytes) && starts(e.residual, e.ldr, e.residual_f32 ? 4 : 2, bytes) &&
          starts(e.pre, e.ldp, 2, bytes) && (!GATED || !e.pre || s.N * 2LL % bytes == 0))
        p.wide = bytes;
    // Boxes for FP32 results, and for BF16 rows that start at multiples of 16 bytes only: 4096 x 7168 x 3584 with an
    // FP32 residual 130 us from 137, the gradients of 181 x 3640 x 6872 51 from 59. Where a store takes 32 bytes of a
    // row they only cost the multiplication its shared memory (BF16 results of 4096 x 7168 x 512 26.7 and 25.1, of
    // 1024 35.7 and 34.5). (BF16 beside FP32 results: 16 columns at a time, no box; nor are a gated pair's.)
    // (A box that ends inside 16 bytes of a row writes all 16: only where rows are whole ones.)
    p.boxes = !GATED && (KIND == kF32 ? p.wide && e.out_f32 : p.wide == 16) && s.N * (e.out_f32 ? 4LL : 2LL) % 16 == 0 &&
              e.ldo < (1LL << 37) && e.ldp < (1LL << 37);
    if (p.boxes) {
      if (!make_out_map(&maps.out[i], e.out, e.ldo, s.M, s.N, e.out_f32)) return MOE_ERR_CUDA;
      if (KIND != kF32 && e.pre && !make_out_map(&maps.pre, e.pre, e.ldp, s.M, s.N, false)) return MOE_ERR_CUDA;
    }
    p.early = KIND == kF32 && p.wide && e.residual && e.act == BF16_ACT_NONE && !e.pre && s.N % 16 == 0;
    const int size = stage_bytes(p.bn, p.b_transposed);
    if (size > parts.stage_bytes) parts.stage_bytes = size;
    if (!make_map(&maps.m[2 * i], s.a, s.M, s.K, 128)) return MOE_ERR_CUDA;
    if (!make_map(&maps.m[2 * i + 1], s.b, GATED ? 2LL * s.N : s.N, s.K, p.bn / 2)) return MOE_ERR_CUDA;
  }
  if (count == 1) maps.m[2] = maps.m[0], maps.m[3] = maps.m[1];
  parts.stages = kStageRoom / parts.stage_bytes;
  if (parts.stages > kMaxStages) parts.stages = kMaxStages;
  static_assert(kStageRoom / (2 * kHalf) >= 6, "");
  auto kern = linear_wide_kernel<KIND>;
  static OncePerDevice once;
  if (!once.allow(reinterpret_cast<const void*>(kern), kSmem)) return MOE_ERR_CUDA;
  return launch_pdl(kern, dim3(2u * (unsigned)pairs), dim3(kThreads), kSmem, stream, maps, parts, err);
}

long long tile_count(const Product& s, bool gated, int bn) {
  return ((s.M - 1) / kRows + 1LL) * ((s.N - 1) / (gated ? bn / 2 : bn) + 1);
}

}  // namespace

WidePlan plan_wide(const Product* products, int count, bool gated, const DeviceInfo& dev) {
  const int pairs = dev.sm_count / 2;
  WidePlan best = {};
  // A product on `n` pairs with tiles of bn: a block of 64 of K in 168 ns at least, 51 + 0.85 bn, or its bytes at 113 a
  // ns; a tile's epilogue, by what its columns load and store, under the next tile's multiplication. (Fitted to 550
  // points, T 1 to 1500, tiles of 64 to 256: 12 % off (rms), the choice 2.7 % slower than the best on average. That was
  // before the epilogue's last steps, without bias or activation, which the estimate does not count: with both an FP32
  // gelu's time over a short K more than doubles.)
  auto time = [&](const Product& s, int bn, long long n) {
    const Epilogue& e = s.e;
    const double waves = (double)((tile_count(s, gated, bn) - 1) / n + 1);
    double block = 51 + 0.85 * bn, feed = stage_bytes(bn, s.b.transposed) / 113.0;
    if (block < 168) block = 168;
    if (block < feed) block = feed;
    const double main = block * ((s.K - 1) / kBlockK + 1);
    const double column = (e.out_f32 ? 19 : 12) + (e.residual ? (e.residual_f32 ? 20 : 10) : 0) + (e.pre ? 10 : 0);
    const double end = 700 + column * (gated ? bn / 2 + bn / 4 : bn);
    return waves * (main > end ? main : end) + 0.45 * end;
  };
  auto bytes = [&] {
    double sum = 0;
    for (int i = 0; i < count; ++i) {
      const Product& s = products[i];
      sum += 2.0 * s.M * s.K + 2.0 * (gated ? 2 : 1) * s.N * s.K + (double)s.M * s.N * ((s.e.out_f32 ? 4 : 2) + (s.e.residual ? (s.e.residual_f32 ? 4 : 2) : 0));
    }
    return sum / 6100;
  };
  const double hbm = bytes();
  if (count == 1) {
    for (int bn = kMaxCols; bn >= 64; bn -= 32) {
      const long long tiles = tile_count(products[0], gated, bn), n = tiles < pairs ? tiles : pairs;
      const double t = time(products[0], bn, n), ns = 2600 + (t > hbm ? t : hbm);
      if (best.bn[0] == 0 || ns < best.ns) best = {{bn, 0}, {(int)n, 0}, ns};
    }
    return best;
  }
  for (int b0 = kMaxCols; b0 >= 64; b0 -= 64)
    for (int b1 = kMaxCols; b1 >= 64; b1 -= 64) {
      // all tiles at once, or pairs in the proportion of the work, and some more or fewer
      const long long t0 = tile_count(products[0], gated, b0), t1 = tile_count(products[1], gated, b1);
      const double w0 = t0 * time(products[0], b0, t0), w1 = t1 * time(products[1], b1, t1);
      const int mid = t0 + t1 <= pairs ? (int)t0 : (int)(pairs * w0 / (w0 + w1));
      for (int n = mid - 3; n <= mid + 4; ++n) {
        if (n < 1 || n >= pairs) continue;
        const long long n0 = t0 < n ? t0 : n, n1 = t1 < pairs - n ? t1 : pairs - n;
        const double e0 = time(products[0], b0, n0), e1 = time(products[1], b1, n1), t = e0 > e1 ? e0 : e1;
        const double ns = 2600 + (t > hbm ? t : hbm);
        if (best.bn[0] == 0 || ns < best.ns) best = {{b0, b1}, {(int)n0, (int)n1}, ns};
      }
    }
  return best;
}

int launch_wide(const Product* products, int count, bool gated, const WidePlan& plan, const DeviceInfo& dev, cudaStream_t stream) {
  for (int i = 0; i < count; ++i)
    if (tile_count(products[i], gated, plan.bn[i]) >= (1LL << 31) - (1 << 16)) return MOE_ERR_CAPACITY;
  bool runs = false;
  for (int i = 0; i < count; ++i) runs = runs || products[i].e.out_f32 || products[i].K > kWhole * kBlockK;
  if (gated) return runs ? launch<kGatedRuns>(products, count, plan, stream, dev.error_word) : launch<kGated>(products, count, plan, stream, dev.error_word);
  return runs ? launch<kF32>(products, count, plan, stream, dev.error_word) : launch<kBf16>(products, count, plan, stream, dev.error_word);
}

}  // namespace linear_impl
}  // namespace moe
