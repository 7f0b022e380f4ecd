// Gradients of the BF16 products' epilogues: dz = dout act'(pre), or [dg | du] of the gated pair,
// in BF16 for the products that follow, and the sum of dz's rows (the bias's gradient) in FP32.
//
// dz is rounded once to BF16, the type the tensor core multiplies (the products' results are then 1.7e-3 of the
// whole off, rms, beside their own rounding); the sums are of the FP32 values before that. Bound by HBM (4 bytes in and 2 out per value; gated 6 and 4).
//
// A CTA takes a strip of 64 columns, eight to a thread (16 bytes a load; where rows do not start at
// multiples of that, every eighth column, one by one), 32 rows at a time. For the column sums the
// CTAs of a strip are a cluster: each adds its rows in registers, its 32 row lanes in order and then
// the CTAs in order through distributed shared memory, so that the sums need neither scratch nor
// atomics and do not change from run to run.
#include "linear.cuh"

namespace moe {
namespace linear_impl {
namespace {

constexpr int kThreads = 256;
constexpr int kStrip = 64;              // columns of a CTA, eight a thread
constexpr int kRowLanes = kThreads / 8;
constexpr int kMaxCluster = 8;

struct DzArgs {
  const uint16_t *dout, *pre;
  uint16_t* dz;
  float* dbias;
  long long ldd, ldp, ldz;
  int T, N;  // N: columns of dout
};

// A thread's eight values of a row, as they are stored. VEC: columns 8 lane.., as 16 bytes; else
// columns lane + 8 i, those below N, one by one (eight lanes then read what lies together).
struct Raw {
  uint32_t w[4];
};
template <bool VEC>
__device__ __forceinline__ Raw load8(const uint16_t* row, int lane, int cols) {
  Raw r;
  if (VEC) {
    const uint4 q = ld_nc16(row + 8 * lane);
    r.w[0] = q.x, r.w[1] = q.y, r.w[2] = q.z, r.w[3] = q.w;
  } else {
    uint16_t u[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) u[i] = lane + 8 * i < cols ? __ldg(row + lane + 8 * i) : (uint16_t)0;
#pragma unroll
    for (int i = 0; i < 4; ++i) r.w[i] = u[2 * i] | (uint32_t)u[2 * i + 1] << 16;
  }
  return r;
}
__device__ __forceinline__ float value(const Raw& r, int i) { return i & 1 ? bf16_hi(r.w[i / 2]) : bf16_lo(r.w[i / 2]); }
template <bool VEC>
__device__ __forceinline__ void store8(uint16_t* row, int lane, int cols, const float (&v)[8]) {
  if (VEC) {
    st16(row + 8 * lane, make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7])));
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (lane + 8 * i < cols) row[lane + 8 * i] = f32_to_bf16(v[i]);
  }
}

// (One for each activation: a choice for every value took three times as long.)
template <int ACT, bool GATED, bool VEC>
__global__ void __launch_bounds__(kThreads, 4) dz_kernel(const DzArgs g) {
  constexpr int kUnroll = 2;  // rows of a thread in flight
  constexpr bool PRE = GATED || ACT != BF16_ACT_NONE;
  __shared__ float part[kRowLanes][kStrip];
  __shared__ float strip[kStrip];
  const int lane = threadIdx.x & 7, r = threadIdx.x >> 3, c0 = blockIdx.x * kStrip, cols = min(kStrip, g.N - c0);
  grid_wait();
  grid_launch_dependents();
  float sum[8] = {};
  const long long step = (long long)kRowLanes * gridDim.y;
  if (VEC ? 8 * lane < cols : lane < cols) {
    for (long long t0 = (long long)blockIdx.y * kRowLanes + r; t0 < g.T; t0 += kUnroll * step) {
      Raw d[kUnroll], z[kUnroll], u[GATED ? kUnroll : 1];
#pragma unroll
      for (int j = 0; j < kUnroll; ++j) {
        const long long t = t0 + j * step;
        if (t >= g.T) continue;
        d[j] = load8<VEC>(g.dout + t * g.ldd + c0, lane, cols);
        if (PRE) z[j] = load8<VEC>(g.pre + t * g.ldp + c0, lane, cols);
        if (GATED) u[j] = load8<VEC>(g.pre + t * g.ldp + g.N + c0, lane, cols);
      }
#pragma unroll
      for (int j = 0; j < kUnroll; ++j) {
        const long long t = t0 + j * step;
        if (t >= g.T) continue;
        float a[8], b[8];
#pragma unroll
        for (int i = 0; i < 8; i += 2) {
          float val[2], slope[2];
          if (PRE) act_impl::with_slope(ACT, {value(z[j], i), value(z[j], i + 1)}, val, slope);
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            float& v = a[i + h];
            v = value(d[j], i + h);
            if (GATED) b[i + h] = v * val[h];
            if (PRE) v *= GATED ? value(u[j], i + h) * slope[h] : slope[h];
            sum[i + h] += v;
          }
        }
        if (g.dz) store8<VEC>(g.dz + t * g.ldz + c0, lane, cols, a);
        if (GATED) store8<VEC>(g.dz + t * g.ldz + g.N + c0, lane, cols, b);
      }
    }
  }
  if (!g.dbias) return;
  __syncwarp();  // (the lanes of a warp end their rows apart)
#pragma unroll
  for (int i = 0; i < 8; ++i) part[r][VEC ? 8 * lane + i : lane + 8 * i] = sum[i];
  __syncthreads();
  if (threadIdx.x < kStrip) {
    float s = 0.f;
    for (int i = 0; i < kRowLanes; ++i) s += part[i][threadIdx.x];
    strip[threadIdx.x] = s;
  }
  __syncwarp();
  cluster_sync();  // (the cluster is the strip's CTAs, ranks in the order of blockIdx.y)
  if (blockIdx.y == 0 && threadIdx.x < kStrip) {
    float s = 0.f;
    for (int q = 0; q < (int)gridDim.y; ++q) {
      float v;
      asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(map_rank(smem_u32(strip + threadIdx.x), q)) : "memory");
      s += v;
    }
    const int n = blockIdx.x * kStrip + threadIdx.x;
    if (n < g.N) g.dbias[n] = s;
  }
  __syncwarp();
  cluster_sync();  // no CTA leaves while its sums may be read
}

template <bool GATED>
int launch(const DzArgs& g, int act, const DeviceInfo& dev, cudaStream_t stream) {
  auto rows16 = [](const void* p, long long ld) { return !p || (aligned(p, 16) && ld % 8 == 0); };
  const bool vec = g.N % 8 == 0 && rows16(g.dout, g.ldd) && rows16(g.pre, g.ldp) && rows16(g.dz, g.ldz);
  const long long strips = ((long long)g.N - 1) / kStrip + 1;
  // CTAs for eight an SM (with the sums four, at most a cluster's of a strip), no more than there are rows
  long long chunks = ((g.dbias ? 4LL : 8LL) * dev.sm_count + strips - 1) / strips;
  const long long most = ((long long)g.T - 1) / kRowLanes + 1;
  chunks = chunks < most ? chunks : most;
  if (g.dbias && chunks > kMaxCluster) chunks = kMaxCluster;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)strips, (unsigned)chunks);
  cfg.blockDim = dim3(kThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = 1, attr[1].val.clusterDim.y = (unsigned)chunks, attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = g.dbias ? 2 : 1;
  using Kernel = void (*)(const DzArgs);
  static const Kernel kernels[2][5] = {
      {dz_kernel<0, GATED, false>, dz_kernel<1, GATED, false>, dz_kernel<2, GATED, false>, dz_kernel<3, GATED, false>, dz_kernel<4, GATED, false>},
      {dz_kernel<0, GATED, true>, dz_kernel<1, GATED, true>, dz_kernel<2, GATED, true>, dz_kernel<3, GATED, true>, dz_kernel<4, GATED, true>}};
  const Kernel kern = kernels[vec][act];
  if (prefer_max_shared(reinterpret_cast<const void*>(kern)) != MOE_OK) return MOE_ERR_CUDA;
  return cudaLaunchKernelEx(&cfg, kern, g) == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

}  // namespace

int launch_dz(const uint16_t* dout, long long ldd, const uint16_t* pre, long long ldp, int act, int T, int N, uint16_t* dz,
              long long ldz, float* dbias, const DeviceInfo& dev, cudaStream_t stream) {
  return launch<false>({dout, pre, dz, dbias, ldd, ldp, ldz, T, N}, act, dev, stream);
}

int launch_gated_dz(const uint16_t* dout, long long ldd, const uint16_t* pre, long long ldp, int act, int T, int F,
                    uint16_t* dz, long long ldz, const DeviceInfo& dev, cudaStream_t stream) {
  return launch<true>({dout, pre, dz, nullptr, ldd, ldp, ldz, T, F}, act, dev, stream);
}

}  // namespace linear_impl
}  // namespace moe
