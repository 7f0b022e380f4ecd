// BF16 products with an epilogue and their gradients: argument checks and the choice of kernel.
//   linear   z = x w^T + bias, out = act(z) + residual
//   gated    [g | u] = x w^T, out = act(g) u
//   gradients: dz (linear_grad.cu), then dx = dz w and dw = dz^T x, both in one launch
#include "linear.cuh"

namespace moe {
namespace {

using namespace linear_impl;

constexpr long long kMaxSize = (1LL << 31) - (1 << 16);  // (TMA coordinates of a tile that starts inside)

bool dtype_ok(int dt) { return dt == MOE_DTYPE_F32 || dt == MOE_DTYPE_BF16; }
bool act_ok(int act) { return act >= BF16_ACT_NONE && act <= BF16_ACT_GELU_TANH; }
int size_of(int dt) { return dt == MOE_DTYPE_F32 ? 4 : 2; }

// An operand in rows that TMA can read.
int check_rows(const void* p, int64_t ld, long long cols) {
  if (!p || ld < cols || ld % 8 != 0) return MOE_ERR_INVALID_ARGUMENT;
  if (ld >= (1LL << 38)) return MOE_ERR_CAPACITY;
  return aligned(p, 16) ? MOE_OK : MOE_ERR_ALIGNMENT;
}
// Rows that plain loads and stores go to.
int check_plain(const void* p, int64_t ld, long long cols, int size) {
  if (!p || ld < cols) return MOE_ERR_INVALID_ARGUMENT;
  return aligned(p, size) ? MOE_OK : MOE_ERR_ALIGNMENT;
}

int check_sizes(int T, int N, int K, bool gated) {
  if (T < 0 || N < 0 || K < 1) return MOE_ERR_INVALID_ARGUMENT;
  if (T >= kMaxSize || K >= kMaxSize || (gated ? 2LL * N : (long long)N) >= kMaxSize) return MOE_ERR_CAPACITY;
  return MOE_OK;
}

#define MOE_TRY(call)                 \
  do {                                \
    const int st_ = (call);           \
    if (st_ != MOE_OK) return st_;    \
  } while (0)

// The plans of the sizes that a thread asked for last: the search takes 1 to 4 us of the host, half of what is
// left of a call.
struct Choice {
  int M, N, K, kind, device;  // kind: what else a plan depends on (0: an empty entry)
  bool narrow;
  NarrowPlan n;
  WidePlan both, one;  // (forward: one)
};
int kind_of(const Product& p) {
  const Epilogue& e = p.e;
  return (e.out_f32 ? 1 : 0) | (e.residual ? (e.residual_f32 ? 4 : 2) : 0) | (e.pre ? 8 : 0);
}
template <typename Make>
int choose(int M, int N, int K, int kind, int device, const Choice** choice, Make make) {
  static thread_local Choice known[64];
  const uint32_t h = ((uint32_t)M * 2654435761u) ^ ((uint32_t)N * 2246822519u) ^ ((uint32_t)K * 3266489917u) ^ ((uint32_t)kind * 668265263u);
  Choice& c = known[(h ^ h >> 15) & 63];
  if (c.M != M || c.N != N || c.K != K || c.kind != kind || c.device != device) {
    c.kind = 0;
    MOE_TRY(make(&c));
    c.M = M, c.N = N, c.K = K, c.kind = kind, c.device = device;
  }
  *choice = &c;
  return MOE_OK;
}

int forward(const Product& p, bool gated, cudaStream_t stream) {
  DeviceInfo dev;
  MOE_TRY(current_device(&dev));
  const Choice* c;
  MOE_TRY(choose(p.M, p.N, p.K, 64 | (gated ? 128 : 0) | kind_of(p), dev.device, &c, [&](Choice* c) {
    MOE_TRY(plan_narrow(p, gated, dev, &c->n));
    c->one = plan_wide(&p, 1, gated, dev);
    c->narrow = c->n.ns < c->one.ns;
    return MOE_OK;
  }));
  return c->narrow ? launch_narrow(p, gated, c->n, dev, stream) : launch_wide(&p, 1, gated, c->one, dev, stream);
}

// Rows of dz start at multiples of 128 bytes, so that a box's rows are whole lines (129 x 2072 x 2064 10.2 us, 12.4 with
// rows of 4144 bytes).
long long padded(long long n) { return (n + 63) / 64 * 64; }
size_t dz_bytes(int T, long long n) { return T > 0 && n > 0 ? (size_t)T * padded(n) * 2 : 0; }

struct Grads {
  void* dx;
  int64_t ldx;
  int dx_dtype;
  void* dw;
  int64_t ldw;
  int dw_dtype;
  float* dbias;
};

int check_grads(const Grads& g, long long N, int K) {
  if (g.dx && !dtype_ok(g.dx_dtype)) return MOE_ERR_INVALID_ARGUMENT;
  if (g.dw && !dtype_ok(g.dw_dtype)) return MOE_ERR_INVALID_ARGUMENT;
  if (g.dx) MOE_TRY(check_plain(g.dx, g.ldx, K, size_of(g.dx_dtype)));
  if (g.dw) MOE_TRY(check_plain(g.dw, g.ldw, K, size_of(g.dw_dtype)));
  return aligned(g.dbias, 4) ? MOE_OK : MOE_ERR_ALIGNMENT;
}

// A sum over no rows: zeros.
int zero_rows(void* p, int64_t ld, int dtype, long long rows, int cols, cudaStream_t stream) {
  const size_t size = size_of(dtype);
  if (ld == cols || rows == 1) return cudaMemsetAsync(p, 0, (size_t)rows * cols * size, stream) == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
  return cudaMemset2DAsync(p, ld * size, 0, cols * size, rows, stream) == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

// dx and dw from dz [T, n].
int backward_products(const uint16_t* dz, long long ldz, const uint16_t* x, int64_t ldx, const uint16_t* w, int64_t ldw,
                      const Grads& g, int T, int n, int K, const DeviceInfo& dev, cudaStream_t stream) {
  Product p[2] = {};
  Product &px = p[0], &pw = p[1];
  px.a = {dz, ldz, false}, px.b = {w, ldw, true};
  px.M = T, px.N = K, px.K = n;
  px.e.out = g.dx, px.e.ldo = g.ldx, px.e.out_f32 = g.dx && g.dx_dtype == MOE_DTYPE_F32;
  pw.a = {dz, ldz, true}, pw.b = {x, ldx, true};
  pw.M = n, pw.N = K, pw.K = T;
  pw.e.out = g.dw, pw.e.ldo = g.ldw, pw.e.out_f32 = g.dw && g.dw_dtype == MOE_DTYPE_F32;
  // Both in one launch, or dx by the narrow kernel and dw after it (a launch more, of which the first one's end hides
  // some). Whether dw is asked for does not enter: dx alone is what it is beside a dw in BF16.
  const Choice* found;
  MOE_TRY(choose(T, n, K, 256 | kind_of(px) | kind_of(pw) << 4, dev.device, &found, [&](Choice* c) {
    c->both = plan_wide(p, 2, false, dev), c->one = plan_wide(&pw, 1, false, dev);
    MOE_TRY(plan_narrow(px, false, dev, &c->n));
    c->narrow = c->n.ns + c->one.ns - 1000 < c->both.ns;
    return MOE_OK;
  }));
  const Choice& c = *found;
  if (g.dx && g.dw && !c.narrow) return launch_wide(p, 2, false, c.both, dev, stream);
  if (g.dx) MOE_TRY(c.narrow ? launch_narrow(px, false, c.n, dev, stream) : launch_wide(&px, 1, false, plan_wide(&px, 1, false, dev), dev, stream));
  return g.dw ? launch_wide(&pw, 1, false, c.one, dev, stream) : MOE_OK;
}

int empty_grads(const Grads& g, int T, long long n, int K, cudaStream_t stream) {
  DeviceInfo dev;
  MOE_TRY(current_device(&dev));
  if (n == 0 && T > 0 && g.dx) MOE_TRY(zero_rows(g.dx, g.ldx, g.dx_dtype, T, K, stream));
  if (T == 0 && n > 0 && g.dw) MOE_TRY(zero_rows(g.dw, g.ldw, g.dw_dtype, n, K, stream));
  if (T == 0 && n > 0 && g.dbias) MOE_TRY(zero_rows(g.dbias, n, MOE_DTYPE_F32, 1, (int)n, stream));
  return MOE_OK;
}

}  // namespace
}  // namespace moe

extern "C" int bf16_linear(const uint16_t* x, int64_t ldx, const uint16_t* w, int64_t ldw, const void* bias,
                           int bias_dtype, const void* residual, int64_t ldr, int residual_dtype, int activation, int T,
                           int N, int K, void* out, int64_t ldo, int out_dtype, uint16_t* pre, int64_t ldp,
                           moe_stream_t stream) {
  using namespace moe;
  MOE_TRY(check_sizes(T, N, K, false));
  if (!act_ok(activation) || !dtype_ok(out_dtype)) return MOE_ERR_INVALID_ARGUMENT;
  if ((bias && !dtype_ok(bias_dtype)) || (residual && !dtype_ok(residual_dtype))) return MOE_ERR_INVALID_ARGUMENT;
  if (T == 0 || N == 0) return MOE_OK;
  MOE_TRY(check_rows(x, ldx, K));
  MOE_TRY(check_rows(w, ldw, K));
  MOE_TRY(check_plain(out, ldo, N, size_of(out_dtype)));
  if (bias) MOE_TRY(check_plain(bias, N, N, size_of(bias_dtype)));
  if (residual) MOE_TRY(check_plain(residual, ldr, N, size_of(residual_dtype)));
  if (pre) MOE_TRY(check_plain(pre, ldp, N, 2));
  Product p = {};
  p.a = {x, ldx, false}, p.b = {w, ldw, false};
  p.M = T, p.N = N, p.K = K;
  p.e.bias = bias, p.e.bias_f32 = bias_dtype == MOE_DTYPE_F32;
  p.e.residual = residual, p.e.ldr = ldr, p.e.residual_f32 = residual_dtype == MOE_DTYPE_F32;
  p.e.out = out, p.e.ldo = ldo, p.e.out_f32 = out_dtype == MOE_DTYPE_F32;
  p.e.pre = pre, p.e.ldp = ldp, p.e.act = activation;
  return forward(p, false, as_cuda(stream));
}

extern "C" int bf16_gated_linear(const uint16_t* x, int64_t ldx, const uint16_t* w, int64_t ldw, int activation, int T,
                                 int F, int K, uint16_t* out, int64_t ldo, uint16_t* pre, int64_t ldp,
                                 moe_stream_t stream) {
  using namespace moe;
  MOE_TRY(check_sizes(T, F, K, true));
  if (!act_ok(activation)) return MOE_ERR_INVALID_ARGUMENT;
  if (T == 0 || F == 0) return MOE_OK;
  MOE_TRY(check_rows(x, ldx, K));
  MOE_TRY(check_rows(w, ldw, K));
  MOE_TRY(check_plain(out, ldo, F, 2));
  if (pre) MOE_TRY(check_plain(pre, ldp, 2LL * F, 2));
  Product p = {};
  p.a = {x, ldx, false}, p.b = {w, ldw, false};
  p.M = T, p.N = F, p.K = K;
  p.e.out = out, p.e.ldo = ldo, p.e.pre = pre, p.e.ldp = ldp, p.e.act = activation;
  return forward(p, true, as_cuda(stream));
}

extern "C" size_t bf16_linear_backward_workspace(int T, int N) { return moe::dz_bytes(T, N); }

extern "C" int bf16_linear_backward(const uint16_t* dout, int64_t ldd, const uint16_t* x, int64_t ldx, const uint16_t* w,
                                    int64_t ldw, const uint16_t* pre, int64_t ldp, int activation, int T, int N, int K,
                                    void* dx, int64_t lddx, int dx_dtype, void* dw, int64_t lddw, int dw_dtype,
                                    float* dbias, void* workspace, size_t workspace_bytes, moe_stream_t stream) {
  using namespace moe;
  MOE_TRY(check_sizes(T, N, K, false));
  if (!act_ok(activation)) return MOE_ERR_INVALID_ARGUMENT;
  const Grads g = {dx, lddx, dx_dtype, dw, lddw, dw_dtype, dbias};
  MOE_TRY(check_grads(g, N, K));
  if (T == 0 || N == 0) return empty_grads(g, T, N, K, as_cuda(stream));
  MOE_TRY(check_plain(dout, ldd, N, 2));
  if (dw) MOE_TRY(check_rows(x, ldx, K));
  if (dx) MOE_TRY(check_rows(w, ldw, K));
  const bool slope = activation != BF16_ACT_NONE;
  if (slope) MOE_TRY(check_plain(pre, ldp, N, 2));
  // dout itself serves where it is dz, in rows that TMA can read
  const bool made = (dx || dw) && (slope || !aligned(dout, 16) || ldd % 8 != 0);
  if (made && (!workspace || workspace_bytes < dz_bytes(T, N))) return MOE_ERR_WORKSPACE;
  if (!aligned(workspace, 16)) return MOE_ERR_ALIGNMENT;
  DeviceInfo dev;
  MOE_TRY(current_device(&dev));
  const long long ldz = made ? padded(N) : ldd;
  if (made || dbias)
    MOE_TRY(launch_dz(dout, ldd, slope ? pre : nullptr, ldp, activation, T, N, made ? static_cast<uint16_t*>(workspace) : nullptr,
                      ldz, dbias, dev, as_cuda(stream)));
  return backward_products(made ? static_cast<const uint16_t*>(workspace) : dout, ldz, x, ldx, w, ldw, g, T, N, K, dev,
                           as_cuda(stream));
}

extern "C" size_t bf16_gated_linear_backward_workspace(int T, int F) { return moe::dz_bytes(T, 2LL * F); }

extern "C" int bf16_gated_linear_backward(const uint16_t* dout, int64_t ldd, const uint16_t* x, int64_t ldx,
                                          const uint16_t* w, int64_t ldw, const uint16_t* pre, int64_t ldp,
                                          int activation, int T, int F, int K, void* dx, int64_t lddx, int dx_dtype,
                                          void* dw, int64_t lddw, int dw_dtype, void* workspace, size_t workspace_bytes,
                                          moe_stream_t stream) {
  using namespace moe;
  MOE_TRY(check_sizes(T, F, K, true));
  if (!act_ok(activation)) return MOE_ERR_INVALID_ARGUMENT;
  const Grads g = {dx, lddx, dx_dtype, dw, lddw, dw_dtype, nullptr};
  MOE_TRY(check_grads(g, 2LL * F, K));
  if (T == 0 || F == 0) return empty_grads(g, T, 2LL * F, K, as_cuda(stream));
  MOE_TRY(check_plain(dout, ldd, F, 2));
  if (dw) MOE_TRY(check_rows(x, ldx, K));
  if (dx) MOE_TRY(check_rows(w, ldw, K));
  MOE_TRY(check_plain(pre, ldp, 2LL * F, 2));
  if (!dx && !dw) return MOE_OK;
  if (!workspace || workspace_bytes < dz_bytes(T, 2LL * F)) return MOE_ERR_WORKSPACE;
  if (!aligned(workspace, 16)) return MOE_ERR_ALIGNMENT;
  DeviceInfo dev;
  MOE_TRY(current_device(&dev));
  uint16_t* const dz = static_cast<uint16_t*>(workspace);
  MOE_TRY(launch_gated_dz(dout, ldd, pre, ldp, activation, T, F, dz, padded(2LL * F), dev, as_cuda(stream)));
  return backward_products(dz, padded(2LL * F), x, ldx, w, ldw, g, T, 2 * F, K, dev, as_cuda(stream));
}
