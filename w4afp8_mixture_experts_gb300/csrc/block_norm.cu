// The norms after and before a block in one pass over a token's row, with the block's gate and residual:
//   u = norm_post(f)      h = residual_scale * r + branch_scale * gate * u      y = norm_pre(h)
// norm in {none, rms, layer}; sums and the values between the two norms stay in fp32 registers, h and y are
// each rounded once (y from the unrounded h).
//
// A row is held by the threads of one block (or one warp, for short rows: several rows to a block); the row's
// sums are one block reduction each (the mean first, then the squared differences, for a LayerNorm).
#include "common.cuh"
#include "block_ops.cuh"

namespace w4a8 {
namespace {

constexpr int kMaxH = 32768;

struct NormParams {
  const void* f;
  const void* r;       // nullptr: no residual
  const void* gate;    // nullptr: 1
  const void* w_post;  // nullptr: 1
  const void* b_post;  // nullptr: 0
  const void* w_pre;
  const void* b_pre;
  void* h;  // nullptr: not wanted
  void* y;  // nullptr: not wanted
  int64_t ldf, ldr, ldg, ldh, ldy;
  int T, H;
  int post, pre;      // w4a8_norm
  int rows_per_gate;  // row t uses gate row t / rows_per_gate
  int gate_scalar;    // one gate value per gate row
  int gate_f32, w_f32;
  float branch_scale, residual_scale, eps;
};

template <typename T, int V>
struct alignas(V * sizeof(T) > 16 ? 16 : V * sizeof(T)) Pack {
  T v[V];
};

template <typename T, int V>
__device__ __forceinline__ void load_vec(const T* p, float (&o)[V]) {
  const Pack<T, V> a = *reinterpret_cast<const Pack<T, V>*>(p);
#pragma unroll
  for (int i = 0; i < V; ++i) o[i] = to_f32(a.v[i]);
}
template <typename T, int V>
__device__ __forceinline__ void store_vec(T* p, const float (&o)[V]) {
  Pack<T, V> a;
#pragma unroll
  for (int i = 0; i < V; ++i) a.v[i] = from_f32<T>(o[i]);
  *reinterpret_cast<Pack<T, V>*>(p) = a;
}
// a parameter vector: fp32 or the activations' type
template <typename X, int V>
__device__ __forceinline__ void load_param(const void* p, int f32, int64_t at, float (&o)[V]) {
  if (f32)
    load_vec<float, V>(static_cast<const float*>(p) + at, o);
  else
    load_vec<X, V>(static_cast<const X*>(p) + at, o);
}

// Sum over the row's threads; the same value on all of them.  `slot` alternates between two halves of the
// scratch so that one barrier per reduction is enough.
__device__ __forceinline__ float row_sum(float v, float* scratch, int& slot) {
  v = warp_sum(v);
  const int warps = blockDim.x >> 5;
  if (warps == 1) return v;
  float* s = scratch + slot;
  slot ^= 32;
  if ((threadIdx.x & 31) == 0) s[threadIdx.x >> 5] = v;
  __syncthreads();
  const int lane = threadIdx.x & 31;
  return warp_sum(lane < warps ? s[lane] : 0.f);
}

template <int V, int VPT>
__device__ __forceinline__ void normalise(float (&u)[VPT][V], int kind, int H, float eps, float* scratch, int& slot) {
  float s = 0.f;
  if (kind == W4A8_NORM_LAYER) {
#pragma unroll
    for (int j = 0; j < VPT; ++j)
#pragma unroll
      for (int i = 0; i < V; ++i) s += u[j][i];
    const float mean = row_sum(s, scratch, slot) / H;
    s = 0.f;
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
      const bool in = (j * blockDim.x + threadIdx.x) * V < H;
#pragma unroll
      for (int i = 0; i < V; ++i) u[j][i] = in ? u[j][i] - mean : 0.f;
    }
  }
#pragma unroll
  for (int j = 0; j < VPT; ++j)
#pragma unroll
    for (int i = 0; i < V; ++i) s = fmaf(u[j][i], u[j][i], s);
  const float inv = rsqrtf(row_sum(s, scratch, slot) / H + eps);
#pragma unroll
  for (int j = 0; j < VPT; ++j)
#pragma unroll
    for (int i = 0; i < V; ++i) u[j][i] *= inv;
}

template <typename X, int V, int VPT>
__device__ __forceinline__ void scale_shift(float (&u)[VPT][V], const void* w, const void* b, int f32, int H) {
#pragma unroll
  for (int j = 0; j < VPT; ++j) {
    const int c = (j * blockDim.x + threadIdx.x) * V;
    if (c >= H) continue;
    float a[V];
    if (w) {
      load_param<X, V>(w, f32, c, a);
#pragma unroll
      for (int i = 0; i < V; ++i) u[j][i] *= a[i];
    }
    if (b) {
      load_param<X, V>(b, f32, c, a);
#pragma unroll
      for (int i = 0; i < V; ++i) u[j][i] += a[i];
    }
  }
}

// blockDim.x threads hold a row (VPT vectors of V elements each), blockDim.y rows to a block (only with
// blockDim.x = 32, where no barrier is needed).
template <typename X, typename R, int V, int VPT>
__global__ void __launch_bounds__(1024) block_norm_kernel(const NormParams p) {
  __shared__ float scratch[64];
  pdl_trigger();
  pdl_wait();
  int slot = 0;
  const int64_t step = static_cast<int64_t>(gridDim.x) * blockDim.y;
  for (int64_t t = static_cast<int64_t>(blockIdx.x) * blockDim.y + threadIdx.y; t < p.T; t += step) {
    float u[VPT][V];
    const X* f = static_cast<const X*>(p.f) + t * p.ldf;
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
      const int c = (j * blockDim.x + threadIdx.x) * V;
#pragma unroll
      for (int i = 0; i < V; ++i) u[j][i] = 0.f;
      if (c < p.H) load_vec<X, V>(f + c, u[j]);
    }
    if (p.post != W4A8_NORM_NONE) {
      normalise<V, VPT>(u, p.post, p.H, p.eps, scratch, slot);
      scale_shift<X, V, VPT>(u, p.w_post, p.b_post, p.w_f32, p.H);
    }
    const int64_t grow = p.gate ? (t / p.rows_per_gate) * p.ldg : 0;
    float gs = p.branch_scale;
    if (p.gate && p.gate_scalar) {
      float a[1];
      load_param<X, 1>(p.gate, p.gate_f32, grow, a);
      gs *= a[0];
    }
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
      const int c = (j * blockDim.x + threadIdx.x) * V;
      if (c >= p.H) continue;
      float a[V];
      if (p.gate && !p.gate_scalar) {
        load_param<X, V>(p.gate, p.gate_f32, grow + c, a);
#pragma unroll
        for (int i = 0; i < V; ++i) u[j][i] *= a[i];
      }
#pragma unroll
      for (int i = 0; i < V; ++i) u[j][i] *= gs;
      if (p.r) {
        load_vec<R, V>(static_cast<const R*>(p.r) + t * p.ldr + c, a);
#pragma unroll
        for (int i = 0; i < V; ++i) u[j][i] = fmaf(p.residual_scale, a[i], u[j][i]);
      }
      if (p.h) store_vec<R, V>(static_cast<R*>(p.h) + t * p.ldh + c, u[j]);
    }
    if (!p.y) continue;
    if (p.pre != W4A8_NORM_NONE) {
      normalise<V, VPT>(u, p.pre, p.H, p.eps, scratch, slot);
      scale_shift<X, V, VPT>(u, p.w_pre, p.b_pre, p.w_f32, p.H);
    }
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
      const int c = (j * blockDim.x + threadIdx.x) * V;
      if (c < p.H) store_vec<X, V>(static_cast<X*>(p.y) + t * p.ldy + c, u[j]);
    }
  }
}

template <typename X, typename R, int V, int VPT>
int launch_norm(const NormParams& p, cudaStream_t st) {
  const int64_t per = ceil_div(ceil_div(p.H, V * VPT), 32) * 32;  // threads of a row
  const int rows = per == 32 ? 8 : 1;
  const int64_t blocks = ceil_div(p.T, rows);
  return launch_pdl("block_norm_kernel", block_norm_kernel<X, R, V, VPT>, dim3(static_cast<unsigned>(blocks)),
                    dim3(static_cast<unsigned>(per), rows), 0, st, p);
}

template <typename X, typename R>
int dispatch(const NormParams& p, bool vec, cudaStream_t st) {
  if (vec) {
    if (p.H <= 8192) return launch_norm<X, R, 8, 1>(p, st);
    if (p.H <= 16384) return launch_norm<X, R, 8, 2>(p, st);
    return launch_norm<X, R, 8, 4>(p, st);
  }
  if (p.H <= 2048) return launch_norm<X, R, 1, 4>(p, st);
  if (p.H <= 8192) return launch_norm<X, R, 1, 8>(p, st);
  return launch_norm<X, R, 1, 32>(p, st);
}

}  // namespace
}  // namespace w4a8

extern "C" int block_norm(const void* f, int64_t ldf, int dtype, const void* residual, int64_t ldr, int residual_dtype,
                          int post, const void* w_post, const void* b_post, const void* gate, int64_t ldg,
                          int64_t gate_rows, int64_t gate_cols, int gate_dtype, float branch_scale,
                          float residual_scale, int pre, const void* w_pre, const void* b_pre, int param_dtype,
                          float eps, int64_t T, int64_t H, void* h, int64_t ldh, void* y, int64_t ldy, void* stream) {
  using namespace w4a8;
  W4A8_REQUIRE(dtype >= W4A8_DTYPE_BF16 && dtype <= W4A8_DTYPE_F32, "dtype=%d is not a w4a8_dtype", dtype);
  W4A8_REQUIRE(residual_dtype == dtype || residual_dtype == W4A8_DTYPE_F32,
               "residual_dtype=%d must be dtype=%d or fp32", residual_dtype, dtype);
  W4A8_REQUIRE(param_dtype == dtype || param_dtype == W4A8_DTYPE_F32, "param_dtype=%d must be dtype=%d or fp32",
               param_dtype, dtype);
  W4A8_REQUIRE(post >= W4A8_NORM_NONE && post <= W4A8_NORM_LAYER && pre >= W4A8_NORM_NONE && pre <= W4A8_NORM_LAYER,
               "post=%d and pre=%d must be 0 (none), 1 (rms) or 2 (layer)", post, pre);
  W4A8_REQUIRE(T >= 0 && T < (1ll << 31), "T=%lld out of range", (long long)T);
  W4A8_REQUIRE(H >= 1 && H <= kMaxH, "H=%lld must be in [1, %d]", (long long)H, kMaxH);
  W4A8_REQUIRE(eps >= 0.f, "eps must not be negative");
  W4A8_REQUIRE(ldf >= H && (!residual || ldr >= H) && (!h || ldh >= H) && (!y || ldy >= H),
               "leading dimensions must be at least H=%lld", (long long)H);
  W4A8_REQUIRE((post != W4A8_NORM_NONE || (!w_post && !b_post)) && (pre != W4A8_NORM_NONE || (!w_pre && !b_pre)),
               "weights given for a norm that is none");
  if (gate) {
    W4A8_REQUIRE(gate_dtype == dtype || gate_dtype == W4A8_DTYPE_F32, "gate_dtype=%d must be dtype=%d or fp32",
                 gate_dtype, dtype);
    W4A8_REQUIRE(gate_cols == 1 || gate_cols == H, "gate_cols=%lld must be 1 or H=%lld", (long long)gate_cols,
                 (long long)H);
    W4A8_REQUIRE(gate_rows >= 1 && (T == 0 || (gate_rows <= T && T % gate_rows == 0)),
                 "gate_rows=%lld must divide T=%lld", (long long)gate_rows, (long long)T);
    W4A8_REQUIRE(ldg >= gate_cols, "ldg=%lld must be at least gate_cols=%lld", (long long)ldg, (long long)gate_cols);
  }
  if (T == 0) return W4A8_OK;
  W4A8_REQUIRE(f, "null pointer");
  W4A8_REQUIRE(h || y, "h and y are both null: nothing to compute");
  const int64_t sx = static_cast<int64_t>(dtype_size(dtype)), sr = static_cast<int64_t>(dtype_size(residual_dtype));
  const int64_t sp = static_cast<int64_t>(dtype_size(param_dtype)), sg = static_cast<int64_t>(dtype_size(gate_dtype));
  bool vec = H % 8 == 0;
  bool elem = true;
  auto look = [&](const void* q, int64_t ld, int64_t size) {
    if (!q) return;
    const uintptr_t a = reinterpret_cast<uintptr_t>(q);
    elem = elem && a % size == 0;
    vec = vec && a % 16 == 0 && ld * size % 16 == 0;
  };
  look(f, ldf, sx);
  look(residual, ldr, sr);
  look(h, ldh, sr);
  look(y, ldy, sx);
  look(w_post, 0, sp);
  look(b_post, 0, sp);
  look(w_pre, 0, sp);
  look(b_pre, 0, sp);
  if (gate && gate_cols == 1)
    elem = elem && reinterpret_cast<uintptr_t>(gate) % sg == 0;
  else
    look(gate, ldg, sg);
  W4A8_REQUIRE(elem, "every pointer must be aligned to its element size");
  NormParams p;
  p.f = f;
  p.r = residual;
  p.gate = gate;
  p.w_post = w_post;
  p.b_post = b_post;
  p.w_pre = w_pre;
  p.b_pre = b_pre;
  p.h = h;
  p.y = y;
  p.ldf = ldf;
  p.ldr = ldr;
  p.ldg = ldg;
  p.ldh = ldh;
  p.ldy = ldy;
  p.T = static_cast<int>(T);
  p.H = static_cast<int>(H);
  p.post = post;
  p.pre = pre;
  p.rows_per_gate = gate ? static_cast<int>(T / gate_rows) : 1;
  p.gate_scalar = gate && gate_cols == 1 && H != 1;
  p.gate_f32 = gate_dtype == W4A8_DTYPE_F32;
  p.w_f32 = param_dtype == W4A8_DTYPE_F32;
  p.branch_scale = branch_scale;
  p.residual_scale = residual_scale;
  p.eps = eps;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const bool r32 = residual_dtype == W4A8_DTYPE_F32;
  if (dtype == W4A8_DTYPE_F32) return dispatch<float, float>(p, vec, st);
  if (dtype == W4A8_DTYPE_F16) return r32 ? dispatch<__half, float>(p, vec, st) : dispatch<__half, __half>(p, vec, st);
  return r32 ? dispatch<__nv_bfloat16, float>(p, vec, st) : dispatch<__nv_bfloat16, __nv_bfloat16>(p, vec, st);
}
