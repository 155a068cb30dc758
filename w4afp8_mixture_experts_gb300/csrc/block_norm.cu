// block_norm: argument checks and the fp32 kernels (block_norm.cuh).
#include "block_norm.cuh"

namespace w4a8 {
int launch_norm_f32(const NormParams& p, bool vec, cudaStream_t st) { return dispatch<float, float>(p, vec, st); }
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
  bool vec = true;  // rows start on 16-byte boundaries
  bool elem = true;
  auto look = [&](const void* q, int64_t ld, int64_t size) {
    if (!q) return;
    const uintptr_t a = reinterpret_cast<uintptr_t>(q);
    elem = elem && a % size == 0;
    vec = vec && a % 16 == 0 && (T == 1 || ld * size % 16 == 0);
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
  if (dtype == W4A8_DTYPE_F32) return launch_norm_f32(p, vec, st);
  return dtype == W4A8_DTYPE_F16 ? launch_norm_f16(p, r32, vec, st) : launch_norm_bf16(p, r32, vec, st);
}
