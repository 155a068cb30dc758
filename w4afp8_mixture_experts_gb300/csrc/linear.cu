// dense_linear: argument checks and the choice of kernel (linear_stream.cu, linear_tc.cu).
#include "linear.cuh"

extern "C" int dense_linear(const void* x, int64_t ldx, const void* w, int64_t ldw, int dtype, const void* bias,
                            int bias_dtype, int act, int gated, const void* residual, int64_t ldr, void* out,
                            int64_t ldo, int out_dtype, int64_t M, int64_t N, int64_t K, void* ws, size_t ws_bytes,
                            void* stream) {
  using namespace w4a8;
  W4A8_REQUIRE(dtype == W4A8_DTYPE_BF16 || dtype == W4A8_DTYPE_F16, "dtype=%d must be bf16 or f16", dtype);
  W4A8_REQUIRE(out_dtype == dtype || out_dtype == W4A8_DTYPE_F32, "out_dtype=%d must be dtype=%d or fp32", out_dtype,
               dtype);
  W4A8_REQUIRE(!bias || bias_dtype == dtype || bias_dtype == W4A8_DTYPE_F32, "bias_dtype=%d must be dtype=%d or fp32",
               bias_dtype, dtype);
  W4A8_REQUIRE(act >= W4A8_ACT_NONE && act <= W4A8_ACT_GELU_TANH, "act=%d is not a w4a8_act", act);
  W4A8_REQUIRE(M >= 0 && M <= (1 << 20) && N >= 0 && N <= (1 << 20) && K >= 1 && K <= (1 << 20),
               "M=%lld, N=%lld, K=%lld: M and N must be in [0, 2^20], K in [1, 2^20]", (long long)M, (long long)N,
               (long long)K);
  W4A8_REQUIRE(!gated || N % 2 == 0, "N=%lld must be even when gated", (long long)N);
  const int64_t n_out = gated ? N / 2 : N;
  W4A8_REQUIRE(ldx >= K && ldw >= K, "ldx=%lld and ldw=%lld must be at least K=%lld", (long long)ldx, (long long)ldw,
               (long long)K);
  W4A8_REQUIRE(ldo >= n_out && (!residual || ldr >= n_out), "ldo=%lld and ldr=%lld must be at least %lld",
               (long long)ldo, (long long)ldr, (long long)n_out);
  if (M == 0 || N == 0) return W4A8_OK;
  W4A8_REQUIRE(x && w && out, "null pointer");
  const auto at = [](const void* q, int dt) { return reinterpret_cast<uintptr_t>(q) % dtype_size(dt) == 0; };
  W4A8_REQUIRE(at(x, dtype) && at(w, dtype) && at(out, out_dtype) && at(residual, out_dtype) && at(bias, bias_dtype),
               "every pointer must be aligned to its element size");
  LinearParams p;
  p.x = x;
  p.w = w;
  p.bias = bias;
  p.residual = residual;
  p.out = out;
  p.ldx = ldx;
  p.ldw = ldw;
  p.ldr = ldr;
  p.ldo = ldo;
  p.M = static_cast<int>(M);
  p.N = static_cast<int>(N);
  p.K = static_cast<int>(K);
  p.n_out = static_cast<int>(n_out);
  p.dtype = dtype;
  p.out_dtype = out_dtype;
  p.bias_f32 = bias_dtype == W4A8_DTYPE_F32;
  p.act = act;
  p.gated = gated != 0;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  // A few rows of x: streaming starts sooner (1 x 256 x 7168: 3.6 us, the tensor-memory kernels 6.2), but these reach a
  // higher bandwidth on large weights when streaming has two row fragments (gated) or two token tiles to carry (1 x 4096
  // x 7168 gated: 16.6 and 13.0 us; 16 x 2048 x 4096: 8.4 and 6.7; 16 x 256 x 7168: 4.4 and 6.4).  They copy unaligned
  // operands first, which streaming does not.
  const int64_t w_bytes = 2 * N * K, limit = M > 8 ? 12 << 20 : gated ? 24 << 20 : INT64_MAX;
  const bool aligned = aligned16(x) && aligned16(w) && ldx % 8 == 0 && ldw % 8 == 0;
  if (M <= kStreamRows && (w_bytes < limit || !aligned)) return launch_linear_stream(p, st);
  return launch_linear_tc(p, ws, ws_bytes, st);
}

extern "C" size_t dense_linear_workspace_bytes(int64_t M, int64_t N, int64_t K) {
  if (M <= w4a8::kStreamRows || N <= 0 || K <= 0) return 0;
  return static_cast<size_t>(M + N) * w4a8::ceil_div(K, 8) * 16;
}
