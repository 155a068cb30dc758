// Declarations shared by the translation units of dense_linear.
#pragma once

#include "block_ops.cuh"
#include "common.cuh"

namespace w4a8 {

// What every kernel of dense_linear gets.  w has N rows; with `gated`, N = 2 * n_out and rows [0, n_out) are
// the gate half, [n_out, N) the other.
struct LinearParams {
  const void* x;
  const void* w;
  const void* bias;      // [N] or nullptr
  const void* residual;  // [M][n_out] of the output's type, or nullptr
  void* out;
  int64_t ldx, ldw, ldr, ldo;
  int M, N, K, n_out;
  int dtype, out_dtype, bias_f32, act, gated;
};

constexpr int kStreamRows = 16;  // rows of x up to which the weights are streamed through mma.sync

int launch_linear_stream(const LinearParams& p, cudaStream_t st);  // M <= kStreamRows
int launch_linear_tc(LinearParams p, void* ws, size_t ws_bytes, cudaStream_t st);

// z / (1 + exp(-y)).  The IEEE division took longer than the rest of an epilogue (its slow path most of all, which
// z = 0 takes: 24 against 5 us for one tile of zeros), the approximate one is good to 2 units in the last place;
// where exp overflows it gives 0 as the exact one does.
__device__ __forceinline__ float times_sigmoid(float z, float y) { return __fdividef(z, 1.0f + __expf(-y)); }

// z * Phi(z) = max(z, 0) - |z| / 2 * erfc(|z| / sqrt 2), erfc by formula 7.1.26 of Abramowitz and Stegun, Handbook of
// Mathematical Functions (absolute error 1.5e-7, so 0.75e-7 |z| here, about one unit of fp32; no cancellation on the
// negative side).  erff took 4.2 us of a tile's epilogue, which then no longer fitted under the products of K = 1024.
__device__ __forceinline__ float gelu(float z) {
  const float a = fabsf(z), x = a * 0.70710678f;
  const float t = __fdividef(1.0f, fmaf(0.3275911f, x, 1.0f));
  float q = fmaf(t, 1.061405429f, -1.453152027f);
  q = fmaf(t, q, 1.421413741f);
  q = fmaf(t, q, -0.284496736f);
  q = fmaf(t, q, 0.254829592f);
  q *= t * __expf(-x * x);
  return (z < 0.f ? 0.f : z) - 0.5f * fminf(a, 64.f) * q;  // q = 0 long before 64: infinities give infinity and 0
}

__device__ __forceinline__ float activate(float z, int act) {
  switch (act) {
    case W4A8_ACT_RELU: return z < 0.f ? 0.f : z;  // keeps NaN
    case W4A8_ACT_SILU: return times_sigmoid(z, z);
    case W4A8_ACT_GELU: return gelu(z);
    // 1/2 (1 + tanh(t)) = 1 / (1 + exp(-2t)), without the cancellation of 1 + tanh
    case W4A8_ACT_GELU_TANH: return times_sigmoid(z, 1.59576912f * (z + 0.044715f * z * z * z));
    default: return z;
  }
}

// out[m][n] from the accumulated products z (gate half) and z2 (other half, gated only)
__device__ __forceinline__ void finish(const LinearParams& p, int m, int n, float z, float z2) {
  const int bd = p.bias_f32 ? W4A8_DTYPE_F32 : p.dtype;
  if (p.bias) z += load_any(p.bias, n, bd);
  float v = activate(z, p.act);
  if (p.gated) {
    if (p.bias) z2 += load_any(p.bias, p.n_out + n, bd);
    v *= z2;
  }
  if (p.residual) v += load_any(p.residual, m * p.ldr + n, p.out_dtype);
  store_any(p.out, m * p.ldo + n, v, p.out_dtype);
}

}  // namespace w4a8
