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

__device__ __forceinline__ float activate(float z, int act) {
  switch (act) {
    case W4A8_ACT_RELU: return fmaxf(z, 0.f);
    case W4A8_ACT_SILU: return z / (1.0f + expf(-z));
    case W4A8_ACT_GELU: return 0.5f * z * (1.0f + erff(z * 0.70710678f));
    case W4A8_ACT_GELU_TANH: return 0.5f * z * (1.0f + tanhf(0.79788456f * (z + 0.044715f * z * z * z)));
    default: return z;
  }
}

__device__ __forceinline__ float load_any(const void* p, int64_t at, int dtype) {
  if (dtype == W4A8_DTYPE_F32) return static_cast<const float*>(p)[at];
  if (dtype == W4A8_DTYPE_F16) return __half2float(static_cast<const __half*>(p)[at]);
  return __bfloat162float(static_cast<const __nv_bfloat16*>(p)[at]);
}
__device__ __forceinline__ void store_any(void* p, int64_t at, float v, int dtype) {
  if (dtype == W4A8_DTYPE_F32)
    static_cast<float*>(p)[at] = v;
  else if (dtype == W4A8_DTYPE_F16)
    static_cast<__half*>(p)[at] = __float2half_rn(v);
  else
    static_cast<__nv_bfloat16*>(p)[at] = __float2bfloat16_rn(v);
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
