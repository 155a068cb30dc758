// Device helpers shared by the operators around the routed experts (block norm, dense linear, grouped routing).
#pragma once

#include <type_traits>

#include "common.cuh"

namespace w4a8 {

__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ float to_f32(__half v) { return __half2float(v); }
__device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }

template <typename T>
__device__ __forceinline__ T from_f32(float v);
template <>
__device__ __forceinline__ float from_f32<float>(float v) { return v; }
template <>
__device__ __forceinline__ __half from_f32<__half>(float v) { return __float2half_rn(v); }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}

// two fp32 values rounded to T and packed (16-bit types)
template <typename T>
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  if constexpr (std::is_same<T, __half>::value) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
  } else {
    return bf16x2_bits(lo, hi);
  }
}

// one element of a w4a8_dtype known at run time
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

inline size_t dtype_size(int dtype) { return dtype == W4A8_DTYPE_F32 ? 4 : 2; }

}  // namespace w4a8
