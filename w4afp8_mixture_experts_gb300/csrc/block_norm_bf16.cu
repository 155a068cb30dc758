// block_norm's kernels for bf16 (block_norm.cuh), in a translation unit of their own.
#include "block_norm.cuh"

namespace w4a8 {
int launch_norm_bf16(const NormParams& p, bool residual_f32, bool vec, cudaStream_t st) {
  return residual_f32 ? dispatch<__nv_bfloat16, float>(p, vec, st) : dispatch<__nv_bfloat16, __nv_bfloat16>(p, vec, st);
}
}  // namespace w4a8
