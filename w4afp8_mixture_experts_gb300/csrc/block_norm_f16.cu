// block_norm's kernels for f16 (block_norm.cuh), in a translation unit of their own.
#include "block_norm.cuh"

namespace w4a8 {
int launch_norm_f16(const NormParams& p, bool residual_f32, bool vec, cudaStream_t st) {
  return residual_f32 ? dispatch<__half, float>(p, vec, st) : dispatch<__half, __half>(p, vec, st);
}
}  // namespace w4a8
