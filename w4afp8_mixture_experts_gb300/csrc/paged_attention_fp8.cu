// paged_attention_decode over caches of E4M3, queries of bf16 (paged_attention.cuh).
#include "paged_attention.cuh"

namespace w4a8 {
int launch_attend_fp8_f16(const AttendParams& p, cudaStream_t st);
int launch_attend_fp8(const AttendParams& p, bool q_f16, cudaStream_t st) {
  return q_f16 ? launch_attend_fp8_f16(p, st) : launch_attend_kind<2>(p, st);
}
}  // namespace w4a8
