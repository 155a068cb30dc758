// paged_attention_decode over caches of bf16 (paged_attention.cuh).
#include "paged_attention.cuh"

namespace w4a8 {
int launch_attend_bf16(const AttendParams& p, cudaStream_t st) { return launch_attend_kind<0>(p, st); }
}  // namespace w4a8
