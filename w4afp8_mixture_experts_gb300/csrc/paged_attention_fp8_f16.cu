// paged_attention_decode over caches of E4M3, queries of f16 (paged_attention.cuh).
#include "paged_attention.cuh"

namespace w4a8 {
int launch_attend_fp8_f16(const AttendParams& p, cudaStream_t st) { return launch_attend_kind<3>(p, st); }
}  // namespace w4a8
