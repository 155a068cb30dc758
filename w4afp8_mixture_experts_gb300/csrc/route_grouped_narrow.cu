// Grouped expert routing with 8 or 16 lanes to a token (route_grouped.cuh), in a translation unit of their own.
#include "route_grouped.cuh"

namespace w4a8 {
int launch_route_8(const RouteParams& p, cudaStream_t st) { return launch_lanes<8>(p, st); }
int launch_route_16(const RouteParams& p, cudaStream_t st) { return launch_lanes<16>(p, st); }
}  // namespace w4a8
