// Grouped expert routing: argument checks, the choice of lanes, and the 32-lane instances (route_grouped.cuh).
#include "route_grouped.cuh"

namespace w4a8 {
int launch_route_32(const RouteParams& p, cudaStream_t st) { return launch_lanes<32>(p, st); }
}  // namespace w4a8

extern "C" int moe_route_grouped_topk(const void* logits, int logits_dtype, int64_t ld, int64_t T, int64_t E, int k,
                                      int score, const float* bias, int n_group, int topk_group, int group_top,
                                      int renormalize, float scale, int32_t* topk_ids, float* topk_w, void* stream) {
  using namespace w4a8;
  W4A8_REQUIRE(logits_dtype >= W4A8_DTYPE_BF16 && logits_dtype <= W4A8_DTYPE_F32, "logits_dtype=%d is not a w4a8_dtype",
               logits_dtype);
  W4A8_REQUIRE(score == W4A8_SCORE_SOFTMAX || score == W4A8_SCORE_SIGMOID, "score=%d must be 0 (softmax) or 1 (sigmoid)",
               score);
  W4A8_REQUIRE(T >= 0 && T < (1ll << 26), "T=%lld out of range", (long long)T);
  W4A8_REQUIRE(E >= 1 && E <= 1024, "E=%lld must be in [1, 1024]", (long long)E);
  W4A8_REQUIRE(k >= 1 && k <= 32 && k <= E, "k=%d must be in [1, min(E, 32)]", k);
  W4A8_REQUIRE(ld >= E, "ld=%lld must be >= E=%lld", (long long)ld, (long long)E);
  W4A8_REQUIRE(n_group >= 1 && n_group <= 32 && E % n_group == 0, "n_group=%d must be in [1, 32] and divide E=%lld",
               n_group, (long long)E);
  W4A8_REQUIRE(topk_group >= 1 && topk_group <= n_group, "topk_group=%d must be in [1, n_group=%d]", topk_group, n_group);
  W4A8_REQUIRE((group_top == 1 || group_top == 2) && group_top <= E / n_group,
               "group_top=%d must be 1 or 2 and at most E / n_group", group_top);
  W4A8_REQUIRE(k <= topk_group * (E / n_group), "k=%d exceeds the %lld experts of topk_group=%d groups", k,
               (long long)(topk_group * (E / n_group)), topk_group);
  if (T == 0) return W4A8_OK;
  W4A8_REQUIRE(logits && topk_ids && topk_w, "null pointer");
  W4A8_REQUIRE(reinterpret_cast<uintptr_t>(logits) % (logits_dtype == W4A8_DTYPE_F32 ? 4 : 2) == 0 &&
                   reinterpret_cast<uintptr_t>(bias) % 4 == 0 && reinterpret_cast<uintptr_t>(topk_ids) % 4 == 0 &&
                   reinterpret_cast<uintptr_t>(topk_w) % 4 == 0,
               "logits, bias, topk_ids and topk_w must be aligned to their element size");
  RouteParams p;
  p.logits = logits;
  p.bias = bias;
  p.ids = topk_ids;
  p.w = topk_w;
  p.ld = ld;
  p.lowest = logits_dtype == W4A8_DTYPE_F32   ? -FLT_MAX
             : logits_dtype == W4A8_DTYPE_F16 ? -65504.0f
                                              : -3.389531390e38f;  // exactly the bf16 value 0xFF7F
  p.scale = scale;
  p.T = static_cast<int>(T);
  p.E = static_cast<int>(E);
  p.k = k;
  p.dtype = logits_dtype;
  p.softmax = score == W4A8_SCORE_SOFTMAX;
  p.renorm = renormalize != 0;
  p.n_group = topk_group == n_group ? 1 : n_group;  // when all groups are kept, nothing depends on them
  p.gs = static_cast<int>(E / p.n_group);
  p.topk_group = topk_group;
  p.group_top = group_top;
  p.live = p.n_group == 1 ? static_cast<int>(E) : topk_group * p.gs;
  const auto lay_out = [&](int lanes) {  // experts a lane holds with this many lanes to a token
    p.lpg_log = 0;
    while ((2 << p.lpg_log) * p.n_group <= lanes) ++p.lpg_log;
    p.epl = static_cast<int>(ceil_div(p.gs, 1ll << p.lpg_log));
    // every lane's logits are whole vectors of 4
    const int64_t size = static_cast<int64_t>(dtype_size(logits_dtype));
    p.vec = p.epl % 4 == 0 && p.gs % 4 == 0 && ld % 4 == 0 && reinterpret_cast<uintptr_t>(logits) % (4 * size) == 0;
    return p.epl;
  };
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  // the fewest lanes that hold the groups and the k choices and leave a lane few experts
  const int least = std::max(k, p.n_group);
  if (least <= 8 && lay_out(8) <= 8) return launch_route_8(p, st);
  if (least <= 16 && lay_out(16) <= 10) return launch_route_16(p, st);
  lay_out(32);
  return launch_route_32(p, st);
}
