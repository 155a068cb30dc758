// Grouped expert routing: softmax or sigmoid scores, a balance bias that only takes part in the choice, the
// best groups of experts, the best experts of those groups, renormalised and scaled weights.
//
// One warp per token.  A group's experts lie on LPG = 2^lpg_log lanes (the largest power of two with
// LPG * n_group <= 32), so a group's largest scores are found by log2(LPG) shuffles; lane (g, sub) holds
// experts g*gs + i*LPG + sub, i < EPL.  The choice values are kept as 32-bit keys in unsigned order, so a
// maximum over the warp is one redux instruction and its index another one (the smallest expert id among
// the lanes that hold it): ties go to the lowest id without a second comparison.
//   key 0            no expert, or already chosen
//   key of -inf      an expert that is out (masked logit, NaN) or whose group was not kept: it only fills
//                    places when fewer than k experts are left, and weighs nothing
#include <cfloat>

#include "block_ops.cuh"
#include "common.cuh"

namespace w4a8 {
namespace {

constexpr uint32_t kKeyOut = 0x007FFFFFu;  // order_key(-inf)
constexpr int kWarps = 8;

// Monotone map of a float (no NaN, no -0) to unsigned integers.
__device__ __forceinline__ uint32_t order_key(float f) {
  const uint32_t u = __float_as_uint(f);
  return u ^ (static_cast<uint32_t>(static_cast<int32_t>(u) >> 31) | 0x80000000u);
}
__device__ __forceinline__ float key_value(uint32_t k) {
  return __uint_as_float(k & 0x80000000u ? k ^ 0x80000000u : ~k);
}

struct RouteParams {
  const void* logits;
  const float* bias;  // [E] or nullptr
  int32_t* ids;
  float* w;
  int64_t ld;
  float lowest;  // logits at or below it take their expert out
  float scale;
  int T, E, k, softmax, renorm;
  int n_group, gs, lpg_log, topk_group, group_top;
};

// 1 / (1 + exp(-l)), every operation rounded once: the same value on every path that reads it.
__device__ __forceinline__ float sigmoid_score(float l) { return __fdiv_rn(1.0f, __fadd_rn(1.0f, expf(-l))); }

// exp(l - max), also where both are +inf.
__device__ __forceinline__ float softmax_term(float l, float mx) { return l == mx ? 1.0f : expf(l - mx); }

template <int EPL, typename L>
__global__ void __launch_bounds__(kWarps * 32) route_grouped_kernel(const RouteParams p) {
  pdl_trigger();
  pdl_wait();
  const int lane = threadIdx.x & 31;
  const int lpg = 1 << p.lpg_log;
  const int g = lane >> p.lpg_log, sub = lane & (lpg - 1);
  const int base = g * p.gs + sub;  // expert of slot i: base + i * lpg, while sub + i * lpg < gs
  const int mine = g < p.n_group ? p.gs - sub : 0;
  const int stride = gridDim.x * (blockDim.x >> 5);
  for (int64_t t = blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5); t < p.T; t += stride) {
    const L* row = static_cast<const L*>(p.logits) + t * p.ld;
    float l[EPL];
    float mx = -INFINITY;
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
      l[i] = -INFINITY;
      if (i * lpg < mine) l[i] = to_f32(row[base + i * lpg]);
      if (!(l[i] > p.lowest)) l[i] = -INFINITY;  // masked, or NaN
      mx = fmaxf(mx, l[i]);
    }
    float total = 0.f;
    if (p.softmax) {
      mx = warp_max(mx);
#pragma unroll
      for (int i = 0; i < EPL; ++i)
        if (l[i] > -INFINITY) total += softmax_term(l[i], mx);
      total = warp_sum(total);
    }
    uint32_t key[EPL];
    uint32_t k1 = 0, k2 = 0;  // this lane's two largest keys
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
      key[i] = 0;
      if (i * lpg < mine) {
        float c = l[i];
        if (c > -INFINITY) {
          if (!p.softmax) c = sigmoid_score(c);
          if (p.bias) {
            // a softmax without a bias is ranked by its logits: the same order, without ties made by rounding
            if (p.softmax) c = __fdiv_rn(softmax_term(c, mx), total);
            c = __fadd_rn(c, p.bias[base + i * lpg]);
            if (!(c >= -INFINITY)) c = -INFINITY;  // NaN bias
          }
        }
        key[i] = order_key(c + 0.0f);  // -0 and +0 are equal
        k2 = max(k2, min(k1, key[i]));
        k1 = max(k1, key[i]);
      }
    }
    if (p.n_group > 1 && p.topk_group < p.n_group) {
      for (int o = 1; o < lpg; o <<= 1) {
        const uint32_t o1 = __shfl_xor_sync(0xffffffffu, k1, o), o2 = __shfl_xor_sync(0xffffffffu, k2, o);
        k2 = max(min(k1, o1), max(k2, o2));
        k1 = max(k1, o1);
      }
      float sc = key_value(k1);
      if (p.group_top == 2) {
        sc = __fadd_rn(sc, key_value(k2));
        if (!(sc >= -INFINITY)) sc = -INFINITY;
      }
      const uint32_t gk = g < p.n_group ? order_key(sc + 0.0f) : 0;
      int rank = 0;  // groups before this one: a larger score, or the same at a lower index
      for (int h = 0; h < p.n_group; ++h) {
        const uint32_t hk = __shfl_sync(0xffffffffu, gk, h << p.lpg_log);
        rank += hk > gk || (hk == gk && h < g);
      }
      if (rank >= p.topk_group) {
#pragma unroll
        for (int i = 0; i < EPL; ++i) key[i] = min(key[i], kKeyOut);
      }
    }
    int my_e = 0;
    uint32_t my_k = 0;
    for (int j = 0; j < p.k; ++j) {
      uint32_t m = 0;
#pragma unroll
      for (int i = 0; i < EPL; ++i) m = max(m, key[i]);
      m = __reduce_max_sync(0xffffffffu, m);
      int e = 0x7fffffff;
#pragma unroll
      for (int i = EPL - 1; i >= 0; --i)
        if (key[i] == m) e = base + i * lpg;
      e = static_cast<int>(__reduce_min_sync(0xffffffffu, static_cast<unsigned>(e)));
#pragma unroll
      for (int i = 0; i < EPL; ++i)
        if (base + i * lpg == e) key[i] = key[i] == m ? 0u : key[i];
      if (lane == j) {
        my_e = e;
        my_k = m;
      }
    }
    float s = 0.f;
    if (lane < p.k && my_k > kKeyOut) {
      const float lj = to_f32(row[my_e]);
      s = p.softmax ? __fdiv_rn(softmax_term(lj, mx), total) : sigmoid_score(lj);
    }
    if (p.renorm) s = __fdiv_rn(s, __fadd_rn(warp_sum(s), 1e-20f));
    if (lane < p.k) {
      const int64_t o = t * p.k + lane;
      p.ids[o] = my_e;
      p.w[o] = __fmul_rn(s, p.scale);
    }
  }
}

template <int EPL>
int launch_route(const RouteParams& p, int dtype, cudaStream_t st) {
  auto kern = dtype == W4A8_DTYPE_F32   ? route_grouped_kernel<EPL, float>
              : dtype == W4A8_DTYPE_F16 ? route_grouped_kernel<EPL, __half>
                                        : route_grouped_kernel<EPL, __nv_bfloat16>;
  const int64_t blocks = ceil_div(p.T, kWarps);
  return launch_pdl("route_grouped_kernel", kern, dim3(static_cast<unsigned>(blocks)), dim3(kWarps * 32), 0, st, p);
}

}  // namespace
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
                                              : -3.389531390e38f;
  p.scale = scale;
  p.T = static_cast<int>(T);
  p.E = static_cast<int>(E);
  p.k = k;
  p.softmax = score == W4A8_SCORE_SOFTMAX;
  p.renorm = renormalize != 0;
  p.n_group = n_group;
  p.gs = static_cast<int>(E / n_group);
  p.lpg_log = 0;
  while ((2 << p.lpg_log) * n_group <= 32) ++p.lpg_log;
  p.topk_group = topk_group;
  p.group_top = group_top;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const int64_t epl = ceil_div(p.gs, 1ll << p.lpg_log);  // experts a lane holds
  if (epl <= 2) return launch_route<2>(p, logits_dtype, st);
  if (epl <= 4) return launch_route<4>(p, logits_dtype, st);
  if (epl <= 5) return launch_route<5>(p, logits_dtype, st);
  if (epl <= 8) return launch_route<8>(p, logits_dtype, st);
  if (epl <= 16) return launch_route<16>(p, logits_dtype, st);
  if (epl <= 32) return launch_route<32>(p, logits_dtype, st);
  return launch_route<64>(p, logits_dtype, st);
}
