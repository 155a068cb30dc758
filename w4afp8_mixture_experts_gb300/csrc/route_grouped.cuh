// Grouped expert routing: softmax or sigmoid scores, a balance bias that only takes part in the choice, the
// best groups of experts, the best experts of those groups, renormalised and scaled weights.
//
// The bytes are few (8192 x 256 fp32 logits: 1.3 us); what bounds it is instructions and their latency (8192 x 256 sigmoid,
// 8 groups, k = 8: 11.1 us, 852 a token or 6 us of issue; 65531 x 160 softmax, k = 6: 30.6 us), so every step is made to
// cost few of them per token:
//   * a token has S = 8, 16 or 32 lanes of a warp, the fewest that leave a lane few experts: what a step costs across
//     lanes is then shared by up to four tokens;
//   * a group's experts lie on LPG = 2^lpg_log of them (the largest power of two with LPG * n_group <= S), EPL
//     neighbours to a lane, so a group's largest scores take log2(LPG) shuffles;
//   * choice values become 32-bit keys in unsigned order, which integer maxima (redux over a whole warp) rank;
//   * the kept groups' experts are dealt out evenly to the lanes again (through shared memory), L to a lane, as
//     (key, ~position) pairs, and each lane sorts its own.  A round then looks at the lanes' first pairs only:
//     the largest key, then the position (ties go to the lowest expert), and the lane that held it moves on.
//     (Scanning all of a lane's keys in every round took twice the instructions: 1183 a token at E = 256, k = 8.)
//   key 0            nothing
//   key of -inf      an expert that is out (masked logit, NaN); it only fills places when fewer than k are left
#pragma once

#include <algorithm>
#include <cfloat>

#include "block_ops.cuh"
#include "common.cuh"

namespace w4a8 {

struct RouteParams {
  const void* logits;
  const float* bias;  // [E] or nullptr
  int32_t* ids;
  float* w;
  int64_t ld;
  float lowest;  // logits at or below it take their expert out
  float scale;
  int T, E, k, dtype, softmax, renorm;
  int n_group, gs, lpg_log, epl, topk_group, group_top;
  int live;      // experts of the kept groups
  int vec;       // a lane's logits take 16-byte loads (fp32) or 8-byte ones
};

// S lanes to a token; the layout fields of p are set for it
int launch_route_8(const RouteParams& p, cudaStream_t st);
int launch_route_16(const RouteParams& p, cudaStream_t st);
int launch_route_32(const RouteParams& p, cudaStream_t st);

namespace {

constexpr uint32_t kKeyOut = 0x007FFFFFu;  // order_key(-inf)

// Monotone map of a float (no NaN, no -0) to unsigned integers.
__device__ __forceinline__ uint32_t order_key(float f) {
  const uint32_t u = __float_as_uint(f);
  return u ^ (static_cast<uint32_t>(static_cast<int32_t>(u) >> 31) | 0x80000000u);
}
__device__ __forceinline__ float key_value(uint32_t k) {
  return __uint_as_float(k & 0x80000000u ? k ^ 0x80000000u : ~k);
}

// 1 / (1 + exp(-l)), every operation rounded to nearest: the value that any other path gets from the same steps, so
// that equal choices stay equal and close ones keep their order.
__device__ __forceinline__ float sigmoid_score(float l) { return __frcp_rn(__fadd_rn(1.0f, expf(-l))); }

// exp(l - max), also where both are +inf.  (l - max <= 0: the fast exponential is off by 2 + 1.2 |l - max| units in
// the last place.)
__device__ __forceinline__ float softmax_term(float l, float mx) { return l == mx ? 1.0f : __expf(l - mx); }

// Ranks groups by the sum of two softmax scores, given their logits a >= b and the token's largest logit: the sum's
// logarithm (up to the token's denominator), which neither overflows nor leaves small sums equal.  With infinite logits,
// the sum itself: how many of the two are.
__device__ __forceinline__ float pair_score(float a, float b, float mx) {
  if (b == -INFINITY) return -INFINITY;
  if (mx == INFINITY) return softmax_term(a, mx) + softmax_term(b, mx);
  return fmaxf(a - mx + log1pf(expf(b - a)), -FLT_MAX);
}

// Sorts v[0 .. N) in descending order: merge exchange (Batcher; Knuth, TAOCP vol. 3, algorithm 5.2.2M).
template <int N>
__device__ __forceinline__ void sort_descending(uint64_t (&v)[N]) {
  constexpr int kTop = N <= 2 ? 1 : N <= 4 ? 2 : N <= 8 ? 4 : N <= 16 ? 8 : 16;
#pragma unroll
  for (int p = kTop; p > 0; p >>= 1)
#pragma unroll
    for (int q = kTop; q >= p; q >>= 1) {
      const int r = q == kTop ? 0 : p, d = q == kTop ? p : 2 * q - p;
#pragma unroll
      for (int i = 0; i + d < N; ++i)
        if ((i & p) == r) {
          const uint64_t a = v[i], b = v[i + d];
          v[i] = a < b ? b : a;
          v[i + d] = a < b ? a : b;
        }
    }
}

// Over the S lanes of a token (aligned parts of the warp); the same on all of them.
template <int S>
__device__ __forceinline__ uint32_t lanes_max(uint32_t v) {
  if constexpr (S == 32) {
    return __reduce_max_sync(0xffffffffu, v);
  } else {
#pragma unroll
    for (int o = S / 2; o > 0; o >>= 1) v = max(v, __shfl_xor_sync(0xffffffffu, v, o));
    return v;
  }
}
template <int S>
__device__ __forceinline__ float lanes_max(float v) {
#pragma unroll
  for (int o = S / 2; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}
template <int S>
__device__ __forceinline__ float lanes_sum(float v) {
#pragma unroll
  for (int o = S / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
// bit i: the predicate of the token's lane i
template <int S>
__device__ __forceinline__ uint32_t lanes_ballot(bool b) {
  const uint32_t all = __ballot_sync(0xffffffffu, b);
  if constexpr (S == 32)
    return all;
  else
    return all >> (threadIdx.x & 31 & ~(S - 1)) & ((1u << S) - 1);
}

// The k rounds over the lanes' keys; lane j ends up with the j-th choice.  Position q is the place among the live
// experts in ascending order.
template <int S, int L>
__device__ __forceinline__ void choose(uint64_t (&v)[L], int k, int lane, uint32_t& my_key, int& my_pos) {
  if constexpr (L <= 8) {
    sort_descending<L>(v);
    for (int j = 0; j < k; ++j) {
      const uint32_t key = static_cast<uint32_t>(v[0] >> 32), low = static_cast<uint32_t>(v[0]);
      const uint32_t m = lanes_max<S>(key);
      const uint32_t c = lanes_max<S>(key == m ? low : 0u);
      if (lane == j) {
        my_key = m;
        my_pos = static_cast<int>(~c);
      }
      if (key == m && low == c) {
#pragma unroll
        for (int i = 0; i + 1 < L; ++i) v[i] = v[i + 1];
        v[L - 1] = 0;
      }
    }
  } else {  // several sorted lists: sorting as one would cost more than comparing their heads
    constexpr int kLists = L <= 16 ? 2 : L / 8, kLen = (L + kLists - 1) / kLists;
    uint64_t w[kLists][kLen];
#pragma unroll
    for (int a = 0; a < kLists; ++a) {
#pragma unroll
      for (int i = 0; i < kLen; ++i) w[a][i] = a * kLen + i < L ? v[a * kLen + i] : 0;
      sort_descending<kLen>(w[a]);
    }
    for (int j = 0; j < k; ++j) {
      uint64_t best = w[0][0];
#pragma unroll
      for (int a = 1; a < kLists; ++a) best = w[a][0] > best ? w[a][0] : best;
      const uint32_t key = static_cast<uint32_t>(best >> 32), low = static_cast<uint32_t>(best);
      const uint32_t m = lanes_max<S>(key);
      const uint32_t c = lanes_max<S>(key == m ? low : 0u);
      if (lane == j) {
        my_key = m;
        my_pos = static_cast<int>(~c);
      }
#pragma unroll
      for (int a = 0; a < kLists; ++a)
        if (w[a][0] == (static_cast<uint64_t>(m) << 32 | c)) {
#pragma unroll
          for (int i = 0; i + 1 < kLen; ++i) w[a][i] = w[a][i + 1];
          w[a][kLen - 1] = 0;
        }
    }
  }
}

// EPL experts to a lane while the groups are scored, L while the experts are chosen (without groups, or when all are
// kept, the lanes keep their own: L = EPL).
template <int S, int EPL, int L, bool GROUPS>
__global__ void __launch_bounds__(256) route_grouped_kernel(const RouteParams p) {
  static_assert(GROUPS || L == EPL, "without groups the lanes choose among their own experts");
  extern __shared__ uint2 deal[];  // [tokens of the block][live] (expert, key)
  constexpr int kTokens = 32 / S;  // of a warp
  pdl_trigger();
  pdl_wait();
  const int lane = threadIdx.x & (S - 1);  // among the token's lanes
  const int slot = threadIdx.x / S;        // the token's place in the block
  uint2* mine = deal + slot * p.live;
  const int lpg = 1 << p.lpg_log;
  const int g = lane >> p.lpg_log, sub = lane & (lpg - 1);
  const int base = g * p.gs + sub * p.epl;  // expert of slot i: base + i, for i < n
  const int n = g < p.n_group ? max(0, min(p.epl, p.gs - sub * p.epl)) : 0;
  float bias[EPL];
  if (p.bias) {
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
      const float b = i < n ? p.bias[base + i] : 0.f;
      bias[i] = b >= -INFINITY ? b : -INFINITY;  // a NaN takes the expert out as -inf does
    }
  }
  // this lane's logits of a token; -inf where there is none
  auto load = [&](int64_t t, float (&l)[EPL]) {
    const int64_t at = t * p.ld + base;
    const int have = t < p.T ? n : 0;
    if (p.dtype == W4A8_DTYPE_F32) {
      const float* row = static_cast<const float*>(p.logits) + at;
      if (EPL % 4 == 0 && p.vec) {
#pragma unroll
        for (int i = 0; i < EPL / 4; ++i) {
          const float4 a = 4 * i < have ? reinterpret_cast<const float4*>(row)[i]
                                        : make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
          l[4 * i] = a.x, l[4 * i + 1] = a.y, l[4 * i + 2] = a.z, l[4 * i + 3] = a.w;
        }
      } else {
#pragma unroll
        for (int i = 0; i < EPL; ++i) l[i] = i < have ? row[i] : -INFINITY;
      }
    } else {
      const uint16_t* row = static_cast<const uint16_t*>(p.logits) + at;
      const bool bf16 = p.dtype == W4A8_DTYPE_BF16;
      uint32_t h[EPL];
      if (EPL % 4 == 0 && p.vec) {
#pragma unroll
        for (int i = 0; i < EPL / 4; ++i) {
          const uint2 a = 4 * i < have ? reinterpret_cast<const uint2*>(row)[i] : make_uint2(0, 0);
          h[4 * i] = a.x & 0xFFFFu, h[4 * i + 1] = a.x >> 16, h[4 * i + 2] = a.y & 0xFFFFu, h[4 * i + 3] = a.y >> 16;
        }
      } else {
#pragma unroll
        for (int i = 0; i < EPL; ++i) h[i] = i < have ? row[i] : 0;
      }
#pragma unroll
      for (int i = 0; i < EPL; ++i) {
        const float f = bf16 ? __uint_as_float(h[i] << 16) : __half2float(__ushort_as_half(static_cast<uint16_t>(h[i])));
        l[i] = i < have ? f : -INFINITY;
      }
    }
  };
  const int64_t stride = static_cast<int64_t>(gridDim.x) * (blockDim.x / S);
  int64_t t = static_cast<int64_t>(blockIdx.x) * (blockDim.x / S) + slot;
  const int64_t first = t - slot % kTokens;  // the warp's first token: its lanes stay together
  float ahead[EPL];
  load(t, ahead);
  for (int64_t tw = first; tw < p.T; tw += stride, t += stride) {
    float l[EPL];
#pragma unroll
    for (int i = 0; i < EPL; ++i) l[i] = ahead[i] > p.lowest ? ahead[i] : -INFINITY;  // masked, or NaN
    if (tw + stride < p.T) load(t + stride, ahead);
    float mx = 0.f, total = 1.f;
    if (p.softmax) {
      mx = l[0];
#pragma unroll
      for (int i = 1; i < EPL; ++i) mx = fmaxf(mx, l[i]);
      mx = lanes_max<S>(mx);
      total = 0.f;
      if (mx < INFINITY) {
#pragma unroll
        for (int i = 0; i < EPL; ++i) total += __expf(l[i] - mx);
      } else {
#pragma unroll
        for (int i = 0; i < EPL; ++i) total += softmax_term(l[i], mx);
      }
      if (mx == -INFINITY) total = 0.f;  // nothing is left
      total = lanes_sum<S>(total);
    }
    uint32_t key[EPL];
    if (p.softmax && !p.bias) {
      // ranked by its logits: the same order as the scores', without ties made by rounding
#pragma unroll
      for (int i = 0; i < EPL; ++i) key[i] = order_key(l[i] + 0.0f);  // -0 and +0 are equal
    } else {
#pragma unroll
      for (int i = 0; i < EPL; ++i) {
        float c = p.softmax ? __fdiv_rn(softmax_term(l[i], mx), total) : sigmoid_score(l[i]);
        if (p.bias) c = __fadd_rn(c, bias[i]);  // never -0: scores are not negative
        key[i] = l[i] > -INFINITY ? order_key(c) : kKeyOut;
      }
    }
    uint64_t v[L];
    if constexpr (GROUPS) {
      uint32_t k1 = kKeyOut, k2 = kKeyOut;  // the group's two largest keys (places without an expert have kKeyOut)
      if (p.group_top == 1) {
#pragma unroll
        for (int i = 0; i < EPL; ++i) k1 = max(k1, key[i]);
        for (int o = 1; o < lpg; o <<= 1) k1 = max(k1, __shfl_xor_sync(0xffffffffu, k1, o));
      } else {
#pragma unroll
        for (int i = 0; i < EPL; ++i) {
          k2 = max(k2, min(k1, key[i]));
          k1 = max(k1, key[i]);
        }
        for (int o = 1; o < lpg; o <<= 1) {
          const uint32_t o1 = __shfl_xor_sync(0xffffffffu, k1, o), o2 = __shfl_xor_sync(0xffffffffu, k2, o);
          k2 = max(min(k1, o1), max(k2, o2));
          k1 = max(k1, o1);
        }
      }
      uint32_t gk = 0;  // on a group's first lane: its score
      if (sub == 0 && g < p.n_group) {
        float sc = key_value(k1);
        if (p.group_top == 2) {
          const float sc2 = key_value(k2);
          if (p.softmax && !p.bias)
            sc = pair_score(sc, sc2, mx);
          else
            sc = __fadd_rn(sc, sc2);
          if (!(sc >= -INFINITY)) sc = -INFINITY;  // inf + -inf
        }
        gk = order_key(sc + 0.0f);
      }
      uint32_t kept = 0;  // first lanes of the kept groups
      for (int j = 0; j < p.topk_group; ++j) {
        const uint32_t m = lanes_max<S>(gk);
        const uint32_t who = lanes_ballot<S>(gk == m);
        const uint32_t lead = who & (0u - who);  // the lowest group of an equal score
        kept |= lead;
        if ((1u << lane) == lead) gk = 0;
      }
      const uint32_t head = 1u << (g << p.lpg_log);
      __syncwarp();
      if (kept & head) {
        uint2* to = mine + __popc(kept & (head - 1)) * p.gs + sub * p.epl;
#pragma unroll
        for (int i = 0; i < EPL; ++i)
          if (i < n) to[i] = make_uint2(static_cast<uint32_t>(base + i), key[i]);
      }
      __syncwarp();
#pragma unroll
      for (int i = 0; i < L; ++i) {
        const int q = lane + S * i;
        v[i] = q < p.live ? static_cast<uint64_t>(mine[q].y) << 32 | ~static_cast<uint32_t>(q) : 0;
      }
    } else {
#pragma unroll
      for (int i = 0; i < L; ++i)
        v[i] = i < n ? static_cast<uint64_t>(key[i]) << 32 | ~static_cast<uint32_t>(base + i) : 0;
    }
    uint32_t my_key = 0;
    int my_e = 0;
    choose<S, L>(v, p.k, lane, my_key, my_e);
    const bool real = lane < p.k && my_key > kKeyOut;
    if (GROUPS && real) my_e = static_cast<int>(mine[my_e].x);
    float s = 0.f;
    if (real) {
      const float lj = load_any(p.logits, t * p.ld + my_e, p.dtype);
      s = p.softmax ? __fdividef(softmax_term(lj, mx), total) : sigmoid_score(lj);
    }
    if (__any_sync(0xffffffffu, lane < p.k && !real)) {
      // fewer than k experts were left: the lowest ids that were not chosen take the places, with weight 0 (they are
      // below 64: k <= 32)
      uint64_t taken = real && my_e < 64 ? 1ull << my_e : 0;
#pragma unroll
      for (int o = S / 2; o > 0; o >>= 1) taken |= __shfl_xor_sync(0xffffffffu, taken, o);
      const int found = __popc(lanes_ballot<S>(real));
      if (lane < p.k && !real) {
        uint64_t free = ~taken;
        for (int j = found; j < lane; ++j) free &= free - 1;
        my_e = __ffsll(static_cast<long long>(free)) - 1;
      }
    }
    if (p.renorm) s = __fdividef(s, lanes_sum<S>(s) + 1e-20f);
    if (lane < p.k && t < p.T) {
      const int64_t o = t * p.k + lane;
      p.ids[o] = my_e;
      p.w[o] = __fmul_rn(s, p.scale);
    }
  }
}

template <int S, int EPL, int L, bool GROUPS>
int launch_route(const RouteParams& p, cudaStream_t st) {
  // few tokens are spread over the SMs, many walk through four blocks of 8 warps an SM
  constexpr int kTokens = 32 / S;
  const int64_t groups = ceil_div(p.T, kTokens);
  const int warps = groups <= num_sms() ? 1 : groups <= 4 * num_sms() ? 4 : 8;
  const int64_t blocks = std::min<int64_t>(ceil_div(groups, warps), 4 * num_sms());
  const size_t smem = GROUPS ? sizeof(uint2) * warps * kTokens * p.live : 0;
  if (smem > 48 * 1024) {
    static DeviceOnce once;
    if (int rc = once.run([] {
          if (cudaFuncSetAttribute(route_grouped_kernel<S, EPL, L, GROUPS>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                   64 * 1024) != cudaSuccess)
            return check_launch("cudaFuncSetAttribute(route_grouped)");
          return static_cast<int>(W4A8_OK);
        }))
      return rc;
  }
  return launch_pdl("route_grouped_kernel", route_grouped_kernel<S, EPL, L, GROUPS>, dim3(static_cast<unsigned>(blocks)),
                    dim3(warps * 32), smem, st, p);
}

// L: the live experts over S lanes, rounded up to a power of two, 2 at least (at most 32 for 1024 experts)
template <int S, int EPL, int L = 2>
int launch_epl(const RouteParams& p, cudaStream_t st) {
  if (L == 2 && p.n_group == 1) return launch_route<S, EPL, EPL, false>(p, st);
  if constexpr (L < EPL && L < 32) {
    if (p.live > S * L) return launch_epl<S, EPL, 2 * L>(p, st);
  }
  return launch_route<S, EPL, L, true>(p, st);
}

template <int S>
int launch_lanes(const RouteParams& p, cudaStream_t st) {
  switch (p.epl) {
    case 1: return launch_epl<S, 1>(p, st);
    case 2: return launch_epl<S, 2>(p, st);
    case 3: return launch_epl<S, 3>(p, st);
    case 4: return launch_epl<S, 4>(p, st);
    case 5: return launch_epl<S, 5>(p, st);
    case 6: return launch_epl<S, 6>(p, st);
    default: break;
  }
  if (p.epl <= 8) return launch_epl<S, 8>(p, st);
  if constexpr (S == 16) return launch_epl<S, 10>(p, st);
  if constexpr (S == 32) {
    if (p.epl <= 12) return launch_epl<S, 12>(p, st);
    if (p.epl <= 16) return launch_epl<S, 16>(p, st);
    if (p.epl <= 32) return launch_epl<S, 32>(p, st);
    return launch_epl<S, 64>(p, st);
  }
  return launch_epl<S, 8>(p, st);
}

}  // namespace
}  // namespace w4a8
