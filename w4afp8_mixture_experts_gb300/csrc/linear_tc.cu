// dense_linear on the 5th-generation tensor cores: out = act(x W^T + bias) [* other half] + residual.
//
// Two kernels, both fed by TMA (128-byte swizzle, 64 k per stage) with fp32 accumulators in tensor memory:
//
//   pair kernel (many rows): a cluster of two CTAs computes a 256 x 256 tile with tcgen05.mma.cta_group::2 (x
//   rows on M, 128 per CTA; W rows on N, each CTA loads half of them).  Persistent, the accumulator double
//   buffered over the whole tensor memory, so that the epilogue of one tile runs under the products of the
//   next.  When gated, one CTA loads 128 gate rows and the other the 128 matching rows of the other half: both
//   CTAs then hold, for their 128 tokens, the two halves of 128 output columns side by side.  With few tiles, two or
//   four pairs of a cluster share a tile by pieces of K.
//     8192 x 4096 x 7168 gated: 240 us, 2.0 PFLOP/s, by itself, and 1.7 PFLOP/s under the power limit (products);
//     8192 x 7168 x 2048 with a residual: 133-145 us (products, then the residual's read and the output's write);
//     8192 x 256 x 7168, fp32 out, two pieces of K: 33 us (x at 4 TB/s, then 6 us of exchange and epilogue).
//
//   split kernel (few rows, or few tiles): a CTA computes a 128 x BN tile with W rows on M and tokens on N over
//   one piece of K; the CTAs of a cluster take the pieces of one tile, push their partial products into the
//   shared memory of the CTA that owns a token, and every owner adds its parts in rank order and finishes its
//   tokens.  One launch, no workspace, and a result that does not depend on timing.
//     64 x 4096 x 7168 gated: 14.3 us, W at 4.1 TB/s; 64 x 256 x 7168: 6.2 us (8 pieces of K; launch and latency).
//
// Every wait is bounded: on expiry the CTA raises its abort flag and the device error word, lets its copies and
// products in flight finish (again with a limit), frees its tensor memory and returns.
#include <algorithm>
#include <atomic>

#include "linear.cuh"

namespace w4a8 {
namespace {

constexpr uint64_t kTimeoutNs = 2000000000ull;  // 2 s: no legitimate wait comes close
constexpr int kBK = 64;                         // k per stage: one 128-byte swizzled row of 16-bit values
constexpr int kATile = 128 * kBK * 2;           // bytes of 128 rows of a stage
constexpr int kMaxSmem = 227 * 1024;

__device__ unsigned int g_linear_error;

// Waits for a phase of `bar`, at most limit_ns; gives up early when another role of the CTA has given up.  A thread that
// was away for longer than the limit looks at the phase once more before it gives up.
__device__ __forceinline__ bool wait_bar(uint64_t* bar, uint32_t parity, volatile int* abort_flag,
                                         uint64_t limit_ns = kTimeoutNs) {
  if (mbar_try_wait(bar, parity)) return true;
  const uint64_t t0 = globaltimer_ns();
  for (uint32_t n = 0;; ++n) {
    if (mbar_try_wait(bar, parity)) return true;
    if ((n & 127u) == 127u) {
      if (*abort_flag) return false;
      if (globaltimer_ns() - t0 > limit_ns) {
        if (mbar_try_wait(bar, parity)) return true;
        *abort_flag = 1;
        atomicOr(&g_linear_error, 1u);
        return false;
      }
    }
  }
}

// Waits for an operation in flight after an abort, whatever the abort flag; bit 2 of the error word on expiry.
__device__ __forceinline__ void drain_bar(uint64_t* bar, uint32_t parity) {
  if (mbar_try_wait(bar, parity)) return;
  const uint64_t t0 = globaltimer_ns();
  while (!mbar_try_wait(bar, parity)) {
    if (globaltimer_ns() - t0 > kTimeoutNs) {
      atomicOr(&g_linear_error, 4u);
      return;
    }
  }
}

// The same by a whole warp; the same answer on all its lanes.
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, volatile int* abort_flag) {
  return __all_sync(0xffffffffu, wait_bar(bar, parity, abort_flag));
}
// Whether the waits of all THREADS threads (whole warps) were satisfied: the same answer on all of them, once each has
// arrived.  Warps that share a step decide on it together: one that gave up by itself would leave the others at their next
// barrier for good.
template <int THREADS>
__device__ __forceinline__ bool all_satisfied(bool ok) {
  uint32_t bad;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.eq.u32 p, %1, 0;\n\t"
      "barrier.cta.red.or.aligned.pred q, 1, %2, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(bad)
      : "r"(static_cast<uint32_t>(ok)), "n"(THREADS)
      : "memory");
  return bad == 0;
}
// One lane of a converged warp.  The producer and product warps run their loops as whole warps and elect a lane
// around each TMA or tcgen05 instruction: with the loop inside a single-lane branch the operands of those
// instructions are not known to be uniform over the warp, and every product cost its issuer ~120 cycles.
__device__ __forceinline__ bool elect_one() {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xffffffff;\n\t"
      "selp.b32 %0, 1, 0, p;\n\t}"
      : "=r"(ok));
  return ok != 0;
}

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }
__device__ __forceinline__ uint32_t map_to_cta(uint32_t saddr, uint32_t cta) {
  uint32_t r;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(saddr), "r"(cta));
  return r;
}
// An arrival on a barrier of another CTA that hands over tensor memory only (ordered by the tcgen05 fences): with a
// release at cluster scope each arrival waited for the warp's outstanding global stores as well.
__device__ __forceinline__ void remote_arrive(uint32_t cluster_addr) {
  asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(cluster_addr) : "memory");
}

// shared-memory operand: K-major, 128-byte swizzle, 8-row groups 1024 B apart
__device__ __forceinline__ uint64_t operand_desc(uint32_t saddr) {
  return static_cast<uint64_t>((saddr >> 4) & 0x3FFFu) | (static_cast<uint64_t>(1u) << 16) |
         (static_cast<uint64_t>(1024u >> 4) << 32) | (static_cast<uint64_t>(1u) << 46) |
         (static_cast<uint64_t>(2u) << 61);
}
// fp32 accumulator, both operands f16 or both bf16, K-major
__host__ __device__ constexpr uint32_t idesc_f16(bool bf16, uint32_t m, uint32_t n) {
  return (1u << 4) | ((bf16 ? 1u : 0u) << 7) | ((bf16 ? 1u : 0u) << 10) | ((n >> 3) << 17) | ((m >> 4) << 24);
}

template <int CG>
__device__ __forceinline__ void mma_f16(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
  if constexpr (CG == 2)
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
        : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
        : "memory");
}
// arrives on `bar` of both CTAs of the pair when every product issued so far has completed
__device__ __forceinline__ void commit_pair(uint64_t* bar, uint16_t ctas) {
  asm volatile(
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
          smem_u32(bar)),
      "h"(ctas)
      : "memory");
}
// a box of a matrix into this CTA's shared memory, signalled on a barrier of either CTA of the pair
__device__ __forceinline__ void tma_load_pair(void* dst, const CUtensorMap* m, uint32_t bar, int32_t x, int32_t y) {
  asm volatile(
      "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4}], [%2];" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(m)), "r"(bar), "r"(x), "r"(y)
      : "memory");
}

// Asks L2 for a block of the residual, `rows` x `cols` at (m, n), with `count` threads of which this is number `i`:
// issued before the products, it takes the memory's latency out of the epilogue's loads.
__device__ __forceinline__ void prefetch_residual(const LinearParams& p, int m, int n, int rows, int cols, int i, int count) {
  const int size = p.out_dtype == W4A8_DTYPE_F32 ? 4 : 2;
  rows = min(rows, p.M - m);
  const int bytes = min(cols, p.n_out - n) * size;
  if (bytes <= 0) return;
  const int segs = (bytes + 127) / 128 + 1;  // a row may start anywhere in a 128-byte line
  for (; i < rows * segs; i += count) {
    const int row = i / segs, at = min(i % segs * 128, bytes - 1);
    asm volatile("prefetch.global.L2 [%0];" ::"l"(static_cast<const char*>(p.residual) +
                                                  ((m + row) * p.ldr + n) * size + at));
  }
}

template <int N>
__device__ __forceinline__ void activate_all(float (&v)[N], int act) {
  switch (act) {  // one branch for the N values
    case W4A8_ACT_RELU:
#pragma unroll
      for (int i = 0; i < N; ++i) v[i] = activate(v[i], W4A8_ACT_RELU);
      break;
    case W4A8_ACT_SILU:
#pragma unroll
      for (int i = 0; i < N; ++i) v[i] = activate(v[i], W4A8_ACT_SILU);
      break;
    case W4A8_ACT_GELU:
#pragma unroll
      for (int i = 0; i < N; ++i) v[i] = activate(v[i], W4A8_ACT_GELU);
      break;
    case W4A8_ACT_GELU_TANH:
#pragma unroll
      for (int i = 0; i < N; ++i) v[i] = activate(v[i], W4A8_ACT_GELU_TANH);
      break;
    default: break;
  }
}

// 32 bytes of one row, as two 16-byte accesses or one
__device__ __forceinline__ void load32b(const void* p, bool whole, uint32_t (&w)[8]) {
  if (whole) {
    asm volatile("ld.global.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]), "=r"(w[4]), "=r"(w[5]), "=r"(w[6]), "=r"(w[7])
                 : "l"(p)
                 : "memory");
  } else {
    const uint4 a = static_cast<const uint4*>(p)[0], b = static_cast<const uint4*>(p)[1];
    w[0] = a.x, w[1] = a.y, w[2] = a.z, w[3] = a.w, w[4] = b.x, w[5] = b.y, w[6] = b.z, w[7] = b.w;
  }
}
__device__ __forceinline__ void store32b(void* p, bool whole, const uint32_t (&w)[8]) {
  if (whole) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(w[0]), "r"(w[1]), "r"(w[2]),
                 "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                 : "memory");
  } else {
    static_cast<uint4*>(p)[0] = make_uint4(w[0], w[1], w[2], w[3]);
    static_cast<uint4*>(p)[1] = make_uint4(w[4], w[5], w[6], w[7]);
  }
}

// --- pair kernel ---------------------------------------------------------------------------------------------

constexpr int kPairStages = 6;
constexpr int kPairEpiWarps = 8;
constexpr int kPairThreads = 128 + kPairEpiWarps * 32;
constexpr int kPairStageBytes = 2 * kATile;  // of one CTA: 128 rows of x, 128 rows of W
constexpr int kStageRow = 17;                // fp32 row of a warp's 32 x 16 transposing block, padded
constexpr int kPairOffBias = kPairStages * kPairStageBytes;
constexpr int kPairOffStg = kPairOffBias + kPairEpiWarps * 128 * 4;
constexpr int kPairOffBar = kPairOffStg + kPairEpiWarps * 32 * kStageRow * 4;
constexpr int kPairSmem = kPairOffBar + (2 * kPairStages + 5) * 8 + 16 + 1024;
static_assert(kPairSmem <= kMaxSmem, "shared memory");
static_assert(kPairOffBar % 8 == 0, "barrier alignment");

struct PairPlan {
  int tiles_m, tiles_n, tiles, kblocks;
  int out_cols;  // output columns of a tile: 256, or 128 when gated
  int vec_out;   // out and residual rows take 16-byte accesses (1) or 32-byte ones (2)
};

// Tiles in an order that keeps the rows and columns in flight compact: bands of 8 row blocks, columns in turn.
__device__ __forceinline__ void pair_tile(const PairPlan& pl, int i, int& tm, int& tn) {
  constexpr int kBand = 8;
  const int per_band = kBand * pl.tiles_n;
  const int band = i / per_band, in = i - band * per_band;
  const int rows = min(kBand, pl.tiles_m - band * kBand);
  tn = in / rows;
  tm = band * kBand + in - tn * rows;
}

// N (16 or 32) output columns of this thread's row m0 + lane, from column n on; `res`: the residual's 32-byte
// pieces when `have` (a 16-bit residual read ahead).  Otherwise it is loaded here (LOADS: a 16-bit one too); an fp32 one ATONCE pieces before the
// first of them is used: one by one each costs a latency (7582 x 6592 x 128: 147 us, 113 with 4; 8192 x 7168 x 2048: 218 and 193;
// read ahead into registers like a 16-bit one it cost launches without a residual more than it gave, 44 -> 55 us).
template <int N, int ATONCE, bool LOADS>
__device__ __forceinline__ void store_row(const LinearParams& p, const PairPlan& pl, float (&v)[N], int m0, int n,
                                          bool have, const uint32_t (*res)[8], float* stg) {
  const int lane = threadIdx.x & 31;
  const bool whole = pl.vec_out == 2;
  if (pl.vec_out && n + N <= p.n_out) {
    const int m = m0 + lane;
    if (m >= p.M) return;
    uint32_t w[8];
    if (p.out_dtype == W4A8_DTYPE_F32) {
      float* o = static_cast<float*>(p.out) + m * p.ldo + n;
      const float* r = static_cast<const float*>(p.residual) + (p.residual ? m * p.ldr + n : 0);
#pragma unroll
      for (int i0 = 0; i0 < N / 8; i0 += ATONCE) {
        static_assert(N / 8 % ATONCE == 0);
        if (p.residual) {
          uint32_t f[ATONCE][8];
#pragma unroll
          for (int i = 0; i < ATONCE; ++i) load32b(r + 8 * (i0 + i), whole, f[i]);
#pragma unroll
          for (int i = 0; i < 8 * ATONCE; ++i) v[8 * i0 + i] += __uint_as_float(f[i / 8][i % 8]);
        }
#pragma unroll
        for (int i = i0; i < i0 + ATONCE; ++i) {
#pragma unroll
          for (int j = 0; j < 8; ++j) w[j] = __float_as_uint(v[8 * i + j]);
          store32b(o + 8 * i, whole, w);
        }
      }
      return;
    }
    uint16_t* o = static_cast<uint16_t*>(p.out) + m * p.ldo + n;
    const bool bf16 = p.out_dtype == W4A8_DTYPE_BF16;
#pragma unroll
    for (int i = 0; i < N / 16; ++i) {
      if (have || (LOADS && p.residual)) {
        uint32_t own[8];
        if (LOADS) load32b(static_cast<const uint16_t*>(p.residual) + m * p.ldr + n + 16 * i, whole, own);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const uint32_t q = LOADS ? own[j] : res[i][j];
          const float2 f = bf16 ? make_float2(__uint_as_float(q << 16), __uint_as_float(q & 0xFFFF0000u))
                                : __half22float2(*reinterpret_cast<const __half2*>(&q));
          v[16 * i + 2 * j] += f.x;
          v[16 * i + 2 * j + 1] += f.y;
        }
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        if (bf16) {
          w[j] = bf16x2_bits(v[16 * i + 2 * j], v[16 * i + 2 * j + 1]);
        } else {
          const __half2 h = __floats2half2_rn(v[16 * i + 2 * j], v[16 * i + 2 * j + 1]);
          w[j] = *reinterpret_cast<const uint32_t*>(&h);
        }
      }
      store32b(o + 16 * i, whole, w);
    }
    return;
  }
  // rows without alignment, or a tile's last columns: 16 columns at a time through shared memory, so that the
  // lanes of a warp touch neighbouring columns of two rows instead of 32 rows
#pragma unroll
  for (int h = 0; h < N / 16; ++h) {
    __syncwarp();
#pragma unroll
    for (int i = 0; i < 16; ++i) stg[lane * kStageRow + i] = v[16 * h + i];
    __syncwarp();
    const int c = n + 16 * h + (lane & 15);
    if (c >= p.n_out) continue;
    const int row = lane >> 4;  // rows row, row + 2, ...
    float a[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) a[i] = stg[(row + 2 * i) * kStageRow + (lane & 15)];
    // every load before the first use, and the type's branch around all of them
    if (p.out_dtype == W4A8_DTYPE_F32) {
      if (p.residual) {
        const float* r = static_cast<const float*>(p.residual) + c;
        float f[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) f[i] = m0 + row + 2 * i < p.M ? r[(m0 + row + 2 * i) * p.ldr] : 0.f;
#pragma unroll
        for (int i = 0; i < 16; ++i) a[i] += f[i];
      }
      float* o = static_cast<float*>(p.out) + c;
#pragma unroll
      for (int i = 0; i < 16; ++i)
        if (m0 + row + 2 * i < p.M) o[(m0 + row + 2 * i) * p.ldo] = a[i];
    } else {
      const bool bf16 = p.out_dtype == W4A8_DTYPE_BF16;
      if (p.residual) {
        const uint16_t* r = static_cast<const uint16_t*>(p.residual) + c;
        uint16_t f[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) f[i] = m0 + row + 2 * i < p.M ? r[(m0 + row + 2 * i) * p.ldr] : 0;
#pragma unroll
        for (int i = 0; i < 16; ++i) a[i] += bf16 ? bf16_bits_to_float(f[i]) : __half2float(__ushort_as_half(f[i]));
      }
      uint16_t* o = static_cast<uint16_t*>(p.out) + c;
#pragma unroll
      for (int i = 0; i < 16; ++i)
        if (m0 + row + 2 * i < p.M)
          o[(m0 + row + 2 * i) * p.ldo] = bf16 ? float_to_bf16_bits(a[i]) : __half_as_ushort(__float2half_rn(a[i]));
    }
  }
}

// The tensor core cuts off what does not fit the accumulator at every addition, so a sum of n products of 16 k is off by
// about n / 2 units of 2^-24 to one side (3.8e-6 of the result at K = 3584, where plain fp32 sums have 0.9e-6; 8.5e-4 with
// positive terms at K = 2^20).  A sum in one accumulator is therefore as long as its output's type hides that, and longer
// ones are added up in registers every kChunk stages, rounded to nearest:
//   fp32   kChunk stages, 1024 products (n / 2 = 32 units)
//   f16    256 stages, 16384 products: off by at most 2^-15, a sixteenth of the output's own rounding (2^-11)
//   bf16   2048 stages, 131072 products: 2^-12, a sixteenth of 2^-8
constexpr int kChunk = 16;
constexpr int longest_sum(int out_dtype) {  // in stages
  return out_dtype == W4A8_DTYPE_F32 ? kChunk : out_dtype == W4A8_DTYPE_F16 ? 256 : 2048;
}
constexpr int kPrefetchStages = 16;  // K up to which the pair kernel's epilogue prefetches the next residual
constexpr int kRegsLaunch = 168;  // of a thread at launch (checked on the host)
constexpr int kRegsRoles = 40, kRegsSums = 232;  // registers of warps 0-3 and of the epilogue's, which hold 128 sums
static_assert(128 * kRegsRoles + 32 * kPairEpiWarps * kRegsSums <= kPairThreads * kRegsLaunch, "within the launch's registers");

// PARTS = 1: persistent over tiles, the accumulator double buffered.  PARTS > 1: a cluster of PARTS pairs computes
// one tile, each pair a piece of K, and finishes 1 / PARTS of its columns: the other pairs push their partial
// products of those columns into its (by then idle) operand stages.  CHUNKED: sums in pieces of kChunk stages.
template <bool GATED, int PARTS, bool CHUNKED>
__global__ void __launch_bounds__(kPairThreads, 1)
    linear_pair_kernel(const __grid_constant__ CUtensorMap tx, const __grid_constant__ CUtensorMap tw,
                       const LinearParams p, const PairPlan pl) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + kPairOffBar);  // the pair's first CTA counts for both
  uint64_t* empty = full + kPairStages;
  uint64_t* tfull = empty + kPairStages;  // [2] accumulator ready, in both CTAs
  uint64_t* tempty = tfull + 2;           // [2] accumulator read by both CTAs (the first CTA's)
  uint64_t* mdrain = tempty + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(mdrain + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  const int crank = static_cast<int>(cluster_rank());
  const int rank = crank & 1, part = crank >> 1, lead = crank & ~1;
  pdl_trigger();
  if (warp == 0 && lane == 0) {
    tma_prefetch_desc(&tx);
    tma_prefetch_desc(&tw);
    for (int i = 0; i < kPairStages; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&tfull[i], 1);
      mbar_init(&tempty[i], 2 * kPairEpiWarps);
    }
    mbar_init(mdrain, 1);
    *abort_flag = 0;
    mbar_fence_init();
  }
  if (warp == 2) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_u32(tmem_slot)));
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;");
  }
  tc_fence_before();
  __syncthreads();
  cluster_arrive();
  cluster_wait();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  pdl_wait();
  const int first = blockIdx.x / (2 * PARTS), stride = PARTS > 1 ? pl.tiles : gridDim.x / 2;
  const int kb0 = static_cast<int>(static_cast<int64_t>(part) * pl.kblocks / PARTS);
  const int kb1 = static_cast<int>(static_cast<int64_t>(part + 1) * pl.kblocks / PARTS);
  // no CTA of the cluster leaves while another may still signal it or read its operands
  auto leave = [&] {
    __syncwarp();
    tc_fence_before();
    cluster_arrive();
    cluster_wait();
  };
  // Warps 0-3 end inside this branch: with CHUNKED they hold fewer registers than the code behind it is built for.
  if (warp < 4) {
    if constexpr (CHUNKED) regs_release<kRegsRoles>();
    if (warp == 0) {  // TMA producer of this CTA's half of every stage
      uint32_t it = 0;
      bool ok = true;
      for (int i = first; ok && i < pl.tiles; i += stride) {
        int tm, tn;
        pair_tile(pl, i, tm, tn);
        const int m = tm * 256 + rank * 128;
        const int n = GATED ? rank * p.n_out + tn * 128 : tn * 256 + rank * 128;
        for (int kb = kb0; kb < kb1; ++kb, ++it) {
          const int s = it % kPairStages;
          if (!(ok = warp_wait(&empty[s], ((it / kPairStages) & 1) ^ 1, abort_flag))) break;
          if (elect_one()) {
            uint8_t* at = smem + s * kPairStageBytes;
            const uint32_t bar = map_to_cta(smem_u32(&full[s]), lead);
            if (rank == 0) mbar_arrive_expect_tx(&full[s], 2 * kPairStageBytes);
            tma_load_pair(at, &tx, bar, kb * kBK, m);
            tma_load_pair(at + kATile, &tw, bar, kb * kBK, n);
          }
          __syncwarp();
        }
      }
      // the last stages' slots are released before the CTA may go (and, after an abort, their loads have landed)
      const uint32_t n = it < kPairStages ? it : kPairStages;
      for (uint32_t j = it - n; j < it; ++j) {
        const uint32_t s = j % kPairStages, ph = (j / kPairStages) & 1;
        if (!(ok && (ok = warp_wait(&empty[s], ph, abort_flag))) && rank == 0) drain_bar(&full[s], ph);
      }
    } else if (warp == 1 && rank == 0) {  // the pair's products
      const uint32_t idesc = idesc_f16(p.dtype == W4A8_DTYPE_BF16, 256, 256);
      const uint16_t both = static_cast<uint16_t>(3 << lead);
      uint32_t it = 0;
      int n = 0;  // accumulator fills so far
      bool ok = true;
      for (int i = first; ok && i < pl.tiles; i += stride) {
        for (int kb = kb0; kb < kb1; ++kb, ++it) {
          const int s = it % kPairStages, at_chunk = CHUNKED ? (kb - kb0) % kChunk : kb - kb0;
          const int buf = n & 1;
          if (at_chunk == 0) {
            if (!(ok = warp_wait(&tempty[buf], ((n >> 1) & 1) ^ 1, abort_flag))) break;
            tc_fence_after();
          }
          if (!(ok = warp_wait(&full[s], (it / kPairStages) & 1, abort_flag))) break;
          tc_fence_after();
          const uint32_t at = smem_u32(smem + s * kPairStageBytes);
          const uint64_t a = operand_desc(at), b = operand_desc(at + kATile);
          const bool last = kb + 1 == kb1 || (CHUNKED && at_chunk == kChunk - 1);
          if (elect_one()) {
#pragma unroll
            for (int k = 0; k < kBK / 16; ++k)
              mma_f16<2>(tmem + buf * 256, a + 2 * k, b + 2 * k, idesc, at_chunk > 0 || k > 0);
            commit_pair(&empty[s], both);
            if (last) commit_pair(&tfull[buf], both);
          }
          __syncwarp();
          n += last;
        }
      }
      if (!ok) {
        if (elect_one())
          asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_u32(mdrain))
                       : "memory");
        __syncwarp();
        drain_bar(mdrain, 0);
      }
    }

    if (PARTS > 1 && (warp == 2 || warp == 3) && p.residual && !pl.vec_out) {  // aligned rows are read ahead below
      int tm, tn;
      pair_tile(pl, first, tm, tn);
      prefetch_residual(p, tm * 256 + rank * 128, tn * pl.out_cols + part * (pl.out_cols / PARTS), 128,
                        pl.out_cols / PARTS, threadIdx.x - 64, 64);
    }
    if constexpr (PARTS > 1) {  // the exchange's two barriers
      __syncwarp();
      for (int i = 0; i < 2; ++i) {
        cluster_arrive();
        cluster_wait();
      }
    }
    leave();
    if (warp == 2) {
      tc_fence_after();
      asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, 512;" ::"r"(tmem));
    }
    return;
  }
  if constexpr (CHUNKED) regs_claim<kRegsSums>();

  // epilogue: warp e reads lane quarter e % 4 (its tokens) and, by e / 4, one half of the columns that this CTA
  // finishes; a turn is kN columns
  constexpr int kCols = (GATED ? 64 : 128) / PARTS;  // output columns of a warp
  constexpr int kN = kCols < 32 ? kCols : 32;
  constexpr int kHalf = GATED ? 128 : 0;             // where the other half's products lie
  const int e = warp - 4, quarter = warp & 3, half = e >> 2;
  float* bias = reinterpret_cast<float*>(smem + kPairOffBias) + e * 128;
  float* stg = reinterpret_cast<float*>(smem + kPairOffStg) + e * 32 * kStageRow;
  const uint32_t lanes = static_cast<uint32_t>(quarter * 32) << 16;
  const int bd = p.bias_f32 ? W4A8_DTYPE_F32 : p.dtype;
  const int nh = part * 2 * kCols + half * kCols;  // first column of this warp within the tile

  auto load_bias = [&](int n0) {
    __syncwarp();
    for (int c = lane; c < (GATED ? 2 : 1) * kCols; c += 32) {
      const int other = GATED && c >= kCols;
      const int col = n0 + c - other * kCols;
      bias[c] = col < p.n_out ? load_any(p.bias, col + other * p.n_out, bd) : 0.f;
    }
    __syncwarp();
  };
  // bias, activation and gating of columns c ... of this warp
  auto apply = [&](float (&v)[kN], float (&u)[kN], int c) {
    if (p.bias) {
#pragma unroll
      for (int j = 0; j < kN; ++j) v[j] += bias[c + j];
    }
    activate_all<kN>(v, p.act);
    if (GATED) {
#pragma unroll
      for (int j = 0; j < kN; ++j) v[j] *= p.bias ? u[j] + bias[kCols + c + j] : u[j];
    }
  };
  constexpr int kPieces = kCols / 16;  // 32-byte pieces of a 16-bit residual
  auto read_ahead = [&](int m, int n0, uint32_t (&res)[kPieces][8]) {
    const uint16_t* r = static_cast<const uint16_t*>(p.residual) + m * p.ldr + n0;
#pragma unroll
    for (int i = 0; i < kPieces; ++i)
      if (m < p.M && n0 + 16 * i + 16 <= p.n_out) load32b(r + 16 * i, pl.vec_out == 2, res[i]);
  };
  const bool ahead = !CHUNKED && p.residual && pl.vec_out && p.out_dtype != W4A8_DTYPE_F32;  // CHUNKED: registers hold the sums
  const uint32_t tempty0 = map_to_cta(smem_u32(tempty), lead);
  int n = 0;  // accumulator fills so far
  // Waits for the products of a tile and returns the accumulator that holds them (-1 after an abort).  CHUNKED: every
  // thread adds up 128 columns of its row over the chunks and puts the sums back into the last chunk's accumulator, where
  // the epilogue warps read one another's columns: each of them arrives at their barrier once per tile, at its last chunk or
  // when it gives up, and all go on or none.
  auto products = [&]() -> int {
    if constexpr (CHUNKED) {
      const int chunks = (kb1 - kb0 + kChunk - 1) / kChunk;
      float sum[4][32];
      bool ok = true;
      for (int ch = 0; ch < chunks; ++ch, ++n) {
        const int buf = n & 1;
        if (!(ok = warp_wait(&tfull[buf], (n >> 1) & 1, abort_flag))) break;
        tc_fence_after();
        if (chunks == 1) break;
        const uint32_t at = tmem + buf * 256 + lanes + half * 128;
#pragma unroll
        for (int q = 0; q < 8; ++q) {
          float v[16];
          tmem_ld16(at + 16 * q, reinterpret_cast<uint32_t*>(v));
          tmem_wait_ld_pin<16>(reinterpret_cast<uint32_t*>(v));
#pragma unroll
          for (int j = 0; j < 16; ++j) sum[q / 2][q % 2 * 16 + j] = ch > 0 ? sum[q / 2][q % 2 * 16 + j] + v[j] : v[j];
        }
        if (ch + 1 < chunks) {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) remote_arrive(tempty0 + buf * 8);
          continue;
        }
#pragma unroll
        for (int q = 0; q < 4; ++q) tmem_st32(at + 32 * q, reinterpret_cast<const uint32_t*>(sum[q]));
        tmem_wait_st();
        tc_fence_before();
        break;
      }
      if (chunks > 1) {
        ok = all_satisfied<32 * kPairEpiWarps>(ok);
        tc_fence_after();
      }
      return ok ? n++ & 1 : -1;
    } else {
      const int buf = n & 1;
      if (!warp_wait(&tfull[buf], (n >> 1) & 1, abort_flag)) return -1;
      tc_fence_after();
      ++n;
      return buf;
    }
  };

  if constexpr (PARTS == 1) {
    for (int i = first; i < pl.tiles; i += stride) {
      int tm, tn;
      pair_tile(pl, i, tm, tn);
      const int n0 = tn * pl.out_cols + nh;
      const int m0 = tm * 256 + rank * 128 + quarter * 32;
      uint32_t res[kPieces][8];
      if (ahead) read_ahead(m0 + lane, n0, res);
      if (p.bias) load_bias(n0);
      const int buf = products();
      if (buf < 0) break;
      // With a short K the epilogue is the longer part, and the residual's latency shows: the next tile's goes to L2
      // now (8192 x 7168 x 512: 73.8 -> 68.6 us, K = 1024: 84.6 -> 82.1; K = 1536: 104.3 -> 106.9, so not there).
      if (p.residual && pl.kblocks <= kPrefetchStages && i + stride < pl.tiles) {
        int um, un;
        pair_tile(pl, i + stride, um, un);
        prefetch_residual(p, um * 256 + rank * 128 + quarter * 32, un * pl.out_cols + nh, 32, kCols, lane, 32);
      }
      const uint32_t at = tmem + buf * 256 + lanes + nh;
#pragma unroll 1
      for (int c = 0; c < kCols; c += 32) {
        float v[32], u[32];
        __syncwarp();
        tmem_ld32(at + c, reinterpret_cast<uint32_t*>(v));
        if (GATED) tmem_ld32(at + kHalf + c, reinterpret_cast<uint32_t*>(u));
        tmem_wait_ld_pin<32>(reinterpret_cast<uint32_t*>(v));
        if (GATED) tmem_wait_ld_pin<32>(reinterpret_cast<uint32_t*>(u));
        if (c + 32 == kCols) {  // every value is in registers: the accumulator is free
          tc_fence_before();
          __syncwarp();
          if (lane == 0) remote_arrive(tempty0 + buf * 8);
        }
        if (n0 + c >= p.n_out) continue;
        apply(v, u, c);
        store_row<32, 4, CHUNKED>(p, pl, v, m0, n0 + c, ahead, res, stg);
#pragma unroll
        for (int j = 0; j + 2 < kPieces; ++j)
#pragma unroll
          for (int q = 0; q < 8; ++q) res[j][q] = res[j + 2][q];
      }
    }
  } else {
    constexpr int kPart = 2 * kCols * (GATED ? 2 : 1);  // columns of products that a CTA finishes: 256 / PARTS
    // [PARTS - 1][kPart / 4][128 tokens][4]: a thread pushes and takes 4 columns of its token at a time
    float4* recv = reinterpret_cast<float4*>(smem);
    static_assert((PARTS - 1) * kPart * 128 * 4 <= kPairStages * kPairStageBytes, "partial products in the stages");
    int tm, tn;
    pair_tile(pl, first, tm, tn);
    const int n0 = tn * pl.out_cols + nh;
    const int m0 = tm * 256 + rank * 128 + quarter * 32;
    uint32_t res[kPieces][8];
    if (ahead) read_ahead(m0 + lane, n0, res);
    if (p.bias) load_bias(n0);
    const int buf = products();
    const bool ok = buf >= 0;
    const uint32_t acc = tmem + lanes + max(buf, 0) * 256;
    __syncwarp();
    tc_fence_before();
    cluster_arrive();  // every pair's products are done: no operand stage is in use any more
    cluster_wait();
    tc_fence_after();
    if (ok) {
      const uint32_t to0 = smem_u32(recv) + (quarter * 32 + lane) * 16;
#pragma unroll 1
      for (int q = 0; q < PARTS; ++q) {
        if (q == part) continue;
        const uint32_t to = map_to_cta(to0 + (part < q ? part : part - 1) * kPart * 512, 2 * q + rank);
#pragma unroll 1
        for (int c = 0; c < kCols; c += kN) {
#pragma unroll
          for (int h = 0; h < (GATED ? 2 : 1); ++h) {
            float v[kN];
            __syncwarp();
            const uint32_t at = acc + h * kHalf + q * 2 * kCols + half * kCols + c;
            if constexpr (kN == 32)
              tmem_ld32(at, reinterpret_cast<uint32_t*>(v));
            else
              tmem_ld16(at, reinterpret_cast<uint32_t*>(v));
            tmem_wait_ld_pin<kN>(reinterpret_cast<uint32_t*>(v));
#pragma unroll
            for (int j = 0; j < kN; j += 4)
              asm volatile("st.shared::cluster.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(
                               to + (h * 2 * kCols + half * kCols + c + j) * 512),
                           "f"(v[j]), "f"(v[j + 1]), "f"(v[j + 2]), "f"(v[j + 3])
                           : "memory");
          }
        }
      }
    }
    cluster_arrive();
    cluster_wait();
    if (ok && n0 < p.n_out) {
      const float4* mine = recv + quarter * 32 + lane;
#pragma unroll 1
      for (int c = 0; c < kCols; c += kN) {
        float v[kN], u[kN];
        __syncwarp();
        const uint32_t at = acc + nh + c;
        if constexpr (kN == 32) {
          tmem_ld32(at, reinterpret_cast<uint32_t*>(v));
          if (GATED) tmem_ld32(at + kHalf, reinterpret_cast<uint32_t*>(u));
        } else {
          tmem_ld16(at, reinterpret_cast<uint32_t*>(v));
          if (GATED) tmem_ld16(at + kHalf, reinterpret_cast<uint32_t*>(u));
        }
        tmem_wait_ld_pin<kN>(reinterpret_cast<uint32_t*>(v));
        if (GATED) tmem_wait_ld_pin<kN>(reinterpret_cast<uint32_t*>(u));
#pragma unroll
        for (int q = 0; q < PARTS - 1; ++q)
#pragma unroll
          for (int j = 0; j < kN; j += 4) {
            const float4 a = mine[(q * kPart + half * kCols + c + j) / 4 * 128];
            v[j] += a.x, v[j + 1] += a.y, v[j + 2] += a.z, v[j + 3] += a.w;
            if (GATED) {
              const float4 b = mine[(q * kPart + 2 * kCols + half * kCols + c + j) / 4 * 128];
              u[j] += b.x, u[j + 1] += b.y, u[j + 2] += b.z, u[j + 3] += b.w;
            }
          }
        if (n0 + c >= p.n_out) continue;
        apply(v, u, c);
        store_row<kN, 1, CHUNKED>(p, pl, v, m0, n0 + c, ahead, res, stg);
#pragma unroll
        for (int j = 0; j + kN / 16 < kPieces; ++j)
#pragma unroll
          for (int q = 0; q < 8; ++q) res[j][q] = res[j + kN / 16][q];
      }
    }
  }
  leave();
}

// --- split kernel --------------------------------------------------------------------------------------------

constexpr int kSplitMma = 2;
// accumulators that share the sums over a CTA's piece of K
__host__ __device__ constexpr int split_accumulators(int out_dtype) {
  return (out_dtype == W4A8_DTYPE_F32 ? 2 : 1) * kSplitMma;
}

template <int BN>
struct SplitCfg {
  // 16 warps share the epilogue's latencies (128 x 7168 x 2048: 13.0 us with 8 warps, 11.5 with 16), but for 32 tokens it
  // is short, and the larger launch costs more (64 x 256 x 7168: 6.25 and 6.7 us)
  static constexpr int kThreads = BN == 32 ? 256 : 512;
  static constexpr int kStageBytes = kATile + BN * kBK * 2;
  static constexpr int kStages = BN == 128 ? 4 : BN == 64 ? 6 : 8;
  static constexpr int kOffRed = kStages * kStageBytes;       // [source CTA][token of mine][128 W rows] fp32
  static constexpr int kOffBar = kOffRed + BN * 128 * 4;
  static constexpr int kSmem = kOffBar + (2 * kStages + 5) * 8 + 16 + 1024;
  // MMA warps (kSplitMma): warp m issues the products of stages it % kMma == m into an accumulator of its own.  One warp spends
  // ~330 cycles a stage on the hand-over (wait, fence, commit), several times what the products take; together they
  // overlap it, and the sums over K are shorter.
  static constexpr int kMma = kSplitMma;
  // A warp waits for every phase of the slots that it uses, in order, only if a slot always falls to the same warp:
  // otherwise its parity wait is satisfied by the phase before the one it needs.
  static_assert(kStages % kMma == 0, "ring depth a multiple of the MMA warps");
  static constexpr int kTurns = BN * 16 / kThreads;  // tokens of a thread in the epilogue, at most
  static constexpr uint32_t kTmemCols = 2 * kMma * BN;  // an fp32 output spreads its sums over two accumulators a warp
  static_assert(kSmem <= kMaxSmem, "shared memory");
};

// The epilogue's threads: with aligned rows a thread finishes 8 neighbouring columns of every kStep-th token, without
// alignment one column of them (so that a warp touches neighbours).
template <int BN, bool GATED>
struct SplitMap {
  static constexpr int kOutCols = GATED ? 64 : 128;
  static constexpr int kOct = kOutCols / 8;
  static constexpr int kOctStep = SplitCfg<BN>::kThreads / kOct, kColStep = SplitCfg<BN>::kThreads / kOutCols;
};

// The biases of this thread's columns and the aligned 16-bit residual of all its tokens.
template <int BN, bool GATED>
__device__ __forceinline__ void read_ahead_split(const LinearParams& p, int m, int n0, int own, int vec_out,
                                                 float (&bias)[8], float (&bias2)[8], uint4 (&res)[SplitCfg<BN>::kTurns]) {
  using Map = SplitMap<BN, GATED>;
  const int n = n0 + (vec_out ? threadIdx.x % Map::kOct * 8 : threadIdx.x % Map::kOutCols);
  const int bd = p.bias_f32 ? W4A8_DTYPE_F32 : p.dtype;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const bool in = p.bias && n + j < p.n_out && (vec_out || j == 0);
    bias[j] = in ? load_any(p.bias, n + j, bd) : 0.f;
    bias2[j] = in && GATED ? load_any(p.bias, p.n_out + n + j, bd) : 0.f;
  }
  if (!p.residual || !vec_out || p.out_dtype == W4A8_DTYPE_F32 || n + 8 > p.n_out) return;
  const int left = min(own, p.M - m);
  const uint16_t* r = static_cast<const uint16_t*>(p.residual) + n;
#pragma unroll
  for (int i = 0; i < SplitCfg<BN>::kTurns; ++i) {
    const int tok = threadIdx.x / Map::kOct + i * Map::kOctStep;
    if (tok < left) res[i] = *reinterpret_cast<const uint4*>(r + (m + tok) * p.ldr);
  }
}

// Adds a CTA's partial products for its tokens in rank order and writes them: red [split][own][128 W rows].
template <int BN, bool GATED, typename T>
__device__ __forceinline__ void finish_tokens(const LinearParams& p, const float* red, int splits, int own, int left, int m,
                                              int n0, int vec_out, const float (&bias)[8], const float (&bias2)[8],
                                              const uint4 (&res)[SplitCfg<BN>::kTurns]) {
  using Map = SplitMap<BN, GATED>;
  const T* residual = static_cast<const T*>(p.residual);
  T* out = static_cast<T*>(p.out);
  if (!vec_out) {
    constexpr int kN = 16;  // tokens at a time: every load before the first use
    const int f = threadIdx.x % Map::kOutCols, n = n0 + f;
    if (n >= p.n_out) return;
#pragma unroll 1
    for (int tok0 = threadIdx.x / Map::kOutCols; tok0 < left; tok0 += kN * Map::kColStep) {
      const int64_t row = m + tok0;
      const int count = (left - tok0 + Map::kColStep - 1) / Map::kColStep;  // tokens of this turn, if fewer than kN
      float v[kN], u[kN];
      T r[kN];
      if (p.residual) {
        const T* rp = residual + row * p.ldr + n;
#pragma unroll
        for (int j = 0; j < kN; ++j)
          if (j < count) r[j] = rp[j * Map::kColStep * p.ldr];
      }
#pragma unroll
      for (int j = 0; j < kN; ++j) {
        v[j] = bias[0];
        u[j] = bias2[0];
      }
#pragma unroll 1
      for (int s = 0; s < splits; ++s) {
        const float* src = red + (s * own + tok0) * 128 + f;
#pragma unroll
        for (int j = 0; j < kN; ++j)
          if (j < count) {
            v[j] += src[j * Map::kColStep * 128];
            if (GATED) u[j] += src[j * Map::kColStep * 128 + 64];
          }
      }
      activate_all<kN>(v, p.act);
      T* o = out + row * p.ldo + n;
#pragma unroll
      for (int j = 0; j < kN; ++j)
        if (j < count) {
          if (GATED) v[j] *= u[j];
          if (p.residual) v[j] += to_f32(r[j]);
          o[j * Map::kColStep * p.ldo] = from_f32<T>(v[j]);
        }
    }
    return;
  }
  const int col = threadIdx.x % Map::kOct * 8, n = n0 + col;
  if (n >= p.n_out) return;
  const bool whole = n + 8 <= p.n_out;
#pragma unroll
  for (int i = 0; i < SplitCfg<BN>::kTurns; ++i) {
    const int tok = threadIdx.x / Map::kOct + i * Map::kOctStep;
    if (tok >= left) break;
    float v[8], u[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      v[j] = bias[j];
      u[j] = bias2[j];
    }
#pragma unroll 1
    for (int s = 0; s < splits; ++s) {
      const float4* src = reinterpret_cast<const float4*>(red + (s * own + tok) * 128 + col);
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const float4 a = src[j];
        v[4 * j] += a.x, v[4 * j + 1] += a.y, v[4 * j + 2] += a.z, v[4 * j + 3] += a.w;
        if (GATED) {
          const float4 b = src[16 + j];
          u[4 * j] += b.x, u[4 * j + 1] += b.y, u[4 * j + 2] += b.z, u[4 * j + 3] += b.w;
        }
      }
    }
    activate_all<8>(v, p.act);
    if (GATED) {
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] *= u[j];
    }
    const T* r = residual + (p.residual ? (m + tok) * p.ldr + n : 0);
    T* o = out + (m + tok) * p.ldo + n;
    if (!whole) {
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (n + j < p.n_out) o[j] = from_f32<T>(p.residual ? v[j] + to_f32(r[j]) : v[j]);
    } else if constexpr (sizeof(T) == 4) {
      if (p.residual) {
        const float4 a = reinterpret_cast<const float4*>(r)[0], b = reinterpret_cast<const float4*>(r)[1];
        v[0] += a.x, v[1] += a.y, v[2] += a.z, v[3] += a.w, v[4] += b.x, v[5] += b.y, v[6] += b.z, v[7] += b.w;
      }
      reinterpret_cast<float4*>(o)[0] = make_float4(v[0], v[1], v[2], v[3]);
      reinterpret_cast<float4*>(o)[1] = make_float4(v[4], v[5], v[6], v[7]);
    } else {
      if (p.residual) {
        const T* h = reinterpret_cast<const T*>(&res[i]);
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] += to_f32(h[j]);
      }
      *reinterpret_cast<uint4*>(o) = make_uint4(pack2<T>(v[0], v[1]), pack2<T>(v[2], v[3]), pack2<T>(v[4], v[5]),
                                                pack2<T>(v[6], v[7]));
    }
  }
}

template <int BN, bool GATED>
__global__ void __launch_bounds__(SplitCfg<BN>::kThreads, 1)
    linear_split_kernel(const __grid_constant__ CUtensorMap tx, const __grid_constant__ CUtensorMap tw,
                        const LinearParams p, int splits, int kblocks, int vec_out) {
  using C = SplitCfg<BN>;
  constexpr int kOutCols = GATED ? 64 : 128;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::kOffBar);
  uint64_t* empty = full + C::kStages;
  uint64_t* done = empty + C::kStages;
  uint64_t* mdrain = done + 1;  // [4]
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(mdrain + 4);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  const int rank = splits > 1 ? static_cast<int>(cluster_rank()) : 0;
  const int n0 = (blockIdx.x / splits) * kOutCols, m0 = blockIdx.y * BN;
  pdl_trigger();
  if (warp == 0 && lane == 0) {
    tma_prefetch_desc(&tx);
    tma_prefetch_desc(&tw);
    for (int i = 0; i < C::kStages; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], 1);
    }
    mbar_init(done, C::kMma);
    for (int i = 0; i < C::kMma; ++i) mbar_init(&mdrain[i], 1);
    *abort_flag = 0;
    mbar_fence_init();
  }
  if (warp == 2) {
    tmem_alloc(tmem_slot, C::kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (splits > 1) cluster_arrive();  // matched before the first remote store
  const uint32_t tmem = *tmem_slot;
  pdl_wait();

  const int kb0 = static_cast<int>(static_cast<int64_t>(rank) * kblocks / splits);
  const int kb1 = static_cast<int>(static_cast<int64_t>(rank + 1) * kblocks / splits);
  const int own_log = 31 - __clz(BN / splits), own = 1 << own_log;  // tokens that a CTA finishes
  // what the epilogue needs besides the products is read ahead of them
  float bias[8], bias2[8];
  uint4 res[SplitCfg<BN>::kTurns];
  read_ahead_split<BN, GATED>(p, m0 + rank * own, n0, own, vec_out, bias, bias2, res);
  const int accs = split_accumulators(p.out_dtype);
  int issued = 0;  // stages whose loads this warp has issued
  if (warp == 0) {
    for (int kb = kb0; kb < kb1; ++kb, ++issued) {
      const int s = issued % C::kStages;
      if (!warp_wait(&empty[s], ((issued / C::kStages) & 1) ^ 1, abort_flag)) break;
      if (elect_one()) {
        uint8_t* at = smem + s * C::kStageBytes;
        mbar_arrive_expect_tx(&full[s], C::kStageBytes);
        tma_load_2d(at, &tw, &full[s], kb * kBK, n0);
        if (GATED) tma_load_2d(at + kATile / 2, &tw, &full[s], kb * kBK, p.n_out + n0);
        tma_load_2d(at + kATile, &tx, &full[s], kb * kBK, m0);
      }
      __syncwarp();
    }
  } else if (warp == 2 || warp == 3) {
    if (p.residual && (!vec_out || p.out_dtype == W4A8_DTYPE_F32)) prefetch_residual(p, m0 + rank * own, n0, own, kOutCols, threadIdx.x - 64, 64);
  } else if (warp >= 4 && warp < 4 + C::kMma) {
    const uint32_t idesc = idesc_f16(p.dtype == W4A8_DTYPE_BF16, 128, BN);
    const int m = warp - 4, stages = kb1 - kb0;
    const int second = accs > C::kMma ? C::kMma * BN : 0;  // the second accumulator, every other time
    bool ok = true;
    for (int it = m; it < stages; it += C::kMma) {
      const int s = it % C::kStages;
      if (!(ok = warp_wait(&full[s], (it / C::kStages) & 1, abort_flag))) break;
      tc_fence_after();
      const uint32_t at = smem_u32(smem + s * C::kStageBytes);
      const uint64_t a = operand_desc(at), b = operand_desc(at + kATile);
      if (elect_one()) {
#pragma unroll
        for (int k = 0; k < kBK / 16; ++k)
          mma_f16<1>(tmem + m * BN + (it / C::kMma % 2) * second, a + 2 * k, b + 2 * k, idesc, it >= accs || k > 0);
        mma_commit(&empty[s]);
      }
      __syncwarp();
    }
    if (elect_one()) mma_commit(ok ? done : &mdrain[m]);
    __syncwarp();
    if (!ok) drain_bar(&mdrain[m], 0);
  }
  __syncwarp();
  const bool ok = !__any_sync(0xffffffffu, !wait_bar(done, 0, abort_flag));
  if (!ok)
    for (int j = issued < C::kStages ? 0 : issued - C::kStages; j < issued; ++j)
      drain_bar(&full[j % C::kStages], (j / C::kStages) & 1);
  __syncwarp();
  tc_fence_after();
  if (splits > 1) cluster_wait();
  // this CTA's partial products to the owners of their tokens: warp w reads lane quarter w % 4 (W rows) and the tokens
  // of its turn w / 4
  const int quarter = warp & 3, f = quarter * 32 + lane;
  if (ok) {
    constexpr int kCols = BN / (C::kThreads / 128);  // of a warp; its lane quarter is a fourth of the W rows
    constexpr int kStep = kCols < 32 ? kCols : 32;
    const uint32_t red = smem_u32(smem + C::kOffRed);
#pragma unroll 1
    for (int c = (warp >> 2) * kCols; c < (warp >> 2) * kCols + kCols; c += kStep) {
      float v[kStep];
#pragma unroll
      for (int m = 0; m < 2 * C::kMma; ++m) {
        if (m >= accs || (m > 0 && m >= kb1 - kb0)) break;  // fewer stages than accumulators: no products in that one
        float w[kStep];
        const uint32_t at = tmem + (static_cast<uint32_t>(quarter * 32) << 16) + m * BN + c;
        if constexpr (kStep == 32)
          tmem_ld32(at, reinterpret_cast<uint32_t*>(w));
        else if constexpr (kStep == 16)
          tmem_ld16(at, reinterpret_cast<uint32_t*>(w));
        else
          tmem_ld8(at, reinterpret_cast<uint32_t(&)[8]>(w));
        tmem_wait_ld_pin<kStep>(reinterpret_cast<uint32_t*>(w));
#pragma unroll
        for (int j = 0; j < kStep; ++j) v[j] = m > 0 ? v[j] + w[j] : w[j];
      }
#pragma unroll
      for (int j = 0; j < kStep; ++j) {
        const int q = (c + j) >> own_log, tok = (c + j) & (own - 1);
        const uint32_t to = red + ((rank * own + tok) * 128 + f) * 4;
        if (splits > 1)
          asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(map_to_cta(to, q)), "f"(v[j]) : "memory");
        else
          asm volatile("st.shared.f32 [%0], %1;" ::"r"(to), "f"(v[j]) : "memory");
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (splits > 1) {
    cluster_arrive();
    cluster_wait();
  }
  if (warp == 2) {
    tc_fence_after();
    tmem_dealloc(tmem, C::kTmemCols);
  }
  if (!ok) return;
  const float* red = reinterpret_cast<const float*>(smem + C::kOffRed);
  const int left = min(own, p.M - m0 - rank * own);  // tokens of mine that exist
  if (p.out_dtype == W4A8_DTYPE_F32)
    finish_tokens<BN, GATED, float>(p, red, splits, own, left, m0 + rank * own, n0, vec_out, bias, bias2, res);
  else if (p.out_dtype == W4A8_DTYPE_F16)
    finish_tokens<BN, GATED, __half>(p, red, splits, own, left, m0 + rank * own, n0, vec_out, bias, bias2, res);
  else
    finish_tokens<BN, GATED, __nv_bfloat16>(p, red, splits, own, left, m0 + rank * own, n0, vec_out, bias, bias2, res);
}

// --- test of the epilogue warps' common outcome -----------------------------------------------------------------

// The epilogue warps of one CTA, each waiting on a barrier of its own as in a tile's last chunk; that of warp `missing` is
// never completed.  gave_up[w]: warp w was told that the tile is lost.
__global__ void __launch_bounds__(32 * kPairEpiWarps) linear_wait_probe_kernel(int missing, uint64_t limit_ns, int* gave_up) {
  __shared__ uint64_t bars[kPairEpiWarps];
  __shared__ int abort_flag;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int i = 0; i < kPairEpiWarps; ++i) mbar_init(&bars[i], 1);
    abort_flag = 0;
    mbar_fence_init();
  }
  __syncthreads();
  if (lane == 0 && warp != missing) mbar_arrive(&bars[warp]);
  __syncwarp();
  const bool mine = __all_sync(0xffffffffu, wait_bar(&bars[warp], 0, &abort_flag, limit_ns));
  const bool ok = all_satisfied<32 * kPairEpiWarps>(mine);
  if (lane == 0) gave_up[warp] = (ok ? 0 : 1) | (mine ? 0 : 2);
}

// --- operands without 16-byte alignment ------------------------------------------------------------------------

// Rows of x and of w (those of the two that need it) to 16-byte-aligned rows of the workspace, zeros past K; 8 elements
// per thread.  Inside a row they come in as 32-bit words, shifted into place where the row starts in the middle of one;
// a row's ends are read element by element, so that nothing beside it is touched.
__global__ void __launch_bounds__(256) linear_repack_kernel(const uint16_t* x, int64_t ldx, int64_t items_x, uint16_t* px,
                                                            const uint16_t* w, int64_t ldw, int64_t items, uint16_t* pw,
                                                            int K, int k8) {
  pdl_trigger();
  pdl_wait();
  for (int64_t i = blockIdx.x * 256ll + threadIdx.x; i < items; i += gridDim.x * 256ll) {
    const bool is_x = i < items_x;
    const int64_t j = is_x ? i : i - items_x;
    const uint32_t row = static_cast<uint32_t>(static_cast<uint64_t>(j) / static_cast<uint32_t>(k8));
    const int k = static_cast<int>(j - static_cast<int64_t>(row) * k8) * 8;
    const uint16_t* src = (is_x ? x + row * ldx : w + row * ldw) + k;
    uint32_t v[4];
    if (k > 0 && k + 8 < K) {
      const uintptr_t a = reinterpret_cast<uintptr_t>(src);
      const uint32_t* words = reinterpret_cast<const uint32_t*>(a & ~uintptr_t(3));
      uint32_t in[5];
#pragma unroll
      for (int c = 0; c < 4; ++c) in[c] = words[c];
      in[4] = a & 2 ? words[4] : 0;
#pragma unroll
      for (int c = 0; c < 4; ++c) v[c] = __funnelshift_r(in[c], in[c + 1], static_cast<uint32_t>(a & 2) * 8);
    } else {
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const uint32_t lo = k + 2 * c < K ? src[2 * c] : 0, hi = k + 2 * c + 1 < K ? src[2 * c + 1] : 0;
        v[c] = lo | (hi << 16);
      }
    }
    reinterpret_cast<uint4*>(is_x ? px : pw)[j] = make_uint4(v[0], v[1], v[2], v[3]);
  }
}

// --- host side -----------------------------------------------------------------------------------------------

typedef CUresult (*EncodeFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                             const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                             CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeFn encode_fn() {
  static EncodeFn fn = [] {
    void* q = nullptr;
    cudaDriverEntryPointQueryResult r;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &q, 12000, cudaEnableDefault, &r) != cudaSuccess ||
        r != cudaDriverEntryPointSuccess)
      q = nullptr;
    return reinterpret_cast<EncodeFn>(q);
  }();
  return fn;
}

// rows x K 16-bit matrix, boxes of box_rows x 64 k (zeros outside), 128-byte swizzle
int row_map(CUtensorMap* m, const void* base, int dtype, int64_t rows, int64_t K, int64_t ld, int box_rows,
            const char* name) {
  EncodeFn fn = encode_fn();
  if (!fn) return set_error(W4A8_ERR_CUDA, "cuTensorMapEncodeTiled is not available");
  const cuuint64_t dims[2] = {static_cast<cuuint64_t>(K), static_cast<cuuint64_t>(rows)};
  const cuuint64_t strides[1] = {static_cast<cuuint64_t>(ld) * 2};
  const cuuint32_t box[2] = {kBK, static_cast<cuuint32_t>(box_rows)};
  const cuuint32_t estr[2] = {1, 1};
  const CUresult r =
      fn(m, dtype == W4A8_DTYPE_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 2,
         const_cast<void*>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
         CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS)
    return set_error(W4A8_ERR_INVALID_ARG, "tensor map for %s rejected (CUresult %d)", name, static_cast<int>(r));
  return W4A8_OK;
}

int read_linear_error() {
  unsigned int v = 0;
  cudaMemcpyFromSymbol(&v, g_linear_error, sizeof(v));
  const unsigned int zero = 0;
  cudaMemcpyToSymbol(g_linear_error, &zero, sizeof(zero));
  return static_cast<int>(v);
}

struct Registrar {
  Registrar() { register_device_error_reader(&read_linear_error); }
} registrar;

// widest access that out's and the residual's rows take: 2 = 32 bytes, 1 = 16 bytes, 0 = single elements
int vec_rows(const LinearParams& p) {
  const uint64_t size = dtype_size(p.out_dtype);
  uint64_t bits = reinterpret_cast<uintptr_t>(p.out) | p.ldo * size;
  if (p.residual) bits |= reinterpret_cast<uintptr_t>(p.residual) | p.ldr * size;
  return bits % 32 == 0 ? 2 : bits % 16 == 0 ? 1 : 0;
}

// What a launch of one kernel instance needs, and how many of its clusters a device runs at once (clusters of 8 leave
// SMs of a graphics-processing cluster unused, so this is not SMs / size).
class Launcher {
 public:
  template <class... KArgs>
  int prepare(int dev, int* clusters, void (*kern)(KArgs...), size_t smem, int threads, int cluster, int least_regs = 0) {
    const bool known = dev >= 0 && dev < 64;
    if (known && (*clusters = clusters_[dev].load(std::memory_order_acquire)) > 0) return W4A8_OK;
    if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem)) != cudaSuccess)
      return check_launch("cudaFuncSetAttribute(linear)");
    if (least_regs) {  // setmaxnreg.inc waits until the released registers cover the request: they must be there
      cudaFuncAttributes fa;
      if (cudaFuncGetAttributes(&fa, kern) != cudaSuccess) return check_launch("cudaFuncGetAttributes(linear)");
      if (fa.numRegs < least_regs)
        return set_error(W4A8_ERR_UNSUPPORTED, "linear kernel built with %d registers per thread: %d are needed",
                         fa.numRegs, least_regs);
    }
    cudaLaunchAttribute attr[1];
    cudaLaunchConfig_t lc = config(dim3(cluster), threads, smem, cluster, nullptr, attr);
    int n = 0;
    if (cudaOccupancyMaxActiveClusters(&n, kern, &lc) != cudaSuccess)
      return check_launch("cudaOccupancyMaxActiveClusters(linear)");
    *clusters = n > 0 ? n : 1;
    if (known) clusters_[dev].store(*clusters, std::memory_order_release);
    return W4A8_OK;
  }
  static cudaLaunchConfig_t config(dim3 grid, int threads, size_t smem, int cluster, cudaStream_t st,
                                   cudaLaunchAttribute* attr) {
    cudaLaunchConfig_t lc = {};
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = cluster;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    lc.gridDim = grid;
    lc.blockDim = dim3(threads);
    lc.dynamicSmemBytes = smem;
    lc.stream = st;
    lc.attrs = attr;
    lc.numAttrs = 1;
    return lc;
  }
  template <class... KArgs, class... Args>
  static int launch(const char* what, void (*kern)(KArgs...), dim3 grid, int threads, size_t smem, int cluster,
                    cudaStream_t st, Args&&... args) {
    cudaLaunchAttribute attr[2];
    cudaLaunchConfig_t lc = config(grid, threads, smem, cluster, st, attr);
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    lc.numAttrs = 2;
    const cudaError_t e = cudaLaunchKernelEx(&lc, kern, static_cast<KArgs>(args)...);
    if (e != cudaSuccess) return set_error(W4A8_ERR_CUDA, "%s: %s", what, cudaGetErrorString(e));
    return check_launch(what);
  }

 private:
  std::atomic<int> clusters_[64] = {};  // 0: not prepared on that device
};

// One configuration of the two kernels: how many clusters run at once, and the launch itself.
struct Option {
  int (*ready)(int dev, int* clusters);  // status; makes the configuration ready on the current device
  int (*launch)(const LinearParams& p, int dev, cudaStream_t st);
  double fixed_us;  // a launch of one tile per cluster without its stages
  double stage_us;  // a 64-k stage of a CTA by itself
  double l2_rate;   // bytes per us that L2 gives all CTAs together
  int stage_bytes;
  int rows, cols;   // x rows and W rows of a tile
  int parts;        // pieces of K
  int ctas, stages; // CTAs of a cluster, stages of a CTA's ring
  bool persistent;
};

template <bool GATED, int PARTS, bool CHUNKED>
struct Pair {
  static Launcher& launcher() {
    static Launcher l;
    return l;
  }
  static int ready(int dev, int* clusters) {
    return launcher().prepare(dev, clusters, linear_pair_kernel<GATED, PARTS, CHUNKED>, kPairSmem, kPairThreads,
                              2 * PARTS, CHUNKED ? kRegsLaunch : 0);
  }
  static int launch(const LinearParams& p, int dev, cudaStream_t st) {
    if (!CHUNKED && p.K > longest_sum(p.out_dtype) * kBK * PARTS)
      return Pair<GATED, PARTS, true>::launch(p, dev, st);
    CUtensorMap tx, tw;
    int rc, clusters = 1;
    if ((rc = ready(dev, &clusters))) return rc;
    if ((rc = row_map(&tx, p.x, p.dtype, p.M, p.K, p.ldx, 128, "x"))) return rc;
    if ((rc = row_map(&tw, p.w, p.dtype, p.N, p.K, p.ldw, 128, "w"))) return rc;
    PairPlan pl;
    pl.out_cols = GATED ? 128 : 256;
    pl.tiles_m = static_cast<int>(ceil_div(p.M, 256));
    pl.tiles_n = static_cast<int>(ceil_div(p.n_out, pl.out_cols));
    pl.tiles = pl.tiles_m * pl.tiles_n;  // below 2^25 for M, N <= 2^20
    pl.kblocks = static_cast<int>(ceil_div(p.K, kBK));
    pl.vec_out = vec_rows(p);
    const int n = PARTS > 1 || pl.tiles < clusters ? pl.tiles : clusters;
    return Launcher::launch("linear_pair_kernel", linear_pair_kernel<GATED, PARTS, CHUNKED>, dim3(2 * PARTS * n), kPairThreads,
                            kPairSmem, 2 * PARTS, st, tx, tw, p, pl);
  }
};

template <int BN, bool GATED, int SPLITS>
struct Split {
  using C = SplitCfg<BN>;
  static Launcher& launcher() {
    static Launcher l;
    return l;
  }
  static int ready(int dev, int* clusters) {
    return launcher().prepare(dev, clusters, linear_split_kernel<BN, GATED>, C::kSmem, C::kThreads, SPLITS);
  }
  static int launch(const LinearParams& p, int dev, cudaStream_t st) {
    CUtensorMap tx, tw;
    int rc, clusters = 1;
    if ((rc = ready(dev, &clusters))) return rc;
    if ((rc = row_map(&tx, p.x, p.dtype, p.M, p.K, p.ldx, BN, "x"))) return rc;
    if ((rc = row_map(&tw, p.w, p.dtype, p.N, p.K, p.ldw, GATED ? 64 : 128, "w"))) return rc;
    const unsigned nb = static_cast<unsigned>(ceil_div(p.n_out, GATED ? 64 : 128));
    return Launcher::launch("linear_split_kernel", linear_split_kernel<BN, GATED>,
                            dim3(nb * SPLITS, static_cast<unsigned>(ceil_div(p.M, BN))), C::kThreads, C::kSmem, SPLITS,
                            st, tx, tw, p, SPLITS, static_cast<int>(ceil_div(p.K, kBK)), vec_rows(p));
  }
};

template <bool GATED, int PARTS>
Option pair_option(double fixed) {
  return {Pair<GATED, PARTS, false>::ready, Pair<GATED, PARTS, false>::launch, fixed, 0.26, 18e6, kPairStageBytes, 256, 256, PARTS, 2 * PARTS, kPairStages,
          PARTS == 1};
}
template <int BN, bool GATED, int SPLITS>
Option split_option(double fixed) {
  return {Split<BN, GATED, SPLITS>::ready, Split<BN, GATED, SPLITS>::launch, fixed, BN == 32 ? 0.2 : 0.18, 12e6, SplitCfg<BN>::kStageBytes, BN, 128, SPLITS,
          SPLITS,
          SplitCfg<BN>::kStages, false};
}

// Configuration asked for by a test (rows of a tile * 16 + pieces of K), 0: none.
std::atomic<int> g_force{0};

// The configuration with the smallest estimate
//   fixed + max(stage * (64-k stages of a piece), W / rate) * waves + (waves - 1) * (fixed - 3 us, a launch; 0 when
//   persistent)
// stage: what a stage takes where memory does not bound it, 0.26 us in the pair kernel (its products) and 0.18 to 0.2 us
// in the split kernel (its loads), or what L2 needs for the stages of all CTAs (12 TB/s for the split kernel; 18 TB/s for
// the pair kernel, which reads most lines for many CTAs at once).  rate: 6 TB/s of memory, or what the bytes in flight of
// the CTAs give at 1.2 us of latency.  fixed: launches of one wave extrapolated to no stages.  Fitted on a GB300 (M x N
// x K = 64 x 256 x 7168, 64 x 4096 x 7168 and 256 x 4096 x 7168 gated, 128 x 7168 x 2048, 777 x 1001 x 1544,
// 2048 x 256 x 7168, every configuration); of 24 other shapes it is within 10 % of the best on 22, and at worst 1.35 times
// it (258 x 3776 x 1536: 12.5 us, 9.3 with tiles of 64 rows).
template <bool GATED>
int launch_best(const LinearParams& p, cudaStream_t st) {
  static const Option options[] = {
      pair_option<GATED, 1>(8.0),          pair_option<GATED, 2>(8.0),          pair_option<GATED, 4>(10.5),
      split_option<128, GATED, 1>(7.4),    split_option<128, GATED, 2>(7.4),    split_option<128, GATED, 4>(7.4),
      split_option<64, GATED, 1>(4.2),     split_option<64, GATED, 2>(4.2),     split_option<64, GATED, 4>(4.2),
      split_option<64, GATED, 8>(4.3),     split_option<32, GATED, 1>(3.3),     split_option<32, GATED, 2>(3.4),
      split_option<32, GATED, 4>(3.4),     split_option<32, GATED, 8>(3.5),
  };
  int dev = -1;
  if (cudaGetDevice(&dev) != cudaSuccess) return check_launch("cudaGetDevice");
  const Option* best = nullptr;
  double best_us = 0.0;
  const int64_t kblocks = ceil_div(p.K, kBK);
  const int force = g_force.load(std::memory_order_relaxed);
  for (const Option& o : options) {
    // sums are kept short (see longest_sum): the split kernel has split_accumulators for a piece of K
    if (!force && o.rows < 256 && kblocks > split_accumulators(p.out_dtype) * longest_sum(p.out_dtype) * o.parts) continue;
    if (o.parts > kblocks || (force && force % 16 <= kblocks && force != o.rows * 16 + o.parts)) continue;
    int clusters = 1;
    if (int rc = o.ready(dev, &clusters)) return rc;
    const int64_t tiles = ceil_div(p.M, o.rows) * ceil_div(p.N, o.cols);
    const int64_t waves = ceil_div(tiles, clusters);
    const double ctas = static_cast<double>(std::min<int64_t>(tiles, clusters)) * o.ctas;
    const double rate = std::min(6.0e6, ctas * o.stages * kATile / 1.2);  // bytes of W per us
    const double w_us = 2.0 * p.N * p.K / rate / static_cast<double>(waves);
    const double stage_us = std::max(o.stage_us, ctas * o.stage_bytes / o.l2_rate);
    const double us = o.fixed_us +
                      std::max(stage_us * static_cast<double>(ceil_div(kblocks, o.parts)), w_us) * waves +
                      (o.persistent ? 0.0 : (waves - 1) * (o.fixed_us - 3.0));
    if (!best || us < best_us) {
      best = &o;
      best_us = us;
    }
  }
  if (!best) return set_error(W4A8_ERR_UNSUPPORTED, "no configuration for K=%d", p.K);
  return best->launch(p, dev, st);
}

}  // namespace

int launch_linear_tc(LinearParams p, void* ws, size_t ws_bytes, cudaStream_t st) {
  const bool x_ok = aligned16(p.x) && p.ldx % 8 == 0, w_ok = aligned16(p.w) && p.ldw % 8 == 0;
  if (!x_ok || !w_ok) {  // TMA takes rows on 16-byte boundaries only
    const int64_t k8 = ceil_div(p.K, 8), items_x = x_ok ? 0 : p.M * k8, items = items_x + (w_ok ? 0 : p.N * k8);
    const size_t need = static_cast<size_t>(items) * 16;
    W4A8_REQUIRE(ws && ws_bytes >= need && aligned16(ws),
                 "x and w without 16-byte alignment need %zu bytes of 16-byte aligned workspace", need);
    uint16_t* px = static_cast<uint16_t*>(ws);
    uint16_t* pw = px + items_x * 8;
    const int64_t blocks = ceil_div(items, 256);
    if (int rc = launch_pdl("linear_repack_kernel", linear_repack_kernel,
                            dim3(static_cast<unsigned>(blocks < 32 * num_sms() ? blocks : 32 * num_sms())), dim3(256), 0,
                            st, static_cast<const uint16_t*>(p.x), p.ldx, items_x, px,
                            static_cast<const uint16_t*>(p.w), p.ldw, items, pw, p.K, static_cast<int>(k8)))
      return rc;
    if (!x_ok) {
      p.x = px;
      p.ldx = k8 * 8;
    }
    if (!w_ok) {
      p.w = pw;
      p.ldw = k8 * 8;
    }
  }
  return p.gated ? launch_best<true>(p, st) : launch_best<false>(p, st);
}

}  // namespace w4a8

extern "C" int w4a8_test_linear_config(int rows, int pieces) {
  w4a8::g_force.store(rows > 0 ? rows * 16 + pieces : 0);
  return W4A8_OK;
}

extern "C" int w4a8_test_linear_wait(int missing, uint64_t limit_ns, int* gave_up, void* stream) {
  using namespace w4a8;
  W4A8_REQUIRE(gave_up != nullptr && (reinterpret_cast<uintptr_t>(gave_up) & 3) == 0, "gave_up must be an int[8]");
  W4A8_REQUIRE(missing >= -1 && missing < kPairEpiWarps, "missing=%d must be in [-1, 8)", missing);
  W4A8_REQUIRE(limit_ns > 0 && limit_ns <= kTimeoutNs, "limit_ns must be in (0, 2e9]");
  linear_wait_probe_kernel<<<1, 32 * kPairEpiWarps, 0, static_cast<cudaStream_t>(stream)>>>(missing, limit_ns, gave_up);
  return check_launch("linear_wait_probe_kernel");
}
