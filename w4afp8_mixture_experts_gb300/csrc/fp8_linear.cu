// fp8_block_linear: E4M3 x E4M3 with a scale per token and 128 k, and per 128 x 128 weights, on the 5th-generation tensor
// cores.
//
// A group of 128 k is one 128-byte swizzled row: one stage of the TMA ring, four products of 32 k, and one accumulator
// fill in tensor memory.  The scales change with every group, so an accumulator is read back after each: sum += product *
// (a_scale * b_scale) in fp32 registers, while the next group's products run into another accumulator.
//
//   pair kernel (many rows): a cluster of two CTAs computes a 256 x 256 tile with tcgen05.mma.cta_group::2, tokens on M,
//   persistent.  A thread holds 128 columns of one token, so that a group's scale is one number to it; 8 warps read 128 x
//   256 values of a group in the time that its products take.
//
//   split kernel (few rows, or few tiles): a CTA computes a 128 x BN tile, W rows on M and tokens on N, over one piece of
//   K; the tokens' scales come with each stage.  The CTAs of a cluster take the pieces of one tile and push their sums
//   into the shared memory of the CTA that owns a token, which adds them up in rank order: one launch, no workspace, a
//   result that does not depend on timing.
//
// Every wait is bounded: on expiry the CTA raises its abort flag and the device error word, lets its copies and products
// in flight finish (again with a limit), frees its tensor memory and returns.
#include <algorithm>
#include <atomic>

#include "block_ops.cuh"
#include "linear_tc.cuh"

namespace w4a8 {
namespace {

constexpr int kTile = 128 * 128;  // bytes of 128 rows of a stage

struct Fp8Params {
  const float *a_s, *b_s;
  void* out;
  int64_t lda_s, ldo;
  int M, N, groups;  // K / 128
  int out_dtype;
  int vec_out;       // out's rows lie on 16-byte boundaries
};

// fp32 accumulator, E4M3 operands, K-major
__host__ __device__ constexpr uint32_t idesc_fp8(uint32_t m, uint32_t n) {
  return (1u << 4) | ((n >> 3) << 17) | ((m >> 4) << 24);
}
__device__ __forceinline__ void mma_fp8_pair(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
      : "memory");
}
// two fp32 sums += two products * one scale, in one instruction
__device__ __forceinline__ void fma2(uint64_t& sum, uint32_t v0, uint32_t v1, uint64_t scale2) {
  asm("{\n\t.reg .b64 v;\n\tmov.b64 v, {%1, %2};\n\tfma.rn.f32x2 %0, v, %3, %0;\n\t}"
      : "+l"(sum)
      : "r"(v0), "r"(v1), "l"(scale2));
}
__device__ __forceinline__ uint64_t mul2(float x, float y, uint64_t scale2) {
  uint64_t r;
  asm("{\n\t.reg .b64 v;\n\tmov.b64 v, {%1, %2};\n\tmul.rn.f32x2 %0, v, %3;\n\t}" : "=l"(r) : "f"(x), "f"(y), "l"(scale2));
  return r;
}
__device__ __forceinline__ uint64_t twice(float v) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %1};" : "=l"(r) : "f"(v));
  return r;
}
__device__ __forceinline__ float2 halves(uint64_t v) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
  return r;
}

// --- pair kernel ---------------------------------------------------------------------------------------------

constexpr int kPairStages = 6;
constexpr int kPairEpiWarps = 8;
constexpr int kPairThreads = 128 + kPairEpiWarps * 32;
constexpr int kPairStageBytes = 2 * kTile;  // of one CTA: 128 rows of A, 128 rows of B
constexpr int kStageRow = 17;               // fp32 row of a warp's 32 x 16 transposing block, padded
constexpr int kStgBytes = 4096;             // of an epilogue warp: a box of 32 rows x 128 bytes on its way out
constexpr int kPairOffStg = kPairStages * kPairStageBytes;
constexpr int kPairOffBar = kPairOffStg + kPairEpiWarps * kStgBytes;
static_assert(32 * kStageRow * 4 <= kStgBytes, "transposing block");
constexpr int kPairSmem = kPairOffBar + (2 * kPairStages + 5) * 8 + 16 + 1024;
static_assert(kPairSmem <= kMaxSmem, "shared memory");
static_assert(kPairOffBar % 8 == 0, "barrier alignment");
constexpr int kRegsLaunch = 168;                 // of a thread at launch (checked on the host)
constexpr int kRegsRoles = 40, kRegsSums = 232;  // registers of warps 0-3 and of the epilogue's, which hold 128 sums
static_assert(128 * kRegsRoles + 32 * kPairEpiWarps * kRegsSums <= kPairThreads * kRegsLaunch, "within the launch's registers");

struct PairPlan {
  int tiles_m, tiles_n, tiles;
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

// 16 columns, from n on, of this thread's token m0 + lane, where out's rows are not aligned for copies: through shared memory,
// so that the lanes of a warp touch neighbouring columns of two rows instead of 32 rows.
__device__ __forceinline__ void store16(const Fp8Params& p, const float (&v)[16], int m0, int n, float* stg) {
  const int lane = threadIdx.x & 31;
  __syncwarp();
#pragma unroll
  for (int i = 0; i < 16; ++i) stg[lane * kStageRow + i] = v[i];
  __syncwarp();
  const int c = n + (lane & 15);
  if (c < p.N) {
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const int row = (lane >> 4) + 2 * i;
      if (m0 + row < p.M) store_any(p.out, (m0 + row) * p.ldo + c, stg[row * kStageRow + (lane & 15)], p.out_dtype);
    }
  }
}

__device__ __forceinline__ void tma_store_2d(const CUtensorMap* m, const void* src, int32_t x, int32_t y) {
  asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.bulk_group [%0, {%1, %2}], [%3];" ::"l"(
                   reinterpret_cast<uint64_t>(m)),
               "r"(x), "r"(y), "r"(smem_u32(src))
               : "memory");
}
__device__ __forceinline__ void bulk_commit() { asm volatile("cp.async.bulk.commit_group;" ::: "memory"); }
__device__ __forceinline__ void bulk_wait_read() { asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory"); }
__device__ __forceinline__ void bulk_wait() { asm volatile("cp.async.bulk.wait_group 0;" ::: "memory"); }

// A warp's 32 tokens x 128 columns as boxes of 128 bytes a row, written to shared memory (128-byte swizzle: no two of 8
// lanes on one bank) and copied out by TMA, which leaves out what lies behind the last row or column.  The copies run
// under the next tile's products.
template <typename T>
__device__ __forceinline__ void store_boxes(const Fp8Params& p, const CUtensorMap* to, const uint64_t (&sum)[64], int m0, int n,
                                            uint8_t* stg) {
  constexpr int kVec = 16 / sizeof(T), kBoxes = 128 * sizeof(T) / 128, kCols = 128 / sizeof(T);  // columns of a box
  int lane;  // read here, so that no address of these stores is held during the products
  asm volatile("mov.u32 %0, %%laneid;" : "=r"(lane));
#pragma unroll
  for (int b = 0; b < kBoxes; ++b) {
    if (lane == 0) bulk_wait_read();  // the last box has left
    __syncwarp();
#pragma unroll
    for (int c = 0; c < 8; ++c) {
      const int j = (b * kCols + c * kVec) / 2;
      uint4 w;
      if constexpr (sizeof(T) == 4) {
        const float2 x = halves(sum[j]), y = halves(sum[j + 1]);
        w = make_uint4(__float_as_uint(x.x), __float_as_uint(x.y), __float_as_uint(y.x), __float_as_uint(y.y));
      } else {
        const float2 x = halves(sum[j]), y = halves(sum[j + 1]), z = halves(sum[j + 2]), u = halves(sum[j + 3]);
        w = make_uint4(pack2<T>(x.x, x.y), pack2<T>(y.x, y.y), pack2<T>(z.x, z.y), pack2<T>(u.x, u.y));
      }
      *reinterpret_cast<uint4*>(stg + lane * 128 + ((c ^ (lane & 7)) << 4)) = w;
    }
    fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) {
      if (m0 < p.M && n + b * kCols < p.N) tma_store_2d(to, stg, n + b * kCols, m0);
      bulk_commit();
    }
  }
}

__global__ void __launch_bounds__(kPairThreads, 1)
    fp8_pair_kernel(const __grid_constant__ CUtensorMap ta, const __grid_constant__ CUtensorMap tb,
                    const __grid_constant__ CUtensorMap to, const Fp8Params p, const PairPlan pl) {
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
  const int rank = static_cast<int>(cluster_rank());
  pdl_trigger();
  if (warp == 0 && lane == 0) {
    tma_prefetch_desc(&ta);
    tma_prefetch_desc(&tb);
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
  const int first = blockIdx.x / 2, stride = gridDim.x / 2;
  // no CTA of the pair leaves while the other may still signal it or read its operands
  auto leave = [&] {
    __syncwarp();
    tc_fence_before();
    cluster_arrive();
    cluster_wait();
  };
  // Warps 0-3 end inside this branch: they hold fewer registers than the code behind it is built for.
  if (warp < 4) {
    regs_release<kRegsRoles>();
    if (warp == 0) {  // TMA producer of this CTA's half of every stage
      uint32_t it = 0;
      bool ok = true;
      for (int i = first; ok && i < pl.tiles; i += stride) {
        int tm, tn;
        pair_tile(pl, i, tm, tn);
        const int m = tm * 256 + rank * 128, n = tn * 256 + rank * 128;
        for (int g = 0; g < p.groups; ++g, ++it) {
          const int s = it % kPairStages;
          if (!(ok = warp_wait(&empty[s], ((it / kPairStages) & 1) ^ 1, abort_flag))) break;
          if (elect_one()) {
            uint8_t* at = smem + s * kPairStageBytes;
            const uint32_t bar = map_to_cta(smem_u32(&full[s]), 0);
            if (rank == 0) mbar_arrive_expect_tx(&full[s], 2 * kPairStageBytes);
            tma_load_pair(at, &ta, bar, g * 128, m);
            tma_load_pair(at + kTile, &tb, bar, g * 128, n);
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
      const uint32_t idesc = idesc_fp8(256, 256);
      uint32_t it = 0;
      bool ok = true;
      for (int i = first; ok && i < pl.tiles; i += stride) {
        for (int g = 0; g < p.groups; ++g, ++it) {
          const int s = it % kPairStages, buf = it & 1;
          if (!(ok = warp_wait(&tempty[buf], ((it >> 1) & 1) ^ 1, abort_flag))) break;
          if (!(ok = warp_wait(&full[s], (it / kPairStages) & 1, abort_flag))) break;
          tc_fence_after();
          const uint32_t at = smem_u32(smem + s * kPairStageBytes);
          const uint64_t a = operand_desc(at), b = operand_desc(at + kTile);
          if (elect_one()) {
#pragma unroll
            for (int k = 0; k < 4; ++k) mma_fp8_pair(tmem + buf * 256, a + 2 * k, b + 2 * k, idesc, k > 0);
            commit_pair(&empty[s], 3);
            commit_pair(&tfull[buf], 3);
          }
          __syncwarp();
        }
      }
      // no product is in flight when the tensor memory goes back, also where the epilogue has given up
      if (elect_one())
        asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_u32(mdrain))
                     : "memory");
      __syncwarp();
      drain_bar(mdrain, 0);
    }
    leave();
    if (warp == 2) {
      tc_fence_after();
      asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, 512;" ::"r"(tmem));
    }
    return;
  }
  regs_claim<kRegsSums>();

  // epilogue: warp e reads lane quarter e % 4 (its tokens) and, by e / 4, one half of the columns, which have one scale
  const int e = warp - 4, quarter = warp & 3, half = e >> 2;
  uint8_t* stg = smem + kPairOffStg + e * kStgBytes;
  const uint32_t lanes = (static_cast<uint32_t>(quarter * 32) << 16) + half * 128;
  const uint32_t tempty0 = map_to_cta(smem_u32(tempty), 0);
  const int nb_end = (p.N + 127) / 128;
  uint32_t it = 0;
  bool ok = true;
  for (int i = first; ok && i < pl.tiles; i += stride) {
    int tm, tn;
    pair_tile(pl, i, tm, tn);
    const int m0 = tm * 256 + rank * 128 + quarter * 32, nb = tn * 2 + half;
    const float* as = p.a_s + m0 + lane;
    const float* bs = p.b_s + static_cast<int64_t>(nb) * p.groups;
    const bool row = m0 + lane < p.M, cols = nb < nb_end;
    // scales are loaded two groups ahead
    auto load_a = [&](int g) { return row && g < p.groups ? as[g * p.lda_s] : 0.f; };
    auto load_b = [&](int g) { return cols && g < p.groups ? bs[g] : 0.f; };
    float a0 = load_a(0), b0 = load_b(0), a1 = load_a(1), b1 = load_b(1);
    uint64_t sum[64];
#pragma unroll
    for (int j = 0; j < 64; ++j) sum[j] = 0;
#pragma unroll 1
    for (int g = 0; g < p.groups; ++g, ++it) {
      const uint64_t scale = twice(a0 * b0);
      a0 = a1, b0 = b1;
      a1 = load_a(g + 2), b1 = load_b(g + 2);
      const int buf = it & 1;
      if (!(ok = warp_wait(&tfull[buf], (it >> 1) & 1, abort_flag))) break;
      tc_fence_after();
      const uint32_t at = tmem + buf * 256 + lanes;
      uint32_t v[2][32];
      tmem_ld32(at, v[0]);
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        tmem_wait_ld_pin<32>(v[q & 1]);
        if (q < 3) {
          tmem_ld32(at + 32 * (q + 1), v[(q + 1) & 1]);
        } else {  // every value is in registers: the accumulator is free
          tc_fence_before();
          __syncwarp();
          if (lane == 0) remote_arrive(tempty0 + buf * 8);
        }
#pragma unroll
        for (int j = 0; j < 16; ++j) fma2(sum[16 * q + j], v[q & 1][2 * j], v[q & 1][2 * j + 1], scale);
      }
    }
    if (!ok) break;
    if (!cols) continue;
    if (p.vec_out) {
      if (p.out_dtype == W4A8_DTYPE_BF16)
        store_boxes<__nv_bfloat16>(p, &to, sum, m0, nb * 128, stg);
      else if (p.out_dtype == W4A8_DTYPE_F16)
        store_boxes<__half>(p, &to, sum, m0, nb * 128, stg);
      else
        store_boxes<float>(p, &to, sum, m0, nb * 128, stg);
      continue;
    }
#pragma unroll
    for (int q = 0; q < 8; ++q) {
      float f[16];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float2 t = halves(sum[8 * q + j]);
        f[2 * j] = t.x;
        f[2 * j + 1] = t.y;
      }
      if (nb * 128 + 16 * q < p.N) store16(p, f, m0, nb * 128 + 16 * q, reinterpret_cast<float*>(stg));
    }
  }
  if (lane == 0) bulk_wait();
  leave();
}

// --- split kernel --------------------------------------------------------------------------------------------

template <int BN>
struct SplitCfg {
  static constexpr int kThreads = 384;
  static constexpr int kStageBytes = kTile + BN * 128;
  static constexpr int kBlocks = BN == 128 ? 1 : 2;  // of an SM
  static constexpr int kStages = BN == 128 ? 6 : BN == 64 ? 4 : 5;
  static constexpr int kBufs = BN == 128 ? 2 : 4;    // accumulators
  static constexpr int kCols = BN / 2;               // of a warp: tokens whose sums it holds
  static constexpr int kScaleBytes = (BN * 4 + 127) / 128 * 128;
  static constexpr int kOffScale = kStages * kStageBytes;
  static constexpr int kOffBar = kOffScale + kStages * kScaleBytes;
  static constexpr int kSmem = kOffBar + (2 * kStages + 2 * kBufs + 1) * 8 + 16 + 1024;
  static constexpr uint32_t kTmemCols = kBufs * BN < 32 ? 32 : kBufs * BN;
  static_assert((kSmem + 1024) * kBlocks <= 228 * 1024, "shared memory");
  static_assert(kTmemCols * kBlocks <= 512, "tensor memory");
  static_assert((BN + 8) * 512 <= kStages * kStageBytes, "partial sums in the ring");
};

template <int N>
__device__ __forceinline__ void tmem_load(uint32_t at, uint32_t (&v)[N]) {
  if constexpr (N == 64) {
    tmem_ld32(at, v);
    tmem_ld32(at + 32, v + 32);
  } else if constexpr (N == 32)
    tmem_ld32(at, v);
  else if constexpr (N == 16)
    tmem_ld16(at, v);
  else
    tmem_ld8(at, v);
}

template <int BN>
__global__ void __launch_bounds__(SplitCfg<BN>::kThreads, SplitCfg<BN>::kBlocks)
    fp8_split_kernel(const __grid_constant__ CUtensorMap ta, const __grid_constant__ CUtensorMap tb,
                     const __grid_constant__ CUtensorMap ts, const Fp8Params p, int splits) {
  using C = SplitCfg<BN>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::kOffBar);
  uint64_t* empty = full + C::kStages;     // products done and scales read
  uint64_t* tfull = empty + C::kStages;
  uint64_t* tempty = tfull + C::kBufs;
  uint64_t* mdrain = tempty + C::kBufs;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(mdrain + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  const int rank = splits > 1 ? static_cast<int>(cluster_rank()) : 0;
  const int nb = blockIdx.x / splits, n0 = nb * 128, m0 = blockIdx.y * BN;
  pdl_trigger();
  if (warp == 0 && lane == 0) {
    tma_prefetch_desc(&ta);
    tma_prefetch_desc(&tb);
    tma_prefetch_desc(&ts);
    for (int i = 0; i < C::kStages; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], 1 + 8);
    }
    for (int i = 0; i < C::kBufs; ++i) {
      mbar_init(&tfull[i], 1);
      mbar_init(&tempty[i], 8);
    }
    mbar_init(mdrain, 1);
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
  const uint32_t tmem = *tmem_slot;
  pdl_wait();

  const int g0 = static_cast<int>(static_cast<int64_t>(rank) * p.groups / splits);
  const int count = static_cast<int>(static_cast<int64_t>(rank + 1) * p.groups / splits) - g0;
  bool ok = true;
  uint64_t sum[C::kCols / 2];  // two tokens each
  const int quarter = warp & 3, half = (warp >> 2) - 1, f = quarter * 32 + lane;
  if (warp == 0) {
    int it = 0;
    for (; it < count; ++it) {
      const int s = it % C::kStages;
      if (!(ok = warp_wait(&empty[s], ((it / C::kStages) & 1) ^ 1, abort_flag))) break;
      if (elect_one()) {
        uint8_t* at = smem + s * C::kStageBytes;
        mbar_arrive_expect_tx(&full[s], C::kStageBytes + BN * 4);
        tma_load_2d(at, &tb, &full[s], (g0 + it) * 128, n0);
        tma_load_2d(at + kTile, &ta, &full[s], (g0 + it) * 128, m0);
        tma_load_2d(smem + C::kOffScale + s * C::kScaleBytes, &ts, &full[s], m0, g0 + it);
      }
      __syncwarp();
    }
    // every load has landed before the ring is used for the exchange, also after an abort
    for (int j = it < C::kStages ? 0 : it - C::kStages; j < it; ++j) drain_bar(&full[j % C::kStages], (j / C::kStages) & 1);
  } else if (warp == 1) {
    const uint32_t idesc = idesc_fp8(128, BN);
    for (int it = 0; it < count; ++it) {
      const int s = it % C::kStages, buf = it % C::kBufs;
      if (!(ok = warp_wait(&tempty[buf], ((it / C::kBufs) & 1) ^ 1, abort_flag))) break;
      if (!(ok = warp_wait(&full[s], (it / C::kStages) & 1, abort_flag))) break;
      tc_fence_after();
      const uint32_t at = smem_u32(smem + s * C::kStageBytes);
      const uint64_t a = operand_desc(at), b = operand_desc(at + kTile);
      if (elect_one()) {
#pragma unroll
        for (int k = 0; k < 4; ++k) mma_f8f6f4_ss(tmem + buf * BN, a + 2 * k, b + 2 * k, idesc, k > 0);
        mma_commit(&empty[s]);
        mma_commit(&tfull[buf]);
      }
      __syncwarp();
    }
    // no product is in flight when the ring and the tensor memory go on, also where the sums' warps have given up
    if (elect_one()) mma_commit(mdrain);
    __syncwarp();
    drain_bar(mdrain, 0);
  } else if (warp >= 4) {
    const float* bs = p.b_s + static_cast<int64_t>(nb) * p.groups + g0;
    float b0 = count > 0 ? bs[0] : 0.f, b1 = count > 1 ? bs[1] : 0.f;  // loaded two groups ahead
#pragma unroll
    for (int j = 0; j < C::kCols / 2; ++j) sum[j] = 0;
    for (int it = 0; it < count; ++it) {
      const int s = it % C::kStages, buf = it % C::kBufs;
      const uint64_t b = twice(b0);
      b0 = b1;
      b1 = it + 2 < count ? bs[it + 2] : 0.f;
      // the scales come with the stage's copies, which this warp waits for as the products do
      if (!(ok = warp_wait(&full[s], (it / C::kStages) & 1, abort_flag))) break;
      const float4* as = reinterpret_cast<const float4*>(smem + C::kOffScale + s * C::kScaleBytes) + half * (C::kCols / 4);
      float4 scale[C::kCols / 4];
      if constexpr (C::kCols <= 16) {  // read under the products; with more columns there are no registers for that
#pragma unroll
        for (int j = 0; j < C::kCols / 4; ++j) scale[j] = as[j];
      }
      if (!(ok = warp_wait(&tfull[buf], (it / C::kBufs) & 1, abort_flag))) break;
      tc_fence_after();
      constexpr int kStep = BN == 128 ? 64 : BN == 16 ? 8 : 16;  // columns on their way at a time
#pragma unroll
      for (int c = 0; c < C::kCols; c += kStep) {
        uint32_t v[kStep];
        tmem_load<kStep>(tmem + (static_cast<uint32_t>(quarter * 32) << 16) + buf * BN + half * C::kCols + c, v);
        tmem_wait_ld_pin<kStep>(v);
#pragma unroll
        for (int j = 0; j < kStep; j += 4) {
          const float4 a = C::kCols <= 16 ? scale[(c + j) / 4] : as[(c + j) / 4];
          fma2(sum[(c + j) / 2], v[j], v[j + 1], mul2(a.x, a.y, b));
          fma2(sum[(c + j) / 2 + 1], v[j + 2], v[j + 3], mul2(a.z, a.w, b));
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(&tempty[buf]);
        mbar_arrive(&empty[s]);
      }
    }
  }
  __syncwarp();
  // the tensor memory goes back when every warp has read it
  const auto leave = [&] {
    tc_fence_before();
    __syncthreads();
    if (warp == 2) {
      tc_fence_after();
      tmem_dealloc(tmem, C::kTmemCols);
    }
  };
  if (splits == 1) {
    if (warp >= 4 && ok && n0 + f < p.N) {  // the lanes of a warp hold neighbouring columns of one token
#pragma unroll
      for (int j = 0; j < C::kCols; ++j) {
        const int m = m0 + half * C::kCols + j;
        const float2 v = halves(sum[j / 2]);
        if (m < p.M) store_any(p.out, m * p.ldo + n0 + f, j % 2 ? v.y : v.x, p.out_dtype);
      }
    }
    leave();
    return;
  }
  cluster_arrive();
  cluster_wait();  // every CTA of the tile is done with its ring: its loads and products
  // tokens [q BN / splits, (q + 1) BN / splits) belong to CTA q: red [source][token][128 W rows]
  const int most = (BN + splits - 1) / splits;
  if (warp >= 4 && ok) {
    const uint32_t red = smem_u32(smem);
    int q = (half * C::kCols + 1) * splits - 1;  // owner of the first token: the last CTA that starts at or before it
    q /= BN;
    int begin = q * BN / splits, end = (q + 1) * BN / splits;
#pragma unroll
    for (int j = 0; j < C::kCols; ++j) {
      const int tok = half * C::kCols + j;
      if (tok >= end) {
        ++q;
        begin = end;
        end = (q + 1) * BN / splits;
      }
      const uint32_t to = map_to_cta(red + ((rank * most + tok - begin) * 128 + f) * 4, q);
      const float2 v = halves(sum[j / 2]);
      asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(to), "f"(j % 2 ? v.y : v.x) : "memory");
    }
  }
  __syncwarp();
  cluster_arrive();
  leave();
  cluster_wait();
  if (*abort_flag) return;
  const int begin = rank * BN / splits, own = (rank + 1) * BN / splits - begin;
  const float* red = reinterpret_cast<const float*>(smem);
  const int left = min(own, p.M - m0 - begin);  // tokens of mine that exist
  if (p.vec_out) {
    for (int i = threadIdx.x; i < left * 32; i += C::kThreads) {  // 4 columns each
      const int tok = i >> 5, c = (i & 31) * 4, n = n0 + c;
      if (n >= p.N) continue;
      float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
      for (int s = 0; s < splits; ++s) {
        const float4 a = *reinterpret_cast<const float4*>(red + (s * most + tok) * 128 + c);
        v.x += a.x, v.y += a.y, v.z += a.z, v.w += a.w;
      }
      const int64_t at = (m0 + begin + tok) * p.ldo + n;
      if (n + 4 > p.N) {
        const float e[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (n + j < p.N) store_any(p.out, at + j, e[j], p.out_dtype);
      } else if (p.out_dtype == W4A8_DTYPE_F32) {
        *reinterpret_cast<float4*>(static_cast<float*>(p.out) + at) = v;
      } else if (p.out_dtype == W4A8_DTYPE_BF16) {
        *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.out) + at) =
            make_uint2(pack2<__nv_bfloat16>(v.x, v.y), pack2<__nv_bfloat16>(v.z, v.w));
      } else {
        *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.out) + at) =
            make_uint2(pack2<__half>(v.x, v.y), pack2<__half>(v.z, v.w));
      }
    }
    return;
  }
  for (int i = threadIdx.x; i < left * 128; i += C::kThreads) {
    const int tok = i >> 7, c = i & 127;
    if (n0 + c >= p.N) continue;
    float v = 0.f;
    for (int s = 0; s < splits; ++s) v += red[(s * most + tok) * 128 + c];
    store_any(p.out, (m0 + begin + tok) * p.ldo + n0 + c, v, p.out_dtype);
  }
}

// --- host side -----------------------------------------------------------------------------------------------

// a matrix of `rows` rows of 8-bit codes, boxes of box_rows x 128 (zeros outside), 128-byte swizzle
int code_map(CUtensorMap* m, const void* base, int64_t rows, int64_t K, int box_rows, const char* name) {
  EncodeFn fn = encode_fn();
  if (!fn) return set_error(W4A8_ERR_CUDA, "cuTensorMapEncodeTiled is not available");
  const cuuint64_t dims[2] = {static_cast<cuuint64_t>(K), static_cast<cuuint64_t>(rows)};
  const cuuint64_t strides[1] = {static_cast<cuuint64_t>(K)};
  const cuuint32_t box[2] = {128, static_cast<cuuint32_t>(box_rows)};
  const cuuint32_t estr[2] = {1, 1};
  const CUresult r = fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(base), dims, strides, box, estr,
                        CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                        CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS)
    return set_error(W4A8_ERR_INVALID_ARG, "tensor map for %s rejected (CUresult %d)", name, static_cast<int>(r));
  return W4A8_OK;
}

// the tokens' scales of a group, BN at a time (zeros behind the last token)
int scale_map(CUtensorMap* m, const Fp8Params& p, int box) {
  EncodeFn fn = encode_fn();
  if (!fn) return set_error(W4A8_ERR_CUDA, "cuTensorMapEncodeTiled is not available");
  const cuuint64_t dims[2] = {static_cast<cuuint64_t>(p.M), static_cast<cuuint64_t>(p.groups)};
  const cuuint64_t strides[1] = {static_cast<cuuint64_t>(p.lda_s) * 4};
  const cuuint32_t boxes[2] = {static_cast<cuuint32_t>(box), 1};
  const cuuint32_t estr[2] = {1, 1};
  const CUresult r = fn(m, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 2, const_cast<float*>(p.a_s), dims, strides, boxes, estr,
                        CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_NONE,
                        CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS)
    return set_error(W4A8_ERR_INVALID_ARG, "tensor map for a_scales rejected (CUresult %d)", static_cast<int>(r));
  return W4A8_OK;
}

// the output in boxes of 32 rows x 128 bytes, 128-byte swizzle
int out_map(CUtensorMap* m, const Fp8Params& p) {
  EncodeFn fn = encode_fn();
  if (!fn) return set_error(W4A8_ERR_CUDA, "cuTensorMapEncodeTiled is not available");
  const cuuint64_t size = dtype_size(p.out_dtype);
  const cuuint64_t dims[2] = {static_cast<cuuint64_t>(p.N), static_cast<cuuint64_t>(p.M)};
  const cuuint64_t strides[1] = {p.M > 1 ? p.ldo * size : (p.N * size + 15) / 16 * 16};  // one row needs none
  const cuuint32_t box[2] = {static_cast<cuuint32_t>(128 / size), 32};
  const cuuint32_t estr[2] = {1, 1};
  const CUtensorMapDataType type = p.out_dtype == W4A8_DTYPE_BF16  ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16
                                   : p.out_dtype == W4A8_DTYPE_F16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16
                                                                   : CU_TENSOR_MAP_DATA_TYPE_FLOAT32;
  const CUresult r = fn(m, type, 2, p.out, dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                        CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_NONE, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS)
    return set_error(W4A8_ERR_INVALID_ARG, "tensor map for out rejected (CUresult %d)", static_cast<int>(r));
  return W4A8_OK;
}

struct Call {
  const uint8_t *A, *B;
  Fp8Params p;
  int64_t K;
};

// One configuration: how many clusters run at once, the launch, and what launch_best needs to know of it.
struct Option {
  int (*ready)(int dev, int* clusters);
  int (*launch)(const Call& c, int dev, cudaStream_t st);
  int rows, cols, parts;              // tokens and W rows of a tile, pieces of K
  int stages, stage_bytes;            // of a CTA's ring
  double fixed_us, stage_us, wave_us; // a launch without its stages, a stage, a further wave of tiles
};

struct Pair {
  static Launcher& launcher() {
    static Launcher l;
    return l;
  }
  static int ready(int dev, int* clusters) {
    return launcher().prepare(dev, clusters, fp8_pair_kernel, kPairSmem, kPairThreads, 2, kRegsLaunch);
  }
  static int launch(const Call& c, int dev, cudaStream_t st) {
    CUtensorMap ta, tb, to = {};
    int rc, clusters = 1;
    if ((rc = ready(dev, &clusters))) return rc;
    if ((rc = code_map(&ta, c.A, c.p.M, c.K, 128, "A"))) return rc;
    if ((rc = code_map(&tb, c.B, c.p.N, c.K, 128, "B"))) return rc;
    if (c.p.vec_out && (rc = out_map(&to, c.p))) return rc;
    PairPlan pl;
    pl.tiles_m = static_cast<int>(ceil_div(c.p.M, 256));
    pl.tiles_n = static_cast<int>(ceil_div(c.p.N, 256));
    pl.tiles = pl.tiles_m * pl.tiles_n;  // at most 2^24
    return Launcher::launch("fp8_pair_kernel", fp8_pair_kernel, dim3(2 * std::min(pl.tiles, clusters)), kPairThreads,
                            kPairSmem, 2, st, ta, tb, to, c.p, pl);
  }
};

template <int BN, int SPLITS>
struct Split {
  using C = SplitCfg<BN>;
  static Launcher& launcher() {
    static Launcher l;
    return l;
  }
  static int ready(int dev, int* clusters) {
    return launcher().prepare(dev, clusters, fp8_split_kernel<BN>, C::kSmem, C::kThreads, SPLITS);
  }
  static int launch(const Call& c, int dev, cudaStream_t st) {
    CUtensorMap ta, tb, ts;
    int rc, clusters = 1;
    if ((rc = ready(dev, &clusters))) return rc;
    if ((rc = code_map(&ta, c.A, c.p.M, c.K, BN, "A"))) return rc;
    if ((rc = code_map(&tb, c.B, c.p.N, c.K, 128, "B"))) return rc;
    if ((rc = scale_map(&ts, c.p, BN))) return rc;
    return Launcher::launch("fp8_split_kernel", fp8_split_kernel<BN>,
                            dim3(static_cast<unsigned>(ceil_div(c.p.N, 128)) * SPLITS,
                                 static_cast<unsigned>(ceil_div(c.p.M, BN))),
                            C::kThreads, C::kSmem, SPLITS, st, ta, tb, ts, c.p, SPLITS);
  }
};

template <int BN, int SPLITS>
constexpr Option split_option() {
  using C = SplitCfg<BN>;
  // the exchange of the pieces' sums: its barriers, and its bytes
  constexpr double fixed = BN == 128 ? 4.4 : BN == 64 ? 3.6 : BN == 32 ? 3.0 : 2.7, exchange = SPLITS > 1 ? 1.35 + 0.82 * BN / 64 : 0;
  return {Split<BN, SPLITS>::ready, Split<BN, SPLITS>::launch, BN, 128, SPLITS, C::kStages, C::kStageBytes, fixed + exchange,
          BN == 128 ? 0.48 : BN == 64 ? 0.44 : BN == 32 ? 0.33 : 0.30, BN == 128 ? 5.7 : BN == 64 ? 4.4 : BN == 32 ? 4.0 : 3.3};
}

// Configuration asked for by a test (rows of a tile * 16 + pieces of K), 0: none; and rows of a tile whose configurations a
// test takes for not available, 0: none.
std::atomic<int> g_force{0}, g_without{0};

// The configuration with the smallest estimate
//   fixed + max(waves * stages of a piece * stage, bytes of W / rate) + (waves - 1) * wave
// stage: what a stage takes by itself, longer by half where two CTAs share every SM, or what L2 needs for the stages of all
// CTAs (13.9 TB/s).  rate: 6.2 TB/s of memory, or what the bytes of W in flight give at 1.95 us of latency.  Fitted on a GB300
// to 22 configurations of 110 shapes, drawn over 1 to 4096 rows, 64 to 24576 columns and K of 128 to 18432: its choice takes
// 1.9 % more than the best on average and is within 10 % of it on 103 (659 x 1984 x 3456: 19.9 us, best 17.0).
int launch_best(const Call& c, cudaStream_t st) {
  static const Option options[] = {
      {Pair::ready, Pair::launch, 256, 256, 1, kPairStages, kPairStageBytes, 5.1, 0.43, 1.8},
      split_option<128, 1>(), split_option<128, 2>(), split_option<128, 4>(),
      split_option<64, 1>(), split_option<64, 2>(), split_option<64, 3>(), split_option<64, 4>(), split_option<64, 5>(), split_option<64, 8>(),
      split_option<32, 1>(), split_option<32, 2>(), split_option<32, 3>(), split_option<32, 4>(), split_option<32, 5>(), split_option<32, 8>(),
      split_option<16, 1>(), split_option<16, 2>(), split_option<16, 3>(), split_option<16, 4>(), split_option<16, 5>(), split_option<16, 8>(),
  };
  int dev = -1;
  if (cudaGetDevice(&dev) != cudaSuccess) return check_launch("cudaGetDevice");
  const int force = g_force.load(std::memory_order_relaxed);
  const double sms = num_sms();
  const Option* best = nullptr;
  double best_us = 0.0;
  int missing = W4A8_OK;  // status of configurations that this build or device does not have
  for (const Option& o : options) {
    if (o.parts > c.p.groups || ceil_div(c.p.M, o.rows) > 65535) continue;
    if (force && force % 16 <= c.p.groups && force != o.rows * 16 + o.parts) continue;
    int clusters = 1, rc = W4A8_OK;
    if (o.rows == g_without.load(std::memory_order_relaxed))
      rc = set_error(W4A8_ERR_UNSUPPORTED, "configurations of %d rows are left out", o.rows);
    else
      rc = o.ready(dev, &clusters);
    if (rc == W4A8_ERR_UNSUPPORTED) {
      missing = rc;
      continue;
    }
    if (rc) return rc;
    const int64_t tiles = ceil_div(c.p.M, o.rows) * ceil_div(c.p.N, o.cols), waves = ceil_div(tiles, clusters);
    const double ctas = static_cast<double>(std::min<int64_t>(tiles, clusters)) * (o.rows == 256 ? 2 : o.parts);
    const double stage = std::max(o.stage_us * (1.0 + 0.45 * std::max(0.0, ctas / sms - 1.0)), ctas * o.stage_bytes / 13.9e6);
    const double rate = std::min(6.2e6, ctas * o.stages * kTile / 1.95);  // bytes of W per us
    const double us = o.fixed_us +
                      std::max(static_cast<double>(waves * ceil_div(c.p.groups, o.parts)) * stage,
                               static_cast<double>(c.p.N) * static_cast<double>(c.K) / rate) +
                      static_cast<double>(waves - 1) * o.wave_us;
    if (!best || us < best_us) {
      best = &o;
      best_us = us;
    }
  }
  if (!best) return missing ? missing : set_error(W4A8_ERR_UNSUPPORTED, "no configuration for M=%d, N=%d", c.p.M, c.p.N);
  return best->launch(c, dev, st);
}

}  // namespace
}  // namespace w4a8

extern "C" int fp8_block_linear(const uint8_t* A, const float* a_scales, int64_t lda_s, const uint8_t* B,
                                const float* b_scales, int64_t M, int64_t N, int64_t K, void* out, int64_t ldo,
                                int out_dtype, void* stream) {
  using namespace w4a8;
  W4A8_REQUIRE(out_dtype >= W4A8_DTYPE_BF16 && out_dtype <= W4A8_DTYPE_F32, "out_dtype=%d must be bf16, f16 or fp32",
               out_dtype);
  W4A8_REQUIRE(M >= 0 && M <= (1 << 20) && N >= 0 && N <= (1 << 20), "M=%lld and N=%lld must be in [0, 2^20]", (long long)M,
               (long long)N);
  W4A8_REQUIRE(K >= 128 && K <= (1 << 20) && K % 128 == 0, "K=%lld must be a multiple of 128 up to 2^20", (long long)K);
  W4A8_REQUIRE(lda_s >= M && lda_s % 4 == 0, "lda_s=%lld must be at least M=%lld and a multiple of 4", (long long)lda_s,
               (long long)M);
  W4A8_REQUIRE(ldo >= N, "ldo=%lld must be at least N=%lld", (long long)ldo, (long long)N);
  if (M == 0 || N == 0) return W4A8_OK;
  W4A8_REQUIRE(A && a_scales && B && b_scales && out, "null pointer");
  W4A8_REQUIRE(aligned16(A) && aligned16(B) && aligned16(a_scales), "A, B and a_scales must be 16-byte aligned");
  W4A8_REQUIRE(reinterpret_cast<uintptr_t>(b_scales) % 4 == 0 &&
                   reinterpret_cast<uintptr_t>(out) % dtype_size(out_dtype) == 0,
               "b_scales and out must be aligned to their element size");
  Call c;
  c.A = A;
  c.B = B;
  c.K = K;
  c.p.a_s = a_scales;
  c.p.b_s = b_scales;
  c.p.out = out;
  c.p.lda_s = lda_s;
  c.p.ldo = ldo;
  c.p.M = static_cast<int>(M);
  c.p.N = static_cast<int>(N);
  c.p.groups = static_cast<int>(K / 128);
  c.p.out_dtype = out_dtype;
  const uint64_t bits = reinterpret_cast<uintptr_t>(out) | (M > 1 ? static_cast<uint64_t>(ldo) * dtype_size(out_dtype) : 0);
  c.p.vec_out = bits % 16 == 0;
  return launch_best(c, static_cast<cudaStream_t>(stream));
}

extern "C" int w4a8_test_fp8_linear_config(int rows, int pieces) {
  w4a8::g_force.store(rows > 0 ? rows * 16 + pieces : 0);
  return W4A8_OK;
}

extern "C" int w4a8_test_fp8_linear_without(int rows) {
  w4a8::g_without.store(rows);
  return W4A8_OK;
}
