// paged_attention_decode: one query token per sequence against its cached keys and values.
//
// The work is a list of units: a unit is 4 * NT neighbouring tokens of one sequence for one key-value head and up to
// 16 * MT of its query heads, and the list goes through all sequences, heads and units in order.  A launch has as many
// blocks as stay resident, and each takes an equal run of the list, so that long and short sequences fill the machine
// alike.  Its 4 warps take NT tokens of each unit.  A warp has its own ring of key and value tiles in shared memory,
// filled by asynchronous 16-byte copies through the page table and read by ldmatrix, and walks on into the next sequence
// without a pause: scores S = Q K^T by mma.sync (16 query heads to a fragment), running maximum and sum per row, weights
// in registers as the next product's left operand, O += P V.  Where a sequence ends (or the block's run does) the
// 4 warps join their rows in shared memory; a sequence's only block writes the result, others leave (m, l, O) in the
// workspace, which a second kernel joins in the order of the blocks.
//
// Bound by memory: 2 D bytes a token and key-value head are read once and meet 4 G D operations for G query heads.  mma.sync
// covers that: a tile of 16 rows by 16 tokens costs 48 products of 16 x 8 x 16 for 8 KB of cache.
//
// Weights are exponentials relative to the running maximum.  With a 16-bit cache a weight is taken to the product as the
// sum of two 16-bit numbers, as one rounding (2^-9 in bf16) would add as much again to the output's own: the first is cut
// off a little below the weight, so that the second is positive too and an infinite value stays one (with a rest of 0, or
// below it, the two products would make a NaN); together they are within 2^-15 of it (bf16) or 2^-21 (f16).  With an 8-bit
// cache and bf16 outputs a single f16 (2^-11) is well below the output's rounding.  Where weights are f16 all carry a factor
// of 2^15, which the sums share: small ones then keep their bits.
#pragma once

#include <algorithm>

#include "paged.cuh"

namespace w4a8 {

struct AttendParams {
  const void* q;
  const void *k, *v;
  void* out;
  float* lse;
  const int32_t *table, *lens;
  const float *k_scale, *v_scale;
  int64_t q_b, q_h, o_b, o_h;
  int64_t k_page, k_slot, k_head, v_page, v_slot, v_head;  // bytes
  int64_t table_ld, pages, max_len;  // max_len: positions that the table reaches
  int64_t* prefix;                   // [B + 1] units before each sequence
  float2* part_ml;                   // [blocks][2][16 MT]
  float* part_o;                     // [blocks][2][16 MT][D]
  int B, Hq, Hkv, G, D, HB;          // HB: groups of up to 16 MT query heads for a key-value head
  int blocks, window;
  float scale;                       // times log2 e
  FastDiv by_page;
  bool q_f16;
};

int launch_attend_bf16(const AttendParams& p, cudaStream_t st);
int launch_attend_f16(const AttendParams& p, cudaStream_t st);
int launch_attend_fp8(const AttendParams& p, cudaStream_t st);

// The instances: head dimensions up to DT, query heads of a group in MT fragments of 16.
__host__ __device__ constexpr int attend_mt(int DT, int G) { return G > 16 && DT <= 128 ? 2 : 1; }
__host__ __device__ constexpr int attend_dt(int64_t D) { return D <= 64 ? 64 : D <= 128 ? 128 : 256; }
// blocks of a launch at most (their partial results have room for it)
inline int attend_blocks(int DT) { return num_sms() * (DT <= 128 ? 2 : 1); }

namespace {

constexpr int kWarps = 4;
constexpr int kStages = 3;
constexpr float kLn2 = 0.69314718056f;

__device__ unsigned int g_attend_error;

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool there) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(there ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t a) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(a)
               : "memory");
}
__device__ __forceinline__ void ldsm4_t(uint32_t (&r)[4], uint32_t a) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(a)
               : "memory");
}
template <bool BF16>
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  if constexpr (BF16)
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ float exp2_fast(float x) {  // 2 units in the last place, 0 below 2^-126
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
// two E4M3 codes (low half of a 32-bit word) -> f16 pair, exact
__device__ __forceinline__ uint32_t f16x2_of_e4m3x2(uint32_t w) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(static_cast<uint16_t>(w)));
  return r;
}

// kind of a cache: 0 bf16, 1 f16, 2 E4M3 (its operands are f16)
template <int KIND, int DT, int MT>
struct AttendCfg {
  static constexpr bool kFp8 = KIND == 2, kBf16 = KIND == 0;
  static constexpr int kSize = kFp8 ? 1 : 2;
  static constexpr int kRow = DT * kSize;               // bytes of a token's row in a tile
  static constexpr int NT = kFp8 || DT == 64 ? 32 : 16;  // tokens of a tile
  static constexpr int kTile = NT * kRow;
  static constexpr int kStage = 2 * kTile;              // keys, values
  static constexpr int kRows = 16 * MT;
  static constexpr float kShift = kBf16 ? 0.f : 15.f;   // weights are 2^kShift times the exponentials
  static constexpr int kQRow = DT * 2 + 16;             // padded: 8 rows at one column lie in different banks
  static constexpr int kOffQ = kWarps * kStages * kStage;
  static constexpr int kOffRow = kOffQ + kRows * kQRow;       // fp32 [rows]: factor of a row's scores
  static constexpr int kOffMl = kOffRow + kRows * 4;          // float2 [warps][rows]
  static constexpr int kSmem = kOffMl + kWarps * kRows * 8;
  static constexpr int kBlocks = DT <= 128 ? 2 : 1;     // of an SM
  static_assert((kSmem + 2048) * kBlocks <= 228 * 1024, "shared memory");
  static_assert(kStage >= 16 * DT * 4, "16 rows of fp32 sums in a ring slot");
  // place of 16-byte chunk c of row r: chunks are exchanged within 128 bytes so that 8 rows at one column lie in
  // different banks
  static __device__ __forceinline__ uint32_t at(int r, int c) {
    if constexpr (kRow >= 128)
      return static_cast<uint32_t>(r * kRow + ((c ^ (r & 7)) << 4));
    else
      return static_cast<uint32_t>(r * kRow + ((c ^ ((r >> 1) & 3)) << 4));
  }
};

// Sequence b's tokens and units.
struct SeqSpan {
  int lo, hi, units;
};
template <int UNIT>
__device__ __forceinline__ SeqSpan span_of(const AttendParams& p, int b) {
  SeqSpan s;
  const int64_t len = p.lens[b];
  if (len > p.max_len) atomicOr(&g_attend_error, 2u);
  s.hi = static_cast<int>(min(len, p.max_len));
  s.lo = p.window > 0 ? max(0, s.hi - p.window) : 0;
  s.units = s.hi > s.lo ? (s.hi - s.lo + UNIT - 1) / UNIT : 0;
  return s;
}

// A place in the list of units.
struct Cursor {
  int b, hh, u;  // sequence, head and group of query heads, unit
  SeqSpan s;
};

template <int KIND, int DT, int MT>
__global__ void __launch_bounds__(kWarps * 32, AttendCfg<KIND, DT, MT>::kBlocks)
    paged_attention_kernel(const __grid_constant__ AttendParams p) {
  using C = AttendCfg<KIND, DT, MT>;
  constexpr int NT = C::NT, UNIT = kWarps * NT;
  constexpr bool kFp8 = C::kFp8;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ int64_t chunk_sum[kWarps * 32 + 1];  // units before the sequences of each thread
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  pdl_trigger();
  pdl_wait();

  // units before each run of sequences; the first block leaves those of every sequence for the second kernel
  const int HH = p.Hkv * p.HB, per = (p.B + kWarps * 32 - 1) / (kWarps * 32);
  int64_t mine = 0;
  for (int b = tid * per; b < min(p.B, (tid + 1) * per); ++b) mine += static_cast<int64_t>(span_of<UNIT>(p, b).units) * HH;
  {
    int64_t up = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t x = __shfl_up_sync(0xffffffffu, up, o);
      if (lane >= o) up += x;
    }
    chunk_sum[tid + 1] = up;
    if (tid == 0) chunk_sum[0] = 0;
    __syncthreads();
    int64_t before = 0;
    for (int w = 0; w < warp; ++w) before += chunk_sum[(w + 1) * 32];
    __syncthreads();
    chunk_sum[tid + 1] = up + before;
    if (blockIdx.x == 0) {
      int64_t at = up + before - mine;
      for (int b = tid * per; b < min(p.B, (tid + 1) * per); ++b) {
        p.prefix[b] = at;
        at += static_cast<int64_t>(span_of<UNIT>(p, b).units) * HH;
      }
      if (tid == kWarps * 32 - 1) p.prefix[p.B] = up + before;
    }
    __syncthreads();
  }
  const int64_t total = chunk_sum[kWarps * 32];
  const int64_t runs = min(total, static_cast<int64_t>(p.blocks));  // blocks with work: each has a unit at least
  if (blockIdx.x >= runs) return;
  const int64_t start = blockIdx.x * total / runs, stop = (blockIdx.x + 1) * total / runs;
  const int count = static_cast<int>(stop - start);

  Cursor here;  // of the unit that is computed next
  {
    int c = 0;  // the last thread whose sequences begin at or before start
#pragma unroll
    for (int step = kWarps * 16; step > 0; step >>= 1)
      if (chunk_sum[c + step] <= start) c += step;
    int64_t at = chunk_sum[c];
    here.b = c * per;
    here.s = span_of<UNIT>(p, here.b);
    while (at + static_cast<int64_t>(here.s.units) * HH <= start) {
      at += static_cast<int64_t>(here.s.units) * HH;
      here.s = span_of<UNIT>(p, ++here.b);
    }
    const int64_t in = start - at;
    here.hh = static_cast<int>(in / here.s.units);
    here.u = static_cast<int>(in - static_cast<int64_t>(here.hh) * here.s.units);
  }
  const auto advance = [&](Cursor& c) {
    if (++c.u < c.s.units) return;
    c.u = 0;
    if (++c.hh < HH) return;
    c.hh = 0;
    do {
      if (++c.b >= p.B) return;
      c.s = span_of<UNIT>(p, c.b);
    } while (c.s.units == 0);
  };

  const uint32_t ring = smem_u32(smem) + warp * kStages * C::kStage;
  constexpr int kChunks = C::kRow / 16, kRowsPer = 32 / kChunks > 0 ? 32 / kChunks : 1;  // rows of one copy by the warp
  static_assert(kChunks <= 32, "a warp copies whole rows");
  // The page of this lane's token of a unit (-1: none), one unit ahead of its copies.
  const auto page_of = [&](const Cursor& c, int& slot) {
    const int t = c.s.lo + c.u * UNIT + warp * NT + (lane & (NT - 1));
    int page = -1;
    slot = 0;
    if (t < c.s.hi) {
      const int n = p.by_page.div(t, slot);
      page = p.table[c.b * p.table_ld + n];
      if (page < 0 || page >= p.pages) {
        atomicOr(&g_attend_error, 2u);
        page = -1;
      }
    }
    return page;
  };
  const auto copy_unit = [&](int hh, int page, int slot, int stage) {
    const int h = hh / p.HB;
    const int64_t k_at = page < 0 ? -1 : page * p.k_page + slot * p.k_slot + h * p.k_head;
    const int64_t v_at = page < 0 ? -1 : page * p.v_page + slot * p.v_slot + h * p.v_head;
    const int c = lane % kChunks, r0 = lane / kChunks;
    const bool in_row = c * 16 < p.D * C::kSize;
    const uint32_t kt = ring + stage * C::kStage, vt = kt + C::kTile;
    const char *k = static_cast<const char*>(p.k) + c * 16, *v = static_cast<const char*>(p.v) + c * 16;
#pragma unroll
    for (int r = 0; r < NT; r += kRowsPer) {
      const int64_t ka = __shfl_sync(0xffffffffu, k_at, r + r0), va = __shfl_sync(0xffffffffu, v_at, r + r0);
      const bool there = in_row && ka >= 0;
      const uint32_t to = C::at(r + r0, c);
      cp_async16(kt + to, there ? k + ka : static_cast<const char*>(p.k), there);
      cp_async16(vt + to, there ? v + va : static_cast<const char*>(p.v), there);
    }
  };

  // fill the ring: kStages - 1 units on their way, the next one's pages known
  Cursor ahead = here;
  int issued = 0, page, slot;
  page = page_of(ahead, slot);
  int ahead_hh = ahead.hh;
#pragma unroll
  for (int i = 0; i < kStages - 1; ++i) {
    if (issued < count) {
      copy_unit(ahead_hh, page, slot, i);
      if (++issued < count) {
        advance(ahead);
        ahead_hh = ahead.hh;
        page = page_of(ahead, slot);
      }
    }
    cp_async_commit();
  }

  constexpr int kNt = DT / 8;  // column fragments of O
  float o[MT][kNt][4], m[MT][2], l[MT][2];
  const int g = lane >> 2, j2 = (lane & 3) * 2;
  const uint32_t q_s = smem_u32(smem) + C::kOffQ;
  float* row_scale = reinterpret_cast<float*>(smem + C::kOffRow);
  float2* join_ml = reinterpret_cast<float2*>(smem + C::kOffMl);

  int done = 0, stage = 0;
  while (done < count) {
    // --- a run of units of one sequence and head ---
    const int run = min(here.s.units - here.u, count - done);
    const bool whole = run == here.s.units;
    const int h = here.hh / p.HB, head0 = h * p.G + (here.hh % p.HB) * C::kRows;
    const int live = min(C::kRows, (h + 1) * p.G - head0);  // query heads of this group
    __syncthreads();  // nobody reads the last run's queries or rows any more
    {
      const float ks = kFp8 && p.k_scale ? p.k_scale[h] : 1.f;
      for (int r = warp; r < C::kRows; r += kWarps) {
        const uint16_t* src = static_cast<const uint16_t*>(p.q) + here.b * p.q_b + (head0 + r) * p.q_h;
        uint16_t* dst = reinterpret_cast<uint16_t*>(smem + C::kOffQ + r * C::kQRow);
        uint16_t e[DT / 32];
#pragma unroll
        for (int i = 0; i < DT / 32; ++i) e[i] = r < live && lane + 32 * i < p.D ? src[lane + 32 * i] : 0;
        float factor = 1.f;
        if constexpr (kFp8) {
          // f16 operands: a bf16 row is scaled by a power of two so that its largest element lies in [2^14, 2^15), where
          // elements down to 2^-29 of it stay exact
          if (!p.q_f16) {
            float top = 0.f;
#pragma unroll
            for (int i = 0; i < DT / 32; ++i) top = fmaxf(top, fabsf(bf16_bits_to_float(e[i])));
            top = warp_max(top);
            const int ex = static_cast<int>(__float_as_uint(top) >> 23) - 127;
            // powers of two beyond fp32's range (tiny rows) are capped; infinities keep their place
            const int by = top > 0.f && ex < 128 ? min(14 - ex, 126) : 0;
            const float up = __uint_as_float(static_cast<uint32_t>(by + 127) << 23);
            factor = __uint_as_float(static_cast<uint32_t>(127 - by) << 23);
#pragma unroll
            for (int i = 0; i < DT / 32; ++i) e[i] = __half_as_ushort(__float2half_rn(bf16_bits_to_float(e[i]) * up));
          }
#pragma unroll
          for (int i = 0; i < DT / 32; ++i) {
            // the order of d within 16 in which a key's codes come out of ldmatrix: four neighbours to a lane
            const int d = lane + 32 * i, in = d & 15, to = (in >> 2) * 2 + (in & 1) + ((in & 2) << 2);
            dst[(d & ~15) + to] = e[i];
          }
        } else {
#pragma unroll
          for (int i = 0; i < DT / 32; ++i) dst[lane + 32 * i] = e[i];
        }
        if (lane == 0) row_scale[r] = factor * p.scale * ks;
      }
    }
    __syncthreads();
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
#pragma unroll
      for (int i = 0; i < kNt; ++i)
#pragma unroll
        for (int x = 0; x < 4; ++x) o[mt][i][x] = 0.f;
      m[mt][0] = m[mt][1] = -INFINITY;
      l[mt][0] = l[mt][1] = 0.f;
    }

    for (int i = 0; i < run; ++i) {
      if (issued < count) {
        int to = stage + kStages - 1;
        if (to >= kStages) to -= kStages;
        copy_unit(ahead_hh, page, slot, to);
        if (++issued < count) {
          advance(ahead);
          ahead_hh = ahead.hh;
          page = page_of(ahead, slot);
        }
      }
      cp_async_commit();
      cp_async_wait<kStages - 1>();
      __syncwarp();
      const uint32_t kt = ring + stage * C::kStage, vt = kt + C::kTile;
      if (++stage == kStages) stage = 0;
      const int left = here.s.hi - (here.s.lo + (here.u + i) * UNIT + warp * NT);  // tokens of this tile
      if (left > 0) {
        // scores
        float s[MT][NT / 8][4];
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
          for (int n = 0; n < NT / 8; ++n)
#pragma unroll
            for (int x = 0; x < 4; ++x) s[mt][n][x] = 0.f;
        if constexpr (!kFp8) {
#pragma unroll
          for (int kk = 0; kk < DT / 16; ++kk) {
            uint32_t a[MT][4];
#pragma unroll
            for (int mt = 0; mt < MT; ++mt)
              ldsm4(a[mt], q_s + (mt * 16 + (lane & 15)) * C::kQRow + kk * 32 + (lane >> 4) * 16);
#pragma unroll
            for (int n = 0; n < NT / 16; ++n) {
              uint32_t b[4];  // tokens 0-7 and 8-15, d 0-7 and 8-15 each
              ldsm4(b, kt + C::at(n * 16 + (lane & 7) + ((lane >> 4) << 3), kk * 2 + ((lane >> 3) & 1)));
#pragma unroll
              for (int mt = 0; mt < MT; ++mt) {
                mma16816<C::kBf16>(s[mt][2 * n], a[mt], b[0], b[1]);
                mma16816<C::kBf16>(s[mt][2 * n + 1], a[mt], b[2], b[3]);
              }
            }
          }
        } else {
#pragma unroll
          for (int kk = 0; kk < DT / 32; ++kk) {
            uint32_t a[2][MT][4];
#pragma unroll
            for (int x = 0; x < 2; ++x)
#pragma unroll
              for (int mt = 0; mt < MT; ++mt)
                ldsm4(a[x][mt], q_s + (mt * 16 + (lane & 15)) * C::kQRow + (2 * kk + x) * 32 + (lane >> 4) * 16);
#pragma unroll
            for (int n = 0; n < NT / 16; ++n) {
              uint32_t b[4];  // tokens 0-7 and 8-15, d 0-15 and 16-31 each
              ldsm4(b, kt + C::at(n * 16 + (lane & 7) + ((lane >> 4) << 3), kk * 2 + ((lane >> 3) & 1)));
#pragma unroll
              for (int x = 0; x < 4; ++x) {
                const uint32_t b0 = f16x2_of_e4m3x2(b[x]), b1 = f16x2_of_e4m3x2(b[x] >> 16);
#pragma unroll
                for (int mt = 0; mt < MT; ++mt) mma16816<false>(s[mt][2 * n + (x >> 1)], a[x & 1][mt], b0, b1);
              }
            }
          }
        }
        // running maximum and sum, weights
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
          const float f0 = row_scale[mt * 16 + g], f1 = row_scale[mt * 16 + g + 8];
          float top0 = m[mt][0], top1 = m[mt][1];
#pragma unroll
          for (int n = 0; n < NT / 8; ++n) {
#pragma unroll
            for (int x = 0; x < 2; ++x) {
              const bool in = n * 8 + j2 + x < left;
              s[mt][n][x] = in ? s[mt][n][x] * f0 : -INFINITY;
              s[mt][n][2 + x] = in ? s[mt][n][2 + x] * f1 : -INFINITY;
              top0 = fmaxf(top0, s[mt][n][x]);
              top1 = fmaxf(top1, s[mt][n][2 + x]);
            }
          }
          top0 = fmaxf(top0, __shfl_xor_sync(0xffffffffu, top0, 1));
          top1 = fmaxf(top1, __shfl_xor_sync(0xffffffffu, top1, 1));
          top0 = fmaxf(top0, __shfl_xor_sync(0xffffffffu, top0, 2));
          top1 = fmaxf(top1, __shfl_xor_sync(0xffffffffu, top1, 2));
          const float base0 = top0 == -INFINITY ? 0.f : top0, base1 = top1 == -INFINITY ? 0.f : top1;
          if (__any_sync(0xffffffffu, top0 > m[mt][0] || top1 > m[mt][1])) {
            const float c0 = exp2_fast(m[mt][0] - base0), c1 = exp2_fast(m[mt][1] - base1);
            l[mt][0] *= c0;
            l[mt][1] *= c1;
#pragma unroll
            for (int n = 0; n < kNt; ++n) {
              o[mt][n][0] *= c0;
              o[mt][n][1] *= c0;
              o[mt][n][2] *= c1;
              o[mt][n][3] *= c1;
            }
            m[mt][0] = top0;
            m[mt][1] = top1;
          }
#pragma unroll
          for (int n = 0; n < NT / 8; ++n)
#pragma unroll
            for (int x = 0; x < 2; ++x) {
              s[mt][n][x] = exp2_fast(s[mt][n][x] - base0 + C::kShift);
              s[mt][n][2 + x] = exp2_fast(s[mt][n][2 + x] - base1 + C::kShift);
              l[mt][0] += s[mt][n][x];
              l[mt][1] += s[mt][n][2 + x];
            }
        }
        // O += P V, 16 tokens at a time
        const bool split = !kFp8 || p.q_f16;
#pragma unroll
        for (int n = 0; n < NT / 16; ++n) {
          uint32_t hi[MT][4], lo[MT][4];
#pragma unroll
          for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int x = 0; x < 4; ++x) {
              const float* w = &s[mt][2 * n + (x >> 1)][(x & 1) * 2];
              if constexpr (C::kBf16) {
                const uint32_t c0 = __float_as_uint(w[0] * (1.f - 0x1p-8f)), c1 = __float_as_uint(w[1] * (1.f - 0x1p-8f));
                hi[mt][x] = prmt(c0, c1, 0x7632);
                lo[mt][x] = pack2<__nv_bfloat16>(w[0] - __uint_as_float(c0 & 0xFFFF0000u),
                                                 w[1] - __uint_as_float(c1 & 0xFFFF0000u));
              } else if (split) {
                const __half2 c = __halves2half2(__float2half_rz(w[0] * (1.f - 0x1p-10f)),
                                                 __float2half_rz(w[1] * (1.f - 0x1p-10f)));
                hi[mt][x] = *reinterpret_cast<const uint32_t*>(&c);
                lo[mt][x] = pack2<__half>(w[0] - __low2float(c), w[1] - __high2float(c));
              } else {
                hi[mt][x] = pack2<__half>(w[0], w[1]);
              }
            }
          if constexpr (!kFp8) {
#pragma unroll
            for (int c = 0; c < DT / 16; ++c) {
              uint32_t b[4];  // d 0-7: tokens 0-7 and 8-15; d 8-15 likewise
              ldsm4_t(b, vt + C::at(n * 16 + (lane & 15), 2 * c + (lane >> 4)));
#pragma unroll
              for (int mt = 0; mt < MT; ++mt) {
                mma16816<C::kBf16>(o[mt][2 * c], hi[mt], b[0], b[1]);
                mma16816<C::kBf16>(o[mt][2 * c + 1], hi[mt], b[2], b[3]);
                mma16816<C::kBf16>(o[mt][2 * c], lo[mt], b[0], b[1]);
                mma16816<C::kBf16>(o[mt][2 * c + 1], lo[mt], b[2], b[3]);
              }
            }
          } else {
#pragma unroll
            for (int c = 0; c < DT / 32; ++c) {
              uint32_t b[4];  // d 0-15: tokens 0-7 and 8-15; d 16-31 likewise; each word two tokens of two neighbours
              ldsm4_t(b, vt + C::at(n * 16 + (lane & 15), 2 * c + (lane >> 4)));
#pragma unroll
              for (int x = 0; x < 2; ++x) {
                const uint32_t w0 = prmt(b[2 * x], 0, 0x3120), w1 = prmt(b[2 * x + 1], 0, 0x3120);
                const uint32_t e0 = f16x2_of_e4m3x2(w0), e1 = f16x2_of_e4m3x2(w1);
                const uint32_t d0 = f16x2_of_e4m3x2(w0 >> 16), d1 = f16x2_of_e4m3x2(w1 >> 16);
#pragma unroll
                for (int mt = 0; mt < MT; ++mt) {  // even and odd d
                  mma16816<false>(o[mt][4 * c + 2 * x], hi[mt], e0, e1);
                  mma16816<false>(o[mt][4 * c + 2 * x + 1], hi[mt], d0, d1);
                  if (split) {
                    mma16816<false>(o[mt][4 * c + 2 * x], lo[mt], e0, e1);
                    mma16816<false>(o[mt][4 * c + 2 * x + 1], lo[mt], d0, d1);
                  }
                }
              }
            }
          }
        }
      }
      __syncwarp();  // the tile's slot is free
    }

    // --- join the warps: rows brought to the common maximum, added up in the order (0 + 2) + (1 + 3) ---
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        l[mt][x] += __shfl_xor_sync(0xffffffffu, l[mt][x], 1);
        l[mt][x] += __shfl_xor_sync(0xffffffffu, l[mt][x], 2);
        if ((lane & 3) == 0) join_ml[warp * C::kRows + mt * 16 + g + 8 * x] = make_float2(m[mt][x], l[mt][x]);
      }
    __syncthreads();
    float top[MT][2], sum[MT][2];
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        float2 ml[kWarps];
        float t = -INFINITY;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
          ml[w] = join_ml[w * C::kRows + mt * 16 + g + 8 * x];
          t = fmaxf(t, ml[w].x);
        }
        const float base = t == -INFINITY ? 0.f : t;
        float r = 0.f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) r += ml[w].y * exp2_fast(ml[w].x - base);
        const float c = exp2_fast(m[mt][x] - base);
#pragma unroll
        for (int n = 0; n < kNt; ++n) {
          o[mt][n][2 * x] *= c;
          o[mt][n][2 * x + 1] *= c;
        }
        top[mt][x] = t;
        sum[mt][x] = r;
      }
    // Through the slot that the sender read last: its next copy is issued behind the next run's first barrier.
    const int last = stage == 0 ? kStages - 1 : stage - 1;
    const auto exchange = [&](int from, int mt, bool take) {
      float2* buf = reinterpret_cast<float2*>(smem + (from * kStages + last) * C::kStage) + lane;
#pragma unroll
      for (int n = 0; n < kNt; ++n)
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          float2* at = buf + (n * 2 + x) * 32;
          if (take) {
            const float2 v = *at;
            o[mt][n][2 * x] += v.x;
            o[mt][n][2 * x + 1] += v.y;
          } else {
            *at = make_float2(o[mt][n][2 * x], o[mt][n][2 * x + 1]);
          }
        }
    };
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
      if (mt > 0) __syncthreads();
      if (warp >= 2) exchange(warp, mt, false);
      __syncthreads();
      if (warp < 2) exchange(warp + 2, mt, true);
      if (warp == 1) exchange(1, mt, false);
      __syncthreads();
      if (warp == 0) exchange(1, mt, true);
    }
    if (warp == 0) {
      const int slot_of = done == 0 ? 0 : 1;
      const int64_t part = (static_cast<int64_t>(blockIdx.x) * 2 + slot_of) * C::kRows;
      const float vs = kFp8 && p.v_scale ? p.v_scale[h] : 1.f;
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          const int r = mt * 16 + g + 8 * x;
          if (r >= live) continue;
          const float inv = sum[mt][x] == 0.f ? 0.f : vs / sum[mt][x];
          if ((lane & 3) == 0) {
            if (whole) {
              if (p.lse)
                p.lse[static_cast<int64_t>(here.b) * p.Hq + head0 + r] =
                    sum[mt][x] == 0.f ? -INFINITY : (top[mt][x] - C::kShift + log2f(sum[mt][x])) * kLn2;
            } else {
              p.part_ml[part + r] = make_float2(top[mt][x], sum[mt][x]);
            }
          }
          const int64_t out = here.b * p.o_b + (head0 + r) * p.o_h;
#pragma unroll
          for (int n = 0; n < kNt; ++n)
#pragma unroll
            for (int y = 0; y < 2; ++y) {
              // with E4M3 the fragments hold even and odd columns of 16
              const int d = kFp8 ? (n >> 1) * 16 + 2 * (j2 + y) + (n & 1) : n * 8 + j2 + y;
              const float val = o[mt][n][2 * x + y];
              if (d >= p.D) continue;
              if (!whole)
                p.part_o[(part + r) * p.D + d] = val;
              else if (C::kBf16 || (kFp8 && !p.q_f16))
                static_cast<__nv_bfloat16*>(p.out)[out + d] = __float2bfloat16_rn(val * inv);
              else
                static_cast<__half*>(p.out)[out + d] = __float2half_rn(val * inv);
            }
        }
    }
    done += run;
    here.u += run - 1;
    if (done < count) advance(here);
  }
}

// Joins the parts of what several blocks computed: a block for (sequence, head, group), its threads as [parts'
// turns][rows][columns in fours].  Empty sequences get zeros here.
constexpr int kJoinThreads = 256;
template <int KIND, int DT, int MT>
__global__ void __launch_bounds__(kJoinThreads) paged_attention_join_kernel(const __grid_constant__ AttendParams p) {
  using C = AttendCfg<KIND, DT, MT>;
  pdl_trigger();
  pdl_wait();
  const int HH = p.Hkv * p.HB;
  const int64_t item = blockIdx.x;
  const int b = static_cast<int>(item / HH), hh = static_cast<int>(item - static_cast<int64_t>(b) * HH);
  const int64_t first = p.prefix[b], units = (p.prefix[b + 1] - first) / HH, total = p.prefix[p.B];
  const int h = hh / p.HB, head0 = h * p.G + (hh % p.HB) * C::kRows;
  const int live = min(C::kRows, (h + 1) * p.G - head0);
  const bool bf16 = C::kBf16 || (C::kFp8 && !p.q_f16);
  const auto store = [&](int r, int d, float v) {
    const int64_t at = b * p.o_b + (head0 + r) * p.o_h + d;
    if (bf16)
      static_cast<__nv_bfloat16*>(p.out)[at] = __float2bfloat16_rn(v);
    else
      static_cast<__half*>(p.out)[at] = __float2half_rn(v);
  };
  if (units == 0) {
    for (int i = threadIdx.x; i < live * p.D; i += kJoinThreads) store(i / p.D, i % p.D, 0.f);
    if (p.lse)
      for (int r = threadIdx.x; r < live; r += kJoinThreads) p.lse[static_cast<int64_t>(b) * p.Hq + head0 + r] = -INFINITY;
    return;
  }
  const int64_t i0 = first + hh * units, i1 = i0 + units;
  const int64_t runs = min(total, static_cast<int64_t>(p.blocks));
  // the block that has unit t: start(c) = floor(c total / runs) <= t < start(c + 1)
  const int c0 = static_cast<int>(((i0 + 1) * runs - 1) / total), c1 = static_cast<int>((i1 * runs - 1) / total);
  if (c0 == c1) return;  // written by its only block
  const bool starts = c0 * total / runs == i0;  // the first part is its block's first run
  const float vs = C::kFp8 && p.v_scale ? p.v_scale[h] : 1.f;
  for (int i = threadIdx.x; i < live * (p.D / 4); i += kJoinThreads) {
    const int r = i / (p.D / 4), d = i % (p.D / 4) * 4;
    float top = -INFINITY, sum = 0.f;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int c = c0; c <= c1; ++c) {
      const int64_t part = (static_cast<int64_t>(c) * 2 + (c == c0 && !starts ? 1 : 0)) * C::kRows + r;
      const float2 ml = p.part_ml[part];
      const float4 v = *reinterpret_cast<const float4*>(p.part_o + part * p.D + d);
      const float t = fmaxf(top, ml.x), base = t == -INFINITY ? 0.f : t;
      const float old = exp2_fast(top - base), now = exp2_fast(ml.x - base);
      sum = sum * old + ml.y * now;
      acc.x = acc.x * old + v.x * now;
      acc.y = acc.y * old + v.y * now;
      acc.z = acc.z * old + v.z * now;
      acc.w = acc.w * old + v.w * now;
      top = t;
    }
    const float inv = sum == 0.f ? 0.f : vs / sum;
    store(r, d, acc.x * inv);
    store(r, d + 1, acc.y * inv);
    store(r, d + 2, acc.z * inv);
    store(r, d + 3, acc.w * inv);
    if (p.lse && d == 0)
      p.lse[static_cast<int64_t>(b) * p.Hq + head0 + r] = sum == 0.f ? -INFINITY : (top - C::kShift + log2f(sum)) * kLn2;
  }
}

template <int KIND, int DT, int MT>
int launch_attend(AttendParams p, cudaStream_t st) {
  using C = AttendCfg<KIND, DT, MT>;
  static DeviceOnce once;
  if (int rc = once.run([] {
        return cudaFuncSetAttribute(paged_attention_kernel<KIND, DT, MT>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                    C::kSmem) == cudaSuccess
                   ? static_cast<int>(W4A8_OK)
                   : check_launch("cudaFuncSetAttribute(paged_attention)");
      }))
    return rc;
  p.HB = static_cast<int>(ceil_div(p.G, C::kRows));
  p.blocks = num_sms() * C::kBlocks;
  if (int rc = launch_pdl("paged_attention_kernel", paged_attention_kernel<KIND, DT, MT>, dim3(p.blocks),
                          dim3(kWarps * 32), C::kSmem, st, p))
    return rc;
  return launch_pdl("paged_attention_join_kernel", paged_attention_join_kernel<KIND, DT, MT>,
                    dim3(static_cast<unsigned>(static_cast<int64_t>(p.B) * p.Hkv * p.HB)), dim3(kJoinThreads), 0, st, p);
}

template <int KIND>
int launch_attend_kind(const AttendParams& p, cudaStream_t st) {
  switch (attend_dt(p.D)) {
    case 64: return attend_mt(64, p.G) == 2 ? launch_attend<KIND, 64, 2>(p, st) : launch_attend<KIND, 64, 1>(p, st);
    case 128: return attend_mt(128, p.G) == 2 ? launch_attend<KIND, 128, 2>(p, st) : launch_attend<KIND, 128, 1>(p, st);
    default: return launch_attend<KIND, 256, 1>(p, st);
  }
}

int read_attend_error() {
  unsigned int v = 0;
  cudaMemcpyFromSymbol(&v, g_attend_error, sizeof(v));
  const unsigned int zero = 0;
  cudaMemcpyToSymbol(g_attend_error, &zero, sizeof(zero));
  return static_cast<int>(v);
}

struct AttendRegistrar {
  AttendRegistrar() { register_device_error_reader(&read_attend_error); }
} attend_registrar;

}  // namespace

}  // namespace w4a8
