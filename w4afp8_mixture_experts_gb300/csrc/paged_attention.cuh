// paged_attention_decode: one query token per sequence against its cached keys and values.
//
// The work is a list of tiles: NT neighbouring tokens of one sequence for one key-value head and up to 16 * MT of its query
// heads, through all sequences, heads and tiles in order.  A launch has as many warps as stay resident, and each takes an
// equal run of the list, so that long and short sequences fill the machine alike; the start of an item (a sequence's head)
// counts as kExtra tiles.  A warp works by itself: it has a ring of key and value tiles in shared memory, filled by
// asynchronous 16-byte copies through the page table and read by ldmatrix, and its copies run on into the next item while it
// finishes one: scores S = Q K^T by mma.sync (16 query heads to a fragment), running maximum and sum per row, weights in
// registers as the next product's left operand, O += P V.  What a warp has whole it writes; of an item that several warps
// share each leaves (m, l, O) in the workspace, and a second kernel joins them in the warps' order.
//
// (Blocks whose 4 warps shared a run, joined in shared memory at each item's end: 4.5 us an item, 39 us for 32 sequences of
// up to 1024 tokens, whose bytes take 10.)
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

// An item of the list: its sequence, head and group, its first place and its places.
struct RunStart {
  int64_t first, each;
  int b, hh;
};

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
  int64_t* prefix;                   // [B + 1] places in the list before each sequence (the last: all of them)
  RunStart* starts;                  // [warps] the item in which each run starts
  float2* part_ml;                   // [warps][2][16 MT]
  float* part_o;                     // [warps][2][16 MT][D]
  int B, Hq, Hkv, G, D, HB;          // HB: groups of up to 16 MT query heads for a key-value head
  int warps, window;
  int cluster;                       // blocks of a cluster that shares an item (0: the list)
  bool by_rows;                      // the second kernel goes by rows, through `prefix`; else by the runs' starts
  float scale;                       // times log2 e
  FastDiv by_page;
  bool q_vec, out_pair;  // 16-byte loads of q, 4-byte stores of out
};

int launch_attend_bf16(const AttendParams& p, cudaStream_t st);
int launch_attend_f16(const AttendParams& p, cudaStream_t st);
int launch_attend_fp8(const AttendParams& p, bool q_f16, cudaStream_t st);

// The instances: head dimensions up to DT, query heads of a group in MT fragments of 16.
__host__ __device__ constexpr int attend_mt(int DT, int G) { return G > 16 && DT <= 128 ? 2 : 1; }
__host__ __device__ constexpr int attend_dt(int64_t D) { return D <= 64 ? 64 : D <= 128 ? 128 : 256; }
__host__ __device__ constexpr int attend_tile(bool fp8, int DT) { return fp8 || DT == 64 ? 32 : 16; }  // tokens of a tile
constexpr int kAttendWarps = 4;  // of a block
inline int attend_warps(int DT) { return num_sms() * (DT <= 128 ? 2 : 1) * kAttendWarps; }  // of a launch

namespace {

constexpr int kWarps = kAttendWarps;
constexpr int kExtra = 1;
constexpr float kLn2 = 0.69314718056f;

__device__ unsigned int g_attend_error;

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool there) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(there ? 16 : 0) : "memory");
}
__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t a) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(a));
}
__device__ __forceinline__ void ldsm4_t(uint32_t (&r)[4], uint32_t a) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(a));
}
template <bool BF16>
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  if constexpr (BF16)
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ float exp2_fast(float x) {  // 2 units in the last place, 0 below 2^-126
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
// four E4M3 codes -> two f16 pairs, exact
__device__ __forceinline__ void f16x4_of_e4m3x4(uint32_t w, uint32_t& lo, uint32_t& hi) {
  asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, l;\n\tcvt.rn.f16x2.e4m3x2 %1, h;\n\t}"
      : "=r"(lo), "=r"(hi)
      : "r"(w));
}

// kind of cache and queries: 0 bf16, 1 f16, 2 E4M3 and bf16, 3 E4M3 and f16 (products of E4M3 are taken in f16)
template <int KIND, int DT, int MT>
struct AttendCfg {
  static constexpr bool kFp8 = KIND >= 2, kBf16 = KIND == 0;
  static constexpr bool kBf16Out = KIND == 0 || KIND == 2, kSplit = KIND != 2;  // weights in two pieces
  static constexpr int kSize = kFp8 ? 1 : 2;
  static constexpr int kRow = DT * kSize;               // bytes of a token's row in a tile
  static constexpr int NT = attend_tile(kFp8, DT);      // (E4M3, 16 tokens and 6 slots: 102 -> 128 us)
  static constexpr int kTile = NT * kRow;
  static constexpr int kStage = 2 * kTile;              // keys, values
  static constexpr int kStages = MT == 2 && kStage == 8192 ? 2 : 3;
  // Whether the next tile's scores are computed beside this one's values: two independent rows of products, but the tile has
  // to be there earlier.  64 sequences of up to 8192 tokens, bf16: 184 us without, 181 with it; E4M3: 102 and 110.
  static constexpr bool kPipe = kStages >= 3 && !kFp8;
  static constexpr int kRows = 16 * MT;
  static constexpr float kShift = kBf16 ? 0.f : 15.f;   // weights are 2^kShift times the exponentials
  static constexpr int kQRow = DT * 2;
  static constexpr int kOffQ = kStages * kStage;        // of a warp
  static constexpr int kOffScale = kOffQ + kRows * kQRow;  // fp32 [rows]: factor of a row's scores
  static constexpr int kWarpBytes = kOffScale + 128;
  // a warp's part for its cluster: fp32 rows, padded so that 8 of them lie in different banks, over the ring (and the
  // queries); maxima and sums at the queries' end
  static constexpr int kJoinRow = DT + 8, kOffMl = kOffScale - kRows * 8;
  static_assert(kRows * kJoinRow * 4 <= kOffMl, "room for the part");
  static constexpr int kSmem = kWarps * kWarpBytes;
  static constexpr int kBlocks = DT <= 128 ? 2 : 1;     // of an SM
  static_assert((kSmem + 1024) * kBlocks <= 228 * 1024, "shared memory");
  static_assert(kWarpBytes % 128 == 0 && kRows * 4 <= 128, "tiles on 128 bytes");
  // place of 16-byte chunk c of row r: chunks are exchanged within 128 bytes so that 8 rows at one column lie in
  // different banks
  static __device__ __forceinline__ uint32_t at(int r, int c) {
    if constexpr (kRow >= 128)
      return static_cast<uint32_t>(r * kRow + ((c ^ (r & 7)) << 4));
    else
      return static_cast<uint32_t>(r * kRow + ((c ^ ((r >> 1) & 3)) << 4));
  }
  static __device__ __forceinline__ uint32_t q_at(int r, int c) { return static_cast<uint32_t>(r * kQRow + ((c ^ (r & 7)) << 4)); }
};

// Sequence b's tokens and tiles.  Of a sequence longer than its table the positions behind it are left out; a window lies
// before the length all the same.  CHECK: such a length is reported (not where lengths are only added up: loads wait for
// such a branch).
struct SeqSpan {
  int lo, hi, tiles;
};
template <int NT, bool CHECK = true>
__device__ __forceinline__ SeqSpan span_of(const AttendParams& p, int b) {
  SeqSpan s;
  const int64_t len = p.lens[b];
  if (CHECK && len > p.max_len) atomicOr(&g_attend_error, 2u);
  s.hi = static_cast<int>(min(len, p.max_len));
  s.lo = p.window > 0 ? static_cast<int>(max(static_cast<int64_t>(0), len - p.window)) : 0;
  // the last tile of a sequence may end behind 2^31: unsigned
  s.tiles = s.hi > s.lo ? static_cast<int>((static_cast<uint32_t>(s.hi - s.lo) + (NT - 1)) / NT) : 0;
  return s;
}
// places of a sequence in the list
__device__ __forceinline__ int64_t places_of(const SeqSpan& s, int HH) {
  return s.tiles ? static_cast<int64_t>(s.tiles + kExtra) * HH : 0;
}
// Warps with work: each has a place at least.  The run of warp w is [w total / runs, (w + 1) total / runs), and the warp
// that has place t is floor(((t + 1) runs - 1) / total).
__device__ __forceinline__ int64_t runs_of(const AttendParams& p, int64_t total) {
  return min(total, static_cast<int64_t>(p.warps));
}

// A tile in the list, and how many places the run has from it on.
struct Cursor {
  int b, hh, u;  // sequence, head and group of query heads, tile
  SeqSpan s;
  int left;
};

// Two fp32 columns of a row of the output; `pair`: in one store.
__device__ __forceinline__ void store_out(void* out, int64_t at, float x, float y, bool bf16, bool pair) {
  uint16_t* o = static_cast<uint16_t*>(out) + at;
  const uint32_t w = bf16 ? pack2<__nv_bfloat16>(x, y) : pack2<__half>(x, y);
  if (pair) {
    *reinterpret_cast<uint32_t*>(o) = w;
    return;
  }
  o[0] = static_cast<uint16_t>(w);
  o[1] = static_cast<uint16_t>(w >> 16);
}

// CLUSTER: an item to a cluster of blocks instead, whose warps share its tiles and join their rows through distributed
// shared memory: one launch, no list, no workspace.  For few short sequences.
template <int KIND, int DT, int MT, bool CLUSTER>
__global__ void __launch_bounds__(kWarps * 32, AttendCfg<KIND, DT, MT>::kBlocks)
    paged_attention_kernel(const __grid_constant__ AttendParams p) {
  using C = AttendCfg<KIND, DT, MT>;
  constexpr int NT = C::NT, kStages = C::kStages;
  constexpr bool kFp8 = C::kFp8;
  extern __shared__ __align__(128) uint8_t smem_all[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  pdl_trigger();
  pdl_wait();

  const int HH = p.Hkv * p.HB;
  const int64_t run_id = static_cast<int64_t>(warp) * gridDim.x + blockIdx.x;
  // zeros for the sequences without a tile, each of them a warp's
  const auto zero_empty = [&] {
    const uint32_t D = p.D, all = p.Hq * D;  // below 256 * 2^16 heads of up to 256: past 2^31, within 2^32 - 2^16
    for (int b = static_cast<int>(run_id); b < p.B; b += p.warps) {
      if (span_of<NT>(p, b).tiles) continue;
      for (uint32_t i = lane; i < all; i += 32)
        static_cast<uint16_t*>(p.out)[b * p.o_b + i / D * p.o_h + i % D] = 0;  // bf16's and f16's zero
      if (p.lse)
        for (int i = lane; i < p.Hq; i += 32) p.lse[static_cast<int64_t>(b) * p.Hq + i] = -INFINITY;
    }
  };
  Cursor here;  // of the tile that is computed next
  if constexpr (CLUSTER) {
    const int item = blockIdx.x / p.cluster, worker = (blockIdx.x - item * p.cluster) * kWarps + warp;
    here.b = item / HH;
    here.hh = item - here.b * HH;
    here.s = span_of<NT>(p, here.b);
    const int workers = p.cluster * kWarps;
    here.u = static_cast<int>(static_cast<int64_t>(worker) * here.s.tiles / workers);
    here.left = static_cast<int>(static_cast<int64_t>(worker + 1) * here.s.tiles / workers) - here.u;
  } else {
    // Every warp adds up the places of all sequences for itself (no barrier; the lengths come from L1 after the first warp),
    // in up to 32 chunks of 32 `turns` neighbours, lane k holding the sum of chunk k.
    const auto scan = [&](int64_t v) {
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int64_t x = __shfl_up_sync(0xffffffffu, v, o);
        if (lane >= o) v += x;
      }
      return v;
    };
    const auto places_at = [&](int b) { return b < p.B ? places_of(span_of<NT, false>(p, b), HH) : 0; };
    const int turns = (p.B + 1023) / 1024, chunk = 32 * turns;
    int64_t mine = 0, v = 0;
    int k = 0, turn = 0;
    const auto close = [&] {  // chunk k: the warp's sum in two pieces, each below 2^32 (a list has fewer than 2^38 places)
      const int64_t all = static_cast<int64_t>(__reduce_add_sync(0xffffffffu, static_cast<uint32_t>(v >> 24))) * (1 << 24) +
                          __reduce_add_sync(0xffffffffu, static_cast<uint32_t>(v & 0xFFFFFF));
      if (lane == k) mine = all;
      ++k;
      v = turn = 0;
    };
    for (int t = 0; t * 32 < p.B; t += 8) {
      int64_t x[8];  // on their way together
#pragma unroll
      for (int j = 0; j < 8; ++j) x[j] = places_at((t + j) * 32 + lane);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        v += x[j];
        if (++turn == turns) close();
      }
    }
    if (turn > 0) close();
    int64_t up = scan(mine);
    const int64_t total = __shfl_sync(0xffffffffu, up, 31);
    if (run_id == 0) {
      if (lane == 0) p.prefix[p.B] = total;
      if (p.by_rows) {
        int64_t at = 0;
        for (int b = lane; b < p.B + lane; b += 32) {
          const int64_t v = places_at(b), to = scan(v);
          if (b < p.B) p.prefix[b] = at + to - v;
          at += __shfl_sync(0xffffffffu, to, 31);
        }
      }
    }
    const int64_t runs = runs_of(p, total);
    if (run_id >= runs) {
      zero_empty();
      return;
    }
    const int64_t start = run_id * total / runs, stop = (run_id + 1) * total / runs;
    // the chunk that has place `start`, then the sequence
    const int c = __popc(__ballot_sync(0xffffffffu, up <= start));
    int64_t at_seq = __shfl_sync(0xffffffffu, up - mine, c);
    for (int i = 0; i < turns; ++i) {
      const int b = c * chunk + i * 32 + lane;
      const int64_t v = places_at(b);
      up = at_seq + scan(v);
      const int l = __popc(__ballot_sync(0xffffffffu, up <= start));
      if (l < 32) {
        here.b = c * chunk + i * 32 + l;
        at_seq = __shfl_sync(0xffffffffu, up - v, l);
        break;
      }
      at_seq = __shfl_sync(0xffffffffu, up, 31);
    }
    here.s = span_of<NT, false>(p, here.b);
    const int64_t in = start - at_seq, each = here.s.tiles + kExtra;
    here.hh = static_cast<int>(in / each);
    const int off = static_cast<int>(in - here.hh * each);
    here.u = max(0, off - kExtra);
    here.left = static_cast<int>(stop - start) - max(0, kExtra - off);
    if (lane == 0 && !p.by_rows) p.starts[run_id] = {at_seq + here.hh * each, each, here.b, here.hh};
  }
  const auto advance = [&](Cursor& c) {
    --c.left;
    if (++c.u < c.s.tiles) return;
    c.u = 0;
    c.left -= kExtra;
    if (++c.hh < HH || c.left <= 0) return;
    c.hh = 0;
    do {
      c.s = span_of<NT>(p, ++c.b);  // the run has places left: there is another sequence with tiles
    } while (c.s.tiles == 0);
  };

  uint8_t* smem = smem_all + warp * C::kWarpBytes;
  const uint32_t ring = smem_u32(smem);
  constexpr int kChunks = C::kRow / 16, kRowsPer = 32 / kChunks;  // rows of one copy by the warp
  static_assert(kChunks <= 32, "a warp copies whole rows");
  // Where a tile's tokens lie, looked up one tile ahead of its copies: the page and slot of this lane's token (-1: none).
  struct Places {
    int page, slot, valid;  // tokens of the tile
    bool flat;              // all slots of the tile in one page
  };
  const auto places = [&](const Cursor& c) {
    Places w;
    const int from = c.s.lo + c.u * NT, in = lane & (NT - 1);
    w.valid = c.s.hi - from;
    w.page = -1;
    w.slot = 0;
    if (c.left > 0 && in < w.valid) {  // (from + in may lie behind 2^31 where the tile ends behind the last token)
      const int n = p.by_page.div(from + in, w.slot);
      w.page = p.table[c.b * p.table_ld + n];
      if (w.page < 0 || w.page >= p.pages) {
        atomicOr(&g_attend_error, 2u);
        w.page = -1;
      }
    }
    w.flat = __shfl_sync(0xffffffffu, w.slot, 0) + NT <= static_cast<int>(p.by_page.d);
    return w;
  };
  const auto copy_tile = [&](int h, const Places& w, int stage) {
    const int c = lane % kChunks, r0 = lane / kChunks;
    const bool in_row = c * 16 < p.D * C::kSize;
    const uint32_t kt = ring + stage * C::kStage, vt = kt + C::kTile;
    const int in = in_row ? c * 16 : 0;
    const char *k = static_cast<const char*>(p.k) + in + h * p.k_head, *v = static_cast<const char*>(p.v) + in + h * p.v_head;
    if (w.flat) {  // the same page and neighbouring slots, all of them the cache's own memory
      const int page = __shfl_sync(0xffffffffu, w.page, 0), slot = __shfl_sync(0xffffffffu, w.slot, 0) + r0;
      const int valid = page < 0 || !in_row ? 0 : w.valid - r0;
      k += max(page, 0) * p.k_page + slot * p.k_slot;
      v += max(page, 0) * p.v_page + slot * p.v_slot;
#pragma unroll
      for (int r = 0; r < NT; r += kRowsPer) {
        const uint32_t to = C::at(r + r0, c);
        cp_async16(kt + to, k, r < valid);
        cp_async16(vt + to, v, r < valid);
        k += kRowsPer * p.k_slot;
        v += kRowsPer * p.v_slot;
      }
      return;
    }
    const int64_t k_at = w.page < 0 ? -1 : w.page * p.k_page + w.slot * p.k_slot;
    const int64_t v_at = w.page < 0 ? -1 : w.page * p.v_page + w.slot * p.v_slot;
#pragma unroll
    for (int r = 0; r < NT; r += kRowsPer) {
      const int64_t ka = __shfl_sync(0xffffffffu, k_at, r + r0), va = __shfl_sync(0xffffffffu, v_at, r + r0);
      const bool there = in_row && ka >= 0;
      const uint32_t to = C::at(r + r0, c);
      cp_async16(kt + to, k + (there ? ka : 0), there);
      cp_async16(vt + to, v + (there ? va : 0), there);
    }
  };

  // fill the ring: kStages - 1 tiles on their way, the next one's pages known
  Cursor ahead = here;
  Places where = places(ahead);
  int ahead_h = ahead.hh / p.HB;
  const auto issue = [&](int stage) {
    if (ahead.left > 0) {
      copy_tile(ahead_h, where, stage);
      advance(ahead);
      ahead_h = ahead.hh / p.HB;
      where = places(ahead);
    }
    copy_commit();
  };
#pragma unroll
  for (int i = 0; i < kStages - 1; ++i) issue(i);
  if constexpr (!CLUSTER) zero_empty();  // while the first tiles are on their way

  constexpr int kNt = DT / 8;  // column fragments of O
  float o[MT][kNt][4], m[MT][2], l[MT][2];
  const int g = lane >> 2, j2 = (lane & 3) * 2;
  const uint32_t q_s = ring + C::kOffQ;
  float* row_scale = reinterpret_cast<float*>(smem + C::kOffScale);
  constexpr bool bf16_out = C::kBf16Out;

  int stage = 0;
  bool first = true;
  if constexpr (CLUSTER) {
    if (here.left <= 0) {  // an item of fewer tiles than warps: rows of no weight
      float2* ml = reinterpret_cast<float2*>(smem + C::kOffMl);
      for (int r = lane; r < C::kRows; r += 32) ml[r] = make_float2(-INFINITY, 0.f);
    }
  }
  while (here.left > 0) {
    // --- the tiles of one item ---
    const int run = min(here.s.tiles - here.u, here.left);
    const bool whole = run == here.s.tiles;
    const int h = here.hh / p.HB, head0 = h * p.G + (here.hh % p.HB) * C::kRows;
    const int live = min(C::kRows, (h + 1) * p.G - head0);  // query heads of this group
    {
      const float ks = kFp8 && p.k_scale ? p.k_scale[h] : 1.f;
      constexpr int kLanes = DT / 8, kPer = 32 / kLanes;  // lanes of a row, rows of a turn
      const int c = lane % kLanes, r0 = lane / kLanes;
      const uint16_t* src = static_cast<const uint16_t*>(p.q) + here.b * p.q_b + (head0 + r0) * p.q_h + c * 8;
      uint4 e[C::kRows / kPer];
#pragma unroll
      for (int i = 0; i < C::kRows / kPer; ++i) {
        e[i] = make_uint4(0, 0, 0, 0);
        if (r0 + i * kPer < live && c * 8 < p.D) {
          const uint16_t* at = src + i * kPer * p.q_h;
          if (p.q_vec) {
            e[i] = *reinterpret_cast<const uint4*>(at);
          } else {
            uint32_t w[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) w[j] = at[2 * j] | static_cast<uint32_t>(at[2 * j + 1]) << 16;
            e[i] = make_uint4(w[0], w[1], w[2], w[3]);
          }
        }
      }
      __syncwarp();  // the last item's queries are read
#pragma unroll
      for (int i = 0; i < C::kRows / kPer; ++i) {
        const int r = r0 + i * kPer;
        uint32_t w[4] = {e[i].x, e[i].y, e[i].z, e[i].w};
        float factor = 1.f;
        if constexpr (kFp8) {
          // f16 operands: a bf16 row is scaled by a power of two so that its largest element lies in [2^14, 2^15), where
          // elements down to 2^-29 of it stay exact
          if constexpr (C::kBf16Out) {
            float f[8], top = 0.f;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              f[j] = __uint_as_float(j & 1 ? w[j / 2] & 0xFFFF0000u : w[j / 2] << 16);
              top = fmaxf(top, fabsf(f[j]));
            }
#pragma unroll
            for (int x = 1; x < kLanes; x <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, x));
            const int ex = static_cast<int>(__float_as_uint(top) >> 23) - 127;
            // powers of two beyond fp32's range (tiny rows) are capped; infinities keep their place
            const int by = top > 0.f && ex < 128 ? min(14 - ex, 126) : 0;
            const float up = __uint_as_float(static_cast<uint32_t>(by + 127) << 23);
            factor = __uint_as_float(static_cast<uint32_t>(127 - by) << 23);
#pragma unroll
            for (int j = 0; j < 4; ++j) w[j] = pack2<__half>(f[2 * j] * up, f[2 * j + 1] * up);
          }
          // the order of d within 16 in which a key's codes come out of ldmatrix, four neighbours to a lane: pairs 0 2 4 6
          // of the 16, then 1 3 5 7
          const uint32_t to = (c & 1) * 8;
          *reinterpret_cast<uint2*>(smem + C::kOffQ + C::q_at(r, c & ~1) + to) = make_uint2(w[0], w[2]);
          *reinterpret_cast<uint2*>(smem + C::kOffQ + C::q_at(r, c | 1) + to) = make_uint2(w[1], w[3]);
        } else {
          *reinterpret_cast<uint4*>(smem + C::kOffQ + C::q_at(r, c)) = make_uint4(w[0], w[1], w[2], w[3]);
        }
        if (c == 0) row_scale[r] = factor * p.scale * ks;
      }
      __syncwarp();
    }
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
#pragma unroll
      for (int i = 0; i < kNt; ++i)
#pragma unroll
        for (int x = 0; x < 4; ++x) o[mt][i][x] = 0.f;
      m[mt][0] = m[mt][1] = -INFINITY;
      l[mt][0] = l[mt][1] = 0.f;
    }

    float s[MT][NT / 8][4];
    const auto scores = [&](uint32_t kt) {
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
            ldsm4(a[mt], q_s + C::q_at(mt * 16 + (lane & 15), 2 * kk + (lane >> 4)));
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
              ldsm4(a[x][mt], q_s + C::q_at(mt * 16 + (lane & 15), 2 * (2 * kk + x) + (lane >> 4)));
#pragma unroll
          for (int n = 0; n < NT / 16; ++n) {
            uint32_t b[4];  // tokens 0-7 and 8-15, d 0-15 and 16-31 each
            ldsm4(b, kt + C::at(n * 16 + (lane & 7) + ((lane >> 4) << 3), kk * 2 + ((lane >> 3) & 1)));
#pragma unroll
            for (int x = 0; x < 4; ++x) {
              uint32_t b0, b1;
              f16x4_of_e4m3x4(b[x], b0, b1);
#pragma unroll
              for (int mt = 0; mt < MT; ++mt) mma16816<false>(s[mt][2 * n + (x >> 1)], a[x & 1][mt], b0, b1);
            }
          }
        }
      }
    };
    const auto tile_at = [&](int st) { return ring + st * C::kStage; };
    if constexpr (C::kPipe) {
      copy_wait<kStages - 2>();
      __syncwarp();
      scores(tile_at(stage));
    }
#pragma unroll 1
    for (int i = 0; i < run; ++i) {
      issue(stage == 0 ? kStages - 1 : stage - 1);
      if constexpr (!C::kPipe) {
        copy_wait<kStages - 1>();
        __syncwarp();
        scores(tile_at(stage));
      }
      const uint32_t vt = tile_at(stage) + C::kTile;
      if (++stage == kStages) stage = 0;
      const int left = here.s.hi - (here.s.lo + (here.u + i) * NT);  // tokens of this tile and behind it
      // running maximum and sum, weights
      const bool last = left < NT;
      const auto weigh = [&](int mt, int x) {  // of the fragment's rows g + 8 x
        const float f = row_scale[mt * 16 + g + 8 * x];
        float top = m[mt][x];
#pragma unroll
        for (int n = 0; n < NT / 8; ++n) {
          s[mt][n][2 * x] *= f;
          s[mt][n][2 * x + 1] *= f;
        }
        if (last) {
#pragma unroll
          for (int n = 0; n < NT / 8; ++n) {
            if (n * 8 + j2 >= left) s[mt][n][2 * x] = -INFINITY;
            if (n * 8 + j2 + 1 >= left) s[mt][n][2 * x + 1] = -INFINITY;
          }
        }
#pragma unroll
        for (int n = 0; n < NT / 8; ++n) top = fmaxf(top, fmaxf(s[mt][n][2 * x], s[mt][n][2 * x + 1]));
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
        const float base = top == -INFINITY ? 0.f : top;
        if (__any_sync(0xffffffffu, top > m[mt][x])) {
          const float c = exp2_fast(m[mt][x] - base);
          l[mt][x] *= c;
#pragma unroll
          for (int n = 0; n < kNt; ++n) {
            o[mt][n][2 * x] *= c;
            o[mt][n][2 * x + 1] *= c;
          }
          m[mt][x] = top;
        }
        const float off = C::kShift - base;
        float sum = 0.f;
#pragma unroll
        for (int n = 0; n < NT / 8; ++n) {
          s[mt][n][2 * x] = exp2_fast(s[mt][n][2 * x] + off);
          s[mt][n][2 * x + 1] = exp2_fast(s[mt][n][2 * x + 1] + off);
          sum += s[mt][n][2 * x] + s[mt][n][2 * x + 1];
        }
        l[mt][x] += sum;
      };
      const bool lower = live > 8;  // whether rows 8-15 of the first fragment are heads
#pragma unroll
      for (int mt = 0; mt < MT; ++mt) {
        weigh(mt, 0);
        if (mt > 0 || lower) {
          weigh(mt, 1);
        } else {
#pragma unroll
          for (int n = 0; n < NT / 8; ++n) s[mt][n][2] = s[mt][n][3] = 0.f;
        }
      }
      // the weights as left operands, 16 tokens to one
      uint32_t hi[NT / 16][MT][4], lo[NT / 16][MT][4];
#pragma unroll
      for (int n = 0; n < NT / 16; ++n) {
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            const float* w = &s[mt][2 * n + (x >> 1)][(x & 1) * 2];
            if constexpr (C::kBf16) {
              const uint32_t c0 = __float_as_uint(w[0] * (1.f - 0x1p-8f)), c1 = __float_as_uint(w[1] * (1.f - 0x1p-8f));
              hi[n][mt][x] = prmt(c0, c1, 0x7632);
              lo[n][mt][x] = pack2<__nv_bfloat16>(w[0] - __uint_as_float(c0 & 0xFFFF0000u),
                                               w[1] - __uint_as_float(c1 & 0xFFFF0000u));
            } else if constexpr (C::kSplit) {
              const __half2 c = __halves2half2(__float2half_rz(w[0] * (1.f - 0x1p-10f)),
                                               __float2half_rz(w[1] * (1.f - 0x1p-10f)));
              hi[n][mt][x] = *reinterpret_cast<const uint32_t*>(&c);
              lo[n][mt][x] = pack2<__half>(w[0] - __low2float(c), w[1] - __high2float(c));
            } else {
              hi[n][mt][x] = pack2<__half>(w[0], w[1]);
            }
          }
      }
      // The next tile's scores beside O += P V: two independent rows of products.  Behind the item's last tile they are of no
      // use and left.
      if constexpr (C::kPipe) {
        copy_wait<kStages - 2>();
        __syncwarp();
        scores(tile_at(stage));
      }
#pragma unroll
      for (int n = 0; n < NT / 16; ++n) {
        if constexpr (!kFp8) {
#pragma unroll
          for (int c = 0; c < DT / 16; ++c) {
            uint32_t b[4];  // d 0-7: tokens 0-7 and 8-15; d 8-15 likewise
            ldsm4_t(b, vt + C::at(n * 16 + (lane & 15), 2 * c + (lane >> 4)));
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) {
              mma16816<C::kBf16>(o[mt][2 * c], hi[n][mt], b[0], b[1]);
              mma16816<C::kBf16>(o[mt][2 * c + 1], hi[n][mt], b[2], b[3]);
              mma16816<C::kBf16>(o[mt][2 * c], lo[n][mt], b[0], b[1]);
              mma16816<C::kBf16>(o[mt][2 * c + 1], lo[n][mt], b[2], b[3]);
            }
          }
        } else {
#pragma unroll
          for (int c = 0; c < DT / 32; ++c) {
            uint32_t b[4];  // d 0-15: tokens 0-7 and 8-15; d 16-31 likewise; each word two tokens of two neighbours
            ldsm4_t(b, vt + C::at(n * 16 + (lane & 15), 2 * c + (lane >> 4)));
#pragma unroll
            for (int x = 0; x < 2; ++x) {
              uint32_t e0, e1, d0, d1;
              f16x4_of_e4m3x4(prmt(b[2 * x], 0, 0x3120), e0, d0);
              f16x4_of_e4m3x4(prmt(b[2 * x + 1], 0, 0x3120), e1, d1);
#pragma unroll
              for (int mt = 0; mt < MT; ++mt) {  // even and odd d
                mma16816<false>(o[mt][4 * c + 2 * x], hi[n][mt], e0, e1);
                mma16816<false>(o[mt][4 * c + 2 * x + 1], hi[n][mt], d0, d1);
                if constexpr (C::kSplit) {
                  mma16816<false>(o[mt][4 * c + 2 * x], lo[n][mt], e0, e1);
                  mma16816<false>(o[mt][4 * c + 2 * x + 1], lo[n][mt], d0, d1);
                }
              }
            }
          }
        }
      }
      __syncwarp();  // the tile's slot is free
    }

    if constexpr (CLUSTER) {  // this warp's rows into its ring, which nothing uses any more
      copy_wait<0>();
      __syncwarp();
      float2* ml = reinterpret_cast<float2*>(smem + C::kOffMl);
      float* rows = reinterpret_cast<float*>(smem);
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          float sum = l[mt][x];
          sum += __shfl_xor_sync(0xffffffffu, sum, 1);
          sum += __shfl_xor_sync(0xffffffffu, sum, 2);
          const int r = mt * 16 + g + 8 * x;
          if ((lane & 3) == 0) ml[r] = make_float2(m[mt][x], sum);
          float* row = rows + r * C::kJoinRow;
          if constexpr (kFp8) {
#pragma unroll
            for (int n = 0; n < kNt; n += 2)
              *reinterpret_cast<float4*>(row + n * 8 + 2 * j2) =
                  make_float4(o[mt][n][2 * x], o[mt][n + 1][2 * x], o[mt][n][2 * x + 1], o[mt][n + 1][2 * x + 1]);
          } else {
#pragma unroll
            for (int n = 0; n < kNt; ++n)
              *reinterpret_cast<float2*>(row + n * 8 + j2) = make_float2(o[mt][n][2 * x], o[mt][n][2 * x + 1]);
          }
        }
      break;
    }
    // --- the item's rows, or this warp's part of them ---
    const int64_t part = (run_id * 2 + (first ? 0 : 1)) * C::kRows;
    const float vs = kFp8 && p.v_scale ? p.v_scale[h] : 1.f;
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        l[mt][x] += __shfl_xor_sync(0xffffffffu, l[mt][x], 1);
        l[mt][x] += __shfl_xor_sync(0xffffffffu, l[mt][x], 2);
      }
    // WHOLE, PAIR: chosen once for all stores (chosen at each of them, they took 0.8 us)
    const auto write = [&](auto whole_, auto pair_) {
      constexpr bool WHOLE = decltype(whole_)::value, PAIR = decltype(pair_)::value;
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          const int r = mt * 16 + g + 8 * x;
          if (r >= live) continue;
          const float top = m[mt][x], sum = l[mt][x], inv = sum == 0.f ? 0.f : vs / sum;
          if ((lane & 3) == 0) {
            if (!WHOLE)
              p.part_ml[part + r] = make_float2(top, sum);
            else if (p.lse)
              p.lse[static_cast<int64_t>(here.b) * p.Hq + head0 + r] =
                  sum == 0.f ? -INFINITY : (top - C::kShift + log2f(sum)) * kLn2;
          }
          const int64_t out = here.b * p.o_b + (head0 + r) * p.o_h;
          float* row = p.part_o + (part + r) * p.D;
          if constexpr (kFp8) {  // fragments n and n + 1 hold the even and odd ones of 16 columns: four neighbours to a lane
#pragma unroll
            for (int n = 0; n < kNt; n += 2) {
              const int d = n * 8 + 2 * j2;
              const float v0 = o[mt][n][2 * x], v1 = o[mt][n + 1][2 * x], v2 = o[mt][n][2 * x + 1], v3 = o[mt][n + 1][2 * x + 1];
              if (d >= p.D) continue;
              if (WHOLE) {
                store_out(p.out, out + d, v0 * inv, v1 * inv, bf16_out, PAIR);
                store_out(p.out, out + d + 2, v2 * inv, v3 * inv, bf16_out, PAIR);
              } else {
                *reinterpret_cast<float4*>(row + d) = make_float4(v0, v1, v2, v3);
              }
            }
          } else {
#pragma unroll
            for (int n = 0; n < kNt; ++n) {
              const int d = n * 8 + j2;
              if (d >= p.D) continue;
              if (WHOLE)
                store_out(p.out, out + d, o[mt][n][2 * x] * inv, o[mt][n][2 * x + 1] * inv, bf16_out, PAIR);
              else
                *reinterpret_cast<float2*>(row + d) = make_float2(o[mt][n][2 * x], o[mt][n][2 * x + 1]);
            }
          }
        }
    };
    if (!whole)
      write(std::false_type{}, std::false_type{});
    else if (p.out_pair)
      write(std::true_type{}, std::true_type{});
    else
      write(std::true_type{}, std::false_type{});
    first = false;
    here.u += run - 1;
    here.left -= run - 1;
    advance(here);
  }
  if constexpr (CLUSTER) {
    __syncwarp();
    cluster_arrive();
    cluster_wait();
    // the cluster's threads share the rows' columns in fours, and add up the warps' parts in their order
    const int h = here.hh / p.HB, head0 = h * p.G + (here.hh % p.HB) * C::kRows, live = min(C::kRows, (h + 1) * p.G - head0);
    const int rank = blockIdx.x % p.cluster, fours = p.D / 4;
    const float vs = kFp8 && p.v_scale ? p.v_scale[h] : 1.f;
    const uint32_t base = smem_u32(smem_all);
    const auto part_of = [&](int w, uint32_t at) {  // an address in the part of warp w of the cluster
      return map_to_cta(base + (w & (kWarps - 1)) * C::kWarpBytes + at, w / kWarps);
    };
    for (int i = rank * kWarps * 32 + threadIdx.x; i < live * fours; i += p.cluster * kWarps * 32) {
      const int r = i / fours, d = (i - r * fours) * 4;
      float top = -INFINITY, sum = 0.f;
      float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
      for (int w0 = 0; w0 < p.cluster * kWarps; w0 += kWarps) {  // a block's parts on their way together
        float2 ml[kWarps];
        float4 v[kWarps];
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
          asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];" : "=f"(ml[w].x), "=f"(ml[w].y) : "r"(part_of(w0 + w, C::kOffMl + r * 8)));
          asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                       : "=f"(v[w].x), "=f"(v[w].y), "=f"(v[w].z), "=f"(v[w].w)
                       : "r"(part_of(w0 + w, (r * C::kJoinRow + d) * 4)));
        }
        float t = top;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) t = fmaxf(t, ml[w].x);
        const float to = t == -INFINITY ? 0.f : t, old = exp2_fast(top - to);
        sum *= old, acc.x *= old, acc.y *= old, acc.z *= old, acc.w *= old;
        top = t;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
          if (ml[w].y == 0.f) continue;  // no weight: its rows may hold anything
          const float f = exp2_fast(ml[w].x - to);
          sum = fmaf(ml[w].y, f, sum);
          acc.x = fmaf(v[w].x, f, acc.x);
          acc.y = fmaf(v[w].y, f, acc.y);
          acc.z = fmaf(v[w].z, f, acc.z);
          acc.w = fmaf(v[w].w, f, acc.w);
        }
      }
      const float inv = sum == 0.f ? 0.f : vs / sum;
      const int64_t out = here.b * p.o_b + (head0 + r) * p.o_h + d;
      store_out(p.out, out, acc.x * inv, acc.y * inv, bf16_out, p.out_pair);
      store_out(p.out, out + 2, acc.z * inv, acc.w * inv, bf16_out, p.out_pair);
      if (p.lse && d == 0)
        p.lse[static_cast<int64_t>(here.b) * p.Hq + head0 + r] = sum == 0.f ? -INFINITY : (top - C::kShift + log2f(sum)) * kLn2;
    }
    __syncwarp();
    cluster_arrive();
    cluster_wait();  // no block leaves while another reads its rows
  }
}

// Joins the parts of the items that several warps shared, in the warps' order.
//   ROWS: a block to a row (sequence, query head), its warps each a range of the parts: few items, many parts.
//   else: a block to a run's start; where it is the first one inside an item, the block's warps take the item's rows.  (Looking
//   at all rows instead, of which few need it, took 14 us for 512 sequences of 64 heads.)
constexpr int kJoinWarps = 8;
template <int KIND, int DT, int MT, bool ROWS>
__global__ void __launch_bounds__(kJoinWarps * 32, ROWS || DT > 128 ? 1 : 4)
    paged_attention_join_kernel(const __grid_constant__ AttendParams p) {
  using C = AttendCfg<KIND, DT, MT>;
  constexpr int kV = (DT + 127) / 128;  // float4 of a lane
  constexpr int WPR = ROWS ? kJoinWarps : 1;
  pdl_trigger();
  pdl_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  constexpr bool bf16 = C::kBf16Out;
  const int64_t total = p.prefix[p.B];
  int b, hh, r0;
  int64_t i0, each, runs;
  if constexpr (ROWS) {
    b = static_cast<int>(blockIdx.x / p.Hq);
    const int head = blockIdx.x - b * p.Hq, h = head / p.G, in = head - h * p.G;
    hh = h * p.HB + in / C::kRows;
    r0 = in % C::kRows;
    const int64_t before = p.prefix[b];
    each = (p.prefix[b + 1] - before) / (p.Hkv * p.HB);
    if (each == 0) return;  // an empty sequence
    i0 = before + hh * each;
    runs = runs_of(p, total);
  } else {
    const int64_t c = blockIdx.x + 1;
    const RunStart s = p.starts[c];
    runs = runs_of(p, total);
    if (c >= runs) return;
    b = s.b;
    hh = s.hh;
    i0 = s.first;
    each = s.each;
    r0 = warp;
    // its place is behind the item's first tile, which the run before it has
    if (c * total / runs <= i0 + kExtra || (c - 1) * total / runs > i0 + kExtra) return;
  }
  const int64_t c0 = ((i0 + kExtra + 1) * runs - 1) / total, c1 = ((i0 + each) * runs - 1) / total;
  if (c0 == c1) return;  // written by its only warp
  const int skip = c0 * total / runs >= i0 ? 0 : 1;  // whether the item is behind another one in its first warp's run
  const int h = hh / p.HB, head0 = h * p.G + (hh % p.HB) * C::kRows, live = min(C::kRows, (h + 1) * p.G - head0);
  const int parts = static_cast<int>(c1 - c0) + 1, w = warp % WPR;
  const int from = static_cast<int>(static_cast<int64_t>(w) * parts / WPR), to = static_cast<int>(static_cast<int64_t>(w + 1) * parts / WPR);
  for (int r = r0; r < live; r += ROWS ? live : kJoinWarps) {
    const int64_t row = static_cast<int64_t>(b) * p.Hq + head0 + r, out = b * p.o_b + (head0 + r) * p.o_h;
    const auto at = [&](int i) { return ((c0 + i) * 2 + (i == 0 ? skip : 0)) * C::kRows + r; };
    float top = -INFINITY, sum = 0.f;
    float4 acc[kV];
#pragma unroll
    for (int x = 0; x < kV; ++x) acc[x] = make_float4(0.f, 0.f, 0.f, 0.f);
    constexpr int kAhead = ROWS ? (kV == 1 ? 10 : 5) : 3;  // parts of O asked for at a time
    float4 v[kAhead][kV];
    const auto load = [&](int i) {
#pragma unroll
      for (int y = 0; y < kAhead; ++y)
#pragma unroll
        for (int x = 0; x < kV; ++x) {
          const int d = (x * 32 + lane) * 4;
          v[y][x] = make_float4(0.f, 0.f, 0.f, 0.f);
          if (i + y < to && d < p.D) v[y][x] = *reinterpret_cast<const float4*>(p.part_o + at(i + y) * p.D + d);
        }
    };
    for (int f0 = from; f0 < to; f0 += 32) {  // 32 parts at a time, one maximum and sum to a lane
      load(f0);  // on its way together with the maxima
      const float2 ml = f0 + lane < to ? p.part_ml[at(f0 + lane)] : make_float2(-INFINITY, 0.f);
      const float t = fmaxf(top, warp_max(ml.x)), base = t == -INFINITY ? 0.f : t;
      const float old = exp2_fast(top - base), now = exp2_fast(ml.x - base);
      sum = sum * old + warp_sum(ml.y * now);
#pragma unroll
      for (int x = 0; x < kV; ++x) acc[x].x *= old, acc[x].y *= old, acc[x].z *= old, acc[x].w *= old;
      top = t;
      const int n = min(32, to - f0);
#pragma unroll 1
      for (int j = 0; j < n; j += kAhead) {
        if (j > 0) load(f0 + j);
#pragma unroll
        for (int y = 0; y < kAhead; ++y) {
          const float f = __shfl_sync(0xffffffffu, now, (j + y) & 31);
          if (j + y >= n) continue;
#pragma unroll
          for (int x = 0; x < kV; ++x) {
            acc[x].x = fmaf(v[y][x].x, f, acc[x].x);
            acc[x].y = fmaf(v[y][x].y, f, acc[x].y);
            acc[x].z = fmaf(v[y][x].z, f, acc[x].z);
            acc[x].w = fmaf(v[y][x].w, f, acc[x].w);
          }
        }
      }
    }
    if constexpr (ROWS) {
      __shared__ float2 all_ml[WPR];
      __shared__ float4 all_o[WPR][kV][32];
      if (lane == 0) all_ml[w] = make_float2(top, sum);
#pragma unroll
      for (int x = 0; x < kV; ++x) all_o[w][x][lane] = acc[x];
      __syncthreads();
      if (w) return;
      for (int y = 1; y < WPR; ++y) top = fmaxf(top, all_ml[y].x);
      const float base = top == -INFINITY ? 0.f : top;
      sum = 0.f;
#pragma unroll
      for (int x = 0; x < kV; ++x) acc[x] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int y = 0; y < WPR; ++y) {
        const float f = exp2_fast(all_ml[y].x - base);
        sum += all_ml[y].y * f;
#pragma unroll
        for (int x = 0; x < kV; ++x) {
          const float4 v = all_o[y][x][lane];
          acc[x].x = fmaf(v.x, f, acc[x].x);
          acc[x].y = fmaf(v.y, f, acc[x].y);
          acc[x].z = fmaf(v.z, f, acc[x].z);
          acc[x].w = fmaf(v.w, f, acc[x].w);
        }
      }
    }
    const float vs = C::kFp8 && p.v_scale ? p.v_scale[h] : 1.f, inv = sum == 0.f ? 0.f : vs / sum;
#pragma unroll
    for (int x = 0; x < kV; ++x) {
      const int d = (x * 32 + lane) * 4;
      if (d >= p.D) continue;
      store_out(p.out, out + d, acc[x].x * inv, acc[x].y * inv, bf16, p.out_pair);
      store_out(p.out, out + d + 2, acc[x].z * inv, acc[x].w * inv, bf16, p.out_pair);
    }
    if (p.lse && lane == 0) p.lse[row] = sum == 0.f ? -INFINITY : (top - C::kShift + log2f(sum)) * kLn2;
  }
}

template <int KIND, int DT, int MT>
int launch_attend(AttendParams p, cudaStream_t st) {
  using C = AttendCfg<KIND, DT, MT>;
  static DeviceOnce once;
  if (int rc = once.run([] {
        return cudaFuncSetAttribute(paged_attention_kernel<KIND, DT, MT, false>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                    C::kSmem) == cudaSuccess &&
                       cudaFuncSetAttribute(paged_attention_kernel<KIND, DT, MT, true>,
                                            cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem) == cudaSuccess
                   ? static_cast<int>(W4A8_OK)
                   : check_launch("cudaFuncSetAttribute(paged_attention)");
      }))
    return rc;
  p.HB = static_cast<int>(ceil_div(p.G, C::kRows));
  p.warps = attend_warps(DT);
  if (p.cluster) {
    const int64_t items = static_cast<int64_t>(p.B) * p.Hkv * p.HB;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = p.cluster;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t lc = {};
    lc.gridDim = dim3(static_cast<unsigned>(items * p.cluster));
    lc.blockDim = dim3(kWarps * 32);
    lc.dynamicSmemBytes = C::kSmem;
    lc.stream = st;
    lc.attrs = attr;
    lc.numAttrs = 2;
    const cudaError_t e = cudaLaunchKernelEx(&lc, paged_attention_kernel<KIND, DT, MT, true>, p);
    if (e != cudaSuccess) return set_error(W4A8_ERR_CUDA, "paged_attention_kernel: %s", cudaGetErrorString(e));
    return check_launch("paged_attention_kernel");
  }
  // few items have many parts each
  p.by_rows = static_cast<int64_t>(p.B) * p.Hkv * p.HB * 8 < p.warps;
  if (int rc = launch_pdl("paged_attention_kernel", paged_attention_kernel<KIND, DT, MT, false>, dim3(p.warps / kWarps),
                          dim3(kWarps * 32), C::kSmem, st, p))
    return rc;
  if (p.by_rows)
    return launch_pdl("paged_attention_join_kernel", paged_attention_join_kernel<KIND, DT, MT, true>,
                      dim3(static_cast<unsigned>(p.B * p.Hq)), dim3(kJoinWarps * 32), 0, st, p);
  return launch_pdl("paged_attention_join_kernel", paged_attention_join_kernel<KIND, DT, MT, false>,
                    dim3(static_cast<unsigned>(p.warps - 1)), dim3(kJoinWarps * 32), 0, st, p);
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
