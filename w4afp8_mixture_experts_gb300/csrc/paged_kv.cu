// rotary_embedding and paged_kv_append: rows of heads moved, and rotated by position on the way.
//
// Both are one kernel over rows (token, head): the heads of a token are its queries, then (append) its keys and its
// values.  A block takes a run of neighbouring rows.  A thread has the same places in each of its rows (items: two vectors
// whose elements are turned with one another, or that stay), asks for its first two rows', the block works out where its
// tokens go and the cosines and sines of their angles once for all heads, and then the vectors are turned and stored.
// Bound by memory; the angles of a token cost R / 2 sincospif and are shared by its heads.
//
// An angle is a fraction of a turn: position * freqs modulo 2^64 is the exact remainder of the product by whole turns,
// and its upper 32 bits as a signed number are half-turns in [-1, 1) in units of 2^-31.  In fp32 they are within 2^-25
// half-turns of the angle, 1e-7, whatever the position.
#include <algorithm>

#include "paged.cuh"

namespace w4a8 {
namespace {

constexpr int kMaxDim = 1024;  // of a head
constexpr int kThreads = 128;
constexpr int kBlocks = 8;    // of an SM
constexpr int kRounds = 12;   // rows of a thread, at most
constexpr int kAhead = 2;     // rows of a thread on their way
constexpr int kMaxCs = 2048;  // cosine and sine pairs of a block's tokens
constexpr int kMaxTok = 64;   // tokens of a block

__device__ unsigned int g_paged_error;

struct RowParams {
  const void *q, *k, *v;
  void *qo, *kc, *vc;
  int64_t q_t, q_h, k_t, k_h, v_t, v_h, o_t, o_h;
  int64_t k_page, k_slot, k_head, v_page, v_slot, v_head;
  const int32_t *table, *lens, *indptr;
  int64_t table_ld, pages;
  const void* positions;
  const int64_t* freqs;
  const float *k_scale, *v_scale;
  int64_t rows;  // T * heads of a token
  int T, B, Hq, Hkv, D, R, start, table_pages;
  int rot_items, items;  // of a row: those with pairs to turn, all of them
  int rows_per_block;
  int row_threads;       // threads of a row, each with kItems of its items
  FastDiv by_row, by_heads, by_page, by_half;
  float cos_scale, sin_scale;
  bool interleaved, positions64;
  bool zero_left;  // queries of rows that are left out become zeros (else they stay as they are)
};

// Items of a thread in a row: more where they are narrow, as a row costs a thread as much (8192 x 40 x 101 f16, single
// elements: 81 us with one item, 45 with 4; 8192 x 40 x 80 in 8 bytes: 26 with one, 19 with 2).
template <typename T, int V>
constexpr int kItems = V * sizeof(T) <= 4 ? 4 : V * sizeof(T) == 8 ? 2 : 1;

template <typename T, int V>
struct alignas(sizeof(T) * V) Vec {
  T e[V];
};

// the correctly rounded quotient, r = 1 / scale; where it is past what E4M3 holds its last bits do not matter
__device__ __forceinline__ float over(float v, float scale, float r) {
  const float q = v * r;
  return fabsf(q) >= 512.f && fabsf(r) < INFINITY ? q : div_by_scale(v, scale, r);
}

// Where the two vectors of an item lie in its row; the second may be missing (-1).  Neighbouring items have neighbouring
// vectors, so that a warp's copies are whole lines (8192 x 72 x 128 neighbours: 64 to 70 us with both vectors of an item
// side by side, 47 so).  Turned items: a vector of the turned part's first half and one of its second, which hold pairs
// between them, or pairs of neighbours each (single elements: a pair of neighbours).  Others: one of the first and one of
// the second half of what stays.
template <int V>
__device__ __forceinline__ void places(const RowParams& p, int item, bool value, int& e0, int& e1) {
  if (value) {
    e0 = V * item;
    e1 = V * (item + p.items);
  } else if (item < p.rot_items) {
    const bool side = V == 1 && p.interleaved;
    e0 = p.start + (side ? 2 : V) * item;
    e1 = e0 + (side ? 1 : p.R / 2);
  } else {
    e0 = V * (item - p.rot_items);
    e1 = e0 + V * (p.items - p.rot_items);
    if (e0 >= p.start) e0 += p.R;
    if (e1 >= p.start) e1 += p.R;
  }
  if (e0 >= p.D) e0 = -1;
  if (e1 >= p.D) e1 = -1;
}

template <typename TC, int V>
__device__ __forceinline__ void store_vec(TC* to, const float (&f)[V], float scale, float r) {
  Vec<TC, V> o;
#pragma unroll
  for (int j = 0; j < V; ++j) {
    if constexpr (sizeof(TC) != 1)
      o.e[j] = from_f32<TC>(f[j]);
    else if constexpr (V == 1)
      o.e[j] = static_cast<uint8_t>(e4m3x2(over(f[j], scale, r), 0.f) & 0xFF);
    else if (j % 2 == 0)
      reinterpret_cast<uint16_t*>(o.e)[j / 2] = e4m3x2(over(f[j], scale, r), over(f[j + 1], scale, r));
  }
  *reinterpret_cast<Vec<TC, V>*>(to) = o;
}

__device__ __forceinline__ void turn(float& x, float& y, float2 c) {
  const float re = x * c.x - y * c.y;
  y = y * c.x + x * c.y;
  x = re;
}

// The cosines and sines of a token: its P neighbouring pairs in n vectors, kept two at a time vector by vector, so that the
// threads of a row read side by side (8192 x 72 x 128: 46.6 us, 48.9 in the order of the pairs; 2000 x 40 x 128: 7.8, 10.5).
template <int P>
__device__ __forceinline__ int angle_place(int pair, int n) {
  return P == 1 ? pair : (pair % P / 2 * n + pair / P) * 2 + pair % 2;
}

template <int P>
__device__ __forceinline__ void angles(const float2* cs, int n, int vec, float2 (&c)[P]) {
  if constexpr (P == 1) {
    c[0] = cs[vec];
  } else {
#pragma unroll
    for (int j = 0; j < P; j += 2) {
      const float4 two = *reinterpret_cast<const float4*>(cs + (j / 2 * n + vec) * 2);
      c[j] = make_float2(two.x, two.y);
      c[j + 1] = make_float2(two.z, two.w);
    }
  }
}

template <typename T, typename TC, int V, bool APPEND>
__global__ void __launch_bounds__(kThreads, kBlocks) rotary_rows_kernel(const __grid_constant__ RowParams p) {
  __shared__ __align__(16) float2 cs[kMaxCs];
  __shared__ int64_t at_k[APPEND ? kMaxTok : 1], at_v[APPEND ? kMaxTok : 1];
  __shared__ int at_pos[APPEND ? kMaxTok : 1];
  __shared__ int first_seq;
  const int heads = p.Hq + 2 * p.Hkv;  // of a token
  const int64_t r0 = static_cast<int64_t>(blockIdx.x) * p.rows_per_block;
  const int rows = static_cast<int>(min(static_cast<int64_t>(p.rows_per_block), p.rows - r0));
  const int tok0 = static_cast<int>(r0 / heads), in0 = static_cast<int>(r0 - static_cast<int64_t>(tok0) * heads);
  const int toks = p.by_heads.div(in0 + rows - 1) + 1;
  const int tid = threadIdx.x, half = p.R / 2;
  int item;
  const int lane_row = p.by_row.div(tid, item), step = kThreads / p.row_threads;  // this thread's first row, and the next
  pdl_trigger();
  if (APPEND && tid == 0) first_seq = 0;
  pdl_wait();

  constexpr int K = kItems<T, V>;
  static_assert(K * kThreads * 2 * V >= kMaxDim, "a block holds every item of a row");
  constexpr bool kAsync = sizeof(Vec<T, V>) == 16;  // rows wait in shared memory; narrow ones in registers
  constexpr int kSlots = kAsync ? kAhead : 1;
  __shared__ Vec<T, V> ring[kAsync ? kAhead : 1][kAsync ? 2 * K : 1][kAsync ? kThreads : 1];
  Vec<T, V> wa[K], wb[K];
  int e0[K], e1[K], v0[K], v1[K];  // places of this thread's items, in turned rows and in rows of values
#pragma unroll
  for (int i = 0; i < K; ++i) {
    e0[i] = e1[i] = v0[i] = v1[i] = -1;
    if (item + i * p.row_threads >= p.items) continue;
    places<V>(p, item + i * p.row_threads, false, e0[i], e1[i]);
    if (APPEND) places<V>(p, item + i * p.row_threads, true, v0[i], v1[i]);
  }
  const auto load = [&](int row, int slot) {
    if (row < rows) {
      int head;
      const int64_t t = tok0 + p.by_heads.div(in0 + row, head);
      const T* src;
      bool value = false;
      if (!APPEND || head < p.Hq) {
        src = static_cast<const T*>(p.q) + t * p.q_t + head * p.q_h;
      } else if (head < p.Hq + p.Hkv) {
        src = static_cast<const T*>(p.k) + t * p.k_t + (head - p.Hq) * p.k_h;
      } else {
        src = static_cast<const T*>(p.v) + t * p.v_t + (head - p.Hq - p.Hkv) * p.v_h;
        value = true;
      }
#pragma unroll
      for (int i = 0; i < K; ++i) {
        const int x = value ? v0[i] : e0[i], y = value ? v1[i] : e1[i];
        if constexpr (kAsync) {
          if (x >= 0) copy_async<16>(&ring[slot][2 * i][tid], src + x);
          if (y >= 0) copy_async<16>(&ring[slot][2 * i + 1][tid], src + y);
        } else {
          if (x >= 0) wa[i] = *reinterpret_cast<const Vec<T, V>*>(src + x);
          if (y >= 0) wb[i] = *reinterpret_cast<const Vec<T, V>*>(src + y);
        }
      }
    }
    if constexpr (kAsync) copy_commit();
  };
  const auto finish = [&](int row) {
    int head;
    const int tok = p.by_heads.div(in0 + row, head);  // in the block
    const bool value = APPEND && head >= p.Hq + p.Hkv, query = !APPEND || head < p.Hq;
    const int64_t t = tok0 + tok;
    if (APPEND && (query ? at_pos[tok] < 0 : at_k[tok] < 0)) {  // a row that belongs to no sequence, or has no place
      if (!query || !p.zero_left) return;
      T* out = static_cast<T*>(p.qo) + t * p.o_t + head * p.o_h;
      const Vec<T, V> zeros = {};
#pragma unroll
      for (int i = 0; i < K; ++i) {
        if (e0[i] >= 0) *reinterpret_cast<Vec<T, V>*>(out + e0[i]) = zeros;
        if (e1[i] >= 0) *reinterpret_cast<Vec<T, V>*>(out + e1[i]) = zeros;
      }
      return;
    }
    const int h = head - p.Hq - (value ? p.Hkv : 0);
    T* out = static_cast<T*>(p.qo) + t * p.o_t + head * p.o_h;
    TC* to = nullptr;
    float scale = 1.f, r = 1.f;
    if (APPEND && !query) {
      to = value ? static_cast<TC*>(p.vc) + at_v[tok] + h * p.v_head : static_cast<TC*>(p.kc) + at_k[tok] + h * p.k_head;
      const float* scales = value ? p.v_scale : p.k_scale;
      if (sizeof(TC) == 1 && scales) {
        scale = scales[h];
        r = __frcp_rn(scale);
      }
    }
#pragma unroll
    for (int i = 0; i < K; ++i) {
      float x[V], y[V];
#pragma unroll
      for (int j = 0; j < V; ++j) x[j] = to_f32(wa[i].e[j]), y[j] = to_f32(wb[i].e[j]);
      const int at = item + i * p.row_threads;
      if (!value && at < p.rot_items) {
        const float2* f = cs + tok * half;
        if (p.interleaved && V > 1) {
          constexpr int P = V > 1 ? V / 2 : 1;
          float2 c[P], d[P];
          angles<P>(f, half / P, at, c);
          angles<P>(f, half / P, at + p.rot_items, d);
#pragma unroll
          for (int j = 0; j < P; ++j) {
            turn(x[2 * j], x[(2 * j + 1) % V], c[j]);
            turn(y[2 * j], y[(2 * j + 1) % V], d[j]);
          }
        } else {
          float2 c[V];
          angles<V>(f, half / V, at, c);
#pragma unroll
          for (int j = 0; j < V; ++j) turn(x[j], y[j], c[j]);
        }
      }
      const int p0 = value ? v0[i] : e0[i], p1 = value ? v1[i] : e1[i];
      if (!APPEND || query) {
        if (p0 >= 0) store_vec<T, V>(out + p0, x, 1.f, 1.f);
        if (p1 >= 0) store_vec<T, V>(out + p1, y, 1.f, 1.f);
      } else {
        if (p0 >= 0) store_vec<TC, V>(to + p0, x, scale, r);
        if (p1 >= 0) store_vec<TC, V>(to + p1, y, scale, r);
      }
    }
  };

  const bool mine = lane_row < step;  // the last threads may be no whole row
  const int first = mine ? lane_row : rows;
#pragma unroll
  for (int i = 0; i < kSlots; ++i) load(first + i * step, i);

  if constexpr (APPEND) {
    if (p.indptr) {  // the sequence of the block's first token: how many end before it
      __syncthreads();
      int before = 0;
      for (int j = 1 + tid; j <= p.B; j += kThreads) before += p.indptr[j] <= tok0;
      before = __reduce_add_sync(0xffffffffu, before);
      if ((tid & 31) == 0 && before) atomicAdd(&first_seq, before);
      __syncthreads();
    }
    if (tid < toks) {
      const int t = tok0 + tid;
      int seq = t, end = t + 1;
      bool in = t < p.B;
      if (p.indptr) {
        seq = first_seq;
        while (seq < p.B && p.indptr[seq + 1] <= t) ++seq;
        in = seq < p.B && p.indptr[seq] <= t;
        if (in) end = p.indptr[seq + 1];
      }
      const int pos = in ? max(p.lens[seq], 0) - (end - t) : -1;  // (from a negative length it may pass -2^31)
      int64_t place = -1;
      int slot = 0;
      if (pos >= 0) {
        const int page = p.by_page.div(pos, slot);
        if (page < p.table_pages) place = p.table[seq * p.table_ld + page];
        if (place < 0 || place >= p.pages) {
          atomicOr(&g_paged_error, 2u);
          place = -1;
        }
      }
      at_pos[tid] = pos;
      at_k[tid] = place < 0 ? -1 : place * p.k_page + slot * p.k_slot;
      at_v[tid] = place * p.v_page + slot * p.v_slot;
    }
    __syncthreads();
  }
  for (int i = tid; i < toks * half; i += kThreads) {
    int f;
    const int tok = p.by_half.div(i, f);
    int64_t pos = 0;
    if (p.positions)
      pos = p.positions64 ? static_cast<const int64_t*>(p.positions)[tok0 + tok]
                          : static_cast<const int32_t*>(p.positions)[tok0 + tok];
    else if (APPEND)
      pos = at_pos[tok];
    const uint64_t turns = static_cast<uint64_t>(pos) * static_cast<uint64_t>(p.freqs[f]);
    float s, c;
    sincospif(static_cast<float>(static_cast<int32_t>(turns >> 32)) * 4.656612873e-10f, &s, &c);  // 2^-31
    constexpr int P = V > 1 ? V / 2 : 1;
    const int place = p.interleaved ? angle_place<P>(f, half / P) : angle_place<V>(f, half / V);
    cs[tok * half + place] = make_float2(c * p.cos_scale, s * p.sin_scale);
  }
  __syncthreads();

  // Two rows of a thread on their way through shared memory (8192 x 72 x 128: 46.6 us; about 2 more with one row; 55 with
  // one in registers, where two take room from other warps: 64).  A third finds no room beside the angles.
  int slot = 0;
#pragma unroll 1
  for (int row = first; row < rows; row += step) {
    if constexpr (kAsync) {
      copy_wait<kSlots - 1>();
#pragma unroll
      for (int i = 0; i < K; ++i) wa[i] = ring[slot][2 * i][tid], wb[i] = ring[slot][2 * i + 1][tid];
      load(row + kSlots * step, slot);
      slot = slot + 1 == kSlots ? 0 : slot + 1;
    }
    finish(row);
    if constexpr (!kAsync) load(row + step, 0);
  }
}

template <typename T, typename TC, int V, bool APPEND>
int launch_rows(RowParams p, cudaStream_t st) {
  const int heads = p.Hq + 2 * p.Hkv, half = p.R / 2;
  p.rot_items = half / V;
  p.items = p.rot_items + static_cast<int>(ceil_div(p.D - p.R, 2 * V));
  p.row_threads = static_cast<int>(ceil_div(p.items, kItems<T, V>));
  p.by_row = FastDiv(p.row_threads);
  p.by_heads = FastDiv(heads);
  p.by_half = FastDiv(half > 0 ? half : 1);
  // Rows of a block: as many rounds for each thread as make whole waves of blocks, up to kRounds (a block's start, with its
  // angles, costs about two rounds; 8192 x 72 x 128 takes 46.6 us, 47.3 with up to 16; an append of 16384 x 80 76.3 and 77.5,
  // and 4 more with up to 8), and no more tokens than have room.
  const int tokens = std::min(kMaxTok, half > 0 ? kMaxCs / half : kMaxTok);
  const int64_t step = kThreads / p.row_threads, slots = kBlocks * num_sms();
  const int64_t rounds = ceil_div(ceil_div(p.rows, step), slots), waves = ceil_div(rounds, kRounds);
  int64_t rows = ceil_div(rounds, waves) * step;
  rows = std::min(rows, static_cast<int64_t>(tokens - 1) * heads + 1);  // rows from anywhere in a token touch no more
  p.rows_per_block = static_cast<int>(std::max<int64_t>(1, rows));
  return launch_pdl("rotary_rows_kernel", rotary_rows_kernel<T, TC, V, APPEND>,
                    dim3(static_cast<unsigned>(ceil_div(p.rows, p.rows_per_block))), dim3(kThreads), 0, st, p);
}

// Rows in vectors of 16, 8 or 4 bytes or single elements: the widest that every start, stride and part of a head allows.
template <typename T, typename TC, bool APPEND>
int launch_vec(const RowParams& p, uint64_t starts_t, uint64_t starts_c, uint64_t elems, cudaStream_t st) {
  constexpr int kFull = 16 / sizeof(T), kHalf = 8 / sizeof(T), kFourth = 4 / sizeof(T);
  const auto fits = [&](int v) {
    return starts_t % (v * sizeof(T)) == 0 && starts_c % (v * sizeof(TC)) == 0 && elems % v == 0;
  };
  if (fits(kFull)) return launch_rows<T, TC, kFull, APPEND>(p, st);
  if (fits(kHalf)) return launch_rows<T, TC, kHalf, APPEND>(p, st);
  if (kFourth > 1 && fits(kFourth)) return launch_rows<T, TC, kFourth, APPEND>(p, st);
  return launch_rows<T, TC, 1, APPEND>(p, st);
}

// A gcd by powers of two of everything that a vector's width has to divide: the lowest set bit of the union of the bits.
uint64_t lowest(uint64_t bits) { return bits ? bits & (~bits + 1) : 1ull << 32; }

int check_rotary(const w4a8_rotary* r, int64_t D, bool needs_positions) {
  if (!r || !r->freqs) return W4A8_OK;
  W4A8_REQUIRE(r->R >= 0 && r->R % 2 == 0 && r->start >= 0 && r->start + r->R <= D,
               "R=%lld must be even and start=%lld + R at most D=%lld", (long long)r->R, (long long)r->start, (long long)D);
  W4A8_REQUIRE(r->scale - r->scale == 0.f, "scale must be finite");
  W4A8_REQUIRE(!needs_positions || r->positions, "null pointer: positions");
  W4A8_REQUIRE(bits_of(r->freqs) % 8 == 0 && bits_of(r->positions) % (r->positions64 ? 8 : 4) == 0,
               "freqs and positions must be aligned to their element size");
  return W4A8_OK;
}

void set_rotary(RowParams& p, const w4a8_rotary* r) {
  if (!r || !r->freqs) return;  // p.R stays 0: nothing is turned
  p.R = static_cast<int>(r->R);
  p.start = static_cast<int>(r->start);
  p.freqs = r->freqs;
  p.positions = r->positions;
  p.positions64 = r->positions64 != 0;
  p.interleaved = r->interleaved != 0;
  p.cos_scale = r->scale;
  p.sin_scale = r->inverse ? -r->scale : r->scale;
}

int read_paged_error() {
  unsigned int v = 0;
  cudaMemcpyFromSymbol(&v, g_paged_error, sizeof(v));
  const unsigned int zero = 0;
  cudaMemcpyToSymbol(g_paged_error, &zero, sizeof(zero));
  return static_cast<int>(v);
}

struct Registrar {
  Registrar() { register_device_error_reader(&read_paged_error); }
} registrar;

}  // namespace
}  // namespace w4a8

extern "C" int rotary_embedding(const void* x, int64_t ldx_t, int64_t ldx_h, int dtype, int64_t T, int64_t H, int64_t D,
                                const w4a8_rotary* rotary, void* out, int64_t ldo_t, int64_t ldo_h, void* stream) {
  using namespace w4a8;
  W4A8_REQUIRE(dtype >= W4A8_DTYPE_BF16 && dtype <= W4A8_DTYPE_F32, "dtype=%d must be bf16, f16 or fp32", dtype);
  W4A8_REQUIRE(D >= 1 && D <= kMaxDim, "D=%lld must be in [1, %d]", (long long)D, kMaxDim);
  W4A8_REQUIRE(T >= 0 && H >= 0 && T < (1ll << 31) && H < (1ll << 31) && T * H < (1ll << 31),
               "T=%lld times H=%lld must be below 2^31", (long long)T, (long long)H);
  W4A8_REQUIRE(ldx_t >= 0 && ldx_h >= 0 && ldo_t >= 0 && ldo_h >= 0, "strides must not be negative");
  W4A8_REQUIRE(rotary && rotary->freqs, "null pointer: rotary, freqs");
  if (T == 0 || H == 0) return W4A8_OK;
  if (int rc = check_rotary(rotary, D, true)) return rc;
  W4A8_REQUIRE(x && out, "null pointer");
  const uint64_t size = dtype_size(dtype);
  W4A8_REQUIRE((bits_of(x) | bits_of(out)) % size == 0, "x and out must be aligned to their element size");
  RowParams p = {};
  set_rotary(p, rotary);
  p.q = x;
  p.qo = out;
  p.q_t = ldx_t;
  p.q_h = ldx_h;
  p.o_t = ldo_t;
  p.o_h = ldo_h;
  p.T = static_cast<int>(T);
  p.Hq = static_cast<int>(H);
  p.D = static_cast<int>(D);
  p.rows = T * H;
  const uint64_t starts = lowest(bits_of(x) | bits_of(out) | (T > 1 ? (ldx_t | ldo_t) * size : 0) |
                                 (H > 1 ? (ldx_h | ldo_h) * size : 0));
  const uint64_t elems = lowest(static_cast<uint64_t>(p.D | p.start | p.R / 2));
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (dtype == W4A8_DTYPE_F32) return launch_vec<float, float, false>(p, starts, starts, elems, st);
  if (dtype == W4A8_DTYPE_F16) return launch_vec<__half, __half, false>(p, starts, starts, elems, st);
  return launch_vec<__nv_bfloat16, __nv_bfloat16, false>(p, starts, starts, elems, st);
}

namespace w4a8 {
namespace {

int append(const void* k, int64_t ldk_t, int64_t ldk_h, const void* v, int64_t ldv_t, int64_t ldv_h, int dtype, int64_t T,
           const int32_t* indptr, const w4a8_paged_cache* cache, const w4a8_rotary* rotary, const void* q, int64_t ldq_t,
           int64_t ldq_h, int64_t Hq, void* q_out, int64_t ldqo_t, int64_t ldqo_h, bool zero_left, void* stream) {
  if (int rc = check_cache(cache, dtype)) return rc;
  const int64_t D = cache->D, H = cache->heads;
  W4A8_REQUIRE(D >= 1 && D <= kMaxDim, "D=%lld must be in [1, %d]", (long long)D, kMaxDim);
  W4A8_REQUIRE(Hq >= 0 && Hq < (1 << 16) && (q || Hq == 0), "Hq=%lld must be in [0, 2^16), and 0 without q", (long long)Hq);
  W4A8_REQUIRE(T >= 0 && T < (1ll << 31) && T * (Hq + 2 * H) < (1ll << 31), "T=%lld rows of %lld heads: below 2^31",
               (long long)T, (long long)(Hq + 2 * H));
  W4A8_REQUIRE(indptr || T >= cache->B, "T=%lld must be at least B=%lld without indptr", (long long)T, (long long)cache->B);
  W4A8_REQUIRE(bits_of(indptr) % 4 == 0, "indptr must be aligned to 4 bytes");
  W4A8_REQUIRE(ldk_t >= 0 && ldk_h >= 0 && ldv_t >= 0 && ldv_h >= 0 && ldq_t >= 0 && ldq_h >= 0 && ldqo_t >= 0 && ldqo_h >= 0,
               "strides must not be negative");
  if (int rc = check_rotary(rotary, D, false)) return rc;
  zero_left = zero_left && q && Hq > 0;
  if (T == 0 || (cache->B == 0 && !zero_left)) return W4A8_OK;
  W4A8_REQUIRE(k && v && (cache->B == 0 || cache->seq_lens) && (!q || Hq == 0 || q_out), "null pointer");
  W4A8_REQUIRE(cache->B == 0 || cache->table_pages == 0 || cache->page_table, "null pointer: page_table");
  W4A8_REQUIRE(cache->pages == 0 || (cache->k && cache->v), "null pointer: k and v of the cache");
  const bool fp8 = cache->dtype == W4A8_DTYPE_E4M3;
  const uint64_t size = 2, csize = fp8 ? 1 : 2;
  const uint64_t qs = q && Hq ? bits_of(q) | bits_of(q_out) : 0;
  W4A8_REQUIRE((bits_of(k) | bits_of(v) | qs) % size == 0 && (bits_of(cache->k) | bits_of(cache->v)) % csize == 0,
               "k, v, q, q_out and the cache must be aligned to their element size");
  RowParams p = {};
  p.cos_scale = p.sin_scale = 1.f;
  p.zero_left = zero_left;
  set_rotary(p, rotary);
  p.q = q;
  p.qo = q_out;
  p.k = k;
  p.v = v;
  p.kc = cache->k;
  p.vc = cache->v;
  p.q_t = ldq_t;
  p.q_h = ldq_h;
  p.o_t = ldqo_t;
  p.o_h = ldqo_h;
  p.k_t = ldk_t;
  p.k_h = ldk_h;
  p.v_t = ldv_t;
  p.v_h = ldv_h;
  p.k_page = cache->k_page;
  p.k_slot = cache->k_slot;
  p.k_head = cache->k_head;
  p.v_page = cache->v_page;
  p.v_slot = cache->v_slot;
  p.v_head = cache->v_head;
  p.table = cache->page_table;
  p.table_ld = cache->table_ld;
  p.table_pages = static_cast<int>(cache->table_pages);
  p.pages = cache->pages;
  p.lens = cache->seq_lens;
  p.indptr = indptr;
  p.k_scale = cache->k_scale;
  p.v_scale = cache->v_scale;
  p.by_page = FastDiv(cache->page_size);
  p.T = static_cast<int>(T);
  p.B = static_cast<int>(cache->B);
  p.Hq = q ? static_cast<int>(Hq) : 0;
  p.Hkv = static_cast<int>(H);
  p.D = static_cast<int>(D);
  p.rows = T * (p.Hq + 2 * H);
  const uint64_t starts = lowest(bits_of(k) | bits_of(v) | qs | (ldk_t | ldk_h | ldv_t | ldv_h) * size |
                                 (qs ? (ldq_t | ldq_h | ldqo_t | ldqo_h) * size : 0));
  const uint64_t places = lowest(bits_of(cache->k) | bits_of(cache->v) |
                                 (p.k_page | p.k_slot | p.k_head | p.v_page | p.v_slot | p.v_head) * csize);
  const uint64_t elems = lowest(static_cast<uint64_t>(p.D | p.start | p.R / 2));
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (dtype == W4A8_DTYPE_F16)
    return fp8 ? launch_vec<__half, uint8_t, true>(p, starts, places, elems, st)
               : launch_vec<__half, __half, true>(p, starts, places, elems, st);
  return fp8 ? launch_vec<__nv_bfloat16, uint8_t, true>(p, starts, places, elems, st)
             : launch_vec<__nv_bfloat16, __nv_bfloat16, true>(p, starts, places, elems, st);
}

}  // namespace
}  // namespace w4a8

extern "C" int paged_kv_append(const void* k, int64_t ldk_t, int64_t ldk_h, const void* v, int64_t ldv_t, int64_t ldv_h,
                               int dtype, int64_t T, const int32_t* indptr, const w4a8_paged_cache* cache,
                               const w4a8_rotary* rotary, const void* q, int64_t ldq_t, int64_t ldq_h, int64_t Hq,
                               void* q_out, int64_t ldqo_t, int64_t ldqo_h, void* stream) {
  return w4a8::append(k, ldk_t, ldk_h, v, ldv_t, ldv_h, dtype, T, indptr, cache, rotary, q, ldq_t, ldq_h, Hq, q_out, ldqo_t,
                      ldqo_h, false, stream);
}

extern "C" int paged_kv_append_whole(const void* k, int64_t ldk_t, int64_t ldk_h, const void* v, int64_t ldv_t, int64_t ldv_h,
                                     int dtype, int64_t T, const int32_t* indptr, const w4a8_paged_cache* cache,
                                     const w4a8_rotary* rotary, const void* q, int64_t ldq_t, int64_t ldq_h, int64_t Hq,
                                     void* q_out, int64_t ldqo_t, int64_t ldqo_h, void* stream) {
  return w4a8::append(k, ldk_t, ldk_h, v, ldv_t, ldv_h, dtype, T, indptr, cache, rotary, q, ldq_t, ldq_h, Hq, q_out, ldqo_t,
                      ldqo_h, true, stream);
}
