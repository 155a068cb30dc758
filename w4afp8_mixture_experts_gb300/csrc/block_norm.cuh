// The norms after and before a block in one pass over a token's row, with the block's gate and residual:
//   u = norm_post(f)      h = residual_scale * r + branch_scale * gate * u      y = norm_pre(h)
// norm in {none, rms, layer}; sums and the values between the two norms stay in fp32 registers, h and y are
// each rounded once (y from the unrounded h).  A LayerNorm takes the mean first, then the squared differences from it.
//
// Bound by memory (each of f, r, h and y once).  Two kernels:
//   row kernel: a row to a block, or to 8, 16 or 32 lanes.  64 x 7168 bf16 takes 3.6 us, of which a launch is 2.5.
//   streaming kernel (many rows): blocks stay and copy the rows to come into a ring in shared memory.
//     8192 x 7168 bf16 with a channel gate: 79 us, 5.9 TB/s (a row to a block: 134 us).  3001 x 5119 f16 with an fp32
//     residual, two LayerNorms, a gate per token and no alignment: 44 us, 4.2 TB/s; there it is bound by the latency of
//     four reductions a row, in 10 rounds of two rows to each block.
#pragma once

#include <algorithm>
#include <type_traits>

#include "block_ops.cuh"
#include "common.cuh"

namespace w4a8 {

constexpr int kMaxH = 32768;

struct NormParams {
  const void* f;
  const void* r;       // nullptr: no residual
  const void* gate;    // nullptr: 1
  const void* w_post;  // nullptr: 1
  const void* b_post;  // nullptr: 0
  const void* w_pre;
  const void* b_pre;
  void* h;  // nullptr: not wanted
  void* y;  // nullptr: not wanted
  int64_t ldf, ldr, ldg, ldh, ldy;
  int T, H;
  int post, pre;      // w4a8_norm
  int rows_per_gate;  // row t uses gate row t / rows_per_gate
  int gate_scalar;    // one gate value per gate row
  int gate_f32, w_f32;
  float branch_scale, residual_scale, eps;
};

// the kernels for one type of f and y, and of the residual and h; `vec`: rows start on 16-byte boundaries
int launch_norm_bf16(const NormParams& p, bool residual_f32, bool vec, cudaStream_t st);
int launch_norm_f16(const NormParams& p, bool residual_f32, bool vec, cudaStream_t st);
int launch_norm_f32(const NormParams& p, bool vec, cudaStream_t st);

namespace {

template <typename T, int V>
struct alignas(V * sizeof(T) > 16 ? 16 : V * sizeof(T)) Pack {
  T v[V];
};

template <typename T, int V>
__device__ __forceinline__ void load_vec(const T* p, float (&o)[V]) {
  const Pack<T, V> a = *reinterpret_cast<const Pack<T, V>*>(p);
#pragma unroll
  for (int i = 0; i < V; ++i) o[i] = to_f32(a.v[i]);
}
template <typename T, int V>
__device__ __forceinline__ void store_vec(T* p, const float (&o)[V]) {
  if constexpr (V == 8 && sizeof(T) == 2) {
    *reinterpret_cast<uint4*>(p) = make_uint4(pack2<T>(o[0], o[1]), pack2<T>(o[2], o[3]), pack2<T>(o[4], o[5]),
                                              pack2<T>(o[6], o[7]));
  } else if constexpr (V == 4 && sizeof(T) == 2) {
    *reinterpret_cast<uint2*>(p) = make_uint2(pack2<T>(o[0], o[1]), pack2<T>(o[2], o[3]));
  } else {
    Pack<T, V> a;
#pragma unroll
    for (int i = 0; i < V; ++i) a.v[i] = from_f32<T>(o[i]);
    *reinterpret_cast<Pack<T, V>*>(p) = a;
  }
}
// the V elements at column c of a row of H, zeros from H on (only a row's last vector can be cut short)
template <typename T, int V>
__device__ __forceinline__ void load_cut(const T* row, int c, int H, float (&o)[V]) {
  if (c + V <= H) {
    load_vec<T, V>(row + c, o);
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) o[i] = c + i < H ? to_f32(row[c + i]) : 0.f;
  }
}
template <typename T, int V>
__device__ __forceinline__ void store_cut(T* row, int c, int H, const float (&o)[V]) {
  if (c + V <= H) {
    store_vec<T, V>(row + c, o);
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (c + i < H) row[c + i] = from_f32<T>(o[i]);
  }
}
// a parameter vector: fp32 or the activations' type
template <typename X, int V>
__device__ __forceinline__ void load_param(const void* p, int f32, int64_t at, float (&o)[V]) {
  if (f32)
    load_vec<float, V>(static_cast<const float*>(p) + at, o);
  else
    load_vec<X, V>(static_cast<const X*>(p) + at, o);
}

// Sum over the row's threads (8, 16 or a multiple of 32 of them); the same value on all of them.  `slot` alternates
// between two halves of the scratch so that one barrier per reduction is enough.
__device__ __forceinline__ float row_sum(float v, float* scratch, int& slot) {
  if (blockDim.x < 32) {
    for (int o = blockDim.x >> 1; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
  }
  v = warp_sum(v);
  const int warps = blockDim.x >> 5;
  if (warps == 1) return v;
  float* s = scratch + slot;
  slot ^= 32;
  if ((threadIdx.x & 31) == 0) s[threadIdx.x >> 5] = v;
  __syncthreads();
  const int lane = threadIdx.x & 31;
  return warp_sum(lane < warps ? s[lane] : 0.f);
}

// `count(j)`: how many elements of this thread's vector j are the row's (at least V: all)
template <int V, int VPT, class C>
__device__ __forceinline__ void normalise(float (&u)[VPT][V], int kind, int H, float eps, float* scratch, int& slot,
                                          C&& count) {
  float s = 0.f;
  if (kind == W4A8_NORM_LAYER) {
#pragma unroll
    for (int j = 0; j < VPT; ++j)
#pragma unroll
      for (int i = 0; i < V; ++i) s += u[j][i];
    const float mean = row_sum(s, scratch, slot) / H;
    s = 0.f;
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
      const int left = count(j);
#pragma unroll
      for (int i = 0; i < V; ++i) u[j][i] = i < left ? u[j][i] - mean : 0.f;
    }
  }
#pragma unroll
  for (int j = 0; j < VPT; ++j)
#pragma unroll
    for (int i = 0; i < V; ++i) s = fmaf(u[j][i], u[j][i], s);
  const float inv = rsqrtf(row_sum(s, scratch, slot) / H + eps);
#pragma unroll
  for (int j = 0; j < VPT; ++j)
#pragma unroll
    for (int i = 0; i < V; ++i) u[j][i] *= inv;
}

// Threads of a row where the kernel's code fixes them (0: blockDim.x): with many single elements to a thread, columns
// that are known offsets from the first leave registers for the elements.
__host__ __device__ constexpr int row_threads(int V, int VPT) { return V == 1 && VPT > 8 ? 1024 : 0; }

// A row to a block (or, for short rows, to 8, 16 or 32 threads): VPT vectors of V elements to a thread.
//   V > 1: aligned rows; their last vector may be cut short.
//   V > 1, CUT: rows of any start, as long as f, r, h and y agree on where the row starts within V elements: the whole
//     aligned vectors go to the row's threads, and the up to 2 * (V - 1) elements beside them to one more warp's lanes.
template <typename X, typename R, int V, bool CUT, int VPT>
__global__ void __launch_bounds__(1024) block_norm_row_kernel(const NormParams p) {
  __shared__ float scratch[64];
  pdl_trigger();
  pdl_wait();
  int slot = 0;
  const int H = p.H;
  const int64_t row = static_cast<int64_t>(blockIdx.x) * blockDim.y + threadIdx.y;
  const bool here = row < p.T;  // where several rows share a warp, all of its lanes stay for the shuffles
  const int64_t t = here ? row : p.T - 1;
  const int tx = threadIdx.x, nx = row_threads(V, VPT) ? row_threads(V, VPT) : blockDim.x - (CUT ? 32 : 0);
  const int64_t start = static_cast<int64_t>(reinterpret_cast<uintptr_t>(p.f) / sizeof(X)) + t * p.ldf;
  const int head = CUT ? min(static_cast<int>(-start & (V - 1)), H) : 0;
  const int vectors = (H - head) / V;  // CUT: whole ones
  const bool single = CUT && tx >= nx;
  // this thread's first column
  const int first = !single ? head + tx * V : tx - nx + (tx - nx < head ? 0 : vectors * V);
  const auto col = [&](int j) { return CUT ? first + j * nx * V : (j * nx + tx) * V; };
  const auto count = [&](int j) {  // the row's elements in vector j
    if (!CUT) return H - col(j);
    return single ? (j == 0 && first < H ? 1 : 0) : j * nx + tx < vectors ? V : 0;
  };
  // a vector of a matrix's row, or of a parameter (which CUT may leave unaligned); zeros beside the row
  const auto load = [&](auto type, const void* q, int64_t at, int j, bool aligned, float (&o)[V])
                        __attribute__((always_inline)) {
    using T = decltype(type);
    const T* from = static_cast<const T*>(q) + at;
    if constexpr (!CUT) {
      load_cut<T, V>(from, col(j), H, o);
    } else if (aligned && !single) {
      if (count(j)) {
        load_vec<T, V>(from + col(j), o);
      } else {
#pragma unroll
        for (int i = 0; i < V; ++i) o[i] = 0.f;
      }
    } else {
#pragma unroll
      for (int i = 0; i < V; ++i) o[i] = i < count(j) ? to_f32(from[col(j) + i]) : 0.f;
    }
  };
  const auto store = [&](auto type, void* q, int64_t at, int j, const float (&o)[V]) __attribute__((always_inline)) {
    using T = decltype(type);
    T* to = static_cast<T*>(q) + at;
    if constexpr (!CUT) {
      store_cut<T, V>(to, col(j), H, o);
    } else if (!single) {
      if (count(j)) store_vec<T, V>(to + col(j), o);
    } else {
      if (count(j)) to[first] = from_f32<T>(o[0]);
    }
  };
  // A parameter or matrix row over this thread's columns, given to f(j, values) vector by vector.  Single elements are
  // loaded 8 at a time, inside one branch on the type: a branch around each of them waited for each load by itself.
  const auto with = [&](const void* q, int f32, int64_t at, bool aligned, auto&& f) __attribute__((always_inline)) {
    constexpr int kAtOnce = V > 1 ? 1 : VPT > 8 ? 4 : VPT;
#pragma unroll
    for (int j0 = 0; j0 < VPT; j0 += kAtOnce) {
      float a[kAtOnce][V];
      if (f32) {
#pragma unroll
        for (int j = 0; j < kAtOnce; ++j) load(float(), q, at, j0 + j, aligned, a[j]);
      } else {
#pragma unroll
        for (int j = 0; j < kAtOnce; ++j) load(X(), q, at, j0 + j, aligned, a[j]);
      }
#pragma unroll
      for (int j = 0; j < kAtOnce; ++j) f(j0 + j, a[j]);
    }
  };
  constexpr bool kEarly = V * VPT <= (V > 1 ? 16 : 8);  // the residual is loaded with f, where registers hold both
  float u[VPT][V], r[kEarly ? VPT : 1][V];
#pragma unroll
  for (int j = 0; j < VPT; ++j) load(X(), p.f, t * p.ldf, j, true, u[j]);
  if (kEarly && p.r) {
#pragma unroll
    for (int j = 0; j < VPT; ++j) load(R(), p.r, t * p.ldr, j, true, r[j]);
  }
  const auto scale = [&](const void* q, int f32, int64_t at) __attribute__((always_inline)) {
    if (q)
      with(q, f32, at, false, [&](int j, const float (&a)[V]) {
#pragma unroll
        for (int i = 0; i < V; ++i) u[j][i] *= a[i];
      });
  };
  const auto shift = [&](const void* b) __attribute__((always_inline)) {
    if (b)
      with(b, p.w_f32, 0, false, [&](int j, const float (&a)[V]) {
#pragma unroll
        for (int i = 0; i < V; ++i) u[j][i] += a[i];
      });
  };
  if (p.post != W4A8_NORM_NONE) {
    normalise<V, VPT>(u, p.post, H, p.eps, scratch, slot, count);
    scale(p.w_post, p.w_f32, 0);
    shift(p.b_post);
  }
  float gs = p.branch_scale;
  if (p.gate) {
    const int64_t grow = t / p.rows_per_gate * p.ldg;
    if (p.gate_scalar) {
      float a[1];
      load_param<X, 1>(p.gate, p.gate_f32, grow, a);
      gs *= a[0];
    } else {
      scale(p.gate, p.gate_f32, grow);
    }
  }
#pragma unroll
  for (int j = 0; j < VPT; ++j)
#pragma unroll
    for (int i = 0; i < V; ++i) {
      u[j][i] *= gs;
      if (kEarly && p.r) u[j][i] = fmaf(p.residual_scale, r[kEarly ? j : 0][i], u[j][i]);
    }
  if (!kEarly && p.r)
    with(p.r, sizeof(R) == 4, t * p.ldr, true, [&](int j, const float (&a)[V]) {
#pragma unroll
      for (int i = 0; i < V; ++i) u[j][i] = fmaf(p.residual_scale, a[i], u[j][i]);
    });
#pragma unroll
  for (int j = 0; j < VPT; ++j) {
    if (p.h && here) store(R(), p.h, t * p.ldh, j, u[j]);
  }
  if (!p.y) return;
  if (p.pre != W4A8_NORM_NONE) {
    normalise<V, VPT>(u, p.pre, H, p.eps, scratch, slot, count);
    scale(p.w_pre, p.w_f32, 0);
    shift(p.b_pre);
  }
#pragma unroll
  for (int j = 0; j < VPT; ++j)
    if (here) store(X(), p.y, t * p.ldy, j, u[j]);
}

// Two fp32 operations in one instruction.
__device__ __forceinline__ uint64_t pair(float x, float y) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(x), "f"(y));
  return r;
}
__device__ __forceinline__ float2 split(uint64_t v) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
  return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}

// Copies the aligned 16-byte pieces that cover row t of a matrix.  A piece that reaches outside the matrix (only its
// first and last one can) is copied element by element.
template <typename T>
__device__ __forceinline__ void fetch_window(uint8_t* dst, const void* base, int64_t ld, int64_t rows, int64_t t, int H) {
  const uintptr_t lo = reinterpret_cast<uintptr_t>(base), hi = lo + ((rows - 1) * ld + H) * sizeof(T);
  const uintptr_t b0 = lo + t * ld * sizeof(T), w0 = b0 & ~uintptr_t(15);
  const int pieces = static_cast<int>((b0 - w0 + H * sizeof(T) + 15) >> 4);
  if (w0 >= lo && w0 + 16 * static_cast<uintptr_t>(pieces) <= hi) {
    for (int i = threadIdx.x; i < pieces; i += blockDim.x)
      copy_async<16>(dst + 16 * i, reinterpret_cast<const void*>(w0 + 16 * i));
    return;
  }
  for (int i = threadIdx.x; i < pieces; i += blockDim.x) {
    const uintptr_t a = w0 + 16 * static_cast<uintptr_t>(i);
    if (a >= lo && a + 16 <= hi) {
      copy_async<16>(dst + 16 * i, reinterpret_cast<const void*>(a));
    } else {
      for (uintptr_t e = a; e < a + 16; e += sizeof(T))
        if (e >= lo && e < hi) *reinterpret_cast<T*>(dst + (e - w0)) = *reinterpret_cast<const T*>(e);
    }
  }
}

// Many rows: blocks stay and stride over them, 16 or 8 elements of a row to a thread and ROWS rows at a time (their
// reductions share the barriers and hide each other's latency).  The weights and biases stay in registers (with
// branch_scale, and a gate that all rows share, multiplied into the first pair), and the rows to come are copied to a ring
// of two or three stages in shared memory asynchronously: registers would not hold enough bytes in flight to cover the
// memory's latency beside the rows that are being worked on.
//   V > 1: rows of whole aligned vectors, of 8 elements, or of 4 beside fp32 ones (every access of a warp then covers
//     whole sectors).  Every thread copies its own pieces and alone reads them back, so there is nothing to synchronise.
//   V > 1, CUT: rows of any width and start, as long as f, r, h and y agree on where a row starts within V elements.
//     That repeats after 8 rows at most, and the number of blocks is a multiple of 8: a block's rows all start alike, and
//     the weights still stay in registers.  The whole aligned vectors of a row go to its threads as before, and the up to
//     2 * (V - 1) elements before and after them to the lanes of one more warp.
//   V = 1: rows that start differently in f, r, h and y, and short or very long ones of odd width or start.  The block
//     copies the 16-byte pieces that cover a row, and threads take single elements from there.
// One stage of the ring (ROWS rows): byte offsets of its parts, and of one row within a part.  V > 1: a thread's
// pieces lie threads of them apart.
struct NormStage {
  int stages, bytes, r_at, g_at;
  int f_row, r_row, g_row;
  bool gate_rows;  // the gate differs between rows and has H columns: it goes through the ring too
};

// Threads of an SM that the registers allow with kE elements to a thread (16: two rows of them in registers).
__host__ __device__ constexpr int max_threads(int elems) { return elems == 16 ? 512 : 768; }

template <typename X, typename R, int V, bool CUT, bool BIAS, int kE>
__global__ void __launch_bounds__(max_threads(kE), 1) block_norm_stream_kernel(const NormParams p, const NormStage st) {
  constexpr int kP = kE / 2;  // pairs of a thread's elements
  constexpr int ROWS = 2;
  extern __shared__ uint8_t ring[];
  __shared__ float2 scratch[2][max_threads(kE) / 32];
  const int threads = blockDim.x * blockDim.y, tid = threadIdx.y * blockDim.x + threadIdx.x;
  const int tx = threadIdx.x, nx = blockDim.x - (CUT ? 32 : 0), H = p.H;
  const int64_t step = static_cast<int64_t>(gridDim.x) * blockDim.y;  // between the rows of a thread
  int64_t t0 = static_cast<int64_t>(blockIdx.x) * blockDim.y + threadIdx.y;
  // CUT: elements before the first whole vector, whole vectors, and whether this thread is of the warp for the others
  const int64_t start = static_cast<int64_t>(reinterpret_cast<uintptr_t>(p.f) / sizeof(X)) + t0 * p.ldf;
  const int head = CUT ? min(static_cast<int>(-start & (V - 1)), H) : 0;
  const int vectors = CUT ? (H - head) / V : (H + V - 1) / V;
  const bool single = CUT && tx >= nx;
  // column of element i: V > 1: vectors nx * V apart; V = 1: elements nx apart.  Elements i < mine exist.
  const int first = !single ? head + tx * V : tx - nx + (tx - nx < head ? 0 : vectors * V);
  int mine = single ? first < H : 0;
#pragma unroll
  for (int i = 0; i < kE; i += V) mine += !single && i / V * nx + tx < vectors ? V : 0;
  auto col = [&](int i) { return first + i / V * nx * V + i % V; };
  auto in = [&](int i) { return i / V * V < mine; };  // for single: of element 0 only
  auto valid = [&](int i) { return CUT ? i < mine : in(i); };
  pdl_trigger();
  pdl_wait();
  auto gate_index = [&](int64_t t) { return static_cast<int64_t>(static_cast<uint32_t>(t) / p.rows_per_gate); };
  const bool odd = (start + first) & 1;  // single, 16 bits: the element is the upper half of its four bytes
  // Copies one row of a matrix of T into its place in the ring.  V > 1: each vector is a piece of 8 or 16 bytes, or two.
  auto piece = [&](uint8_t* at, int bytes, int q) { return at + bytes * (q * threads + tid); };
  auto fetch_part = [&](auto type, const void* base, int64_t ld, int64_t rows, int64_t t, uint8_t* at) {
    using T = decltype(type);
    if constexpr (V > 1) {
      constexpr int kBytes = V * sizeof(T), kPiece = kBytes < 16 ? kBytes : 16, Q = kBytes / kPiece;
      const char* src = reinterpret_cast<const char*>(static_cast<const T*>(base) + t * ld + first);
      if (single) {  // the four bytes around the element, but nothing outside the matrix
        if (!mine) return;
        uint8_t* to = piece(at, kPiece, 0);
        const char* word = src - (sizeof(T) == 2 && odd ? 2 : 0);
        const bool out = sizeof(T) == 2 && (odd ? t == 0 && first == 0 : t == rows - 1 && first == H - 1);
        if (out)
          *reinterpret_cast<T*>(to + (odd ? 2 : 0)) = *reinterpret_cast<const T*>(src);
        else
          copy_async<4>(to, word);
        return;
      }
#pragma unroll
      for (int j = 0; j < kE / V; ++j)
        if (in(V * j)) {
#pragma unroll
          for (int q = 0; q < Q; ++q)
            copy_async<kPiece>(piece(at, kPiece, j * Q + q), src + j * nx * kBytes + kPiece * q);
        }
    } else {
      fetch_window<T>(at, base, ld, rows, t, H);
    }
  };
  auto fetch = [&](int64_t t0, uint8_t* at) {
#pragma unroll
    for (int r = 0; r < ROWS; ++r) {
      const int64_t t = t0 + r * step;
      if (t >= p.T) break;
      fetch_part(X(), p.f, p.ldf, p.T, t, at + r * st.f_row);
      if (p.r) fetch_part(R(), p.r, p.ldr, p.T, t, at + st.r_at + r * st.r_row);
      if (st.gate_rows) {
        uint8_t* g = at + st.g_at + r * st.g_row;
        if (p.gate_f32)
          fetch_part(float(), p.gate, p.ldg, p.T / p.rows_per_gate, gate_index(t), g);
        else
          fetch_part(X(), p.gate, p.ldg, p.T / p.rows_per_gate, gate_index(t), g);
      }
    }
    copy_commit();
  };
  // this thread's elements of one row of the ring; zeros where there are none
  auto take = [&](auto type, const void* base, int64_t ld, int64_t t, uint8_t* at, uint64_t* o) {
    using T = decltype(type);
    if constexpr (V > 1) {
      constexpr int kBytes = V * sizeof(T), kPiece = kBytes < 16 ? kBytes : 16, Q = kBytes / kPiece;
      using Piece = std::conditional_t<kPiece == 16, uint4, uint2>;
      if (single) {
        const uint8_t* from = piece(at, kPiece, 0) + (sizeof(T) == 2 && odd ? 2 : 0);
        o[0] = pair(mine ? to_f32(*reinterpret_cast<const T*>(from)) : 0.f, 0.f);
#pragma unroll
        for (int i = 1; i < kP; ++i) o[i] = 0;
        return;
      }
#pragma unroll
      for (int j = 0; j < kE / V; ++j) {
        Pack<T, V> a;
#pragma unroll
        for (int q = 0; q < Q; ++q)
          reinterpret_cast<Piece*>(&a)[q] =
              in(V * j) ? *reinterpret_cast<const Piece*>(piece(at, kPiece, j * Q + q)) : Piece{};
#pragma unroll
        for (int i = 0; i < V / 2; ++i) o[V / 2 * j + i] = pair(to_f32(a.v[2 * i]), to_f32(a.v[2 * i + 1]));
      }
    } else {
      const T* row =
          reinterpret_cast<const T*>(at + ((reinterpret_cast<uintptr_t>(base) + t * ld * sizeof(T)) & 15)) + tx;
#pragma unroll
      for (int i = 0; i < kP; ++i)
        o[i] = pair(in(2 * i) ? to_f32(row[2 * i * nx]) : 0.f, in(2 * i + 1) ? to_f32(row[(2 * i + 1) * nx]) : 0.f);
    }
  };
  auto put = [&](auto type, void* base, int64_t ld, int64_t t, const uint64_t* o) {
    using T = decltype(type);
    T* row = static_cast<T*>(base) + t * ld;
    if constexpr (V > 1) {
      if (single) {
        if (mine) row[first] = from_f32<T>(split(o[0]).x);
        return;
      }
#pragma unroll
      for (int j = 0; j < kE / V; ++j) {
        float v[V];
#pragma unroll
        for (int i = 0; i < V; i += 2) {
          const float2 a = split(o[(V * j + i) / 2]);
          v[i] = a.x;
          v[i + 1] = a.y;
        }
        if (in(V * j)) store_vec<T, V>(row + col(V * j), v);
      }
    } else {
      row += tx;
#pragma unroll
      for (int i = 0; i < kP; ++i) {
        const float2 a = split(o[i]);
        if (in(2 * i)) row[2 * i * nx] = from_f32<T>(a.x);
        if (in(2 * i + 1)) row[(2 * i + 1) * nx] = from_f32<T>(a.y);
      }
    }
  };
  int turn = 0;
  auto reduce = [&](float (&v)[ROWS]) {  // sums over the row's threads, one barrier
#pragma unroll
    for (int r = 0; r < ROWS; ++r) v[r] = warp_sum(v[r]);
    const int warps = blockDim.x >> 5, lane = tx & 31;
    if (warps == 1) return;
    float2* at = scratch[turn];
    turn ^= 1;
    if (lane == 0) at[tx >> 5] = make_float2(v[0], v[ROWS - 1]);
    __syncthreads();
    const float2 a = lane < warps ? at[lane] : make_float2(0.f, 0.f);
    v[0] = warp_sum(a.x);
    if (ROWS == 2) v[ROWS - 1] = warp_sum(a.y);
  };
  const float inv_h = 1.0f / H;
  auto normalise_rows = [&](uint64_t (&u)[ROWS][kP], int kind) {
    float s[ROWS];
    if (kind == W4A8_NORM_LAYER) {
#pragma unroll
      for (int r = 0; r < ROWS; ++r) {
        uint64_t a = u[r][0];
#pragma unroll
        for (int i = 1; i < kP; ++i) a = add2(a, u[r][i]);
        const float2 b = split(a);
        s[r] = b.x + b.y;
      }
      reduce(s);
#pragma unroll
      for (int r = 0; r < ROWS; ++r) {
        const float m = -s[r] * inv_h;
#pragma unroll
        for (int i = 0; i < kP; ++i) u[r][i] = add2(u[r][i], pair(in(2 * i) ? m : 0.f, in(2 * i + 1) ? m : 0.f));
        if (single) {
          u[r][0] = pair(split(u[r][0]).x, 0.f);
#pragma unroll
          for (int i = 1; i < V / 2; ++i) u[r][i] = 0;
        }
      }
    }
#pragma unroll
    for (int r = 0; r < ROWS; ++r) {
      uint64_t a = mul2(u[r][0], u[r][0]);
#pragma unroll
      for (int i = 1; i < kP; ++i) a = fma2(u[r][i], u[r][i], a);
      const float2 b = split(a);
      s[r] = b.x + b.y;
    }
    reduce(s);
#pragma unroll
    for (int r = 0; r < ROWS; ++r) {
      const float inv = rsqrtf(fmaf(s[r], inv_h, p.eps));
#pragma unroll
      for (int i = 0; i < kP; ++i) u[r][i] = mul2(u[r][i], pair(inv, inv));
    }
  };
  auto scale_rows = [&](uint64_t (&u)[ROWS][kP], const uint64_t (&w)[kP], const uint64_t* b) {
#pragma unroll
    for (int i = 0; i < kP; ++i) {
      const uint64_t bi = BIAS ? b[i * threads] : 0;
#pragma unroll
      for (int r = 0; r < ROWS; ++r) u[r][i] = BIAS ? fma2(u[r][i], w[i], bi) : mul2(u[r][i], w[i]);
    }
  };
  // a row's gate value, loaded a round ahead as it is: its conversion would wait for the load at once
  auto gate_bits = [&](int64_t t) -> uint32_t {
    if (!p.gate_scalar || t >= p.T) return 0;
    const int64_t at = gate_index(t) * p.ldg;
    return p.gate_f32 || sizeof(X) == 4 ? static_cast<const uint32_t*>(p.gate)[at]
                                        : static_cast<const uint16_t*>(p.gate)[at];
  };
  auto gate_value = [&](uint32_t bits) {
    if (p.gate_f32 || sizeof(X) == 4) return __uint_as_float(bits);
    X x;
    memcpy(&x, &bits, sizeof(X));
    return to_f32(x);
  };

  for (int s = 0; s < st.stages; ++s) fetch(t0 + s * ROWS * step, ring + s * st.bytes);
  // while the first rows are on their way
  uint64_t w_post[kP], w_pre[kP];
  // the biases: this thread's pairs in shared memory behind the ring, b_post then b_pre (registers hold no more)
  uint64_t* biases = reinterpret_cast<uint64_t*>(ring + st.stages * st.bytes) + tid;
  {
    // a parameter at this thread's columns: all loads inside one branch on the type, so that none waits for another
    auto param = [&](const void* q, int f32, float* a) {
      if (f32) {
#pragma unroll
        for (int i = 0; i < kE; ++i) a[i] = valid(i) ? static_cast<const float*>(q)[col(i)] : 0.f;
      } else {
#pragma unroll
        for (int i = 0; i < kE; ++i) a[i] = valid(i) ? to_f32(static_cast<const X*>(q)[col(i)]) : 0.f;
      }
    };
    auto keep_bias = [&](int at, const void* q, const float* w) {
      float a[kE];
#pragma unroll
      for (int i = 0; i < kE; ++i) a[i] = 0.f;
      if (q) param(q, p.w_f32, a);
#pragma unroll
      for (int j = 0; j < kP; ++j) biases[(at + j) * threads] = pair(a[2 * j] * w[2 * j], a[2 * j + 1] * w[2 * j + 1]);
    };
    float w[kE], a[kE];
#pragma unroll
    for (int i = 0; i < kE; ++i) w[i] = valid(i) ? p.branch_scale : 0.f;
    if (p.gate && !p.gate_scalar && !st.gate_rows) {
      param(p.gate, p.gate_f32, a);
#pragma unroll
      for (int i = 0; i < kE; ++i) w[i] *= a[i];
    }
    if (BIAS) keep_bias(0, p.b_post, w);
    if (p.w_post) {
      param(p.w_post, p.w_f32, a);
#pragma unroll
      for (int i = 0; i < kE; ++i) w[i] *= a[i];
    }
#pragma unroll
    for (int j = 0; j < kP; ++j) w_post[j] = pair(w[2 * j], w[2 * j + 1]);
#pragma unroll
    for (int i = 0; i < kE; ++i) w[i] = valid(i) ? 1.f : 0.f;
    if (BIAS) keep_bias(kP, p.b_pre, w);
    if (p.w_pre) param(p.w_pre, p.w_f32, w);
#pragma unroll
    for (int j = 0; j < kP; ++j) w_pre[j] = pair(w[2 * j], w[2 * j + 1]);
  }
  uint32_t gs[ROWS];
#pragma unroll
  for (int r = 0; r < ROWS; ++r) gs[r] = gate_bits(t0 + r * step);
  int s = 0;
  const uint64_t rs = pair(p.residual_scale, p.residual_scale);
  for (; t0 < p.T; t0 += ROWS * step) {
    uint8_t* at = ring + s * st.bytes;
    if (st.stages == 3)
      copy_wait<2>();
    else
      copy_wait<1>();
    if (V == 1) __syncthreads();
    uint64_t u[ROWS][kP];
#pragma unroll
    for (int r = 0; r < ROWS; ++r) take(X(), p.f, p.ldf, t0 + r * step, at + r * st.f_row, u[r]);
    if (p.post != W4A8_NORM_NONE) normalise_rows(u, p.post);
    scale_rows(u, w_post, biases);
#pragma unroll
    for (int r = 0; r < ROWS; ++r) {
      const int64_t t = t0 + r * step;
      if (p.gate_scalar) {
        const float g = gate_value(gs[r]);
#pragma unroll
        for (int i = 0; i < kP; ++i) u[r][i] = mul2(u[r][i], pair(g, g));
        gs[r] = gate_bits(t + ROWS * step);
      }
      if (st.gate_rows) {
        uint64_t a[kP];
        uint8_t* g = at + st.g_at + r * st.g_row;
        if (p.gate_f32)
          take(float(), p.gate, p.ldg, gate_index(t), g, a);
        else
          take(X(), p.gate, p.ldg, gate_index(t), g, a);
#pragma unroll
        for (int i = 0; i < kP; ++i) u[r][i] = mul2(u[r][i], a[i]);
      }
      if (p.r) {
        uint64_t a[kP];
        take(R(), p.r, p.ldr, t, at + st.r_at + r * st.r_row, a);
#pragma unroll
        for (int i = 0; i < kP; ++i) u[r][i] = fma2(rs, a[i], u[r][i]);
      }
      if (p.h && t < p.T) put(R(), p.h, p.ldh, t, u[r]);
    }
    if (V == 1) __syncthreads();  // every thread has read the stage
    fetch(t0 + st.stages * ROWS * step, at);
    s = s + 1 == st.stages ? 0 : s + 1;
    if (!p.y) continue;
    if (p.pre != W4A8_NORM_NONE) normalise_rows(u, p.pre);
    scale_rows(u, w_pre, biases + kP * threads);
#pragma unroll
    for (int r = 0; r < ROWS; ++r)
      if (t0 + r * step < p.T) put(X(), p.y, p.ldy, t0 + r * step, u[r]);
  }
  copy_wait<0>();
}

template <typename X, typename R, int V, bool CUT, int VPT>
int launch_row(const NormParams& p, cudaStream_t st) {
  const int64_t need = ceil_div(p.H, V * VPT), warps = ceil_div(need, 32);
  const int64_t per = row_threads(V, VPT) ? row_threads(V, VPT)  // threads of a row
                      : CUT               ? warps * 32 + 32
                      : need <= 8         ? 8
                      : need <= 16        ? 16
                                          : warps * 32;
  const int rows = per <= 32 ? 256 / static_cast<int>(per) : 1;
  return launch_pdl("block_norm_row_kernel", block_norm_row_kernel<X, R, V, CUT, VPT>,
                    dim3(static_cast<unsigned>(ceil_div(p.T, rows))), dim3(static_cast<unsigned>(per), rows), 0, st, p);
}

constexpr int kMaxSmem = 227 * 1024;

template <typename X, typename R, int V, bool CUT, bool BIAS, int kE>
int launch_stream(const NormParams& p, const NormStage& stage, int threads, int rows, cudaStream_t st) {
  auto kern = block_norm_stream_kernel<X, R, V, CUT, BIAS, kE>;
  static DeviceOnce once;
  if (int rc = once.run([&] {
        if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxSmem - 1024) != cudaSuccess)
          return check_launch("cudaFuncSetAttribute(block_norm)");
        return static_cast<int>(W4A8_OK);
      }))
    return rc;
  // as many blocks as run at once: max_threads(kE) threads have registers, and shared memory takes the ring (with the
  // kernel's static part and the 1 KB that a block costs)
  const int64_t smem = static_cast<int64_t>(stage.stages) * stage.bytes + (BIAS ? threads * rows * kE * 8 : 0);
  const int64_t per_sm =
      std::max<int64_t>(1, std::min<int64_t>(max_threads(kE) / (threads * rows), kMaxSmem / (smem + 1280)));
  int64_t blocks = std::min(ceil_div(p.T, rows), per_sm * num_sms());
  if (CUT) blocks = std::max<int64_t>(8, blocks / 8 * 8);  // all rows of a block start alike
  return launch_pdl("block_norm_stream_kernel", kern, dim3(static_cast<unsigned>(blocks)), dim3(threads, rows),
                    static_cast<size_t>(smem), st, p, stage);
}

// Whether the rows fit the streaming kernel (two stages of them in shared memory); *rc is the launch's status then.
template <typename X, typename R, int V, bool CUT, int kE>
bool try_stream(const NormParams& p, cudaStream_t st, int* rc) {
  const bool bias = p.b_post || p.b_pre;
  const int threads = static_cast<int>(ceil_div(ceil_div(p.H, kE), 32) * 32) + (CUT ? 32 : 0);
  if (threads > max_threads(kE)) return false;
  const int rows = V > 1 && threads == 32 ? 4 : 1;
  constexpr int turn = 2;  // rows of a stage
  NormStage stage;
  stage.gate_rows = p.gate && !p.gate_scalar && p.rows_per_gate < p.T;
  // one row of a part: the block's vectors, or the 16-byte pieces that cover a row
  const auto part = [&](int size) { return V > 1 ? threads * rows * kE * size : (p.H * size + 15) / 16 * 16 + 16; };
  stage.f_row = part(sizeof(X));
  stage.r_row = p.r ? part(sizeof(R)) : 0;
  stage.g_row = stage.gate_rows ? part(p.gate_f32 ? 4 : static_cast<int>(sizeof(X))) : 0;
  stage.r_at = turn * stage.f_row;
  stage.g_at = stage.r_at + turn * stage.r_row;
  stage.bytes = stage.g_at + turn * stage.g_row;
  // three stages where that leaves an SM as many blocks as two do (8192 x 4096 bf16 with an fp32 residual: one block of
  // 256 threads with three, two with two)
  const auto blocks = [&](int stages) {
    const int smem = stages * stage.bytes + (bias ? threads * rows * kE * 8 : 0) + 1280;
    return std::min(max_threads(kE) / (threads * rows), kMaxSmem / smem);
  };
  if (blocks(2) < 1) return false;
  stage.stages = blocks(3) < blocks(2) ? 2 : 3;
  *rc = bias ? launch_stream<X, R, V, CUT, true, kE>(p, stage, threads, rows, st)
             : launch_stream<X, R, V, CUT, false, kE>(p, stage, threads, rows, st);
  return true;
}

// Whether every row starts at the same place within V elements in all of the row's matrices.
template <typename X, typename R>
bool rows_agree(const NormParams& p, int V) {
  const auto phase = [&](const void* q, int size) { return static_cast<int>(reinterpret_cast<uintptr_t>(q) / size % V); };
  const auto like_f = [&](const void* q, int64_t ld, int size) {
    return !q || (phase(q, size) == phase(p.f, sizeof(X)) && (p.T == 1 || (ld - p.ldf) % V == 0));
  };
  if (!like_f(p.r, p.ldr, sizeof(R)) || !like_f(p.h, p.ldh, sizeof(R)) || !like_f(p.y, p.ldy, sizeof(X))) return false;
  if (!p.gate || p.gate_scalar || p.rows_per_gate >= p.T) return true;
  return like_f(p.gate, p.ldg, p.gate_f32 ? 4 : static_cast<int>(sizeof(X))) && (p.rows_per_gate == 1 || p.ldg % V == 0);
}

template <typename X, typename R>
int dispatch(const NormParams& p, bool vec, cudaStream_t st) {
  // Rows that a block works through in turn pay for the ring from the second one on; with few rows, and with rows too
  // long for it, each gets a block of its own.
  int rc;
  const bool many = p.T > 2 * num_sms();
  constexpr int V = sizeof(R) == 4 ? 4 : 8;
  // (shorter rows leave the warps for whole vectors too little: 20000 x 643 bf16 36.3 us, 34.0 in single elements; 16000 x
  // 771: 30.8 and 35.7)
  const bool whole = vec && p.H % V == 0, cut = p.H > 704 && rows_agree<X, R>(p, V);
  // Rows of up to 256 elements go to a warp each or, up to 128, to a part of one.  From 129 on they go through the ring
  // where a warp gets more than two of them (40000 x 200 bf16: 14.8 us, the row kernel 23.5; 4000 x 200: 4.6 and 4.2;
  // 60000 x 128: 17.9 and 14.8), in single elements where there are many (40000 x 201: 22.1 us, the row kernel 36.1; 60000
  // x 101: 30.0 and 25.4).
  if (p.H <= 256) {
    if (p.H > 128 && whole && p.T > 48 * num_sms() && try_stream<X, R, V, false, 8>(p, st, &rc)) return rc;
    if (vec) return launch_row<X, R, 8, false, 1>(p, st);
    if (p.H <= 128 || !many) return launch_row<X, R, 1, false, 8>(p, st);
  }
  // fp32 rows of whole vectors fill the memory's pipes from registers, and the ring would take the threads' room (2837 x
  // 7680: 54.7 us a row to a block, 62.6 us with the ring; bf16, 16384 x 1024: 35.7 and 23.5 us)
  if (many && !(sizeof(X) == 4 && whole)) {
    if (whole ? try_stream<X, R, V, false, 16>(p, st, &rc) : cut && try_stream<X, R, V, true, 16>(p, st, &rc)) return rc;
    // Single elements cost more instructions and latency each, which twice the warps hide where they fit, but a row to one
    // warp needs no barrier (40000 x 257 bf16: 35.5 us, with two warps 42.0).  Rows that miss the ring above for their
    // length alone are still faster this way without fp32 among them (1596 x 8191 bf16: 35.3 us, 39.3 a row to a block;
    // with an fp32 residual 73.8 and 58.6).
    if (!whole && (!cut || sizeof(R) != 4)) {
      const bool one_warp = p.H > 256 && p.H <= 512;
      if (!one_warp && try_stream<X, R, 1, false, 8>(p, st, &rc)) return rc;
      if (try_stream<X, R, 1, false, 16>(p, st, &rc)) return rc;
    }
  }
  // Few rows: as many threads to a row as possible; many: half as many, so that two rows share an SM.  Many long rows of
  // fp32 alone are read in vectors of 4, where each access covers whole sectors (2837 x 7680: 62.5 us in vectors of 8, 55.2
  // of 4; but 3000 x 4096: 35.4 and 37.9); those beside 16-bit ones are not (1596 x 10048: 47.1 us, of 4 55.7).
  if (vec) {
    if (many && sizeof(X) == 4 && p.H > 4096)
      return p.H <= 8192 ? launch_row<X, R, 4, false, 4>(p, st) : launch_row<X, R, 4, false, 8>(p, st);
    if (p.H <= (many ? 4096 : 8192)) return launch_row<X, R, 8, false, 1>(p, st);
    if (p.H <= (many ? 8192 : 16384)) return launch_row<X, R, 8, false, 2>(p, st);
    return launch_row<X, R, 8, false, 4>(p, st);
  }
  // a block has at most 31 warps for whole vectors (1596 x 10047 bf16 with an fp32 residual: 52.6 us; single elements 134)
  if (cut) {
    if (p.H <= (many ? 3968 : 7936)) return launch_row<X, R, V, true, 8 / V>(p, st);
    if (p.H <= (many ? 7936 : 15872)) return launch_row<X, R, V, true, 16 / V>(p, st);
    if (p.H <= 31744) return launch_row<X, R, V, true, 32 / V>(p, st);
  }
  if (p.H <= 4096) return launch_row<X, R, 1, false, 4>(p, st);
  if (p.H <= 8192) return launch_row<X, R, 1, false, 8>(p, st);
  if (p.H <= 16384) return launch_row<X, R, 1, false, 16>(p, st);
  return launch_row<X, R, 1, false, 32>(p, st);
}

}  // namespace
}  // namespace w4a8

