// dense_linear, weight-streaming form: out = act(x W^T + bias) [* other half] + residual for a few rows of x.
//
// Every weight is read once from memory straight into the operand registers of mma.sync (16 weight rows x
// 8 tokens): the order of k inside a product is free as long as both operands agree, so a lane loads 16
// contiguous bytes (8 k) of its weight rows and of its token, and uses them as the k-pairs of two
// instructions.  No shared memory and no barrier stand between memory and the tensor core; the 8 warps of a
// block take interleaved 64-element pieces of K and their fp32 partial products meet in shared memory.
// With few weight rows K is also cut over the CTAs of a cluster: the partial sums are pushed into the first
// CTA's shared memory and added there in rank order, so results do not depend on timing.
// Bound by memory where W is large (1 x 8192 x 8192: 24 us, 5.6 TB/s), by a launch where it is small (1 x 256 x 7168:
// 3.5 us; the tensor-memory kernels, which set up barriers and tensor memory first, take 6.2).
#include "linear.cuh"

namespace w4a8 {
namespace {

constexpr int kWarps = 8;
constexpr int kStep = 32;  // k per pair of mma instructions

// 8 consecutive elements [k, k + 8) of a row, zeros from K on.  An ordinary load: a non-coherent one asks for memory that
// nothing writes during the kernel's whole life, and this kernel starts while its predecessor may still write x.
template <bool ALIGNED>
__device__ __forceinline__ uint4 load8(const uint16_t* row, int k, int K) {
  if (ALIGNED && k + 8 <= K) return *reinterpret_cast<const uint4*>(row + k);
  uint32_t v[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t lo = k + 2 * i < K ? row[k + 2 * i] : 0;
    const uint32_t hi = k + 2 * i + 1 < K ? row[k + 2 * i + 1] : 0;
    v[i] = lo | (hi << 16);
  }
  return make_uint4(v[0], v[1], v[2], v[3]);
}

template <bool F16>
__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1) {
  if (F16)
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  else
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }

// NT token tiles of 8; a block computes 16 output columns (two row fragments of W when gated).  blockIdx.x =
// column block * splits + split, blockIdx.y = token block.
template <int NT, bool GATED, bool ALIGNED, bool F16>
__global__ void __launch_bounds__(kWarps * 32) linear_stream_kernel(const LinearParams p, int splits) {
  constexpr int R = GATED ? 2 : 1;
  constexpr int kTile = R * 16 * NT * 8;  // fp32 values of the block's result
  extern __shared__ float smem[];         // [kWarps][kTile], then, with splits, [splits][kTile] (first CTA's in use)
  pdl_trigger();
  if (splits > 1) cluster_arrive();  // matched before the first remote store: every CTA runs by then
  pdl_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, t4 = lane & 3;
  const int split = blockIdx.x % splits;
  const int n0 = (blockIdx.x / splits) * 16;
  const int m0 = blockIdx.y * NT * 8;
  const uint16_t* W = static_cast<const uint16_t*>(p.w);
  const uint16_t* X = static_cast<const uint16_t*>(p.x);
  const uint16_t* wrow[R][2];
  bool wok[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int n = n0 + g + 8 * h;
    wok[h] = n < p.n_out;
#pragma unroll
    for (int r = 0; r < R; ++r) wrow[r][h] = W + static_cast<int64_t>(wok[h] ? n + r * p.n_out : 0) * p.ldw;
  }
  const uint16_t* xrow[NT];
#pragma unroll
  for (int j = 0; j < NT; ++j) {
    const int m = m0 + j * 8 + g;
    xrow[j] = m < p.M ? X + m * p.ldx : nullptr;
  }
  float c[R][NT][4];
#pragma unroll
  for (int r = 0; r < R; ++r)
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
      for (int i = 0; i < 4; ++i) c[r][j][i] = 0.f;
  const uint4 zero = make_uint4(0, 0, 0, 0);
  // pieces of 2 * kStep elements, dealt round-robin to the warps of all splits.  The tensor core cuts off at every
  // addition to its accumulator, so long sums drift: every kChunk pieces they move to sums that are rounded to nearest.
  constexpr int kChunk = 16;
  float sum[R][NT][4];
#pragma unroll
  for (int r = 0; r < R; ++r)
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
      for (int i = 0; i < 4; ++i) sum[r][j][i] = 0.f;
  auto flush = [&] {
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          sum[r][j][i] += c[r][j][i];
          c[r][j][i] = 0.f;
        }
  };
  const int pieces = (p.K + 2 * kStep - 1) / (2 * kStep);
  int until_flush = kChunk;
  constexpr int kUnroll = NT == 1 ? 2 : 1;  // with 16 tokens, two pieces at a time take the registers of two more blocks
#pragma unroll kUnroll
  for (int q = split * kWarps + warp; q < pieces; q += splits * kWarps) {
    if (--until_flush < 0) {
      flush();
      until_flush = kChunk - 1;
    }
    uint4 a[2][R][2], b[2][NT];
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      const int k = q * 2 * kStep + s * kStep + t4 * 8;
#pragma unroll
      for (int r = 0; r < R; ++r)
#pragma unroll
        for (int h = 0; h < 2; ++h) a[s][r][h] = wok[h] && k < p.K ? load8<ALIGNED>(wrow[r][h], k, p.K) : zero;
#pragma unroll
      for (int j = 0; j < NT; ++j) b[s][j] = xrow[j] && k < p.K ? load8<ALIGNED>(xrow[j], k, p.K) : zero;
    }
#pragma unroll
    for (int s = 0; s < 2; ++s)
#pragma unroll
      for (int r = 0; r < R; ++r)
#pragma unroll
        for (int j = 0; j < NT; ++j) {
          const uint4 &a0 = a[s][r][0], &a1 = a[s][r][1], &x = b[s][j];
          mma16816<F16>(c[r][j], a0.x, a1.x, a0.y, a1.y, x.x, x.y);
          mma16816<F16>(c[r][j], a0.z, a1.z, a0.w, a1.w, x.z, x.w);
        }
  }
  flush();
  // partial products of the warps: [warp][r][token][16 columns]
  float* mine = smem + warp * kTile;
#pragma unroll
  for (int r = 0; r < R; ++r)
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
      for (int i = 0; i < 4; ++i)
        mine[(r * NT * 8 + j * 8 + 2 * t4 + (i & 1)) * 16 + g + 8 * (i >> 1)] = sum[r][j][i];
  __syncthreads();
  if (splits > 1) {
    cluster_wait();
    const uint32_t at0 = smem_u32(smem + kWarps * kTile + split * kTile);
    for (int i = threadIdx.x; i < kTile; i += kWarps * 32) {
      float s = 0.f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) s += smem[w * kTile + i];
      uint32_t remote;
      asm("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(remote) : "r"(at0 + 4 * i));
      asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(remote), "f"(s) : "memory");
    }
    cluster_arrive();
    cluster_wait();
    if (cluster_rank() != 0) return;
  }
  const float* part = splits > 1 ? smem + kWarps * kTile : smem;
  const int parts = splits > 1 ? splits : kWarps;
  for (int i = threadIdx.x; i < kTile / R; i += kWarps * 32) {
    const int m = m0 + i / 16, n = n0 + i % 16;
    if (m >= p.M || n >= p.n_out) continue;
    float z = 0.f, z2 = 0.f;
    for (int s = 0; s < parts; ++s) {
      z += part[s * kTile + i];
      if (GATED) z2 += part[s * kTile + kTile / 2 + i];
    }
    finish(p, m, n, z, z2);
  }
}

template <int NT, bool GATED, bool ALIGNED, bool F16>
int launch_one(const LinearParams& p, cudaStream_t st) {
  constexpr int kTile = (GATED ? 2 : 1) * 16 * NT * 8;
  const int64_t nb = ceil_div(p.n_out, 16), mb = ceil_div(p.M, NT * 8);
  // cut K until the GPU has two blocks per SM, but keep a 64-element piece for every warp
  int splits = 1;
  while (splits < 8 && nb * mb * splits < 2 * num_sms() && p.K >= 2 * splits * kWarps * 2 * kStep) splits *= 2;
  W4A8_REQUIRE(nb * splits < (1ll << 31) && mb < 65536, "M=%d, N=%d out of range", p.M, p.N);
  const size_t smem = sizeof(float) * kTile * (kWarps + (splits > 1 ? splits : 0));
  auto kern = linear_stream_kernel<NT, GATED, ALIGNED, F16>;
  static DeviceOnce attrs;
  if (int rc = attrs.run([&] {
        if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, sizeof(float) * kTile * 16) !=
            cudaSuccess)
          return check_launch("cudaFuncSetAttribute(linear_stream)");
        return static_cast<int>(W4A8_OK);
      }))
    return rc;
  cudaLaunchConfig_t lc = {};
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = splits;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  lc.gridDim = dim3(static_cast<unsigned>(nb * splits), static_cast<unsigned>(mb));
  lc.blockDim = dim3(kWarps * 32);
  lc.dynamicSmemBytes = smem;
  lc.stream = st;
  lc.attrs = attr;
  lc.numAttrs = splits > 1 ? 2 : 1;
  const cudaError_t e = cudaLaunchKernelEx(&lc, kern, p, splits);
  if (e != cudaSuccess) return set_error(W4A8_ERR_CUDA, "linear_stream_kernel: %s", cudaGetErrorString(e));
  return check_launch("linear_stream_kernel");
}

template <int NT>
int launch_nt(const LinearParams& p, bool aligned, cudaStream_t st) {
  const bool f16 = p.dtype == W4A8_DTYPE_F16;
  if (p.gated) {
    if (aligned) return f16 ? launch_one<NT, true, true, true>(p, st) : launch_one<NT, true, true, false>(p, st);
    return f16 ? launch_one<NT, true, false, true>(p, st) : launch_one<NT, true, false, false>(p, st);
  }
  if (aligned) return f16 ? launch_one<NT, false, true, true>(p, st) : launch_one<NT, false, true, false>(p, st);
  return f16 ? launch_one<NT, false, false, true>(p, st) : launch_one<NT, false, false, false>(p, st);
}

}  // namespace

int launch_linear_stream(const LinearParams& p, cudaStream_t st) {
  const bool aligned = aligned16(p.x) && aligned16(p.w) && p.ldx % 8 == 0 && p.ldw % 8 == 0;
  return p.M <= 8 ? launch_nt<1>(p, aligned, st) : launch_nt<2>(p, aligned, st);
}

}  // namespace w4a8
