// What the tcgen05 kernels of the Linears share: bounded waits, clusters, operands and products of CTA pairs, launches.
// Included once by each translation unit, which has an error word and a reader of its own.
#pragma once

#include <atomic>

#include "common.cuh"

namespace w4a8 {
namespace {

constexpr uint64_t kTimeoutNs = 2000000000ull;  // 2 s: no legitimate wait comes close
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

}  // namespace
}  // namespace w4a8
