// Status plumbing, workspace sizing and the whole-layer entry point.
#include <cstdarg>
#include <cstdio>
#include <mutex>
#include <vector>

#include "common.cuh"

namespace w4a8 {

namespace {
thread_local char g_msg[512] = "";
std::vector<device_error_reader>& readers() {
  static std::vector<device_error_reader> v;
  return v;
}
std::mutex g_mu;
}  // namespace

int set_error(int status, const char* fmt, ...) {
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(g_msg, sizeof(g_msg), fmt, ap);
  va_end(ap);
  return status;
}

int check_launch(const char* what) {
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return set_error(W4A8_ERR_CUDA, "%s: %s", what, cudaGetErrorString(e));
  return W4A8_OK;
}

int num_sms() {
  constexpr int kGb300Sms = 152;  // used only if the device cannot be queried
  static int cache[64] = {0};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return kGb300Sms;
  if (!cache[dev]) {
    int n = 0;
    cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev);
    cache[dev] = n > 0 ? n : kGb300Sms;
  }
  return cache[dev];
}

void register_device_error_reader(device_error_reader f) {
  std::lock_guard<std::mutex> lk(g_mu);
  readers().push_back(f);
}

namespace {
inline size_t align256(size_t v) { return (v + 255) & ~size_t(255); }

int layout_of(int64_t T, int64_t H, int64_t I, int64_t E, int k, w4a8_moe_layout* L) {
  W4A8_REQUIRE(T >= 0 && H > 0 && I > 0 && E >= 1 && k >= 1, "bad layer shape");
  W4A8_REQUIRE(H % 128 == 0 && I % 128 == 0, "H and I must be multiples of 128");
  const int64_t P = T * k;
  const int64_t ld = (P + 3) / 4 * 4 > 0 ? (P + 3) / 4 * 4 : 4;
  size_t o = 0;
  auto take = [&](size_t bytes) {
    const size_t at = o;
    o = align256(o + bytes);
    return at;
  };
  L->topk_ids = take(P * 4);
  L->topk_w = take(P * 4);
  L->seg_indptr = take((E + 1) * 8);
  L->src2dst = take(P * 4);
  L->dst2src = take(P * 4);
  L->xq = take(P * H);
  L->xs = take((H / 128) * ld * 4);
  L->xc = take((H / 128) * ld * 4);
  L->y13 = take(P * 2 * I * 2);
  L->hq = take(P * I);
  L->hs = take((I / 128) * ld * 4);
  L->hc = take((I / 128) * ld * 4);
  L->y2 = take(P * H * 2);
  L->permute_ws = take(permute_ws_bytes(P, E));
  L->scale_ld = ld;
  L->total = o;
  return W4A8_OK;
}
}  // namespace

}  // namespace w4a8

extern "C" const char* w4a8_status_string(int status) {
  switch (status) {
    case W4A8_OK: return "ok";
    case W4A8_ERR_INVALID_ARG: return "invalid argument";
    case W4A8_ERR_UNSUPPORTED: return "unsupported";
    case W4A8_ERR_CUDA: return "CUDA error";
    case W4A8_ERR_TIMEOUT: return "device-side wait timed out";
    default: return "unknown status";
  }
}

extern "C" const char* w4a8_last_error(void) { return w4a8::g_msg; }

extern "C" int w4a8_abi_version(void) { return W4A8MOE_ABI_VERSION; }

extern "C" int w4a8_device_error(void) {
  if (cudaDeviceSynchronize() != cudaSuccess) return -1;
  int v = 0;
  std::lock_guard<std::mutex> lk(w4a8::g_mu);
  for (auto f : w4a8::readers()) v |= f();
  return v;
}

extern "C" size_t w4a8_workspace_bytes(int op, int64_t M, int64_t N, int64_t K, int64_t E) {
  if (op == W4A8_OP_LINEAR) return w4a8::gemm_workspace_bytes(M, N, K, true);
  if (op == W4A8_OP_GROUPED_GEMM) return w4a8::gemm_workspace_bytes(M, N, K, false);
  if (op == W4A8_OP_GROUPED_GEMM_SILU) return w4a8::gemm_silu_workspace_bytes(M, N, K);
  if (op == W4A8_OP_PERMUTE) return w4a8::permute_ws_bytes(M, E);
  return 0;
}

extern "C" int w4a8_moe_workspace_layout(int64_t T, int64_t H, int64_t I, int64_t E, int k,
                                         w4a8_moe_layout* layout) {
  if (!layout) return w4a8::set_error(W4A8_ERR_INVALID_ARG, "layout is null");
  return w4a8::layout_of(T, H, I, E, k, layout);
}

extern "C" size_t w4a8_moe_workspace_bytes(int64_t T, int64_t H, int64_t I, int64_t E, int k) {
  w4a8_moe_layout L;
  if (w4a8::layout_of(T, H, I, E, k, &L) != W4A8_OK) return 0;
  return L.total;
}

namespace w4a8 {
namespace {

// The layer with its routing: topk ids and weights given (ids, tw), or computed into the workspace from logits.
int moe_layer(const uint16_t* x, const float* logits, const int32_t* ids, const float* tw, int64_t T, int64_t H,
              int64_t I, int64_t E, int k, int renormalize, const uint8_t* w13, const float* w13_s, const uint8_t* w2,
              const float* w2_s, uint16_t* out, void* ws, size_t ws_bytes, void* stream) {
  w4a8_moe_layout L;
  int rc = layout_of(T, H, I, E, k, &L);
  if (rc) return rc;
  W4A8_REQUIRE(ws != nullptr && ws_bytes >= L.total, "workspace too small: need %zu bytes", L.total);
  W4A8_REQUIRE((reinterpret_cast<uintptr_t>(ws) & 255) == 0, "workspace must be 256-byte aligned");
  if (T == 0) return W4A8_OK;
  uint8_t* b = static_cast<uint8_t*>(ws);
  int64_t* seg = reinterpret_cast<int64_t*>(b + L.seg_indptr);
  int32_t* s2d = reinterpret_cast<int32_t*>(b + L.src2dst);
  int32_t* d2s = reinterpret_cast<int32_t*>(b + L.dst2src);
  uint8_t* xq = b + L.xq;
  float* xs = reinterpret_cast<float*>(b + L.xs);
  float* xc = reinterpret_cast<float*>(b + L.xc);
  uint16_t* y13 = reinterpret_cast<uint16_t*>(b + L.y13);
  uint8_t* hq = b + L.hq;
  float* hs = reinterpret_cast<float*>(b + L.hs);
  float* hc = reinterpret_cast<float*>(b + L.hc);
  uint16_t* y2 = reinterpret_cast<uint16_t*>(b + L.y2);
  const int64_t P = T * k;
  if (!ids) {
    int32_t* ws_ids = reinterpret_cast<int32_t*>(b + L.topk_ids);
    float* ws_tw = reinterpret_cast<float*>(b + L.topk_w);
    if ((rc = moe_route_topk(logits, T, E, k, renormalize, ws_ids, ws_tw, stream))) return rc;
    ids = ws_ids;
    tw = ws_tw;
  }
  if ((rc = moe_permute(ids, T, k, E, seg, s2d, d2s, b + L.permute_ws, permute_ws_bytes(P, E), stream))) return rc;
  if ((rc = fp8_quant_scatter_per_token_group(x, T, H, s2d, k, P, xq, xs, xc, L.scale_ld, stream))) return rc;
  // w13, then SiLU-and-Mul requantisation in its own kernel: with the requantisation fused into w13's
  // epilogue (w4a8_grouped_gemm_silu) the prefill w13 launch took 5.37 ms against 4.22 + 0.19 ms, since
  // the promotion epilogue is the GEMM's critical role and the SiLU math is cheaper at full occupancy
  if ((rc = w4a8_grouped_gemm(xq, xs, xc, L.scale_ld, w13, w13_s, seg, E, 2 * I, H, P, y13, nullptr, 0, stream)))
    return rc;
  if ((rc = silu_mul_requant(y13, P, I, hq, hs, hc, L.scale_ld, stream))) return rc;
  if ((rc = w4a8_grouped_gemm(hq, hs, hc, L.scale_ld, w2, w2_s, seg, E, H, I, P, y2, nullptr, 0, stream)))
    return rc;
  return moe_unpermute_combine(y2, s2d, tw, T, k, H, out, stream);
}

}  // namespace
}  // namespace w4a8

extern "C" int w4a8_moe_forward(const uint16_t* x, const float* logits, int64_t T, int64_t H, int64_t I, int64_t E,
                                int k, int renormalize, const uint8_t* w13, const float* w13_s, const uint8_t* w2,
                                const float* w2_s, uint16_t* out, void* ws, size_t ws_bytes, void* stream) {
  return w4a8::moe_layer(x, logits, nullptr, nullptr, T, H, I, E, k, renormalize, w13, w13_s, w2, w2_s, out, ws,
                         ws_bytes, stream);
}

extern "C" int w4a8_moe_forward_routed(const uint16_t* x, const int32_t* topk_ids, const float* topk_w, int64_t T,
                                       int64_t H, int64_t I, int64_t E, int k, const uint8_t* w13, const float* w13_s,
                                       const uint8_t* w2, const float* w2_s, uint16_t* out, void* ws, size_t ws_bytes,
                                       void* stream) {
  using namespace w4a8;
  W4A8_REQUIRE(E >= 1 && E <= 1024, "E=%lld must be in [1, 1024]", (long long)E);
  W4A8_REQUIRE(k >= 1 && k <= 32 && k <= E, "k=%d must be in [1, min(E, 32)]", k);
  W4A8_REQUIRE(T == 0 || (topk_ids && topk_w), "null pointer");
  return moe_layer(x, nullptr, topk_ids, topk_w, T, H, I, E, k, 0, w13, w13_s, w2, w2_s, out, ws, ws_bytes, stream);
}

extern "C" int w4a8_moe_forward_ep(const uint16_t* x, const float* logits, int64_t T, int64_t H, int64_t I,
                                   int64_t E, int k, int renormalize, const int32_t* expert_map, int64_t E_local,
                                   const uint8_t* w13, const float* w13_s, const uint8_t* w2, const float* w2_s,
                                   uint16_t* out, void* ws, size_t ws_bytes, void* stream) {
  using namespace w4a8;
  w4a8_moe_layout L;
  int rc = layout_of(T, H, I, E, k, &L);
  if (rc) return rc;
  W4A8_REQUIRE(expert_map != nullptr, "expert_map is null");
  W4A8_REQUIRE(E_local >= 1 && E_local <= E && E_local <= 1024, "E_local=%lld must be in [1, min(E, 1024)]",
               (long long)E_local);
  W4A8_REQUIRE(ws != nullptr && ws_bytes >= L.total, "workspace too small: need %zu bytes", L.total);
  W4A8_REQUIRE((reinterpret_cast<uintptr_t>(ws) & 255) == 0, "workspace must be 256-byte aligned");
  if (T == 0) return W4A8_OK;
  uint8_t* b = static_cast<uint8_t*>(ws);
  int32_t* ids = reinterpret_cast<int32_t*>(b + L.topk_ids);
  float* tw = reinterpret_cast<float*>(b + L.topk_w);
  int64_t* seg = reinterpret_cast<int64_t*>(b + L.seg_indptr);  // [E_local + 1] of the [E + 1] slot
  int32_t* s2d = reinterpret_cast<int32_t*>(b + L.src2dst);
  int32_t* d2s = reinterpret_cast<int32_t*>(b + L.dst2src);
  uint8_t* xq = b + L.xq;
  float* xs = reinterpret_cast<float*>(b + L.xs);
  float* xc = reinterpret_cast<float*>(b + L.xc);
  uint16_t* y13 = reinterpret_cast<uint16_t*>(b + L.y13);
  uint8_t* hq = b + L.hq;
  float* hs = reinterpret_cast<float*>(b + L.hs);
  float* hc = reinterpret_cast<float*>(b + L.hc);
  uint16_t* y2 = reinterpret_cast<uint16_t*>(b + L.y2);
  const int64_t P = T * k;  // upper bound of the local pairs; the count itself is seg[E_local]
  if ((rc = moe_route_topk(logits, T, E, k, renormalize, ids, tw, stream))) return rc;
  if ((rc = moe_permute_ep(ids, T, k, E, expert_map, E_local, seg, s2d, d2s, b + L.permute_ws,
                           permute_ws_bytes(P, E_local), stream)))
    return rc;
  if ((rc = fp8_quant_scatter_per_token_group(x, T, H, s2d, k, P, xq, xs, xc, L.scale_ld, stream))) return rc;
  if ((rc = w4a8_grouped_gemm(xq, xs, xc, L.scale_ld, w13, w13_s, seg, E_local, 2 * I, H, P, y13, nullptr, 0,
                              stream)))
    return rc;
  if ((rc = silu_mul_requant_rows(y13, P, seg + E_local, I, hq, hs, hc, L.scale_ld, stream))) return rc;
  if ((rc = w4a8_grouped_gemm(hq, hs, hc, L.scale_ld, w2, w2_s, seg, E_local, H, I, P, y2, nullptr, 0, stream)))
    return rc;
  return moe_unpermute_combine(y2, s2d, tw, T, k, H, out, stream);
}
