// paged_attention_decode: argument checks, workspace, choice of the instance (paged_attention.cuh).
#include <atomic>

#include "paged_attention.cuh"

namespace w4a8 {
namespace {

std::atomic<int> g_force{0};  // way asked for by a test

// Workspace: places before each sequence, the runs' starts, then (m, l) and O of two parts of every warp.
struct AttendLayout {
  size_t starts, ml, o, total;
};
AttendLayout attend_layout(int64_t B, int64_t G, int64_t D) {
  const auto up = [](size_t v) { return (v + 255) & ~size_t(255); };
  const int DT = attend_dt(D);
  const size_t rows = static_cast<size_t>(attend_warps(DT)) * 2 * 16 * attend_mt(DT, static_cast<int>(G));
  AttendLayout L;
  L.starts = up(static_cast<size_t>(B + 1) * 8);
  L.ml = L.starts + up(static_cast<size_t>(attend_warps(DT)) * sizeof(RunStart));
  L.o = L.ml + up(rows * 8);
  L.total = L.o + up(rows * static_cast<size_t>(D) * 4);
  return L;
}

// Blocks of the cluster that shares an item of up to `longest` tokens, 0 where the list's warps take all items: the smaller
// estimate.  A cluster needs one launch and no joining kernel but has few warps; as many blocks as stay resident are used.
// Per warp's tile of 8 KB 0.8 us alone and 1.15 with every SM busy, 1.05 from the list (where sequences are half as long as
// the table on average); fitted to 1 to 256 sequences of up to 16 to 4096 tokens (16 x 512, 8 heads: 10 us, 16 by the list; 16
// x 1024 14 and 20; 1 x 4096 13.6 both; 64 x 1024 39 and 37).
int attend_cluster(int64_t B, int64_t Hq, int64_t heads, int64_t D, bool fp8, int64_t longest) {
  const int force = g_force.load(std::memory_order_relaxed);
  if (force) return force & 15;
  const int DT = attend_dt(D), G = static_cast<int>(Hq / heads), NT = attend_tile(fp8, DT), warps = attend_warps(DT);
  const int64_t items = B * heads * ceil_div(G, 16 * attend_mt(DT, G)), tiles = ceil_div(longest, NT), resident = warps / kAttendWarps;
  for (int c = 8; c >= 1; c /= 2) {
    if (items * c > resident || (c > 1 && (c - 1) * kAttendWarps >= tiles)) continue;
    const double tile = 2.0 * NT * DT * (fp8 ? 1 : 2) / 8192;
    const double here = 5.5 + tile * static_cast<double>(ceil_div(tiles, c * kAttendWarps)) *
                                  (0.8 + 0.35 * static_cast<double>(items * c) / static_cast<double>(resident));
    const double list = 11.0 + tile * 1.05 * static_cast<double>(ceil_div(items * tiles, warps));
    return here <= list ? c : 0;
  }
  return 0;
}

}  // namespace
}  // namespace w4a8

extern "C" int paged_attention_decode(const void* q, int64_t ldq_b, int64_t ldq_h, int dtype, int64_t Hq,
                                      const w4a8_paged_cache* cache, float scale, int64_t window, void* out,
                                      int64_t ldo_b, int64_t ldo_h, float* lse, void* ws, size_t ws_bytes, void* stream) {
  using namespace w4a8;
  if (int rc = check_cache(cache, dtype)) return rc;
  const bool fp8 = cache->dtype == W4A8_DTYPE_E4M3;
  const int64_t D = cache->D, H = cache->heads, B = cache->B, size = fp8 ? 1 : 2;
  W4A8_REQUIRE(D >= 8 && D <= 256 && D % (fp8 ? 16 : 8) == 0, "D=%lld must be a multiple of %d up to 256", (long long)D,
               fp8 ? 16 : 8);
  W4A8_REQUIRE(Hq >= 1 && Hq % H == 0 && Hq / H <= 256, "Hq=%lld must be a multiple of heads=%lld, at most 256 times it",
               (long long)Hq, (long long)H);
  W4A8_REQUIRE(B * H < (1ll << 24) && B * Hq < (1ll << 31), "B=%lld times heads=%lld must be below 2^24, times Hq=%lld below 2^31",
               (long long)B, (long long)H, (long long)Hq);
  W4A8_REQUIRE(window >= 0, "window=%lld must not be negative", (long long)window);
  W4A8_REQUIRE(scale - scale == 0.f, "scale must be finite");
  W4A8_REQUIRE(ldq_b >= 0 && ldq_h >= 0 && ldo_b >= 0 && ldo_h >= 0, "strides must not be negative");
  const int DT = attend_dt(D), G = static_cast<int>(Hq / H), rows = 16 * attend_mt(DT, G);
  const int64_t max_len = cache->table_pages * cache->page_size;
  W4A8_REQUIRE(B * H * ceil_div(G, rows) * (ceil_div(max_len + 1, 16) + 1) < (1ll << 38),
               "B=%lld sequences of up to %lld tokens are too many for one call", (long long)B, (long long)max_len);
  if (B == 0) return W4A8_OK;
  W4A8_REQUIRE(q && out && cache->seq_lens, "null pointer");
  W4A8_REQUIRE(max_len == 0 || cache->page_table, "null pointer: page_table");
  W4A8_REQUIRE(cache->pages == 0 || (cache->k && cache->v), "null pointer: k and v of the cache");
  W4A8_REQUIRE((bits_of(q) | bits_of(out)) % 2 == 0 && bits_of(lse) % 4 == 0,
               "q, out and lse must be aligned to their element size");
  const uint64_t strides = static_cast<uint64_t>(cache->k_page | cache->k_slot | cache->k_head | cache->v_page |
                                                 cache->v_slot | cache->v_head) * size;
  W4A8_REQUIRE((bits_of(cache->k) | bits_of(cache->v) | strides) % 16 == 0,
               "the cache's pointers and strides must be multiples of 16 bytes");
  const AttendLayout L = attend_layout(B, G, D);
  const int cluster = attend_cluster(B, Hq, H, D, fp8, window > 0 && window < max_len ? window : max_len);
  W4A8_REQUIRE(cluster || (ws && ws_bytes >= L.total && aligned16(ws)), "%zu bytes of 16-byte aligned workspace are needed", L.total);
  AttendParams p = {};
  p.q = q;
  p.k = cache->k;
  p.v = cache->v;
  p.out = out;
  p.lse = lse;
  p.table = cache->page_table;
  p.lens = cache->seq_lens;
  p.k_scale = cache->k_scale;
  p.v_scale = cache->v_scale;
  p.q_b = ldq_b;
  p.q_h = ldq_h;
  p.o_b = ldo_b;
  p.o_h = ldo_h;
  p.k_page = cache->k_page * size;
  p.k_slot = cache->k_slot * size;
  p.k_head = cache->k_head * size;
  p.v_page = cache->v_page * size;
  p.v_slot = cache->v_slot * size;
  p.v_head = cache->v_head * size;
  p.table_ld = cache->table_ld;
  p.pages = cache->pages;
  p.max_len = max_len;
  uint8_t* w = static_cast<uint8_t*>(ws);
  p.prefix = reinterpret_cast<int64_t*>(w);
  p.starts = reinterpret_cast<RunStart*>(w + L.starts);
  p.part_ml = reinterpret_cast<float2*>(w + L.ml);
  p.part_o = reinterpret_cast<float*>(w + L.o);
  p.B = static_cast<int>(B);
  p.Hq = static_cast<int>(Hq);
  p.Hkv = static_cast<int>(H);
  p.G = G;
  p.D = static_cast<int>(D);
  p.window = static_cast<int>(window < INT32_MAX ? window : 0);  // no length is above that: nothing is left out
  p.cluster = cluster;
  p.scale = scale * 1.44269504089f;
  p.by_page = FastDiv(cache->page_size);
  const bool q_f16 = dtype == W4A8_DTYPE_F16;
  p.q_vec = (bits_of(q) | static_cast<uint64_t>(ldq_b | ldq_h) * 2) % 16 == 0;
  p.out_pair = (bits_of(out) | static_cast<uint64_t>(ldo_b | ldo_h) * 2) % 4 == 0;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (fp8) return launch_attend_fp8(p, q_f16, st);
  return q_f16 ? launch_attend_f16(p, st) : launch_attend_bf16(p, st);
}

extern "C" int w4a8_test_paged_attention_way(int way) {
  W4A8_REQUIRE(way == 0 || way == 16 || way == 1 || way == 2 || way == 4 || way == 8, "way=%d must be 0, 1, 2, 4, 8 or 16", way);
  w4a8::g_force.store(way);
  return W4A8_OK;
}

extern "C" size_t paged_attention_workspace_bytes(int64_t B, int64_t Hq, int64_t heads, int64_t D, int cache_dtype,
                                                  int64_t longest) {
  if (B <= 0 || heads <= 0 || Hq < heads || D < 8 || D > 256) return 0;
  if (longest >= 0 && w4a8::attend_cluster(B, Hq, heads, D, cache_dtype == W4A8_DTYPE_E4M3, longest)) return 0;
  return w4a8::attend_layout(B, Hq / heads, D).total;
}
