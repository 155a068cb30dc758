// What the operators of the attention half share: whole-number division by a run-time divisor, places in a paged cache.
#pragma once

#include "block_ops.cuh"

namespace w4a8 {

// n / d for 0 <= n < 2^31 and 1 <= d < 2^31 by a product: with 2^(s-1) < d <= 2^s and m = floor(2^32 (2^s - d) / d) + 1,
// n / d = floor((n + floor(m n / 2^32)) / 2^s) (Granlund and Montgomery, "Division by invariant integers using
// multiplication", PLDI 1994).
struct FastDiv {
  uint32_t d, m, s;
  FastDiv() = default;
  explicit FastDiv(int64_t divisor) {
    d = static_cast<uint32_t>(divisor);
    s = 0;
    while ((1ull << s) < d) ++s;
    m = static_cast<uint32_t>(((1ull << 32) * ((1ull << s) - d)) / d + 1);
  }
  __device__ __forceinline__ int div(int n) const {
    return static_cast<int>((static_cast<uint32_t>(n) + __umulhi(m, static_cast<uint32_t>(n))) >> s);
  }
  __device__ __forceinline__ int div(int n, int& rest) const {
    const int q = div(n);
    rest = n - q * static_cast<int>(d);
    return q;
  }
};

inline uint64_t bits_of(const void* q) { return static_cast<uint64_t>(reinterpret_cast<uintptr_t>(q)); }

// Checks of a cache that its operators share.
inline int check_cache(const w4a8_paged_cache* c, int dtype) {
  W4A8_REQUIRE(c, "null pointer: cache");
  W4A8_REQUIRE(dtype == W4A8_DTYPE_BF16 || dtype == W4A8_DTYPE_F16, "dtype=%d must be bf16 or f16", dtype);
  W4A8_REQUIRE(c->dtype == dtype || c->dtype == W4A8_DTYPE_E4M3, "cache dtype=%d must be dtype=%d or E4M3", c->dtype,
               dtype);
  W4A8_REQUIRE(c->B >= 0 && c->B < (1ll << 24), "B=%lld out of range", (long long)c->B);
  W4A8_REQUIRE(c->pages >= 0 && c->pages < (1ll << 31), "pages=%lld out of range", (long long)c->pages);
  W4A8_REQUIRE(c->page_size >= 1 && c->page_size <= (1 << 20), "page_size=%lld must be in [1, 2^20]",
               (long long)c->page_size);
  W4A8_REQUIRE(c->heads >= 1 && c->heads < (1 << 16), "heads=%lld must be in [1, 2^16)", (long long)c->heads);
  W4A8_REQUIRE(c->table_pages >= 0 && c->table_pages < (1ll << 31) && c->table_pages * c->page_size < (1ll << 31),
               "table_pages=%lld times page_size=%lld must be below 2^31", (long long)c->table_pages,
               (long long)c->page_size);
  W4A8_REQUIRE(c->B <= 1 || c->table_ld >= c->table_pages, "table_ld=%lld must be at least table_pages=%lld",
               (long long)c->table_ld, (long long)c->table_pages);
  const int64_t strides[6] = {c->k_page, c->k_slot, c->k_head, c->v_page, c->v_slot, c->v_head};
  for (int64_t s : strides) W4A8_REQUIRE(s >= 0, "strides of the cache must not be negative");
  W4A8_REQUIRE(c->dtype == W4A8_DTYPE_E4M3 || (!c->k_scale && !c->v_scale), "scales given for a cache of 16 bits");
  const uintptr_t ints = reinterpret_cast<uintptr_t>(c->page_table) | reinterpret_cast<uintptr_t>(c->seq_lens) |
                         reinterpret_cast<uintptr_t>(c->k_scale) | reinterpret_cast<uintptr_t>(c->v_scale);
  W4A8_REQUIRE(ints % 4 == 0, "page_table, seq_lens, k_scale and v_scale must be aligned to 4 bytes");
  return W4A8_OK;
}

}  // namespace w4a8
