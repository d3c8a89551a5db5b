// paged.cuh -- what the paged-cache kernels share: the page pool's geometry
// and the lookup of a slot's pool row.
#pragma once

#include <cstdint>

#include "dsa_internal.h"
#include "sm100.cuh"

namespace dsa {

// A paged cache as the kernels see it.
struct PagePool {
  const int32_t* table;  // row b at table + b * ld
  int64_t ld;
  int64_t n_pages;
  int max_pages;
  int page_size;  // multiple of 16
};

// Longest sequence the page lists can hold.
__device__ __forceinline__ int64_t pool_capacity(const PagePool& p) { return (int64_t)p.max_pages * p.page_size; }

// Pool row of a slot, or -1 where its page number is outside the pool.  The
// slot must lie below the pool's capacity.
__device__ __forceinline__ int64_t pool_row(const PagePool& p, int b, int32_t slot) {
  const int32_t i = slot / p.page_size;
  const int32_t page = __ldg(p.table + (int64_t)b * p.ld + i);
  if (page < 0 || page >= p.n_pages) return -1;
  return (int64_t)page * p.page_size + (slot - i * p.page_size);
}

// The length of sequence b as the kernels use it: 0 where lens[b] is outside
// [0, cap] (bad is then set).
__device__ __forceinline__ int32_t checked_len(int32_t len, int64_t cap, bool& bad) {
  bad = len < 0 || (int64_t)len > cap;
  return bad ? 0 : len;
}

// ceil(a / b); the quotient in 32 bits where they hold it (a 64-bit division
// takes a few hundred cycles).
__device__ __forceinline__ int64_t ceil_div(int64_t a, int b) {
  const int64_t n = a + b - 1;
  return n < ((int64_t)1 << 31) ? (int64_t)((uint32_t)n / (uint32_t)b) : n / b;
}

// NBOX boxes of BOX rows, NBLK column blocks each, into blocks of BYTES.
// Spelled out: an issue then takes about 16 cycles, in a loop over the boxes 45.
template <int BOX, int NBOX, int NBLK, int BYTES>
__device__ __forceinline__ void load_boxes(uint32_t dst, const CUtensorMap* tm, int x0, const int32_t* ys, uint32_t full) {
  int32_t y[NBOX];
#pragma unroll
  for (int i = 0; i < NBOX; ++i) y[i] = ys[i];
#pragma unroll
  for (int i = 0; i < NBOX; ++i)
#pragma unroll
    for (int blk = 0; blk < NBLK; ++blk)
      tma_load_2d(dst + blk * BYTES + i * BOX * 128, tm, x0 + 64 * blk, y[i], full);
}

inline bool is_aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
template <class... Ptr>
bool is_aligned4(Ptr... p) {
  return ((reinterpret_cast<uintptr_t>(p) | ...) & 3u) == 0;
}

// Checks of the arguments that describe the pool (host).
inline int check_pool(const void* kv_pages, const int32_t* table, int64_t ld_table, int max_pages, int page_size,
                      int64_t n_pages) {
  if (!kv_pages || !table || !is_aligned16(kv_pages) || !is_aligned4(table)) return DSA_ERR_INVALID_ARG;
  if (max_pages < 1 || ld_table < max_pages) return DSA_ERR_INVALID_ARG;
  if (page_size < 16 || page_size % 16 != 0 || n_pages < 1) return DSA_ERR_INVALID_ARG;
  if (n_pages > (((int64_t)1 << 31) - 4096) / page_size) return DSA_ERR_INVALID_ARG;
  return DSA_OK;
}

// Checks of the per-slot arrays (host); either may be NULL.
inline int check_slots(const float* acc, const int32_t* pos, int64_t ld_slots) {
  if (!acc && !pos) return DSA_OK;
  if (ld_slots < 1 || (ld_slots & 3) != 0 || ld_slots > ((int64_t)1 << 31) - 4096) return DSA_ERR_INVALID_ARG;
  if (!is_aligned16(acc) || !is_aligned16(pos)) return DSA_ERR_INVALID_ARG;
  return DSA_OK;
}

}  // namespace dsa
