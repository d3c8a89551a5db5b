// paged_cache.cu -- row traffic of the paged latent cache: the write of the
// newest tokens and the row moves of an eviction.
//
// Both only move bytes: a token is one 1152-byte row (576 bf16) read and
// written, plus its acc and pos entries.  HBM bounds them for prompts and
// large evictions, launch latency for single steps.  B200: 8 prompts of 4096
// tokens (75.8 MB) in 14.5 us, 198 K moves of random rows (461 MB) in 94 us, 4.9
// TB/s; loads alone of as many rows in flight as registers hold reach 3.6.
// Four rows in flight per warp instead of one measured the same.
#include <algorithm>

#include "paged.cuh"

namespace dsa {
namespace {

constexpr int kRowPieces = kDQK / 8;  // 16-byte pieces per row: 72

// One warp copies one row: lanes take the pieces l, l + 32, l + 64.
__device__ __forceinline__ void copy_row(uint4* __restrict__ dst, const uint4* __restrict__ src, int lane) {
  const uint4 a = src[lane], b = src[lane + 32];
  uint4 c;
  if (lane < kRowPieces - 64) c = src[lane + 64];
  dst[lane] = a;
  dst[lane + 32] = b;
  if (lane < kRowPieces - 64) dst[lane + 64] = c;
}

// One warp per new token (b, t).
__global__ void __launch_bounds__(256)
    paged_append_kernel(const __nv_bfloat16* __restrict__ kv_new, const int32_t* __restrict__ lens, PagePool pool, int B,
                        int T, __nv_bfloat16* __restrict__ kv, float* __restrict__ acc, int32_t* __restrict__ pos,
                        const int32_t* __restrict__ end_pos, int64_t ld_slots, int32_t* status) {
  grid_dependency_wait();  // the new rows may come from the previous kernel
  allow_dependents_launch();
  const int lane = threadIdx.x & 31;
  const int64_t tok = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
  if (tok >= (int64_t)B * T) return;
  const int b = (int)(tok / T), t = (int)(tok - (int64_t)b * T);
  bool bad;
  int64_t cap = pool_capacity(pool);
  if (acc || pos) cap = min(cap, ld_slots);
  const int32_t len = checked_len(lens[b], cap, bad);
  if (bad || (len > 0 && len < T)) {
    if (lane == 0) report(status, DSA_ERR_BAD_OFFSETS);
    return;
  }
  if (len == 0) return;
  const int32_t slot = len - T + t;
  const int64_t row = pool_row(pool, b, slot);
  if (row < 0) {
    if (lane == 0) report(status, DSA_ERR_BAD_INDEX);
  } else {
    copy_row(reinterpret_cast<uint4*>(kv + row * kDQK), reinterpret_cast<const uint4*>(kv_new + tok * kDQK), lane);
  }
  if (lane == 0) {
    if (acc) acc[(int64_t)b * ld_slots + slot] = 0.f;
    if (pos) pos[(int64_t)b * ld_slots + slot] = end_pos[b] - T + t;
  }
}

// One warp per move.  The moves of 256 sequences form one list, dealt out to
// the warps in turn, because the sequences' lists differ in length and only the
// device knows them: one list of 16K moves among 32 takes 12 us, 72 with a
// thirty-second of the card for each sequence.
constexpr int kMoveThreads = 256, kMoveGroup = kMoveThreads;

__global__ void __launch_bounds__(kMoveThreads)
    paged_move_kernel(__nv_bfloat16* kv, PagePool pool, const int32_t* __restrict__ n_moves,
                      const int32_t* __restrict__ move_dst, const int32_t* __restrict__ move_src, int64_t ld_moves, int B,
                      float* acc, int32_t* pos, int64_t ld_slots, int32_t* status) {
  __shared__ int64_t s_first[kMoveGroup + 1];  // a sequence's first move in the list
  __shared__ int64_t s_sum[kMoveThreads / 32];
  grid_dependency_wait();  // the plan may come from the previous kernel
  allow_dependents_launch();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int64_t cap = pool_capacity(pool);
  if (acc || pos) cap = min(cap, ld_slots);
  for (int64_t b0 = (int64_t)blockIdx.y * kMoveGroup; b0 < B; b0 += (int64_t)gridDim.y * kMoveGroup) {
    int64_t n = b0 + threadIdx.x < B ? n_moves[b0 + threadIdx.x] : 0;
    if (n < 0 || n > ld_moves) {
      if (blockIdx.x == 0) report(status, DSA_ERR_BAD_OFFSETS);
      n = 0;
    }
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t v = __shfl_up_sync(0xffffffffu, n, o);
      if (lane >= o) n += v;
    }
    if (lane == 31) s_sum[warp] = n;
    __syncthreads();
    for (int w = 0; w < warp; ++w) n += s_sum[w];
    s_first[threadIdx.x + 1] = n;
    if (threadIdx.x == 0) s_first[0] = 0;
    __syncthreads();
    const int64_t total = s_first[kMoveGroup];
    const int seqs = (int)min((int64_t)kMoveGroup, B - b0);
    int at = 0;
    for (int64_t i = (int64_t)blockIdx.x * (kMoveThreads / 32) + warp; i < total;
         i += (int64_t)gridDim.x * (kMoveThreads / 32)) {
      for (int end = seqs; end - at > 1;) {  // s_first[at] <= i < s_first[end]
        const int mid = (at + end) >> 1;
        if (s_first[mid] <= i) at = mid;
        else end = mid;
      }
      const int64_t b = b0 + at, m = b * ld_moves + (i - s_first[at]);
      const int32_t d = move_dst[m], s = move_src[m];
      const bool in = d >= 0 && s >= 0 && d < cap && s < cap;
      const int64_t rd = in ? pool_row(pool, (int)b, d) : -1, rs = in ? pool_row(pool, (int)b, s) : -1;
      if (rd < 0 || rs < 0) {
        if (lane == 0) report(status, DSA_ERR_BAD_INDEX);
        continue;
      }
      copy_row(reinterpret_cast<uint4*>(kv + rd * kDQK), reinterpret_cast<const uint4*>(kv + rs * kDQK), lane);
      if (lane == 0) {
        const int64_t o = b * ld_slots;
        if (acc) acc[o + d] = acc[o + s];
        if (pos) pos[o + d] = pos[o + s];
      }
    }
    __syncthreads();  // the list is read
  }
}

}  // namespace
}  // namespace dsa

using namespace dsa;

extern "C" {

int dsa_paged_append(const void* kv_new, const int32_t* lens, const int32_t* page_table, int64_t ld_table,
                     int max_pages, int B, int T, int page_size, int64_t n_pages, void* kv_pages, float* acc,
                     int32_t* pos, const int32_t* end_pos, int64_t ld_slots, int32_t* dev_status, void* stream) {
  if (B <= 0 || T <= 0 || !kv_new || !lens || !is_aligned16(kv_new) || !is_aligned4(lens, end_pos, dev_status))
    return DSA_ERR_INVALID_ARG;
  if ((int64_t)B * T > (int64_t)1 << 24) return DSA_ERR_UNSUPPORTED;
  if (int rc = check_pool(kv_pages, page_table, ld_table, max_pages, page_size, n_pages)) return rc;
  if (int rc = check_slots(acc, pos, ld_slots)) return rc;
  if (pos && !end_pos) return DSA_ERR_INVALID_ARG;
  const PagePool pool{page_table, ld_table, n_pages, max_pages, page_size};
  const int64_t toks = (int64_t)B * T;
  const cudaError_t e =
      launch_pdl(paged_append_kernel, dim3((unsigned)((toks + 7) / 8)), dim3(256), 0,
                 reinterpret_cast<cudaStream_t>(stream), reinterpret_cast<const __nv_bfloat16*>(kv_new), lens, pool, B, T,
                 reinterpret_cast<__nv_bfloat16*>(kv_pages), acc, pos, end_pos, ld_slots, dev_status);
  return e == cudaSuccess ? DSA_OK : DSA_ERR_CUDA;
}

int dsa_paged_move(void* kv_pages, const int32_t* page_table, int64_t ld_table, int max_pages, int page_size,
                   int64_t n_pages, const int32_t* n_moves, const int32_t* move_dst, const int32_t* move_src,
                   int64_t ld_moves, int B, float* acc, int32_t* pos, int64_t ld_slots, int32_t* dev_status,
                   void* stream) {
  if (B <= 0 || !n_moves || !move_dst || !move_src || ld_moves < 1) return DSA_ERR_INVALID_ARG;
  if (!is_aligned4(n_moves, move_dst, move_src, dev_status)) return DSA_ERR_INVALID_ARG;
  if (B > (1 << 24)) return DSA_ERR_UNSUPPORTED;
  if (int rc = check_pool(kv_pages, page_table, ld_table, max_pages, page_size, n_pages)) return rc;
  if (int rc = check_slots(acc, pos, ld_slots)) return rc;
  const PagePool pool{page_table, ld_table, n_pages, max_pages, page_size};
  // Eight CTAs of eight warps per SM over all groups of sequences, fewer where
  // the lists have no room for as many moves.
  const int64_t groups = ((int64_t)B + kMoveGroup - 1) / kMoveGroup, y = std::min<int64_t>(groups, 32768);
  const int64_t room = (std::min<int64_t>(B, kMoveGroup) * ld_moves + kMoveThreads / 32 - 1) / (kMoveThreads / 32);
  const int64_t x = std::min<int64_t>(room, std::max<int64_t>(1, (8 * (int64_t)device_info().sm_count + y - 1) / y));
  const cudaError_t e =
      launch_pdl(paged_move_kernel, dim3((unsigned)x, (unsigned)y), dim3(kMoveThreads), 0, reinterpret_cast<cudaStream_t>(stream),
                 reinterpret_cast<__nv_bfloat16*>(kv_pages), pool, n_moves, move_dst, move_src, ld_moves, B, acc, pos,
                 ld_slots, dev_status);
  return e == cudaSuccess ? DSA_OK : DSA_ERR_CUDA;
}

}  // extern "C"
