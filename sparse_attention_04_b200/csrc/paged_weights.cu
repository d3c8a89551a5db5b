// paged_weights.cu -- the attention weight that every slot of a paged cache
// collects from the newest tokens' heads:
//   acc_out[b,s] = decay * acc[b,s] + sum_{t,h : s <= len-T+t} exp(scale q.k_s - lse)
//
// The cache is read once (1152 bytes a slot), against 2 * 576 flops and one
// exponential per slot and head: HBM bounds it up to 128 (token, head) rows.
//
// S^T = K.Q^T, the slots as the M = 128 rows of the product: a thread of the
// epilogue then owns one slot (TMEM lane) and sums over heads in its own
// registers, in a fixed order, in fp32.  The query rows of a sequence, up to
// 128 (t, h) pairs at a time, stay in shared memory as the B operand; a
// chunk's rows stream through a ring of 128-row x 64-column blocks, as many
// places as fit beside the query.  Every CTA takes an equal, contiguous part of
// the list of all sequences' 128-slot chunks.
//
// Roles: warps 0-3 epilogue, warp 4 loader, warp 5 TMEM allocator and MMA
// issuer.  S^T has two TMEM buffers, so that the exponentials of a chunk run
// beside the products of the next.
#include <cuda.h>
#include <cuda_bf16.h>

#include <algorithm>

#include "paged.cuh"
#include "tmap.h"

namespace dsa {
namespace {

constexpr int kChunk = 128;                  // slots per chunk: the product's M
constexpr int kKB = kDQK / 64;               // 64-column blocks of a row: 9
constexpr int kBlockBytes = kChunk * 128;    // one block of a chunk
constexpr int kMaxCols = 128;                // (t, h) rows per query tile: the product's N
constexpr int kMaxPlaces = 12;
constexpr int kThreads = 192;
constexpr int kLoadWarp = 4, kMmaWarp = 5;
constexpr int kSmemTotal = 232448 - 1024;    // behind the 1024-byte alignment
enum Bar : int { kQFull = 0, kQFree, kKFull, kKEmpty = kKFull + kMaxPlaces, kSFull = kKEmpty + kMaxPlaces, kSEmpty = kSFull + 2, kDrain = kSEmpty + 2, kNumBar };
struct Misc {
  uint64_t bars[kNumBar];
  alignas(16) float lse2[2][kMaxCols];  // lse * log2(e) per column, by query tile parity; +inf where nothing is to be added
  int32_t y[8];             // row coordinates of a chunk's boxes
  int tmem_base, abort, first_seq, pad;
  int64_t first_unit, total_units;
  int64_t warp_sum[kThreads / 32];
};
constexpr int kMiscBytes = (int)((sizeof(Misc) + 1023) / 1024 * 1024);
constexpr int kRingOff = kMiscBytes;         // the ring, then the query's blocks
static_assert(offsetof(Misc, lse2) % 16 == 0 && offsetof(Misc, bars) == 0, "alignment");
static_assert(kSmemTotal - kMiscBytes - kKB * kMaxCols * 128 >= 4 * kBlockBytes, "four places beside the largest query tile");

struct PagedWeightsParams {
  PagePool pool;
  const int32_t* lens;
  const float* lse;
  int B, T, H;
  int cols;     // (t, h) rows per query tile, a multiple of 16
  int places;   // ring places
  int box;      // rows per TMA box
  float scale_log2, decay;
  const float* acc;
  float* acc_out;
  int64_t ld_slots;
  int32_t* status;
  uint64_t wait_limit_ns;
};

__device__ __forceinline__ int32_t seq_len(const PagedWeightsParams& p, int b, bool& bad) {
  return checked_len(__ldg(p.lens + b), min(pool_capacity(p.pool), p.ld_slots), bad);
}
__device__ __forceinline__ int64_t n_chunks_of(int32_t len) { return ((int64_t)len + kChunk - 1) / kChunk; }

// The parts of sequences that fall to this CTA, one after the other; every
// role walks the same list.
struct Walk {
  int64_t u, w0, w1;  // first unit of sequence b; this CTA's units
  int b, n_seq;
  int seq, lo, hi;    // the current part
  int32_t len;

  __device__ __forceinline__ bool next(const PagedWeightsParams& p) {
    while (b < n_seq && u < w1) {
      bool bad;
      len = seq_len(p, b, bad);
      const int64_t c = n_chunks_of(len);
      seq = b;
      lo = (int)min(max(w0 - u, (int64_t)0), c);
      hi = (int)min(w1 - u, c);
      ++b;
      u += c;
      if (lo < hi) return true;
    }
    return false;
  }
};

__global__ void __launch_bounds__(kThreads, 1)
    paged_weights_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                         const PagedWeightsParams p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sbase = smem_u32(smem);
  Misc* misc = reinterpret_cast<Misc*>(smem);
  auto bar = [&](int i) { return sbase + 8u * (uint32_t)i; };
  volatile int* abort = &misc->abort;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t q_off = sbase + kRingOff + p.places * kBlockBytes;
  const int q_block = p.cols * 128;  // one 64-column block of a query tile

  if (threadIdx.x == 0) misc->abort = 0;
  if (warp == kMmaWarp) {
    if (lane == 0) {
      tma_prefetch_desc(&tm_k);
      for (int i = 0; i < kNumBar; ++i) mbar_init(bar(i), i >= kSEmpty && i < kSEmpty + 2 ? 4 : 1);
      fence_mbar_init();
    }
    __syncwarp();
    tmem_alloc(sbase + (uint32_t)offsetof(Misc, tmem_base), 2 * kMaxCols);
    tmem_relinquish();
  }
  grid_dependency_wait();  // everything may come from the previous kernel
  allow_dependents_launch();
  {
    // units (chunks) of all sequences, and the one this CTA's part begins in
    const int per = (p.B + kThreads - 1) / kThreads;
    const int b0 = min((int)threadIdx.x * per, p.B), b1 = min(b0 + per, p.B);
    int64_t mine = 0;
    for (int b = b0; b < b1; ++b) {
      bool bad;
      mine += n_chunks_of(seq_len(p, b, bad));
      if (bad && blockIdx.x == 0) report(p.status, DSA_ERR_BAD_OFFSETS);
    }
    int64_t inc = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t v = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += v;
    }
    if (lane == 31) misc->warp_sum[warp] = inc;
    __syncthreads();
    int64_t before = inc - mine, total = 0;
    for (int w = 0; w < kThreads / 32; ++w) {
      const int64_t v = misc->warp_sum[w];
      if (w < warp) before += v;
      total += v;
    }
    const int64_t w0 = (total + gridDim.x - 1) / gridDim.x * blockIdx.x;
    if (threadIdx.x == 0) {
      misc->total_units = total;
      if (w0 >= total) misc->first_seq = p.B;
    }
    if (before <= w0 && w0 < before + mine) {
      int64_t u = before;
      for (int b = b0; b < b1; ++b) {
        bool bad;
        const int64_t c = n_chunks_of(seq_len(p, b, bad));
        if (w0 < u + c) {
          misc->first_seq = b;
          misc->first_unit = u;
          break;
        }
        u += c;
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = static_cast<uint32_t>(misc->tmem_base);
  Walk wk;
  const int64_t share = (misc->total_units + gridDim.x - 1) / gridDim.x;
  wk.w0 = share * blockIdx.x;
  wk.w1 = min(wk.w0 + share, misc->total_units);
  wk.b = misc->first_seq;
  wk.n_seq = p.B;
  wk.u = wk.b < p.B ? misc->first_unit : 0;
  const int th = p.T * p.H, n_tiles = (th + p.cols - 1) / p.cols;

  if (warp == kLoadWarp) {
    const uint32_t on = elect_one();
    const int nbox = kChunk / p.box;
    const int32_t pool_rows = (int32_t)(p.pool.n_pages * p.pool.page_size);
    uint32_t tiles = 0, fills = 0;  // query tiles and blocks so far
    uint32_t place = 0, round = 0;
    bool ok = true;
    while (ok && wk.next(p)) {
      for (int qt = 0; ok && qt < n_tiles; ++qt, ++tiles) {
        // the query tile, once the products with the one before are complete
        if (tiles > 0 && !(ok = warp_wait(bar(kQFree), (tiles - 1) & 1, abort, p.wait_limit_ns))) break;
        if (on) {
          mbar_arrive_expect_tx(bar(kQFull), kKB * q_block);
#pragma unroll 1
          for (int kb = 0; kb < kKB; ++kb) tma_load_3d(q_off + kb * q_block, &tm_q, kb * 64, qt * p.cols, wk.seq, bar(kQFull));
        }
        __syncwarp();
        for (int i = wk.lo; ok && i < wk.hi; ++i) {
          const int64_t s = (int64_t)i * kChunk + lane * p.box;
          int32_t y = pool_rows;  // outside the pool: zeros
          if (lane < nbox && s < wk.len) {
            const int64_t row = pool_row(p.pool, wk.seq, (int32_t)s);
            if (row >= 0) y = (int32_t)row;
            else report(p.status, DSA_ERR_BAD_INDEX);
          }
          if (lane < 8) misc->y[lane] = y;
          __syncwarp();
#pragma unroll 1
          for (int kb = 0; kb < kKB; ++kb) {
            if (!(ok = warp_wait(bar(kKEmpty + place), (round & 1) ^ 1, abort, p.wait_limit_ns))) break;
            if (on) {
              const uint32_t full = bar(kKFull + place);
              uint32_t dst = sbase + kRingOff + place * kBlockBytes;
              mbar_arrive_expect_tx(full, kBlockBytes);
#pragma unroll 1
              for (int bx = 0; bx < nbox; bx += 2, dst += 2 * p.box * 128) {
                tma_load_2d(dst, &tm_k, kb * 64, misc->y[bx], full);
                tma_load_2d(dst + p.box * 128, &tm_k, kb * 64, misc->y[bx + 1], full);
              }
            }
            __syncwarp();
            ++fills;
            if (++place == (uint32_t)p.places) {
              place = 0;
              ++round;
            }
          }
          __syncwarp();  // the coordinates are read before the next chunk's are written
        }
      }
    }
    if (*abort) {
      // the loads in flight must land before the CTA exits (10 ms at most each)
      volatile int never = 0;
      for (uint32_t k = fills > (uint32_t)p.places ? fills - p.places : 0; k < fills; ++k)
        mbar_wait(bar(kKFull + k % p.places), (k / p.places) & 1, &never, 10000000ull);
      mbar_wait(bar(kQFull), tiles & 1, &never, 10000000ull);
    }
  } else if (warp == kMmaWarp) {
    const uint32_t on = elect_one();
    const uint64_t k0 = smem_desc(sbase + kRingOff, 16, 1024, kSwizzle128B);
    const uint64_t q0 = smem_desc(q_off, 16, 1024, kSwizzle128B);
    const uint32_t idesc = idesc_bf16(kChunk, p.cols);
    auto wait = [&](int which, uint32_t parity) {
      const bool there = warp_wait(bar(which), parity, abort, p.wait_limit_ns);
      tc_fence_after();
      return there;
    };
    uint32_t tiles = 0, g = 0, place = 0, round = 0;
    bool ok = true;
    while (ok && wk.next(p)) {
      for (int qt = 0; ok && qt < n_tiles; ++qt, ++tiles) {
        if (!(ok = wait(kQFull, tiles & 1))) break;
        for (int i = wk.lo; ok && i < wk.hi; ++i, ++g) {
          const int sb = g & 1;
          if (g >= 2 && !(ok = wait(kSEmpty + sb, ((g - 2) >> 1) & 1))) break;
          const uint32_t d = tmem + kMaxCols * sb;
#pragma unroll 1
          for (int kb = 0; kb < kKB; ++kb) {
            if (!(ok = wait(kKFull + place, round & 1))) break;
            const uint64_t ad = k0 + (uint64_t)((place * kBlockBytes) >> 4), bd = q0 + (uint64_t)((kb * q_block) >> 4);
#pragma unroll
            for (int ks = 0; ks < 4; ++ks)
              mma_f16_ss_if(on, d, ad + (uint64_t)ks * 2, bd + (uint64_t)ks * 2, idesc, (kb | ks) ? 1u : 0u);
            if (on) tc_commit(bar(kKEmpty + place));
            if (++place == (uint32_t)p.places) {
              place = 0;
              ++round;
            }
          }
          if (ok && on) tc_commit(bar(kSFull + sb));
        }
        if (ok && on) tc_commit(bar(kQFree));
      }
    }
    if (*abort && on) {  // tensor-core work ends before TMEM is released
      volatile int never = 0;
      tc_commit(bar(kDrain));
      mbar_wait(bar(kDrain), 0, &never, 10000000ull);
    }
  } else {
    // ---- epilogue: thread = slot of the chunk
    const uint32_t lane_addr = tmem + (static_cast<uint32_t>(warp * 32) << 16);
    uint32_t tiles = 0, g = 0;
    bool ok = true, leave = false;
    while (!leave && wk.next(p)) {
      for (int qt = 0; qt < n_tiles; ++qt, ++tiles) {
        float* const lse2 = misc->lse2[tiles & 1];
        {
          const int c = qt * p.cols + threadIdx.x;
          float v = INFINITY;
          if ((int)threadIdx.x < p.cols && c < th) {
            const float l = __ldg(p.lse + (int64_t)wk.seq * th + c);
            v = l == -INFINITY ? INFINITY : l * 1.4426950408889634f;
          }
          lse2[threadIdx.x] = v;
        }
        // the tile's lse2 is written; a warp whose wait ran out takes the others along
        if (named_barrier_or(1, 128, !ok)) {
          leave = true;
          break;
        }
        for (int i = wk.lo; ok && i < wk.hi; ++i, ++g) {
          const int sb = g & 1;
          const int64_t s = (int64_t)i * kChunk + threadIdx.x;
          const bool in = s < wk.len;
          const bool there = in && pool_row(p.pool, wk.seq, (int32_t)s) >= 0;
          const int64_t o = (int64_t)wk.seq * p.ld_slots + s;
          float old = 0.f;
          if (in) old = qt > 0 ? p.acc_out[o] : p.acc ? p.decay * p.acc[o] : 0.f;
          // columns from c_min on see this slot
          const int64_t beyond = s - ((int64_t)wk.len - p.T);
          const int c_min = beyond > 0 && in ? (int)min(beyond * p.H, (int64_t)th) - qt * p.cols : 0;
          const bool masked = __any_sync(0xffffffffu, c_min > 0);
          if (!(ok = warp_wait(bar(kSFull + sb), (g >> 1) & 1, abort, p.wait_limit_ns))) break;
          tc_fence_after();
          float sum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 1
          for (int c0 = 0; c0 < p.cols; c0 += 32) {
            uint32_t sv[32];
            tmem_ld32(lane_addr + kMaxCols * sb + c0, sv);
            tc_wait_ld();
            if (c0 + 32 >= p.cols) {
              tc_fence_before();
              warp_arrive(bar(kSEmpty + sb));
            }
#pragma unroll
            for (int c = 0; c < 32; c += 4) {
              const float4 l = *reinterpret_cast<const float4*>(lse2 + c0 + c);
              const float lv[4] = {l.x, l.y, l.z, l.w};
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                // columns that hold no query row were loaded as zeros: 0 - inf
                float x = fmaf(__uint_as_float(sv[c + e]), p.scale_log2, -lv[e]);
                if (masked && c0 + c + e < c_min) x = -INFINITY;
                if (lv[e] == INFINITY) x = -INFINITY;
                sum[e] += ex2_approx(x);
              }
            }
          }
          if (in) p.acc_out[o] = there ? old + ((sum[0] + sum[1]) + (sum[2] + sum[3])) : old;
        }
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == kMmaWarp) {
    tc_fence_after();
    tmem_dealloc(tmem, 2 * kMaxCols);
  }
  if (threadIdx.x == 0 && *abort) report(p.status, DSA_ERR_TIMEOUT);
}

}  // namespace
}  // namespace dsa

using namespace dsa;

extern "C" int dsa_paged_weights(const void* q, const void* kv_pages, const int32_t* page_table, int64_t ld_table,
                                 int max_pages, const int32_t* lens, const float* lse, int B, int T, int H,
                                 int page_size, int64_t n_pages, float scale, float decay, const float* acc,
                                 float* acc_out, int64_t ld_slots, int32_t* dev_status, void* stream) {
  if (B <= 0 || T <= 0 || H < 1 || !q || !lens || !lse || !acc_out) return DSA_ERR_INVALID_ARG;
  if ((int64_t)B * T > (int64_t)1 << 24 || H > DSA_MAX_HEADS) return DSA_ERR_UNSUPPORTED;
  if (int rc = check_pool(kv_pages, page_table, ld_table, max_pages, page_size, n_pages)) return rc;
  if (int rc = check_slots(acc_out, nullptr, ld_slots)) return rc;
  if (!is_aligned16(acc) || !is_aligned16(q)) return DSA_ERR_INVALID_ARG;
  if (!(scale == scale) || !(decay == decay)) return DSA_ERR_INVALID_ARG;
  PagedWeightsParams p;
  p.pool = PagePool{page_table, ld_table, n_pages, max_pages, page_size};
  p.lens = lens;
  p.lse = lse;
  p.B = B;
  p.T = T;
  p.H = H;
  const int64_t th = (int64_t)T * H;
  p.cols = (int)std::min<int64_t>((th + 15) / 16 * 16, kMaxCols);
  p.places = std::min(kMaxPlaces, (kSmemTotal - kMiscBytes - kKB * p.cols * 128) / kBlockBytes);
  p.box = page_size % 64 == 0 ? 64 : page_size % 32 == 0 ? 32 : 16;
  p.scale_log2 = scale * 1.4426950408889634f;
  p.decay = decay;
  p.acc = acc;
  p.acc_out = acc_out;
  p.ld_slots = ld_slots;
  p.status = dev_status;
  p.wait_limit_ns = kWaitLimitNs;
  CUtensorMap tq, tk;
  // rows behind a sequence's own query rows read as zeros
  const uint64_t dims[3] = {kDQK, (uint64_t)th, (uint64_t)B}, strides[2] = {kDQK * 2, (uint64_t)th * kDQK * 2};
  const uint32_t box[3] = {64, (uint32_t)p.cols, 1};
  if (!make_tmap_3d(&tq, q, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B) ||
      !make_tmap_2d(&tk, kv_pages, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, kDQK, (uint64_t)n_pages * page_size, kDQK * 2, 64,
                    (uint32_t)p.box, CU_TENSOR_MAP_SWIZZLE_128B))
    return DSA_ERR_CUDA;
  static PerDeviceOnce attr;
  if (attr.run([] {
        return cudaFuncSetAttribute(paged_weights_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemTotal + 1024);
      }) != cudaSuccess)
    return DSA_ERR_CUDA;
  const cudaError_t e = launch_pdl(paged_weights_kernel, dim3((unsigned)device_info().sm_count), dim3(kThreads),
                                   (size_t)(kSmemTotal + 1024), reinterpret_cast<cudaStream_t>(stream), tq, tk, p);
  return e == cudaSuccess ? DSA_OK : DSA_ERR_CUDA;
}
