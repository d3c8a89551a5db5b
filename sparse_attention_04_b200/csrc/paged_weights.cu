// paged_weights.cu -- the attention weight that every slot of a paged cache
// collects from the newest tokens' heads:
//   acc_out[b,s] = decay * acc[b,s] + sum_{t,h : s <= len-T+t} exp(scale q.k_s - lse)
//
// The cache is read once (1152 bytes a slot), against 2 * 576 flops and one
// exponential per slot and head: HBM bounds it up to 128 (token, head) rows.
//
// S = Q.K^T with the (token, head) rows of a sequence, up to 128 at a time, as
// the product's M: all but one of the query's 64-column blocks stay in TMEM as
// the A operand, which leaves shared memory to the ring that the cache streams
// through, four places of three 128-row x 64-column blocks (192 KB: HBM answers
// in about 2 us under load, so an SM has to keep 90 KB and more in flight.
// With the query in shared memory as the B operand, 80 KB of ring were left:
// 140 us against 106 for 16 ragged sequences of 560 K slots in all).
// A thread of the epilogue owns a query row (TMEM lane) and half of a chunk's
// slots; the sums over rows run across lanes (a butterfly that halves the
// columns as it halves the rows) and then across the four warps of a half, in
// fp32 and in a fixed order.  Every CTA takes an equal, contiguous part of the
// list of all sequences' 128-slot chunks.
//
// B200: 16 sequences of 1K to 65K slots, 128 heads (560 K slots, 644 MB): 106 us
// in a row, 119 with changing inputs, 6.1 and 5.4 TB/s; one 32K sequence 9.5 us in
// a row, 13 with changing inputs.
//
// Roles: warps 0-7 epilogue, warp 8 loader, warp 9 TMEM allocator and MMA
// issuer.  S has two TMEM buffers, so that the exponentials of a chunk run
// beside the products of the next.
#include <cuda.h>
#include <cuda_bf16.h>

#include <algorithm>

#include "paged.cuh"
#include "tmap.h"

namespace dsa {
namespace {

constexpr int kChunk = 128;                  // slots per chunk: the product's N
constexpr int kKB = kDQK / 64;               // 64-column blocks of a row: 9
constexpr int kBlockBytes = kChunk * 128;    // one block of a chunk, or of a query tile
constexpr int kRows = 128;                   // (token, head) rows per query tile: the product's M
constexpr int kPlaceBlocks = 3;
constexpr int kPlaceBytes = kPlaceBlocks * kBlockBytes;
constexpr int kPlaces = 4;
constexpr int kPerChunk = kKB / kPlaceBlocks;  // places a chunk, or a query tile, goes through
constexpr int kEpiWarps = 8;
constexpr int kThreads = 320;
constexpr int kLoadWarp = 8, kMmaWarp = 9;
constexpr uint32_t kTmemS = 256;             // query blocks 0-7 in [0, 256), S buffers at 256 and 384
constexpr uint32_t kIdesc = idesc_bf16(kRows, kChunk);
enum Bar : int { kQFull = 0, kQFree, kKFull, kKEmpty = kKFull + kPlaces, kSFull = kKEmpty + kPlaces, kSEmpty = kSFull + 2, kDrain = kSEmpty + 2, kNumBar };
struct Misc {
  uint64_t bars[kNumBar];
  alignas(16) int32_t y[8];  // row coordinates of a chunk's boxes
  float part[2][4][kChunk];  // sums over 32 rows each, by chunk parity
  int tmem_base, abort, first_seq, pad;
  int64_t first_unit;
  int64_t warp_sum[kThreads / 32];
};
constexpr int kQ8Off = (int)((sizeof(Misc) + 1023) / 1024 * 1024);
constexpr int kRingOff = kQ8Off + kBlockBytes;
constexpr int kSmemBytes = kRingOff + kPlaces * kPlaceBytes + 1024;
static_assert(kSmemBytes <= 232448 && offsetof(Misc, bars) == 0, "shared memory");

struct PagedWeightsParams {
  PagePool pool;
  const int32_t* lens;
  const float* lse;
  int B, T, H;
  int box;      // rows per TMA box
  float scale_log2, decay;
  const float* acc;
  float* acc_out;
  int64_t ld_slots;
  int32_t* status;
  int debug_stall;
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
                         const __grid_constant__ PagedWeightsParams p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sbase = smem_u32(smem);
  Misc* misc = reinterpret_cast<Misc*>(smem);
  auto bar = [&](int i) { return sbase + 8u * (uint32_t)i; };
  volatile int* abort = &misc->abort;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) misc->abort = 0;
  if (warp == kMmaWarp) {
    if (lane == 0) {
      tma_prefetch_desc(&tm_q);
      tma_prefetch_desc(&tm_k);
      for (int i = 0; i < kNumBar; ++i)
        mbar_init(bar(i), i == kQFull ? 1 + p.debug_stall : i >= kSEmpty && i < kSEmpty + 2 ? kEpiWarps : 1);
      fence_mbar_init();
    }
    __syncwarp();
    tmem_alloc(sbase + (uint32_t)offsetof(Misc, tmem_base), 512);
    tmem_relinquish();
  }
  grid_dependency_wait();  // everything may come from the previous kernel
  allow_dependents_launch();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = static_cast<uint32_t>(misc->tmem_base);
  // ---- units (chunks) of all sequences, and the one this CTA's part begins in
  Walk wk;
  wk.n_seq = p.B;
  int64_t total;
  constexpr int kPer = 4;
  if (p.B <= 32 * kPer) {
    // every warp for itself, a lane takes up to four sequences (one 32K
    // sequence: 9.5 us, with the CTA's threads 9.95)
    const int per = (p.B + 31) >> 5;
    int64_t units[kPer], mine = 0;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int b = lane * per + i;
      bool bad = false;
      units[i] = i < per && b < p.B ? n_chunks_of(seq_len(p, b, bad)) : 0;
      if (bad && blockIdx.x == 0 && warp == 0) report(p.status, DSA_ERR_BAD_OFFSETS);
      mine += units[i];
    }
    int64_t inc = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t v = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += v;
    }
    total = __shfl_sync(0xffffffffu, inc, 31);
    wk.w0 = ceil_div(total, (int)gridDim.x) * blockIdx.x;
    wk.b = p.B;
    wk.u = 0;
    const uint32_t has = __ballot_sync(0xffffffffu, inc - mine <= wk.w0 && wk.w0 < inc);
    if (has) {
      int b = lane * per;
      int64_t u = inc - mine, next = u;
#pragma unroll
      for (int i = 0; i < kPer - 1; ++i) {
        next += units[i];
        if (i + 1 < per && wk.w0 >= next) {
          u = next;
          b = lane * per + i + 1;
        }
      }
      const int src = __ffs((int)has) - 1;
      wk.b = __shfl_sync(0xffffffffu, b, src);
      wk.u = __shfl_sync(0xffffffffu, u, src);
    }
  } else {
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
    // every warp adds the warps' sums up for itself
    total = lane < kThreads / 32 ? misc->warp_sum[lane] : 0;
    int64_t before = lane < warp ? total : 0;
#pragma unroll
    for (int o = 16; o; o >>= 1) {
      total += __shfl_xor_sync(0xffffffffu, total, o);
      before += __shfl_xor_sync(0xffffffffu, before, o);
    }
    before += inc - mine;
    const int64_t w0 = ceil_div(total, (int)gridDim.x) * blockIdx.x;
    if (threadIdx.x == 0 && w0 >= total) misc->first_seq = p.B;
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
    __syncthreads();
    wk.w0 = ceil_div(total, (int)gridDim.x) * blockIdx.x;
    wk.b = misc->first_seq;
    wk.u = wk.b < p.B ? misc->first_unit : 0;
  }
  wk.w1 = min(wk.w0 + ceil_div(total, (int)gridDim.x), total);
  const int th = p.T * p.H, n_tiles = (th + kRows - 1) / kRows;

  if (warp == kLoadWarp) {
    const uint32_t on = elect_one();
    const int nbox = kChunk / p.box;
    const int32_t pool_rows = (int32_t)(p.pool.n_pages * p.pool.page_size);
    uint32_t tiles = 0, fills = 0;  // query tiles asked for and ring places filled so far
    bool ok = true;
    auto place_free = [&]() {
      return warp_wait(bar(kKEmpty + fills % kPlaces), ((fills / kPlaces) & 1) ^ 1, abort, p.wait_limit_ns);
    };
    while (ok && wk.next(p)) {
      for (int qt = 0; ok && qt < n_tiles; ++qt) {
        const int yq = wk.seq * th + qt * kRows;
        // blocks 0-7 of the query tile go through the ring, on their way to TMEM
#pragma unroll 1
        for (int pl = 0; pl < kPerChunk; ++pl) {
          if (!(ok = place_free())) break;
          if (on) {
            const uint32_t place = fills % kPlaces, full = bar(kKFull + place);
            const int kb0 = kPlaceBlocks * pl, kb1 = min(kb0 + kPlaceBlocks, kKB - 1);
            mbar_arrive_expect_tx(full, (kb1 - kb0) * kBlockBytes);
            for (int kb = kb0; kb < kb1; ++kb)
              tma_load_2d(sbase + kRingOff + place * kPlaceBytes + (kb - kb0) * kBlockBytes, &tm_q, kb * 64, yq, full);
          }
          __syncwarp();
          ++fills;
        }
        // block 8, once the products with the tile before are complete
        if (!ok || (tiles > 0 && !(ok = warp_wait(bar(kQFree), (tiles - 1) & 1, abort, p.wait_limit_ns)))) break;
        if (on) {
          mbar_arrive_expect_tx(bar(kQFull), kBlockBytes);
          tma_load_2d(sbase + kQ8Off, &tm_q, (kKB - 1) * 64, yq, bar(kQFull));
        }
        __syncwarp();
        ++tiles;
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
          for (int pl = 0; pl < kPerChunk; ++pl) {
            if (!(ok = place_free())) break;
            if (on) {
              const uint32_t place = fills % kPlaces, full = bar(kKFull + place), dst = sbase + kRingOff + place * kPlaceBytes;
              const int x0 = kPlaceBlocks * pl * 64;
              mbar_arrive_expect_tx(full, kPlaceBytes);
              if (p.box == 64) load_boxes<64, 2, kPlaceBlocks, kBlockBytes>(dst, &tm_k, x0, misc->y, full);
              else if (p.box == 32) load_boxes<32, 4, kPlaceBlocks, kBlockBytes>(dst, &tm_k, x0, misc->y, full);
              else load_boxes<16, 8, kPlaceBlocks, kBlockBytes>(dst, &tm_k, x0, misc->y, full);
            }
            __syncwarp();
            ++fills;
          }
        }
      }
    }
    if (*abort) {
      // the loads in flight must land before the CTA exits (10 ms at most each)
      volatile int never = 0;
      for (uint32_t k = fills > (uint32_t)kPlaces ? fills - kPlaces : 0; k < fills; ++k)
        mbar_wait(bar(kKFull + k % kPlaces), (k / kPlaces) & 1, &never, 10000000ull);
      if (tiles > 0) mbar_wait(bar(kQFull), (tiles - 1) & 1, &never, 10000000ull);
    }
  } else if (warp == kMmaWarp) {
    const uint32_t on = elect_one();
    const uint64_t k0 = smem_desc(sbase + kRingOff, 16, 1024, kSwizzle128B);
    const uint64_t q8 = smem_desc(sbase + kQ8Off, 16, 1024, kSwizzle128B);
    auto wait = [&](int which, uint32_t parity) {
      const bool there = warp_wait(bar(which), parity, abort, p.wait_limit_ns);
      tc_fence_after();
      return there;
    };
    uint32_t tiles = 0, g = 0, fills = 0;
    bool ok = true;
    while (ok && wk.next(p)) {
      for (int qt = 0; ok && qt < n_tiles; ++qt, ++tiles) {
        // the query tile into TMEM, once no product reads the one before
        if (tiles > 0 && !(ok = wait(kQFree, (tiles - 1) & 1))) break;
#pragma unroll 1
        for (int pl = 0; pl < kPerChunk; ++pl, ++fills) {
          const uint32_t place = fills % kPlaces;
          if (!(ok = wait(kKFull + place, (fills / kPlaces) & 1))) break;
          if (on) {
            const uint64_t src = k0 + (uint64_t)((place * kPlaceBytes) >> 4);
            for (int kb = kPlaceBlocks * pl; kb < min(kPlaceBlocks * (pl + 1), kKB - 1); ++kb)
#pragma unroll
              for (int ks = 0; ks < 4; ++ks)
                tmem_cp_128x32b(tmem + kb * 32 + ks * 8,
                                src + (uint64_t)(((kb - kPlaceBlocks * pl) * kBlockBytes) >> 4) + (uint64_t)ks * 2);
            tc_commit(bar(kKEmpty + place));
          }
          __syncwarp();
        }
        if (!ok || !(ok = wait(kQFull, tiles & 1))) break;
        for (int i = wk.lo; ok && i < wk.hi; ++i, ++g) {
          const int sb = g & 1;
          if (g >= 2 && !(ok = wait(kSEmpty + sb, ((g - 2) >> 1) & 1))) break;
          const uint32_t d = tmem + kTmemS + kChunk * sb;
#pragma unroll 1
          for (int pl = 0; pl < kPerChunk - 1; ++pl, ++fills) {
            const uint32_t place = fills % kPlaces;
            if (!(ok = wait(kKFull + place, (fills / kPlaces) & 1))) break;
            const uint64_t bs = k0 + (uint64_t)((place * kPlaceBytes) >> 4);
#pragma unroll
            for (int u = 0; u < 4 * kPlaceBlocks; ++u) {
              const int kb = kPlaceBlocks * pl + u / 4, ks = u % 4;
              mma_f16_ts_if(on, d, tmem + kb * 32 + ks * 8, bs + (uint64_t)(((u / 4) * kBlockBytes) >> 4) + (uint64_t)ks * 2,
                            kIdesc, (kb | ks) ? 1u : 0u);
            }
            if (on) tc_commit(bar(kKEmpty + place));
          }
          const uint32_t place = fills % kPlaces;
          if (!ok || !(ok = wait(kKFull + place, (fills / kPlaces) & 1))) break;
          ++fills;
          const uint64_t bs = k0 + (uint64_t)((place * kPlaceBytes) >> 4);
#pragma unroll
          for (int u = 0; u < 4 * kPlaceBlocks; ++u) {
            const int kb = kKB - kPlaceBlocks + u / 4, ks = u % 4;
            const uint64_t bd = bs + (uint64_t)(((u / 4) * kBlockBytes) >> 4) + (uint64_t)ks * 2;
            if (kb < kKB - 1) mma_f16_ts_if(on, d, tmem + kb * 32 + ks * 8, bd, kIdesc, 1u);
            else mma_f16_ss_if(on, d, q8 + (uint64_t)ks * 2, bd, kIdesc, 1u);
          }
          if (on) {
            tc_commit(bar(kKEmpty + place));
            tc_commit(bar(kSFull + sb));
          }
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
    // ---- epilogue: thread = (query row r, slots 64 * half .. of every chunk)
    const int r = (warp & 3) * 32 + lane, half = warp >> 2;
    const uint32_t s_addr = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16) + kTmemS + 64 * half;
    uint32_t g = 0;
    bool ok = true;
    while (ok && wk.next(p)) {
      for (int qt = 0; ok && qt < n_tiles; ++qt) {
        const int m = min(kRows, th - qt * kRows);  // rows of this tile
        const bool dead = (warp & 3) * 32 >= m;     // a warp without rows only keeps step
        float lse2 = 0.f;
        bool live = r < m;
        if (live) {
          const float l = __ldg(p.lse + (int64_t)wk.seq * th + qt * kRows + r);
          live = l != -INFINITY;  // a row that saw nothing adds nothing
          lse2 = l * 1.4426950408889634f;
        }
        // slots that this row's token sees, and the first token
        const int row_len = wk.len - p.T + 1 + (qt * kRows + r) / p.H, min_len = wk.len - p.T + 1;
        for (int i = wk.lo; ok && i < wk.hi; ++i, ++g) {
          const int sb = g & 1;
          // the first 128 threads finish a slot each
          const int64_t s = (int64_t)i * kChunk + threadIdx.x, o = (int64_t)wk.seq * p.ld_slots + s;
          const bool mine = threadIdx.x < kChunk && s < wk.len;
          float old = 0.f;
          bool there = false;
          if (mine) {
            old = qt > 0 ? p.acc_out[o] : p.acc ? p.decay * p.acc[o] : 0.f;
            there = pool_row(p.pool, wk.seq, (int32_t)s) >= 0;
          }
          ok = warp_wait(bar(kSFull + sb), (g >> 1) & 1, abort, p.wait_limit_ns);
          if (ok) {
            tc_fence_after();
            uint32_t sv[64];
            if (!dead) {
              tmem_ld64(s_addr + kChunk * sb, sv);
              tc_wait_ld();
            }
            tc_fence_before();
            warp_arrive(bar(kSEmpty + sb));
            if (!dead) {
              const int64_t s0 = (int64_t)i * kChunk + 64 * half;
              const int see = s0 + 64 <= min_len ? 64 : (int)min(max(row_len - s0, (int64_t)0), (int64_t)64);
              float v[64];
#pragma unroll
              for (int c = 0; c < 64; ++c) {
                const float x = ex2_approx(fmaf(__uint_as_float(sv[c]), p.scale_log2, -lse2));
                v[c] = live && c < see ? x : 0.f;
              }
              // sums over the warp's rows: lane l ends with columns l and l + 32
#pragma unroll
              for (int grp = 0; grp < 64; grp += 32) {
#pragma unroll
                for (int d = 16; d; d >>= 1) {
                  const bool up = (lane & d) != 0;
#pragma unroll
                  for (int c = 0; c < d; ++c) {
                    const float keep = up ? v[grp + c + d] : v[grp + c], give = up ? v[grp + c] : v[grp + c + d];
                    v[grp + c] = keep + __shfl_xor_sync(0xffffffffu, give, d);
                  }
                }
              }
              misc->part[sb][warp & 3][64 * half + lane] = v[0];
              misc->part[sb][warp & 3][64 * half + 32 + lane] = v[32];
            }
          }
          // every warp's sums are written; all leave together
          if (named_barrier_or(1, 32 * kEpiWarps, !ok)) {
            ok = false;
            break;
          }
          if (mine) {
            float sum = 0.f;
#pragma unroll
            for (int w = 0; w < 4; ++w)
              if (32 * w < m) sum += misc->part[sb][w][threadIdx.x];
            p.acc_out[o] = there ? old + sum : old;
          }
        }
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == kMmaWarp) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
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
  if (!is_aligned16(acc) || !is_aligned16(q) || !is_aligned4(lens, lse, dev_status)) return DSA_ERR_INVALID_ARG;
  if (!(scale == scale) || !(decay == decay)) return DSA_ERR_INVALID_ARG;
  PagedWeightsParams p;
  p.pool = PagePool{page_table, ld_table, n_pages, max_pages, page_size};
  p.lens = lens;
  p.lse = lse;
  p.B = B;
  p.T = T;
  p.H = H;
  p.box = page_size % 64 == 0 ? 64 : page_size % 32 == 0 ? 32 : 16;
  p.scale_log2 = scale * 1.4426950408889634f;
  p.decay = decay;
  p.acc = acc;
  p.acc_out = acc_out;
  p.ld_slots = ld_slots;
  p.status = dev_status;
  MlaParams debug;
  take_attention_debug(debug);
  p.debug_stall = debug.debug_stall;
  p.wait_limit_ns = debug.wait_limit_ns;
  CUtensorMap tq, tk;
  if (!make_tmap_2d(&tq, q, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, kDQK, (uint64_t)B * T * H, kDQK * 2, 64, kRows,
                    CU_TENSOR_MAP_SWIZZLE_128B) ||
      !make_tmap_2d(&tk, kv_pages, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, kDQK, (uint64_t)n_pages * page_size, kDQK * 2, 64,
                    (uint32_t)p.box, CU_TENSOR_MAP_SWIZZLE_128B))
    return DSA_ERR_CUDA;
  static PerDeviceOnce attr;
  if (attr.run([] {
        return cudaFuncSetAttribute(paged_weights_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemBytes);
      }) != cudaSuccess)
    return DSA_ERR_CUDA;
  const cudaError_t e = launch_pdl(paged_weights_kernel, dim3((unsigned)device_info().sm_count), dim3(kThreads),
                                   (size_t)kSmemBytes, reinterpret_cast<cudaStream_t>(stream), tq, tk, p);
  return e == cudaSuccess ? DSA_OK : DSA_ERR_CUDA;
}
