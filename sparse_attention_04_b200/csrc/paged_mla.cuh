// paged_mla.cuh -- what the two kernels for attention over a paged cache
// share: the launch's parameters, the division of the work, and the partials
// that the joining kernel reads.
//
// A tile is as many tokens of a sequence as fit 128 (token, head) rows; its
// slots are read in chunks.  The tiles' units (their chunks, and a few for
// what a tile costs besides) form one list; every worker (a CTA, or a pair)
// takes an equal, contiguous part of it, whatever the sequences' lengths (they
// are read on the device).  A tile that lies in one worker's part is finished
// there; a tile cut by part boundaries leaves one partial per worker.  A worker
// has at most two partials: the tile that begins before its part, and the tile
// that goes on behind it.
#pragma once

#include <cuda.h>

#include <algorithm>

#include "paged.cuh"

namespace dsa {

// A tile that part boundaries cut, as the joining kernel sees it.
struct alignas(16) CutRow {
  int q0;     // first row of out; -1: none
  int first;  // worker of its first partial
  int count;  // partials, one per worker from `first` on
  int m;      // rows
};

struct PagedMlaParams {
  PagePool pool;
  const int32_t* lens;
  int T, H, n_workers;
  int tp;            // tokens per tile
  int tiles;         // tiles per sequence
  int n_rows;        // B * tiles
  int box;           // rows per TMA box
  float scale_log2;
  void* out;
  int out_bf16;
  float* lse;
  CutRow* cut;       // [n_workers]
  float* part_ml;    // [2 * n_workers][2][tp * H]: maximum, sum
  // unnormalised, in 16-byte pieces: [2 * n_workers][128][tp * H][4] fp32 or,
  // from the CTA pair with bf16 output, [2 * n_workers][64][tp * H][8] fp16
  uint4* part_o;
  float* part_sc;    // [2 * n_workers][16][tp * H]: what 32 columns of fp16 are to be multiplied by
  int part_f32;
  int32_t* status;
  int debug_stall;
  uint64_t wait_limit_ns;
};

// Slots that the last token of a tile sees.
__device__ __forceinline__ int32_t tile_len(const PagedMlaParams& p, int seq, int tile, bool& bad) {
  const int32_t len = checked_len(__ldg(p.lens + seq), pool_capacity(p.pool), bad);
  return max(0, len - p.T + min(p.T, (tile + 1) * p.tp));
}
__device__ __forceinline__ int32_t row_len(const PagedMlaParams& p, int r) {
  bool bad;
  const int b = p.tiles == 1 ? r : r / p.tiles;
  return tile_len(p, b, r - b * p.tiles, bad);
}

// One after the other, the parts of tiles that fall to this worker.  Every
// role walks the same list.  CHUNK: slots per chunk; UNITS: what a tile costs
// besides its chunks, in chunks.
template <int CHUNK, int UNITS>
struct MlaWalk {
  int64_t u;       // first unit of tile r
  int64_t w0, w1;  // this worker's units
  int64_t share;   // units per worker
  int r, n_rows;
  int r_seq, r_tile;  // of tile r
  // of the current part:
  int seq, lo, hi, chunks;
  int q0, nt, m;  // first row of q and out, tokens, rows (token, head)
  int32_t len;    // slots the tile's last token sees
  bool bad;

  static __device__ __forceinline__ int64_t chunks_of(int32_t len) { return ((int64_t)len + CHUNK - 1) / CHUNK; }

  __device__ __forceinline__ bool next(const PagedMlaParams& p) {
    while (r < n_rows && u < w1) {
      seq = r_seq;
      len = tile_len(p, seq, r_tile, bad);
      const int64_t c = chunks_of(len), u0 = u + UNITS;
      const int t0 = r_tile * p.tp;
      q0 = (seq * p.T + t0) * p.H;
      nt = min(p.tp, p.T - t0);
      m = nt * p.H;
      chunks = (int)c;
      const bool starts_here = u >= w0;
      lo = (int)min(max(w0 - u0, (int64_t)0), c);
      hi = (int)min(max(w1 - u0, (int64_t)0), c);
      ++r;
      if (++r_tile == p.tiles) {
        r_tile = 0;
        ++r_seq;
      }
      u = u0 + c;
      if (lo < hi || (c == 0 && starts_here)) return true;
    }
    return false;
  }

  // The tile that this worker's first boundary cuts, if its first partial ends
  // there: that boundary describes the tile to the joining kernel.
  __device__ __forceinline__ CutRow cut_row(const PagedMlaParams& p, int worker) const {
    CutRow c{-1, 0, 0, 0};
    MlaWalk first = *this;
    const int64_t u0 = u + UNITS;
    if (first.next(p) && w0 > u0 && w0 - share <= u0) {
      c.q0 = first.q0;
      c.first = worker - 1;
      const int64_t last = u0 + first.chunks - 1 - share * c.first;
      c.count = (int)ceil_div(last + 1, (int)min(share, (int64_t)INT32_MAX));
      c.m = first.m;
    }
    return c;
  }
};

// The units of all tiles, and the tile a worker's part begins in.  By all
// THREADS threads of a CTA; sh needs no values before.
template <int THREADS>
struct MlaScan {
  int64_t first_unit, total_units, warp_sum[THREADS / 32];
  int first_row, pad;
};
// Many tiles: the CTA's threads share them and meet on the way.
template <int CHUNK, int UNITS, int THREADS>
__device__ __noinline__ void scan_many(const PagedMlaParams& p, int worker, MlaScan<THREADS>* sh) {
  using Walk = MlaWalk<CHUNK, UNITS>;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int per = (p.n_rows + THREADS - 1) / THREADS;
  const int r0 = min((int)threadIdx.x * per, p.n_rows), r1 = min(r0 + per, p.n_rows);
  int64_t mine = 0;
  for (int r = r0; r < r1; ++r) mine += UNITS + Walk::chunks_of(row_len(p, r));
  int64_t inc = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t v = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += v;
  }
  if (lane == 31) sh->warp_sum[warp] = inc;
  __syncthreads();
  // every warp adds the warps' sums up for itself
  int64_t total = lane < THREADS / 32 ? sh->warp_sum[lane] : 0, before = lane < warp ? total : 0;
#pragma unroll
  for (int o = 16; o; o >>= 1) {
    total += __shfl_xor_sync(0xffffffffu, total, o);
    before += __shfl_xor_sync(0xffffffffu, before, o);
  }
  before += inc - mine;
  const int64_t w0 = ceil_div(total, p.n_workers) * worker;
  if (threadIdx.x == 0) {
    sh->total_units = total;
    if (w0 >= total) sh->first_row = p.n_rows;
  }
  if (before <= w0 && w0 < before + mine) {  // one thread, if any
    int64_t u = before;
    for (int r = r0; r < r1; ++r) {
      const int64_t c = Walk::chunks_of(row_len(p, r));
      if (w0 < u + UNITS + c) {
        sh->first_row = r;
        sh->first_unit = u;
        break;
      }
      u += UNITS + c;
    }
  }
  __syncthreads();
}
template <int CHUNK, int UNITS, int THREADS>
__device__ __forceinline__ MlaWalk<CHUNK, UNITS> first_part(const PagedMlaParams& p, int worker, MlaScan<THREADS>* sh) {
  using Walk = MlaWalk<CHUNK, UNITS>;
  constexpr int kPer = 4;
  Walk wk;
  int64_t total;
  if (p.n_rows <= 32 * kPer) {
    // every warp for itself, a lane takes up to four tiles (one 2K row of 16
    // heads: 12.7 us, with the CTA's threads 13.2)
    const int lane = threadIdx.x & 31, per = (p.n_rows + 31) >> 5;
    int64_t units[kPer], mine = 0;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int r = lane * per + i;
      units[i] = i < per && r < p.n_rows ? UNITS + Walk::chunks_of(row_len(p, r)) : 0;
      mine += units[i];
    }
    int64_t inc = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t v = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += v;
    }
    total = __shfl_sync(0xffffffffu, inc, 31);
    wk.share = ceil_div(total, p.n_workers);
    wk.w0 = wk.share * worker;
    wk.r = p.n_rows;
    wk.u = 0;
    const int64_t before = inc - mine;
    const uint32_t has = __ballot_sync(0xffffffffu, before <= wk.w0 && wk.w0 < inc);
    if (has) {
      int r = lane * per;
      int64_t u = before, next = before;
#pragma unroll
      for (int i = 0; i < kPer - 1; ++i) {
        next += units[i];
        if (i + 1 < per && wk.w0 >= next) {
          u = next;
          r = lane * per + i + 1;
        }
      }
      const int src = __ffs((int)has) - 1;
      wk.r = __shfl_sync(0xffffffffu, r, src);
      wk.u = __shfl_sync(0xffffffffu, u, src);
    }
  } else {
    scan_many<CHUNK, UNITS, THREADS>(p, worker, sh);
    total = sh->total_units;
    wk.share = ceil_div(total, p.n_workers);
    wk.w0 = wk.share * worker;
    wk.r = sh->first_row;
    wk.u = wk.r < p.n_rows ? sh->first_unit : 0;
  }
  wk.w1 = min(wk.w0 + wk.share, total);
  wk.n_rows = p.n_rows;
  wk.r_seq = p.tiles == 1 ? wk.r : wk.r / p.tiles;
  wk.r_tile = wk.r - wk.r_seq * p.tiles;
  return wk;
}

// The kernel for tiles of up to kFewRows rows, one CTA per worker.
constexpr int kFewRows = 32;
int paged_few_workers();  // workers of a launch: a CTA per SM
cudaError_t launch_paged_mla_few(const PagedMlaParams& p, const void* q, uint64_t q_rows, const void* kv_pages,
                                 uint64_t pool_rows, cudaStream_t s);

}  // namespace dsa
