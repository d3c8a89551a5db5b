// paged_mla_few.cu -- absorbed MLA over a paged cache for tiles of up to 32
// (token, head) rows: few heads, few tokens.
//
// The mathematics is paged_mla.cu's.  With R rows a slot costs 2 * R * 1088
// flops and 1152 bytes: the memory bounds it, so every slot is to enter one
// SM's shared memory once and every SM is to read.  That asks for the products
// the other way round:
//   S^T [64 slots, R] = K . Q^T           K as it lies in shared memory,
//   O^T [512, R]     += V^T . P           V the same bytes, read column-major,
// so that O takes 4 R columns of tensor memory and both products fit one CTA.
// (The products have M = 128; S^T's upper 64 lanes are computed from whatever
// lies behind the chunk and never looked at.)
//
// A chunk is 64 slots: four pieces of 128 columns in a ring of 10 or 11, and
// the rope block, which is free as soon as the scores are computed.  Four warps
// issue: the cache's loads, the query's, S^T, and O^T, each waiting for itself,
// so that a chunk whose P is ready frees its pieces however late the next chunk
// lands.  Eight warps consume: four of them (32 slots each, half of the rows)
// compute P, all eight rescale and write out, 32 of the 128 columns of two
// blocks each.  A row's maximum over 32 slots is one warp reduction; O is
// rescaled only when it rose by more than 2^8.  A row's sum stays per lane
// until the part ends.
//
// What bounds it (B200).  24 sequences of up to 30K slots (423 MB), two tokens
// of 16 heads: 94 us, 65 of them the bytes at the measured copy rate (the CTA
// pair of paged_mla.cu: 117; a ring of eight pieces: 98); 32 sequences of 8K to
// 128K slots, 16 heads: 465 of 451.  A chunk takes about 3400 cycles, 1350 of
// them in the consumers; without loads the first case takes 76.  The rest is
// latency at both ends: one row of 2K takes 12.5 us, one of 32K 17.2 (16 heads,
// ten calls in a graph).
#include "paged_mla.cuh"
#include "tmap.h"

namespace dsa {
namespace {

constexpr int kChunk = 64;
constexpr int kKB = kDQK / 64;  // 64-column blocks of a row: 9
constexpr int kBlockBytes = kChunk * 128;
constexpr int kPieces = 4;      // of a chunk without its rope block: blocks 0-1, 2-3, 4-5, 6-7
constexpr int kPieceBytes = 2 * kBlockBytes;
constexpr int kMaxRing = 11;    // pieces
constexpr int kMaxWorkers = 256;

constexpr int kThreads = 384;
constexpr int kConsumers = 256;
constexpr int kLoadWarp = 8, kScoreWarp = 9, kOutWarp = 10, kQueryWarp = 11;

enum Bar : int {
  kQFull = 0,
  kQFree,                             // a part's score products are complete
  kFull,                              // [ring]
  kEmpty = kFull + kMaxRing,          // [ring]
  kRopeFull = kEmpty + kMaxRing,
  kRopeEmpty,
  kSFull,                             // [2]
  kSEmpty = kSFull + 2,               // [2]
  kMaskFull = kSEmpty + 2,            // [4]: the chunk's validity words are written
  kPReady = kMaskFull + 4,            // [2]: P is written, O rescaled, the tile's tail zero
  kPvDone = kPReady + 2,              // [2]: the product with P is complete
  kDrain = kPvDone + 2,               // [2]
  kNumBar = kDrain + 2
};

struct Misc {
  int tmem_base, abort;
  MlaScan<kThreads> scan;
};

template <int R>
struct Layout {
  static constexpr int kQBlockBytes = R * 128;
  // What a tile costs besides its chunks, in chunks (128 sequences of 500 to
  // 4000 slots: 16 heads 72.5 us, one less 73.7, one more 73.3; 32 heads 78.5,
  // 80.1, 80.0).
  static constexpr int kUnits = R / 16 + 1;
  static constexpr int kRing = R == 16 ? 11 : 10;         // what shared memory holds
  static constexpr int kRopeOff = kRing * kPieceBytes;
  static constexpr int kPOff = kRopeOff + kBlockBytes;    // [2] P [64 slots][64 rows], 128-byte rows, swizzled
  static constexpr int kPBytes = kChunk * 128;
  static constexpr int kQOff = kPOff + 2 * kPBytes;
  static constexpr int kMaxOff = kQOff + kKB * kQBlockBytes;  // [2][2][R]: maxima, at the end sums
  static constexpr int kAlphaOff = kMaxOff + 2 * 2 * R * 4;   // [R]: rescale factors, at the end maxima
  static constexpr int kSeenOff = kAlphaOff + R * 4;          // [R]: slots that a row sees
  static constexpr int kMaskOff = kSeenOff + R * 4;           // [4][2] validity words
  static constexpr int kBoxOff = kMaskOff + 4 * 8;            // [4] row coordinates
  static constexpr int kBarOff = kBoxOff + 4 * 4;
  static constexpr int kMiscOff = kBarOff + kNumBar * 8;
  static constexpr int kSmemBytes = kMiscOff + (int)sizeof(Misc) + 1024;
  // The 128 product rows of the last block end inside shared memory: P and Q
  // lie behind it.  The epilogue stages 2 KB per warp where P was.
  // Fewer places than three chunks have pieces: the scores of chunk g + 2 are
  // computed only after the product of chunk g has freed a piece, that is after
  // all eight consumer warps saw chunk g's scores.  Four of them alone give a
  // score buffer back; the others would miss a phase of its barrier otherwise.
  static_assert(kRing < 3 * kPieces, "a score buffer filled twice behind a waiting warp");
  static_assert(kRing <= kMaxRing && kRing >= 2 * kPieces && kSmemBytes <= 232448 && 2 * kPBytes >= 8 * 2048, "shared memory budget");
  static_assert(kQOff % 1024 == 0 && kMaxOff % 16 == 0 && kAlphaOff % 16 == 0 && kBarOff % 8 == 0 && kMiscOff % 8 == 0,
                "alignment");
  // tensor memory: O^T in four blocks of R columns, then two S^T buffers
  static constexpr uint32_t kTmemS = 4 * R;
  static constexpr uint32_t kIdescS = idesc_bf16(128, R);
  static constexpr uint32_t kIdescO = idesc_bf16(128, R, /*b_mn_major=*/true, /*a_mn_major=*/true);
  static_assert(6 * R <= 512, "tensor memory");
};

template <int R>
__global__ void __launch_bounds__(kThreads, 1)
    paged_mla_few_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                         const __grid_constant__ PagedMlaParams p) {
  using L = Layout<R>;
  constexpr int C = R / 2;  // rows per consumer warp
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sbase = smem_u32(smem);
  auto bar = [&](int i) { return sbase + L::kBarOff + 8u * (uint32_t)i; };
  Misc* misc = reinterpret_cast<Misc*>(smem + L::kMiscOff);
  volatile int* abort = &misc->abort;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  auto wait = [&](int which, uint32_t parity) { return warp_wait(bar(which), parity, abort, p.wait_limit_ns); };

  // ---- prologue: barriers, TMEM
  if (threadIdx.x == 0) misc->abort = 0;
  if (warp == kScoreWarp) {
    if (lane == 0) {
      tma_prefetch_desc(&tm_k);
      tma_prefetch_desc(&tm_q);
      mbar_init(bar(kQFull), 1 + (p.debug_stall & 1));
      mbar_init(bar(kQFree), 1);
      for (int i = 0; i < L::kRing; ++i) {
        mbar_init(bar(kFull + i), 1);
        mbar_init(bar(kEmpty + i), 1);
      }
      mbar_init(bar(kRopeFull), 1);
      mbar_init(bar(kRopeEmpty), 1);
      for (int i = 0; i < 2; ++i) {
        mbar_init(bar(kSFull + i), 1);
        mbar_init(bar(kSEmpty + i), 4);
        mbar_init(bar(kPReady + i), kConsumers / 32 + (i == 0 ? p.debug_stall >> 1 : 0));
        mbar_init(bar(kPvDone + i), 1);
        mbar_init(bar(kDrain + i), 1);
      }
      for (int i = 0; i < 4; ++i) mbar_init(bar(kMaskFull + i), 1);
      fence_mbar_init();
    }
    __syncwarp();
    tmem_alloc(sbase + L::kMiscOff + (uint32_t)offsetof(Misc, tmem_base), 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  grid_dependency_wait();  // lens, q and the cache may come from the previous kernel
  allow_dependents_launch();
  auto wk = first_part<kChunk, L::kUnits, kThreads>(p, blockIdx.x, &misc->scan);
  const uint32_t tmem = static_cast<uint32_t>(misc->tmem_base);
  if (threadIdx.x == kQueryWarp * 32) p.cut[blockIdx.x] = wk.cut_row(p, blockIdx.x);
  const int64_t pool_rows = p.pool.n_pages * p.pool.page_size;

  if (warp == kLoadWarp) {
    // ---- the chunks: lane i < nbox locates box i
    const uint32_t on = elect_one();
    const int nbox = kChunk / p.box;
    int32_t* const yk = reinterpret_cast<int32_t*>(smem + L::kBoxOff);
    uint32_t g = 0, fills = 0, ropes = 0;  // chunks, pieces and rope blocks so far
    bool ok = true;
    while (ok && wk.next(p)) {
      if (wk.bad && lane == 0) report(p.status, DSA_ERR_BAD_OFFSETS);
      // row coordinate and valid slots of this lane's box of chunk i
      auto locate = [&](int i, int32_t& y, int& valid) {
        const int64_t s = (int64_t)i * kChunk + lane * p.box;
        valid = 0;
        y = (int32_t)pool_rows;
        if (lane < nbox && s < wk.len) {
          const int64_t row = pool_row(p.pool, wk.seq, (int32_t)s);
          if (row >= 0) {
            y = (int32_t)row;
            valid = min(p.box, wk.len - (int32_t)s);
          } else {
            report(p.status, DSA_ERR_BAD_INDEX);
          }
        }
      };
      int32_t y = 0, y_next = 0;
      int valid = 0, valid_next = 0;
      if (wk.lo < wk.hi) locate(wk.lo, y, valid);
      for (int i = wk.lo; ok && i < wk.hi; ++i, ++g) {
        if (lane < 4) yk[lane] = y;
        __syncwarp();
#pragma unroll 1
        for (int pc = 0; pc < kPieces; ++pc) {
          const uint32_t at = fills % L::kRing;
          if (!(ok = wait(kEmpty + at, ((fills / L::kRing) & 1) ^ 1))) break;
          if (on) {
            const uint32_t full = bar(kFull + at), dst = sbase + at * kPieceBytes;
            mbar_arrive_expect_tx(full, kPieceBytes);
            if (p.box == 64) load_boxes<64, 1, 2, kBlockBytes>(dst, &tm_k, 128 * pc, yk, full);
            else if (p.box == 32) load_boxes<32, 2, 2, kBlockBytes>(dst, &tm_k, 128 * pc, yk, full);
            else load_boxes<16, 4, 2, kBlockBytes>(dst, &tm_k, 128 * pc, yk, full);
          }
          __syncwarp();
          ++fills;
        }
        if (!ok || !(ok = wait(kRopeEmpty, (ropes & 1) ^ 1))) break;
        if (on) {
          const uint32_t full = bar(kRopeFull), dst = sbase + L::kRopeOff;
          mbar_arrive_expect_tx(full, kBlockBytes);
          if (p.box == 64) load_boxes<64, 1, 1, kBlockBytes>(dst, &tm_k, kDV, yk, full);
          else if (p.box == 32) load_boxes<32, 2, 1, kBlockBytes>(dst, &tm_k, kDV, yk, full);
          else load_boxes<16, 4, 1, kBlockBytes>(dst, &tm_k, kDV, yk, full);
        }
        __syncwarp();
        ++ropes;
        if (i + 1 < wk.hi) locate(i + 1, y_next, valid_next);
        // validity words of the chunk, 16 slots (never more than a box) at a time
        uint32_t word = ~0u;
        if (!__all_sync(0xffffffffu, lane >= nbox || valid == p.box)) {
          word = 0;
#pragma unroll 1
          for (int hh = 0; hh < 2; ++hh) {
            const int k0 = 32 * (lane & 1) + 16 * hh, bx = k0 / p.box;
            const int v = __shfl_sync(0xffffffffu, valid, bx) - (k0 - bx * p.box);
            word |= (v >= 16 ? 0xffffu : v <= 0 ? 0u : (1u << v) - 1u) << (16 * hh);
          }
        }
        if (lane < 2) reinterpret_cast<uint32_t*>(smem + L::kMaskOff)[2 * (g & 3) + lane] = word;
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(kMaskFull + (g & 3)));
        y = y_next;
        valid = valid_next;
      }
    }
    if (*abort) {
      // the loads in flight must land before the CTA exits (10 ms at most each)
      volatile int never = 0;
      for (uint32_t f = fills > (uint32_t)L::kRing ? fills - L::kRing : 0; f < fills; ++f)
        mbar_wait(bar(kFull + f % L::kRing), (f / L::kRing) & 1, &never, 10000000ull);
      if (ropes > 0) mbar_wait(bar(kRopeFull), (ropes - 1) & 1, &never, 10000000ull);
    }
  } else if (warp == kQueryWarp) {
    // ---- the query, once no product reads the one before.  That takes as long
    // as the part before does, so the limit is one per chunk of it.  (A chunk
    // that does not come ends the other warps' waits, and with them this one.)
    const uint32_t on = elect_one();
    uint32_t item = 0;
    uint64_t limit = 0;
    while (wk.next(p)) {
      if (wk.lo >= wk.hi) continue;
      if (item > 0 && !warp_wait(bar(kQFree), (item - 1) & 1, abort, limit)) break;
      limit = p.wait_limit_ns * (uint64_t)(wk.hi - wk.lo + 1);
      if (on) {
        mbar_arrive_expect_tx(bar(kQFull), kKB * L::kQBlockBytes);
        for (int kb = 0; kb < kKB; ++kb) tma_load_2d(sbase + L::kQOff + kb * L::kQBlockBytes, &tm_q, kb * 64, wk.q0, bar(kQFull));
      }
      __syncwarp();
      ++item;
    }
    if (*abort) {
      volatile int never = 0;
      if (item > 0) mbar_wait(bar(kQFull), (item - 1) & 1, &never, 10000000ull);
    }
  } else if (warp == kScoreWarp) {
    // ---- S^T(g) = K(g) . Q^T into buffer g & 1
    const uint32_t on = elect_one();
    const uint64_t kd = smem_desc(sbase, 16, 1024, kSwizzle128B);
    const uint64_t qd = smem_desc(sbase + L::kQOff, 16, 1024, kSwizzle128B);
    uint32_t g = 0, item = 0;
    bool ok = true;
    while (ok && wk.next(p)) {
      if (wk.lo >= wk.hi) continue;
      if (!(ok = wait(kQFull, item & 1))) break;
      ++item;
      for (int i = wk.lo; ok && i < wk.hi; ++i, ++g) {
        const uint32_t sb = g & 1;
        if (g >= 2 && !(ok = wait(kSEmpty + sb, ((g - 2) >> 1) & 1))) break;
        const uint32_t d = tmem + L::kTmemS + R * sb;
#pragma unroll 1
        for (int pc = 0; pc < kPieces; ++pc) {
          const uint32_t f = kPieces * g + pc, at = f % L::kRing;
          if (!(ok = wait(kFull + at, (f / L::kRing) & 1))) break;
          tc_fence_after();
          const uint64_t a = kd + (uint64_t)((at * kPieceBytes) >> 4);
          const uint64_t b = qd + (uint64_t)((pc * 2 * L::kQBlockBytes) >> 4);
#pragma unroll
          for (int u = 0; u < 8; ++u)
            mma_f16_ss_if(on, d, a + (uint64_t)(((u / 4) * kBlockBytes) >> 4) + (uint64_t)(u % 4) * 2,
                          b + (uint64_t)(((u / 4) * L::kQBlockBytes) >> 4) + (uint64_t)(u % 4) * 2, L::kIdescS,
                          (pc | u) ? 1u : 0u);
        }
        if (!ok || !(ok = wait(kRopeFull, g & 1))) break;
        tc_fence_after();
#pragma unroll
        for (int u = 0; u < 4; ++u)
          mma_f16_ss_if(on, d, kd + (uint64_t)(L::kRopeOff >> 4) + (uint64_t)u * 2,
                        qd + (uint64_t)((8 * L::kQBlockBytes) >> 4) + (uint64_t)u * 2, L::kIdescS, 1u);
        if (on) {
          tc_commit(bar(kRopeEmpty));
          tc_commit(bar(kSFull + sb));
        }
      }
      if (ok && on) tc_commit(bar(kQFree));
    }
    if (*abort) {
      volatile int never = 0;  // tensor-core work ends before TMEM is released
      if (on) {
        tc_commit(bar(kDrain));
        mbar_wait(bar(kDrain), 0, &never, 10000000ull);
      }
    }
  } else if (warp == kOutWarp) {
    // ---- O^T[128 n ..] += V^T(g)[128 n ..] . P(g)
    const uint32_t on = elect_one();
    const uint64_t vd = smem_desc(sbase, kBlockBytes, 1024, kSwizzle128B);
    const uint64_t pd = smem_desc(sbase + L::kPOff, kBlockBytes, 1024, kSwizzle128B);
    uint32_t g = 0;
    bool ok = true;
    while (ok && wk.next(p)) {
      for (int i = wk.lo; ok && i < wk.hi; ++i, ++g) {
        if (!(ok = wait(kPReady + (g & 1), (g >> 1) & 1))) break;
#pragma unroll 1
        for (int n = 0; n < 4; ++n) {
          // landed long ago; the wait makes the bytes this warp's to read
          const uint32_t f = kPieces * g + n, at = f % L::kRing;
          if (!(ok = wait(kFull + at, (f / L::kRing) & 1))) break;
          tc_fence_after();
#pragma unroll
          for (int s = 0; s < kChunk / 16; ++s)
            mma_f16_ss_if(on, tmem + R * n, vd + (uint64_t)((at * kPieceBytes + s * 2048) >> 4),
                          pd + (uint64_t)(((g & 1) * L::kPBytes + s * 2048) >> 4), L::kIdescO, (i > wk.lo || s > 0) ? 1u : 0u);
          if (on) tc_commit(bar(kEmpty + at));
        }
        if (ok && on) tc_commit(bar(kPvDone + (g & 1)));
      }
    }
    if (*abort) {
      volatile int never = 0;
      if (on) {
        tc_commit(bar(kDrain + 1));
        mbar_wait(bar(kDrain + 1), 0, &never, 10000000ull);
      }
    }
  } else {
    // ---- softmax (warps with lanes 0-63: thread = slot, rows cb .. cb + C),
    // rescale and epilogue (all: thread = column 32 q + lane of two blocks)
    const int q = warp & 3, half = warp >> 2, cb = half * C;
    const bool scores = q < 2;
    const int slot = 32 * q + lane;
    const uint32_t quarter = tmem + (static_cast<uint32_t>(32 * q) << 16);
    float* const maxima = reinterpret_cast<float*>(smem + L::kMaxOff);
    float* const alphas = reinterpret_cast<float*>(smem + L::kAlphaOff);
    int32_t* const seen = reinterpret_cast<int32_t*>(smem + L::kSeenOff);
    uint32_t g = 0;
    // A warp whose wait ran out says so at the next barrier, and all eight leave
    // there: one that left by itself would be waited for without end.
    bool ok = true, leave = false;
    while (!leave && wk.next(p)) {
      if (threadIdx.x < R) seen[threadIdx.x] = wk.len - max(0, wk.nt - 1 - (int)threadIdx.x / p.H);
      const int min_len = wk.len - (wk.nt - 1);
      float m_run[C], l_run[C];
#pragma unroll
      for (int c = 0; c < C; ++c) {
        m_run[c] = -INFINITY;
        l_run[c] = 0.f;
      }
      named_barrier_sync(1, kConsumers);
      for (int i = wk.lo; i < wk.hi; ++i, ++g) {
        ok = ok && wait(kMaskFull + (g & 3), (g >> 2) & 1) && wait(kSFull + (g & 1), (g >> 1) & 1);
        const int64_t s0 = (int64_t)i * kChunk;
        uint32_t sv[C];
        bool rise = false;
        float* const mx = maxima + (g & 1) * 2 * R;
        if (ok && scores) {
          tc_fence_after();
          tmem_ld(quarter + L::kTmemS + R * (g & 1) + cb, sv);
          tc_wait_ld();
          tc_fence_before();
          warp_arrive(bar(kSEmpty + (g & 1)));
          // x = s * scale * log2(e); masked slots -inf
#pragma unroll
          for (int c = 0; c < C; c += 2) {
            const float2 x = __fmul2_rn(make_float2(__uint_as_float(sv[c]), __uint_as_float(sv[c + 1])),
                                        make_float2(p.scale_log2, p.scale_log2));
            sv[c] = __float_as_uint(x.x);
            sv[c + 1] = __float_as_uint(x.y);
          }
          const uint32_t valid = reinterpret_cast<const uint32_t*>(smem + L::kMaskOff)[2 * (g & 3) + q];
          if (valid != ~0u || s0 + kChunk > min_len) {  // the tile's tokens may see different slots here
            const bool in = (valid >> lane) & 1u;
#pragma unroll
            for (int c = 0; c < C; ++c)
              if (!in || s0 + slot >= seen[cb + c]) sv[c] = 0xff800000u;
          }
#pragma unroll
          for (int c = 0; c < C; c += 4) {
            float4 t;
            t.x = warp_max(__uint_as_float(sv[c]));
            t.y = warp_max(__uint_as_float(sv[c + 1]));
            t.z = warp_max(__uint_as_float(sv[c + 2]));
            t.w = warp_max(__uint_as_float(sv[c + 3]));
            // always in the row's first chunk that holds a finite score
            rise |= t.x > m_run[c] + 8.f || t.y > m_run[c + 1] + 8.f || t.z > m_run[c + 2] + 8.f || t.w > m_run[c + 3] + 8.f;
            if (lane == 0) *reinterpret_cast<float4*>(mx + R * q + cb + c) = t;
          }
        }
        // the product before the last has read this P buffer
        if (ok && g >= 2) ok = wait(kPvDone + (g & 1), ((g - 2) >> 1) & 1);
        // The maxima are written.  A warp that gives up casts 32 votes, one
        // with a maximum that rose casts one; all eight warps go the same way.
        const uint32_t votes = named_barrier_count(1, kConsumers, !ok || (rise && lane == 0));
        if (votes >= 32) {
          leave = true;
          break;
        }
        if (scores) {
          if (votes) {
#pragma unroll
            for (int c = 0; c < C; ++c) {
              const float top = fmaxf(mx[cb + c], mx[R + cb + c]);
              float alpha = 1.f;
              if (top > m_run[c] + 8.f) {
                alpha = exp2f(m_run[c] - top);  // 0 at first
                m_run[c] = top;
                l_run[c] *= alpha;
              }
              if (slot == 0) alphas[cb + c] = alpha;
            }
          }
          uint8_t* const prow = smem + L::kPOff + (g & 1) * L::kPBytes + slot * 128;
#pragma unroll
          for (int c8 = 0; c8 < C / 8; ++c8) {
            uint32_t w4[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const int c = 8 * c8 + 2 * e;
              const float sa = m_run[c] == -INFINITY ? 0.f : m_run[c], sb = m_run[c + 1] == -INFINITY ? 0.f : m_run[c + 1];
              const float2 pv = make_float2(ex2_approx(__uint_as_float(sv[c]) - sa), ex2_approx(__uint_as_float(sv[c + 1]) - sb));
              l_run[c] += pv.x;
              l_run[c + 1] += pv.y;
              const __nv_bfloat162 pb = __floats2bfloat162_rn(pv.x, pv.y);
              w4[e] = *reinterpret_cast<const uint32_t*>(&pb);
            }
            *reinterpret_cast<uint4*>(prow + (((cb / 8 + c8) ^ (slot & 7)) << 4)) = make_uint4(w4[0], w4[1], w4[2], w4[3]);
          }
        }
        if (votes && i > wk.lo) {
          // the factors are written, and O holds the product before
          ok = wait(kPvDone + ((g - 1) & 1), ((g - 1) >> 1) & 1);
          named_barrier_sync(2, kConsumers);
          tc_fence_after();
#pragma unroll 1
          for (int n = 2 * half; n < 2 * half + 2; ++n)
#pragma unroll 1
            for (int r0 = 0; r0 < R; r0 += 16) {
              uint32_t ov[16];
              tmem_ld(quarter + R * n + r0, ov);
              tc_wait_ld();
#pragma unroll
              for (int c = 0; c < 16; ++c) ov[c] = __float_as_uint(__uint_as_float(ov[c]) * alphas[r0 + c]);
              tmem_st16(quarter + R * n + r0, ov);
            }
          tc_wait_st();
        }
        // Two kinds of slots must not meet the product as they are.  Slots
        // behind the end that share the last box with it may hold anything:
        // they become zeros.  Slots that only some of the tile's tokens see
        // have P = 0 for the others, and 0 * NaN is not 0: a slot that is not
        // finite becomes zeros too (the rows that see it have a NaN for a sum
        // already).  The scores are complete: nobody else reads the chunk.
        if (s0 + kChunk > min_len) {
          const int z_begin = (int)max((int64_t)0, min_len - s0);
          const int z_end = (int)min((int64_t)kChunk, (((int64_t)wk.len + p.box - 1) & -(int64_t)p.box) - s0);
          // landed long ago; the waits make the bytes this thread's to read and write
          for (uint32_t f = kPieces * g; f < kPieces * (g + 1); ++f) wait(kFull + f % L::kRing, (f / L::kRing) & 1);
          // this lane's 16 bytes of a slot lie in blocks lane / 8 and 4 + lane / 8
          const uint32_t f = kPieces * g + (lane >> 4), in = ((lane >> 3) & 1) * kBlockBytes + (lane & 7) * 16;
          uint8_t* const a0 = smem + f % L::kRing * kPieceBytes + in;
          uint8_t* const b0 = smem + (f + 2) % L::kRing * kPieceBytes + in;
          // a warp takes a slot: 2 x 4 blocks x 8 pieces of 16 bytes
          for (int z = z_begin + warp; z < z_end; z += 8) {
            uint4* const a = reinterpret_cast<uint4*>(a0 + z * 128);
            uint4* const b = reinterpret_cast<uint4*>(b0 + z * 128);
            bool clear = s0 + z >= wk.len;
            if (!clear) {
              const uint4 va = *a, vb = *b;
              const uint32_t w[8] = {va.x, va.y, va.z, va.w, vb.x, vb.y, vb.z, vb.w};
              bool odd = false;
#pragma unroll
              for (int e = 0; e < 8; ++e) odd |= (w[e] & 0x7f80u) == 0x7f80u || (w[e] & 0x7f800000u) == 0x7f800000u;
              clear = __any_sync(0xffffffffu, odd);
            }
            if (clear) {
              *a = make_uint4(0u, 0u, 0u, 0u);
              *b = make_uint4(0u, 0u, 0u, 0u);
            }
          }
        }
        fence_proxy_async_smem();
        tc_fence_before();
        warp_arrive(bar(kPReady + (g & 1)));
      }
      if (leave) break;
      const bool any = wk.lo < wk.hi;
      if (any && ok) ok = wait(kPvDone + ((g - 1) & 1), ((g - 1) >> 1) & 1);
      // the lanes' sums; the buffers of the maxima and factors are free: all
      // warps have read them (they arrived at kPReady since)
      float* const sums = maxima + (g & 1) * 2 * R;
      if (scores) {
#pragma unroll
        for (int c = 0; c < C; ++c) {
          float t = l_run[c];
#pragma unroll
          for (int o = 16; o; o >>= 1) t += __shfl_xor_sync(0xffffffffu, t, o);
          if (lane == 0) sums[R * q + cb + c] = t;
          if (slot == 0) alphas[cb + c] = m_run[c];
        }
      }
      if (named_barrier_count(1, kConsumers, !ok) != 0) break;
      tc_fence_after();
      const bool whole = wk.hi - wk.lo == wk.chunks;
      const int64_t part = 2 * (int64_t)blockIdx.x + (wk.lo > 0 ? 0 : 1);
      const int pm = p.tp * p.H;  // rows a partial has room for
      if (threadIdx.x < wk.m) {
        const int r = threadIdx.x;
        const float l = sums[r] + sums[R + r], m = alphas[r];
        if (whole) {
          if (p.lse) p.lse[(int64_t)wk.q0 + r] = l == 0.f ? -INFINITY : (m + log2f(l)) * 0.69314718055994531f;
        } else {
          p.part_ml[2 * part * pm + r] = m;
          p.part_ml[(2 * part + 1) * pm + r] = l;
        }
      }
      // 16 rows x 32 columns at a time through shared memory (P's, which no
      // product reads any more): then thread = (row, eight columns).
      float* const stage = reinterpret_cast<float*>(smem + L::kPOff + warp * 2048);
      const int sub = lane & 3;
#pragma unroll 1
      for (int r0 = 0; r0 < wk.m; r0 += 16) {
#pragma unroll 1
        for (int n = 2 * half; n < 2 * half + 2; ++n) {
          const int col = 128 * n + 32 * q;  // the warp's first column
          uint32_t ov[16];
          if (any) {
            tmem_ld(quarter + R * n + r0, ov);
            tc_wait_ld();
          } else {
#pragma unroll
            for (int c = 0; c < 16; ++c) ov[c] = 0u;
          }
#pragma unroll
          for (int c = 0; c < 16; ++c) stage[32 * c + lane] = __uint_as_float(ov[c]);
          __syncwarp();
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            const int r = r0 + 8 * u + (lane >> 2);
            float4 v[2];
            v[0] = *reinterpret_cast<const float4*>(stage + 32 * (8 * u + (lane >> 2)) + 8 * sub);
            v[1] = *reinterpret_cast<const float4*>(stage + 32 * (8 * u + (lane >> 2)) + 8 * sub + 4);
            float* const w = reinterpret_cast<float*>(v);
            if (whole) {
              const float l = sums[r] + sums[R + r];
              const float mul = l == 0.f ? 0.f : 1.f / l;  // a NaN among the scores stays one
#pragma unroll
              for (int e = 0; e < 8; ++e) w[e] *= mul;
              if (r < wk.m) {
                const int64_t at = ((int64_t)wk.q0 + r) * kDV + col + 8 * sub;
                if (p.out_bf16) {
                  uint4 o;
                  __nv_bfloat162* const t = reinterpret_cast<__nv_bfloat162*>(&o);
#pragma unroll
                  for (int e = 0; e < 4; ++e) t[e] = __floats2bfloat162_rn(w[2 * e], w[2 * e + 1]);
                  *reinterpret_cast<uint4*>(reinterpret_cast<__nv_bfloat16*>(p.out) + at) = o;
                } else {
                  float4* const o = reinterpret_cast<float4*>(reinterpret_cast<float*>(p.out) + at);
                  o[0] = v[0];
                  o[1] = v[1];
                }
              }
            } else if (r < wk.m) {
              uint4* const o = p.part_o + (part * (kDV / 4) + col / 4 + 2 * sub) * pm + r;
              o[0] = *reinterpret_cast<const uint4*>(&v[0]);
              o[pm] = *reinterpret_cast<const uint4*>(&v[1]);
            }
          }
          __syncwarp();
        }
      }
      tc_fence_before();  // O is read: the next part's first product (after kPReady) may overwrite it
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == kScoreWarp) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
  if (threadIdx.x == 0 && *abort) report(p.status, DSA_ERR_TIMEOUT);
}

template <int R>
cudaError_t launch(const PagedMlaParams& p, const void* q, uint64_t q_rows, const CUtensorMap& tk, cudaStream_t s) {
  static PerDeviceOnce once;
  const cudaError_t e = once.run([] {
    return cudaFuncSetAttribute(paged_mla_few_kernel<R>, cudaFuncAttributeMaxDynamicSharedMemorySize, Layout<R>::kSmemBytes);
  });
  if (e != cudaSuccess) return e;
  CUtensorMap tq;
  if (!make_tmap_2d(&tq, q, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, kDQK, q_rows, kDQK * 2, 64, R, CU_TENSOR_MAP_SWIZZLE_128B))
    return cudaErrorInvalidValue;
  return launch_pdl(paged_mla_few_kernel<R>, dim3((unsigned)p.n_workers), dim3(kThreads), (size_t)Layout<R>::kSmemBytes, s, tq,
                    tk, p);
}

}  // namespace

int paged_few_workers() { return std::max(1, std::min(device_info().sm_count, kMaxWorkers)); }

cudaError_t launch_paged_mla_few(const PagedMlaParams& p, const void* q, uint64_t q_rows, const void* kv_pages,
                                 uint64_t pool_rows, cudaStream_t s) {
  CUtensorMap tk;
  if (!make_tmap_2d(&tk, kv_pages, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, kDQK, pool_rows, kDQK * 2, 64, (uint32_t)p.box,
                    CU_TENSOR_MAP_SWIZZLE_128B))
    return cudaErrorInvalidValue;
  const int rows = p.tp * p.H;
  return rows <= 16 ? launch<16>(p, q, q_rows, tk, s) : launch<32>(p, q, q_rows, tk, s);
}

}  // namespace dsa
