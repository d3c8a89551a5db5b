// paged_mla.cu -- absorbed MLA of the newest tokens over a whole paged cache.
//
// For query row (b, t) and head h, over the slots s <= lens[b] - T + t:
//   l_s = scale * q . kv_s[:576];  out = softmax(l) . kv[:, :512];  lse = log sum exp(l)
//
// With 128 heads a slot costs 2 * 128 * (576 + 512) flops and 1152 bytes: 242
// flops per byte, the ratio of this card's measured rates, so the kernel has
// to keep the tensor cores and the memory busy at the same time.  With fewer
// heads the memory bounds it; tiles of up to 32 (token, head) rows go to
// paged_mla_few.cu.
//
// Split.  Every cluster of two CTAs is a worker with an equal part of all
// tiles' 128-slot chunks (paged_mla.cuh); paged_mla_combine_kernel joins the
// tiles that part boundaries cut.
//
// Two CTAs.  A 128-head tile's output fills an SM's tensor memory (128 lanes x
// 512 fp32 columns), so the pair divides the work by role:
//   CTA 0 (QK side): query blocks 0-7 (64 columns each) in TMEM, block 8 in
//     shared memory; a chunk's rows arrive by TMA as nine 128 x 64 blocks in a
//     ring of three places of three; S = Q.K^T (N = 128) goes to one of two
//     TMEM buffers.
//     Eight softmax warps, thread = (head, half of the chunk's slots); the
//     halves' maxima meet in shared memory, P is rounded to bf16 (the tensor
//     core's operand; its sum l is kept unrounded in fp32) and two warps store
//     it into CTA 1's shared memory, 64 slots at a time, with the rescale factor.
//   CTA 1 (PV side): O in TMEM.  The rows' first 512 columns arrive by TMA as
//     64-slot x 256-column tiles in a ring of five (they come out of L2, where
//     CTA 0's loads have put them); O += P.V in two N = 256 halves per 64
//     slots.  O is rescaled only when a row's running maximum rose by more
//     than 2^8 (P then stays below 2^8 and keeps its relative precision).
// TMA boxes are the largest of 64, 32, 16 rows that divides the page size, so
// that no box crosses a page.  Boxes behind the row's end, or on a bad page,
// are asked for outside the tensor and arrive as zeros; slots behind the end
// inside the last box are zeroed in CTA 1 before the product (their P is 0,
// but they may hold NaN) and masked in CTA 0.
//
// What bounds it (B200).  32 sequences of 8K to 128K slots, 128 heads: 0.53 ms
// in a short run (4.4 TB/s, 1.06 PFLOP/s) and 0.64 ms in a long one, where the
// 1000 W cap holds the SM clock near 1.2 GHz; a chunk takes about 3400 cycles,
// 2304 of them QK products.  Without the loads the same kernel takes 0.37 ms,
// with all of them answered by L2 0.42 ms.  What the steps to it were worth:
// MMAs issued under an elected-lane predicate, waits that suspend, and small
// code in the two issuing loops (instruction fetch: unrolled nine times they
// took twice as long) 0.83 -> 0.56 ms; no arrival on the partner's barriers on
// the way of a message (it flushes the thread's earlier stores first, 2000
// cycles) 0.70 -> 0.61.  Measured slower: requesting later chunks into L2 ahead
// (0.55 -> 0.63 ms and more), P through the copy engine (behind the block loads
// in its queue).  One 2K row takes 17.3 us and one 32K row 24.7, most of it
// latency: query into TMEM, one chunk through both CTAs, the partial's stores,
// the joining kernel.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "paged_mla.cuh"
#include "tmap.h"

namespace dsa {
namespace {

constexpr int kChunk = 128;              // slots per chunk: the QK product's N
constexpr int kSub = 64;                 // slots per message to CTA 1
constexpr int kKB = kDQK / 64;           // 64-column blocks of a row: 9
constexpr int kQBlockBytes = 128 * 128;             // a 64-column block of the query, 128 heads
constexpr int kVBlockBytes = kSub * 128;            // a 64-column block of 64 rows
constexpr int kRowUnits = 2;             // what a tile costs besides its chunks, in chunks (64 rows of 2K slots: 76.2 us; 1: 79.2, 4: 78.2)

constexpr int kThreads = 384;
constexpr int kLoadWarp = 8, kMmaWarp = 9, kSendWarp = 10;
constexpr int kSoftmaxThreads = 256;
constexpr int kSendThreads = kThreads - 32 * kSendWarp;

constexpr int kPBytes = 128 * kSub * 2;             // P: 128 heads x 64 slots, bf16
constexpr uint32_t kMsgBytes = kPBytes + 3 * 512;   // then alpha, l, m per head
// ---- CTA 0 shared memory
constexpr int kQ8Off = 0;
constexpr int kKBlockBytes = kChunk * 128;          // a 64-column block of a chunk's 128 rows
constexpr int kKSlotBlocks = 3;                     // ring place i: blocks 3i .. 3i + 2 of a chunk
constexpr int kKSlotBytes = kKSlotBlocks * kKBlockBytes;
constexpr int kKSlots = kKB / kKSlotBlocks;
constexpr int kKRingOff = kQBlockBytes;
constexpr int kStages = 3;
constexpr int kStageOff = kKRingOff + kKSlots * kKSlotBytes;      // 163840
constexpr int kMaxOff = kStageOff + kStages * (int)kMsgBytes;     // 217600: maxima [2][2][128]
constexpr int kMaskOff = kMaxOff + 2 * 2 * 128 * 4;               // validity words [4][4]
constexpr int kBoxOff = kMaskOff + 4 * 16;                        // row coordinates [8]
constexpr int kQkEnd = kBoxOff + 8 * 4;
// ---- CTA 1 shared memory
constexpr int kVSlotBytes = kSub * 512;             // 64 slots x 256 columns
constexpr int kVSlots = 5;
constexpr int kPBufs = 3;
constexpr int kPOff = kVSlots * kVSlotBytes;                      // 163840
constexpr int kOutOff = kPOff + kPBufs * (int)kMsgBytes;          // 217600: epilogue staging, 1 KB per warp
constexpr int kPvBoxOff = kOutOff + 8 * 1024;
constexpr int kPvEnd = kPvBoxOff + 4 * 4;
// ---- both
constexpr int kBarOff = (kQkEnd > kPvEnd ? kQkEnd : kPvEnd);
enum Bar : int {
  kQFull = 0,                       // CTA 0: query block 8 has landed
  kQFree,                           // CTA 0: the products of a part are complete
  kKFull,                           // [3] CTA 0
  kKEmpty = kKFull + kKSlots,       // [3] CTA 0
  kSFull = kKEmpty + kKSlots,       // [2] CTA 0
  kSEmpty = kSFull + 2,             // [2] CTA 0
  kMaskFull = kSEmpty + 2,          // [4] CTA 0: the chunk's validity words are written
  kStaged = kMaskFull + 4,          // [3] CTA 0: a message is staged
  kStageFree = kStaged + kStages,   // [3] CTA 0: it is read
  kPvDone = kStageFree + kStages,   // [3] both: the product of a message is complete
  kVFull = kPvDone + kPBufs,        // [5] CTA 1
  kVEmpty = kVFull + kVSlots,       // [5] CTA 1
  kPFull = kVEmpty + kVSlots,       // [3] CTA 1: a message has landed
  kReady = kPFull + kPBufs,         // [3] CTA 1: O is rescaled, the tiles' tails are zero
  kDrain = kReady + kPBufs,
  kNumBar
};
constexpr int kMiscOff = kBarOff + kNumBar * 8;
struct Misc {
  int tmem_base, abort;
  // what a CTA's warps have done when they are through, for settle():
  uint32_t sent[2];  // CTA 0: messages that each sender warp has stored
  uint32_t issued;   // CTA 1: messages whose product is committed
  uint32_t armed;    // CTA 1: messages expected
  MlaScan<kThreads> scan;
};
constexpr int kSmemBytes = kMiscOff + (int)sizeof(Misc) + 1024;
static_assert(kSmemBytes <= 232448, "shared memory budget");
static_assert(kBarOff % 8 == 0 && kMiscOff % 8 == 0 && kMsgBytes % 16 == 0 && kStageOff % 128 == 0 && kPOff % 128 == 0, "alignment");
// Pieces of a message are dealt out to the sender's threads one by one: bytes
// that its warp w stores.
constexpr int kPieces = (int)kMsgBytes / 16;
constexpr uint32_t sender_bytes(int w) {
  const int rest = kPieces % kSendThreads - 32 * w;
  return 16u * (uint32_t)(kPieces / kSendThreads * 32 + (rest < 0 ? 0 : rest > 32 ? 32 : rest));
}
static_assert(kSendThreads == 64 && sender_bytes(0) + sender_bytes(1) == kMsgBytes, "two sender warps");
constexpr int kTmemCols = 512;
constexpr uint32_t kTmemS = 256;  // CTA 0: query blocks 0-7 in [0, 256), S buffers at 256 and 384
constexpr uint32_t kIdescQK = idesc_bf16(128, kChunk);
constexpr uint32_t kIdescPV = idesc_bf16(128, 256, /*b_mn_major=*/true);

// After a timeout, when all warps of both CTAs are done: what the partner still
// has on its way into this CTA's shared memory must land before the CTA exits.
// One thread; every wait ends after 10 ms at most.
__device__ __noinline__ void settle(uint32_t rank, uint32_t bars, const Misc* misc, uint32_t peer_misc) {
  volatile int never = 0;
  if (rank == 0) {  // arrivals of CTA 1's products
    const uint32_t n = ld_cluster_u32(peer_misc + (uint32_t)offsetof(Misc, issued));
    for (uint32_t k = n > kPBufs ? n - kPBufs : 0; k < n; ++k)
      mbar_wait(bars + 8u * (kPvDone + k % kPBufs), (k / kPBufs) & 1, &never, 10000000ull);
    return;
  }
  // Messages, the last three at most: one is sent when the product of the third
  // before it is complete.  A sender warp may have given up before the other,
  // and the message may not be expected yet.
  const uint32_t sent0 = ld_cluster_u32(peer_misc + (uint32_t)offsetof(Misc, sent));
  const uint32_t sent1 = ld_cluster_u32(peer_misc + (uint32_t)offsetof(Misc, sent) + 4u);
  const uint32_t n = max(sent0, sent1);
  for (uint32_t k = n > kPBufs ? n - kPBufs : 0; k < n; ++k) {
    const uint32_t full = bars + 8u * (kPFull + k % kPBufs);
    if (k >= misc->armed) mbar_arrive_expect_tx(full, kMsgBytes);
    if (k >= sent0) mbar_complete_tx(full, sender_bytes(0));
    if (k >= sent1) mbar_complete_tx(full, sender_bytes(1));
    mbar_wait(full, (k / kPBufs) & 1, &never, 10000000ull);
  }
}

__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    paged_mla_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                     const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ PagedMlaParams p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sbase = smem_u32(smem);
  auto bar = [&](int i) { return sbase + kBarOff + 8u * (uint32_t)i; };
  Misc* misc = reinterpret_cast<Misc*>(smem + kMiscOff);
  volatile int* abort = &misc->abort;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();
  const uint32_t peer_misc = mapa_shared(sbase + kMiscOff, rank ^ 1u);
  auto give_up = [&]() {
    *abort = 1;
    st_cluster_u32(peer_misc + (uint32_t)offsetof(Misc, abort), 1u);
  };

  // ---- prologue: barriers, TMEM
  if (threadIdx.x == 0) misc->abort = 0;
  if (warp == kMmaWarp) {
    if (lane == 0) {
      tma_prefetch_desc(rank == 0 ? &tm_k : &tm_v);
      if (rank == 0) tma_prefetch_desc(&tm_q);
      mbar_init(bar(kQFull), 1 + (p.debug_stall & 1));
      mbar_init(bar(kQFree), 1);
      for (int i = 0; i < kKSlots; ++i) {
        mbar_init(bar(kKFull + i), 1);
        mbar_init(bar(kKEmpty + i), 1);
      }
      for (int i = 0; i < 2; ++i) {
        mbar_init(bar(kSFull + i), 1);
        mbar_init(bar(kSEmpty + i), kSoftmaxThreads / 32);
      }
      for (int i = 0; i < 4; ++i) mbar_init(bar(kMaskFull + i), 1);
      for (int i = 0; i < kStages; ++i) {
        mbar_init(bar(kStaged + i), 4);
        mbar_init(bar(kStageFree + i), kSendThreads / 32);
      }
      for (int i = 0; i < kPBufs; ++i) {
        mbar_init(bar(kPvDone + i), 1);
        mbar_init(bar(kPFull + i), 1);
        mbar_init(bar(kReady + i), 8 + (i == 0 ? p.debug_stall >> 1 : 0));
      }
      for (int i = 0; i < kVSlots; ++i) {
        mbar_init(bar(kVFull + i), 1);
        mbar_init(bar(kVEmpty + i), 1);
      }
      mbar_init(bar(kDrain), 1);
      fence_mbar_init();
    }
    __syncwarp();
    tmem_alloc(sbase + kMiscOff + (uint32_t)offsetof(Misc, tmem_base), kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  cluster_arrive_release();  // the barriers are initialised; waited for before the partner's are touched
  grid_dependency_wait();    // lens, q and the cache may come from the previous kernel
  allow_dependents_launch();

  const int cl = blockIdx.x >> 1;
  auto wk = first_part<kChunk, kRowUnits, kThreads>(p, cl, &misc->scan);
  const uint32_t tmem = static_cast<uint32_t>(misc->tmem_base);
  if (rank == 1 && threadIdx.x == kSendWarp * 32) p.cut[cl] = wk.cut_row(p, cl);
  cluster_wait_acquire();
  const uint32_t lane_addr = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16);
  const int nbox64 = kSub / p.box;  // boxes per 64 slots
  const int64_t pool_rows = p.pool.n_pages * p.pool.page_size;

  if (rank == 0) {
    // ================================================================ QK side
    if (warp == kLoadWarp) {
      // ---- the chunks' blocks: lane i < 2 * nbox64 locates box i
      const uint32_t on = elect_one();
      uint32_t g = 0, item = 0;  // chunks and parts so far
      int32_t* const yk = reinterpret_cast<int32_t*>(smem + kBoxOff);  // row coordinates of a chunk's boxes
      int sent = 0;  // places filled for the current query or chunk
      bool ok = true;
      while (ok && wk.next(p)) {
        if (wk.bad && lane == 0) report(p.status, DSA_ERR_BAD_OFFSETS);
        if (wk.lo >= wk.hi) continue;
        const int b = wk.seq;
        const int nbox = 2 * nbox64;
        // row coordinate and valid slots of this lane's box of chunk i
        auto locate = [&](int i, int32_t& y, int& valid) {
          const int64_t s = (int64_t)i * kChunk + lane * p.box;
          valid = 0;
          y = (int32_t)pool_rows;
          if (lane < nbox && s < wk.len) {
            const int64_t row = pool_row(p.pool, b, (int32_t)s);
            if (row >= 0) {
              y = (int32_t)row;
              valid = min(p.box, wk.len - (int32_t)s);
            } else {
              report(p.status, DSA_ERR_BAD_INDEX);
            }
          }
        };
        // the query's blocks 0-7 go through the ring, on their way to TMEM
#pragma unroll 1
        for (int pl = 0; pl < kKSlots; ++pl) {
          if (!(ok = warp_wait(bar(kKEmpty + pl), (g + item + 1) & 1, abort, p.wait_limit_ns))) break;
          if (on) {
            const int kb0 = kKSlotBlocks * pl, kb1 = min(kb0 + kKSlotBlocks, kKB - 1);
            mbar_arrive_expect_tx(bar(kKFull + pl), (kb1 - kb0) * kQBlockBytes);
            for (int kb = kb0; kb < kb1; ++kb)
              tma_load_2d(sbase + kKRingOff + kb * kKBlockBytes, &tm_q, kb * 64, wk.q0, bar(kKFull + pl));
          }
          __syncwarp();
          sent = pl + 1;
        }
        if (!ok) break;
        if (item > 0 && !(ok = warp_wait(bar(kQFree), (item - 1) & 1, abort, p.wait_limit_ns))) break;
        if (on) {
          mbar_arrive_expect_tx(bar(kQFull), kQBlockBytes);
          tma_load_2d(sbase + kQ8Off, &tm_q, (kKB - 1) * 64, wk.q0, bar(kQFull));
        }
        ++item;
        sent = 0;
        int32_t y = 0, y_next = 0;
        int valid = 0, valid_next = 0;
        locate(wk.lo, y, valid);
        for (int i = wk.lo; ok && i < wk.hi; ++i, ++g) {
          if (lane < 8) yk[lane] = y;
          __syncwarp();
#pragma unroll 1
          for (int pl = 0; pl < kKSlots; ++pl) {
            if (!(ok = warp_wait(bar(kKEmpty + pl), (g + item + 1) & 1, abort, p.wait_limit_ns))) break;
            if (on) {
              const uint32_t full = bar(kKFull + pl);
              const uint32_t dst = sbase + kKRingOff + pl * kKSlotBytes;
              mbar_arrive_expect_tx(full, kKSlotBytes);
              const int x0 = kKSlotBlocks * pl * 64;
              if (p.box == 64) load_boxes<64, 2, kKSlotBlocks, kKBlockBytes>(dst, &tm_k, x0, yk, full);
              else if (p.box == 32) load_boxes<32, 4, kKSlotBlocks, kKBlockBytes>(dst, &tm_k, x0, yk, full);
              else load_boxes<16, 8, kKSlotBlocks, kKBlockBytes>(dst, &tm_k, x0, yk, full);
            }
            __syncwarp();
            sent = pl + 1;
          }
          if (!ok) break;  // before g counts a chunk that was not sent
          sent = 0;
          if (i + 1 < wk.hi) locate(i + 1, y_next, valid_next);
          // validity words of the chunk, 16 slots (never more than a box) at a time
          uint32_t word = ~0u;
          if (!__all_sync(0xffffffffu, lane >= nbox || valid == p.box)) {
            word = 0;
#pragma unroll 1
            for (int hh = 0; hh < 2; ++hh) {
              const int k0 = 32 * (lane & 3) + 16 * hh, bx = k0 / p.box;
              const int v = __shfl_sync(0xffffffffu, valid, bx) - (k0 - bx * p.box);
              word |= (v >= 16 ? 0xffffu : v <= 0 ? 0u : (1u << v) - 1u) << (16 * hh);
            }
          }
          if (lane < 4) reinterpret_cast<uint32_t*>(smem + kMaskOff)[4 * (g & 3) + lane] = word;
          __syncwarp();
          if (lane == 0) mbar_arrive(bar(kMaskFull + (g & 3)));
          y = y_next;
          valid = valid_next;
        }
      }
      if (*abort) {
        give_up();
        // The loads in flight must land before the CTA exits: wait (10 ms at
        // most) for the last fill of every place (one per chunk and per part).
        volatile int never = 0;
        for (int pl = 0; pl < kKSlots; ++pl) {
          const uint32_t fills = g + item + (pl < sent ? 1u : 0u);
          if (fills > 0) mbar_wait(bar(kKFull + pl), (fills - 1) & 1, &never, 10000000ull);
        }
        if (item > 0) mbar_wait(bar(kQFull), (item - 1) & 1, &never, 10000000ull);
      }
    } else if (warp == kMmaWarp) {
      // ---- S(g) = Q . K(g)^T into buffer g & 1
      const uint32_t on = elect_one();
      const uint64_t q8 = smem_desc(sbase + kQ8Off, 16, 1024, kSwizzle128B);
      const uint64_t kb0 = smem_desc(sbase + kKRingOff, 16, 1024, kSwizzle128B);
      auto wait = [&](int which, uint32_t parity) {
        const bool there = warp_wait(bar(which), parity, abort, p.wait_limit_ns);
        tc_fence_after();
        return there;
      };
      uint32_t g = 0, item = 0;
      bool ok = true;
      while (ok && wk.next(p)) {
        if (wk.lo >= wk.hi) continue;
        // the query into TMEM, once no product reads the one before
        if (item > 0 && !(ok = wait(kQFree, (item - 1) & 1))) break;
#pragma unroll 1
        for (int pl = 0; pl < kKSlots; ++pl) {
          if (!(ok = wait(kKFull + pl, (g + item) & 1))) break;
          if (on) {
            for (int kb = kKSlotBlocks * pl; kb < min(kKSlotBlocks * (pl + 1), kKB - 1); ++kb)
#pragma unroll
              for (int ks = 0; ks < 4; ++ks)
                tmem_cp_128x32b(tmem + kb * 32 + ks * 8, kb0 + (uint64_t)((kb * kKBlockBytes) >> 4) + (uint64_t)ks * 2);
            tc_commit(bar(kKEmpty + pl));
          }
          __syncwarp();
        }
        if (!ok || !(ok = wait(kQFull, item & 1))) break;
        ++item;
        for (int i = wk.lo; ok && i < wk.hi; ++i, ++g) {
          const int sb = g & 1;
          if (g >= 2 && !(ok = wait(kSEmpty + sb, ((g - 2) >> 1) & 1))) break;
          const uint32_t d = tmem + kTmemS + 128 * sb;
#pragma unroll 1
          for (int pl = 0; pl < kKSlots - 1; ++pl) {
            if (!(ok = wait(kKFull + pl, (g + item) & 1))) break;
#pragma unroll
            for (int u = 0; u < 4 * kKSlotBlocks; ++u) {
              const int kb = kKSlotBlocks * pl + u / 4, ks = u % 4;
              mma_f16_ts_if(on, d, tmem + kb * 32 + ks * 8, kb0 + (uint64_t)((kb * kKBlockBytes) >> 4) + (uint64_t)ks * 2,
                            kIdescQK, (kb | ks) ? 1u : 0u);
            }
            if (on) tc_commit(bar(kKEmpty + pl));
          }
          if (!ok || !(ok = wait(kKFull + kKSlots - 1, (g + item) & 1))) break;
#pragma unroll
          for (int u = 0; u < 4 * kKSlotBlocks; ++u) {
            const int kb = kKB - kKSlotBlocks + u / 4, ks = u % 4;
            const uint64_t bd = kb0 + (uint64_t)((kb * kKBlockBytes) >> 4) + (uint64_t)ks * 2;
            if (kb < kKB - 1) mma_f16_ts_if(on, d, tmem + kb * 32 + ks * 8, bd, kIdescQK, 1u);
            else mma_f16_ss_if(on, d, q8 + (uint64_t)ks * 2, bd, kIdescQK, 1u);
          }
          if (on) tc_commit(bar(kKEmpty + kKSlots - 1));
          if (on) tc_commit(bar(kSFull + sb));
        }
        if (ok && on) tc_commit(bar(kQFree));
      }
      if (*abort) {
        give_up();
        volatile int never = 0;  // tensor-core work ends before TMEM is released
        if (on) {
          tc_commit(bar(kDrain));
          mbar_wait(bar(kDrain), 0, &never, 10000000ull);
        }
      }
    } else if (warp >= kSendWarp) {
      // ---- message j (64 slots of P, alpha, l, m) to CTA 1's buffer j % 3:
      // two warps read the staged message and store it into the partner's
      // shared memory.  (The copy engine would take it too, but behind the
      // block loads in its queue: 2600 cycles a message against 970 without.)
      const uint32_t rem_msg = mapa_shared(sbase + kPOff, 1);
      const uint32_t rem_pfull = mapa_shared(bar(kPFull), 1);
      const int tid = threadIdx.x - kSendWarp * 32;
      constexpr int kBatch = 9;
      static_assert(kPieces <= 2 * kBatch * kSendThreads, "two rounds per message");
      uint32_t j = 0;
      bool ok = true;
      while (ok && wk.next(p)) {
        for (int i = 2 * wk.lo; i < 2 * wk.hi; ++i, ++j) {
          const uint32_t st = j % kStages, pb = j % kPBufs;
          ok = warp_wait(bar(kStaged + st), (j / kStages) & 1, abort, p.wait_limit_ns) &&
               (j < kPBufs || warp_wait<true>(bar(kPvDone + pb), ((j / kPBufs) - 1) & 1, abort, p.wait_limit_ns));
          if (!ok) break;
          const uint32_t full = rem_pfull + 8u * pb, dst = rem_msg + pb * kMsgBytes;
          const uint8_t* const src = smem + kStageOff + st * kMsgBytes;
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            uint4 v[kBatch];
#pragma unroll
            for (int k = 0; k < kBatch; ++k) {
              const int e = (r * kBatch + k) * kSendThreads + tid;
              if (e < kPieces) v[k] = *reinterpret_cast<const uint4*>(src + 16 * e);
            }
#pragma unroll
            for (int k = 0; k < kBatch; ++k) {
              const int e = (r * kBatch + k) * kSendThreads + tid;
              if (e < kPieces) st_async_v4(dst + 16 * e, v[k], full);
            }
          }
          warp_arrive(bar(kStageFree + st));  // the message is read
        }
      }
      // CTA 1's last arrivals here must land before this CTA exits
      for (uint32_t k = j > kPBufs ? j - kPBufs : 0; ok && k < j; ++k)
        ok = warp_wait<true>(bar(kPvDone + k % kPBufs), (k / kPBufs) & 1, abort, p.wait_limit_ns);
      if (lane == 0) misc->sent[warp - kSendWarp] = j;
      if (*abort) give_up();
    } else if (warp < 8) {
      // ---- softmax: thread = (head h, slots 64 * half .. of every chunk)
      const int h = (warp & 3) * 32 + lane, half = warp >> 2;
      uint32_t g = 0;
      bool ok = true;
      while (ok && wk.next(p)) {
        const bool dead = (warp & 3) * 32 >= wk.m;  // a warp without rows only keeps step
        // slots that this row's token sees, and the tile's first token
        const int row_len = wk.len - max(0, wk.nt - 1 - h / p.H), min_len = wk.len - (wk.nt - 1);
        float m_run = -INFINITY, l_run = 0.f;
        for (int i = wk.lo; i < wk.hi; ++i, ++g) {
          const int sb = g & 1;
          const uint32_t j = 2 * g + half, stg = j % kStages;
          ok = warp_wait(bar(kMaskFull + (g & 3)), (g >> 2) & 1, abort, p.wait_limit_ns) &&
               warp_wait(bar(kSFull + sb), (g >> 1) & 1, abort, p.wait_limit_ns);
          uint32_t sv[64];
          float mx = -INFINITY;
          if (ok) {
            tc_fence_after();
            if (!dead) {
              tmem_ld64(lane_addr + kTmemS + 128 * sb + 64 * half, sv);
              tc_wait_ld();
            }
            tc_fence_before();
            const uint32_t* vm = reinterpret_cast<const uint32_t*>(smem + kMaskOff) + 4 * (g & 3) + 2 * half;
            uint32_t vm0 = vm[0], vm1 = vm[1];
            warp_arrive(bar(kSEmpty + sb));
            const int64_t s0 = (int64_t)i * kChunk + 64 * half;
            if (s0 + 64 > min_len) {  // the tile's tokens see different slots here
              const int see = (int)max(row_len - s0, (int64_t)0);
              vm0 &= see >= 32 ? ~0u : (1u << see) - 1u;
              vm1 &= see >= 64 ? ~0u : see <= 32 ? 0u : (1u << (see - 32)) - 1u;
            }
            if (!dead) {
              // x = s * scale * log2(e); masked slots -inf
#pragma unroll
              for (int c = 0; c < 64; c += 2) {
                const float2 x = __fmul2_rn(make_float2(__uint_as_float(sv[c]), __uint_as_float(sv[c + 1])),
                                            make_float2(p.scale_log2, p.scale_log2));
                sv[c] = __float_as_uint(x.x);
                sv[c + 1] = __float_as_uint(x.y);
              }
              if ((vm0 & vm1) != ~0u) {
#pragma unroll
                for (int c = 0; c < 32; ++c) {
                  if (!((vm0 >> c) & 1u)) sv[c] = 0xff800000u;
                  if (!((vm1 >> c) & 1u)) sv[32 + c] = 0xff800000u;
                }
              }
              float m8[8];
#pragma unroll
              for (int c = 0; c < 8; ++c) {
                m8[c] = __uint_as_float(sv[c]);
#pragma unroll
                for (int e = 8 + c; e < 64; e += 8) m8[c] = fmaxf(m8[c], __uint_as_float(sv[e]));
              }
              mx = fmaxf(fmaxf(fmaxf(m8[0], m8[1]), fmaxf(m8[2], m8[3])), fmaxf(fmaxf(m8[4], m8[5]), fmaxf(m8[6], m8[7])));
              reinterpret_cast<float*>(smem + kMaxOff)[256 * sb + 128 * half + h] = mx;
            }
            // the staging buffer is free once message j - 3 is read
            if (j >= kStages) ok = warp_wait(bar(kStageFree + stg), ((j / kStages) - 1) & 1, abort, p.wait_limit_ns);
          }
          // both halves' maxima are written; all eight warps leave together
          if (named_barrier_or(1, kSoftmaxThreads, !ok)) {
            ok = false;
            break;
          }
          uint8_t* const stage = smem + kStageOff + stg * kMsgBytes;
          if (!dead) {
            mx = fmaxf(mx, reinterpret_cast<const float*>(smem + kMaxOff)[256 * sb + 128 * (half ^ 1) + h]);
            float alpha = 1.f;
            if (mx > m_run + 8.f) {  // always in the row's first chunk that holds a finite score
              alpha = exp2f(m_run - mx);  // 0 at first
              m_run = mx;
            }
            const float sub = m_run == -INFINITY ? 0.f : m_run;
            float2 l2[4] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f), make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
            const float2 nm = make_float2(-sub, -sub);
            uint8_t* const prow = stage + (h >> 3) * 1024 + (h & 7) * 16;
#pragma unroll
            for (int c8 = 0; c8 < 8; ++c8) {
              uint32_t w4[4];
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const int c = 8 * c8 + 2 * e;
                const float2 d = __fadd2_rn(make_float2(__uint_as_float(sv[c]), __uint_as_float(sv[c + 1])), nm);
                const float2 pv = make_float2(ex2_approx(d.x), ex2_approx(d.y));
                l2[e] = __fadd2_rn(l2[e], pv);
                const __nv_bfloat162 pb = __floats2bfloat162_rn(pv.x, pv.y);
                w4[e] = *reinterpret_cast<const uint32_t*>(&pb);
              }
              *reinterpret_cast<uint4*>(prow + c8 * 128) = make_uint4(w4[0], w4[1], w4[2], w4[3]);
            }
            const float2 a = __fadd2_rn(l2[0], l2[1]), bb = __fadd2_rn(l2[2], l2[3]);
            l_run = l_run * alpha + ((a.x + bb.x) + (a.y + bb.y));
            float* const tail = reinterpret_cast<float*>(stage + kPBytes);
            tail[h] = alpha;
            tail[128 + h] = l_run;
            tail[256 + h] = m_run;
          } else {
            reinterpret_cast<float*>(stage + kPBytes)[h] = 1.f;
          }
          warp_arrive(bar(kStaged + stg));
        }
      }
      if (*abort) give_up();
    }
  } else {
    // ================================================================ PV side
    if (warp == kLoadWarp) {
      // ---- 64-slot x 256-column tiles: lane i < nbox64 locates box i
      uint32_t ring = 0;
      bool ok = true;
      const uint32_t on = elect_one();
      int32_t* const yv = reinterpret_cast<int32_t*>(smem + kPvBoxOff);  // row coordinates of a tile's boxes
      while (ok && wk.next(p)) {
        const int b = wk.seq;
        auto locate = [&](int i) -> int32_t {  // i counts 64-slot halves
          const int64_t s = (int64_t)i * kSub + lane * p.box;
          if (lane < nbox64 && s < wk.len) {
            const int64_t row = pool_row(p.pool, b, (int32_t)s);
            if (row >= 0) return (int32_t)row;
          }
          return (int32_t)pool_rows;
        };
        int32_t y = 0, y_next = 0;
        if (wk.lo < wk.hi) y = locate(2 * wk.lo);
        for (int i = 2 * wk.lo; ok && i < 2 * wk.hi; ++i) {
          if (i + 1 < 2 * wk.hi) y_next = locate(i + 1);
          if (lane < 4) yv[lane] = y;
          __syncwarp();
#pragma unroll 1
          for (int n = 0; n < 2; ++n, ++ring) {
            const uint32_t slot = ring % kVSlots;
            if (!(ok = warp_wait(bar(kVEmpty + slot), ((ring / kVSlots) & 1) ^ 1, abort, p.wait_limit_ns))) break;
            if (on) {
              mbar_arrive_expect_tx(bar(kVFull + slot), kVSlotBytes);
              const uint32_t full = bar(kVFull + slot);
              const uint32_t dst = sbase + slot * kVSlotBytes;
              if (p.box == 64) {
                tma_load_3d(dst, &tm_v, 0, yv[0], 4 * n, full);
              } else if (p.box == 32) {
                load_boxes<32, 2, 4, kVBlockBytes>(dst, &tm_v, 256 * n, yv, full);
              } else {
                load_boxes<16, 4, 4, kVBlockBytes>(dst, &tm_v, 256 * n, yv, full);
              }
            }
            __syncwarp();
          }
          y = y_next;
        }
      }
      if (*abort) {
        give_up();
        volatile int never = 0;
        for (uint32_t k = ring > kVSlots ? ring - kVSlots : 0; k < ring; ++k)
          mbar_wait(bar(kVFull + k % kVSlots), (k / kVSlots) & 1, &never, 10000000ull);
      }
    } else if (warp == kMmaWarp) {
      // ---- O[:, 256 n ..] += P(j) . V(j)[:, 256 n ..]
      const uint32_t on = elect_one();
      const uint64_t pa0 = smem_desc(sbase + kPOff, 128, 1024, kSwizzleNone);
      const uint64_t vb0 = smem_desc(sbase, kVBlockBytes, 1024, kSwizzle128B);
      auto wait = [&](int which, uint32_t parity) {
        const bool there = warp_wait(bar(which), parity, abort, p.wait_limit_ns);
        tc_fence_after();
        return there;
      };
      uint32_t j = 0, ring = 0, issued = 0;
      bool ok = true;
      while (ok && wk.next(p)) {
        for (int i = 2 * wk.lo; ok && i < 2 * wk.hi; ++i, ++j) {
          const uint32_t pb = j % kPBufs;
          if (!(ok = wait(kReady + pb, (j / kPBufs) & 1))) break;
          const uint64_t ad = pa0 + (uint64_t)((pb * kMsgBytes) >> 4);
#pragma unroll 1
          for (int n = 0; n < 2; ++n, ++ring) {
            const uint32_t slot = ring % kVSlots;
            if (!(ok = wait(kVFull + slot, (ring / kVSlots) & 1))) break;
            const uint64_t bd = vb0 + (uint64_t)((slot * kVSlotBytes) >> 4);
#pragma unroll
            for (int s = 0; s < kSub / 16; ++s)
              mma_f16_ss_if(on, tmem + 256 * n, ad + (uint64_t)((s * 256) >> 4), bd + (uint64_t)((s * 2048) >> 4), kIdescPV,
                            (i > 2 * wk.lo || s > 0) ? 1u : 0u);
            if (on) tc_commit(bar(kVEmpty + slot));
          }
          if (ok && on) tc_commit_mc(bar(kPvDone + pb), 0x3);
          if (ok) ++issued;
        }
      }
      if (lane == 0) misc->issued = issued;
      if (*abort) {
        give_up();
        volatile int never = 0;
        if (on) {
          tc_commit(bar(kDrain));
          mbar_wait(bar(kDrain), 0, &never, 10000000ull);
        }
      }
    } else if (warp == kSendWarp) {
      // ---- expects message j in buffer j % 3 once that buffer is free.  (Done
      // here and not by the sender: an arrival on another CTA's barrier
      // releases the thread's earlier stores first, which took 2000 cycles.)
      uint32_t j = 0, armed = 0;
      bool ok = true;
      while (ok && wk.next(p)) {
        for (int i = 2 * wk.lo; ok && i < 2 * wk.hi; ++i, ++j) {
          const uint32_t pb = j % kPBufs;
          ok = j < kPBufs || warp_wait(bar(kPvDone + pb), ((j / kPBufs) - 1) & 1, abort, p.wait_limit_ns);
          if (ok && lane == 0) mbar_arrive_expect_tx(bar(kPFull + pb), kMsgBytes);
          if (ok) ++armed;
        }
      }
      if (lane == 0) misc->armed = armed;
      if (*abort) give_up();
    } else if (warp < 8) {
      // ---- rescale and epilogue: thread = (head h, half of the columns)
      const int h = (warp & 3) * 32 + lane, col0 = 256 * (warp >> 2);
      uint8_t* const ostage = smem + kOutOff + warp * 1024;
      uint32_t j = 0;
      bool ok = true;
      while (ok && wk.next(p)) {
        const bool dead = (warp & 3) * 32 >= wk.m;
        float l_half[2] = {0.f, 0.f}, m_row = -INFINITY;
        for (int i = 2 * wk.lo; i < 2 * wk.hi; ++i, ++j) {
          const uint32_t pb = j % kPBufs;
          ok = warp_wait<true>(bar(kPFull + pb), (j / kPBufs) & 1, abort, p.wait_limit_ns);
          if (!ok) break;
          const float* tail = reinterpret_cast<const float*>(smem + kPOff + pb * kMsgBytes + kPBytes);
          if (!dead) {
            const float alpha = (i & 1) ? 1.f : tail[h];  // a chunk's factor comes with its first half
            if (i & 1) l_half[1] = tail[128 + h];
            else l_half[0] = tail[128 + h];
            m_row = tail[256 + h];
            if (i > 2 * wk.lo && __any_sync(0xffffffffu, alpha != 1.f)) {
              // every product so far is complete when the last one is
              ok = warp_wait(bar(kPvDone + (j - 1) % kPBufs), ((j - 1) / kPBufs) & 1, abort, p.wait_limit_ns);
              if (!ok) break;
              tc_fence_after();
#pragma unroll 1
              for (int c0 = col0; c0 < col0 + 256; c0 += 32) {
                uint32_t ov[32];
                tmem_ld32(lane_addr + c0, ov);
                tc_wait_ld();
#pragma unroll
                for (int c = 0; c < 32; ++c) ov[c] = __float_as_uint(__uint_as_float(ov[c]) * alpha);
                tmem_st32(lane_addr + c0, ov);
              }
              tc_wait_st();
            }
          }
          // Two kinds of slots must not meet the product as they are.  Slots
          // behind the end that share the last box with it may hold anything:
          // they become zeros.  Slots that only some of the tile's tokens see
          // have P = 0 in the others' rows, and 0 * NaN is not 0: a row that is
          // not finite becomes zeros too (the tokens that see it have a NaN
          // for a sum already).
          const int64_t s0 = (int64_t)i * kSub;
          if (s0 + kSub > wk.len - (wk.nt - 1)) {
            const int z_begin = (int)max((int64_t)0, wk.len - (wk.nt - 1) - s0);
            const int z_end = (int)min((int64_t)kSub, (((int64_t)wk.len + p.box - 1) & -(int64_t)p.box) - s0);
            const uint32_t k0 = (2 * j) % kVSlots, k1 = (2 * j + 1) % kVSlots;
            ok = warp_wait(bar(kVFull + k0), ((2 * j) / kVSlots) & 1, abort, p.wait_limit_ns) &&
                 warp_wait(bar(kVFull + k1), ((2 * j + 1) / kVSlots) & 1, abort, p.wait_limit_ns);
            if (!ok) break;
            // a warp takes a row: 2 x 4 blocks x 8 pieces of 16 bytes
            for (int z = z_begin + warp; z < z_end; z += 8) {
              uint8_t* const row = smem + (lane >> 3) * kVBlockBytes + z * 128 + (lane & 7) * 16;
              uint4* const a = reinterpret_cast<uint4*>(row + k0 * kVSlotBytes);
              uint4* const b = reinterpret_cast<uint4*>(row + k1 * kVSlotBytes);
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
          warp_arrive(bar(kReady + pb));
        }
        if (!ok) break;
        const bool any = wk.lo < wk.hi;
        if (any)
          ok = warp_wait(bar(kPvDone + (j - 1) % kPBufs), ((j - 1) / kPBufs) & 1, abort, p.wait_limit_ns);
        if (!ok) break;
        if (dead) continue;
        tc_fence_after();
        const float l = l_half[0] + l_half[1];
        const bool whole = wk.hi - wk.lo == wk.chunks;
        const float mul = l == 0.f ? 0.f : 1.f / l;  // a NaN among the scores stays one
        const int64_t part = 2 * cl + (wk.lo > 0 ? 0 : 1);
        // Partials: fp32 where the output is.  With bf16 output fp16, each
        // row's 32 columns scaled by the power of two that brings the largest of
        // them to [1, 2): 11 bits, against the 8 that P has and the output
        // keeps, and half the bytes (an SM writes 28 bytes a cycle, however it
        // writes: a 128-row fp32 partial takes 9000 cycles).  With nothing else
        // changed, ten calls in a graph, fp16 against fp32: one 2K row 17.2 us,
        // 18.8; one 32K row 24.7, 26.8; two of 20K-30K 28.8, 32.6; eight of
        // 4K-12K 34.4, 38.4.  (Tiles of up to 32 rows gain nothing and keep
        // fp32: one 2K row of 16 heads 12.9, 12.5.)
        // [column / 8][row][8] or [column / 4][row][4], so that a warp's stores
        // are whole lines.
        // Finished rows: 64 bytes of 16 rows at a time through shared memory,
        // so that four lanes write a row's piece.
        const int pm = p.tp * p.H;  // rows a partial has room for
        uint4* const pout = p.part_o + part * pm * (p.part_f32 ? kDV / 4 : kDV / 8) + h;
        const int elt = p.out_bf16 ? 2 : 4;
        uint8_t* const gout =
            reinterpret_cast<uint8_t*>(p.out) + ((int64_t)wk.q0 + (warp & 3) * 32) * (int64_t)(kDV * elt);
        // 64 bytes of every row (four pieces per lane), 16 rows at a time
        auto put = [&](const uint4 (&piece)[4], int col_byte) {
#pragma unroll
          for (int hf = 0; hf < 2; ++hf) {
            if ((lane >> 4) == hf) {
              const int rr = lane & 15;
#pragma unroll
              for (int c = 0; c < 4; ++c)
                *reinterpret_cast<uint4*>(ostage + rr * 64 + ((c ^ ((rr >> 1) & 3)) << 4)) = piece[c];
            }
            __syncwarp();
#pragma unroll
            for (int u = 0; u < 2; ++u) {
              const int rr = 8 * u + (lane >> 2), c = lane & 3;
              const uint4 v = *reinterpret_cast<const uint4*>(ostage + rr * 64 + ((c ^ ((rr >> 1) & 3)) << 4));
              if ((warp & 3) * 32 + 16 * hf + rr < wk.m)
                *reinterpret_cast<uint4*>(gout + (16 * hf + rr) * (kDV * elt) + col_byte + 16 * c) = v;
            }
            __syncwarp();
          }
        };
#pragma unroll 1
        for (int c0 = col0; c0 < col0 + 256; c0 += 32) {
          uint32_t ov[32];
          if (any) {
            tmem_ld32(lane_addr + c0, ov);
            tc_wait_ld();
#pragma unroll
            for (int c = 0; c < 32; c += 2) {
              if (!whole) break;
              const float2 v = __fmul2_rn(make_float2(__uint_as_float(ov[c]), __uint_as_float(ov[c + 1])), make_float2(mul, mul));
              ov[c] = __float_as_uint(v.x);
              ov[c + 1] = __float_as_uint(v.y);
            }
          } else {
#pragma unroll
            for (int c = 0; c < 32; ++c) ov[c] = 0u;
          }
          if (!whole) {
            if (h < wk.m && p.part_f32) {
#pragma unroll
              for (int c = 0; c < 8; ++c)
                pout[(int64_t)(c0 / 4 + c) * pm] = make_uint4(ov[4 * c], ov[4 * c + 1], ov[4 * c + 2], ov[4 * c + 3]);
            } else if (h < wk.m) {
              float big = 0.f;
#pragma unroll
              for (int c = 0; c < 32; ++c) big = fmaxf(big, fabsf(__uint_as_float(ov[c])));
              if (big == INFINITY) {  // the largest finite one decides; infinities stay what they are
                big = 0.f;
#pragma unroll
                for (int c = 0; c < 32; ++c) {
                  const float v = fabsf(__uint_as_float(ov[c]));
                  if (v < INFINITY) big = fmaxf(big, v);
                }
              }
              const int e = min(max((int)(__float_as_uint(big) >> 23), 1), 253);  // biased exponent
              const float scale = __uint_as_float((uint32_t)(254 - e) << 23);
              p.part_sc[(part * (kDV / 32) + c0 / 32) * pm + h] = __uint_as_float((uint32_t)e << 23);  // 1 / scale
#pragma unroll
              for (int c = 0; c < 4; ++c) {
                uint32_t w4[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                  const float2 v = __fmul2_rn(make_float2(__uint_as_float(ov[8 * c + 2 * e]), __uint_as_float(ov[8 * c + 2 * e + 1])),
                                              make_float2(scale, scale));
                  const __half2 t2 = __floats2half2_rn(v.x, v.y);
                  w4[e] = *reinterpret_cast<const uint32_t*>(&t2);
                }
                pout[(int64_t)(c0 / 8 + c) * pm] = make_uint4(w4[0], w4[1], w4[2], w4[3]);
              }
            }
          } else if (p.out_bf16) {
            uint4 piece[4];
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              uint32_t w4[4];
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const __nv_bfloat162 t2 =
                    __floats2bfloat162_rn(__uint_as_float(ov[8 * c + 2 * e]), __uint_as_float(ov[8 * c + 2 * e + 1]));
                w4[e] = *reinterpret_cast<const uint32_t*>(&t2);
              }
              piece[c] = make_uint4(w4[0], w4[1], w4[2], w4[3]);
            }
            put(piece, c0 * 2);
          } else {
#pragma unroll
            for (int hf = 0; hf < 2; ++hf) {
              uint4 piece[4];
#pragma unroll
              for (int c = 0; c < 4; ++c)
                piece[c] = make_uint4(ov[16 * hf + 4 * c], ov[16 * hf + 4 * c + 1], ov[16 * hf + 4 * c + 2], ov[16 * hf + 4 * c + 3]);
              put(piece, c0 * 4 + hf * 64);
            }
          }
        }
        tc_fence_before();  // O is read: the next row's first product (after Ready) may overwrite it
        if (h < wk.m && col0 == 0) {
          if (whole) {
            if (p.lse) p.lse[(int64_t)wk.q0 + h] = l == 0.f ? -INFINITY : (m_row + log2f(l)) * 0.69314718055994531f;
          } else {
            p.part_ml[2 * part * pm + h] = m_row;
            p.part_ml[(2 * part + 1) * pm + h] = l;
          }
        }
      }
      if (*abort) give_up();
    }
  }

  tc_fence_before();
  __syncthreads();
  // neither CTA leaves while the other may still write into its shared memory
  cluster_sync_all();
  if (*abort) {  // the same in both CTAs: whoever gives up tells the partner
    if (threadIdx.x == 0) settle(rank, bar(0), misc, peer_misc);
    __syncwarp();
    cluster_sync_all();  // the partner has read this CTA's counts
  }
  if (warp == kMmaWarp) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
  if (threadIdx.x == 0 && *abort) report(p.status, DSA_ERR_TIMEOUT);
}

// Joins the partials of the cut rows: out = sum_i 2^(m_i - M) O_i / sum_i 2^(m_i - M) l_i.
// A task is (cut tile, 32 rows, WARPS / SPLIT groups of eight columns); lane = row.
// SPLIT warps share a tile's partials, each with the maximum of its own, and
// the first of them joins their sums in a fixed order: with one long row the
// partials are many and the rows few (64 partials: 8 loads in flight per
// thread instead of 64 one behind the other), with many rows it is the other
// way round.
constexpr int kMaxWorkers = 256;

template <int SPLIT, int WARPS, bool F32>
__global__ void __launch_bounds__(32 * WARPS)
    paged_mla_combine_kernel(const CutRow* __restrict__ cut, const float* __restrict__ part_ml,
                             const float* __restrict__ part_sc, const uint4* __restrict__ part_o, int n_workers, int pm,
                             int64_t rows, void* out, int out_bf16, float* lse, int32_t* status) {
  constexpr int kGroups = WARPS / SPLIT;  // column groups per task
  constexpr int kFlight = 8;              // partials a thread has in flight
  constexpr int kVec = F32 ? 2 : 1;       // 16-byte pieces of eight columns
  __shared__ CutRow s_cut[kMaxWorkers];
  __shared__ int s_count[WARPS];
  __shared__ float s_sum[SPLIT > 1 ? WARPS : 1][10][32];
  grid_dependency_wait();
  allow_dependents_launch();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  // the boundaries that cut a tile, a thread each
  static_assert(kMaxWorkers <= 32 * WARPS, "a thread per worker");
  CutRow mine{-1, 0, 0, 0};
  if (threadIdx.x < n_workers) mine = cut[threadIdx.x];
  // The only addresses that come out of the workspace.  Another call that uses
  // it at the same time may have written them: no access outside this call's
  // own arrays then.
  if (mine.q0 >= 0 && (mine.m < 1 || mine.m > pm || mine.q0 > rows - mine.m || mine.first < 0 || mine.count < 1 ||
                       mine.first > n_workers - mine.count)) {
    mine.q0 = -1;
    if (blockIdx.x == 0) report(status, DSA_ERR_WORKSPACE);
  }
  const uint32_t cuts = __ballot_sync(0xffffffffu, mine.q0 >= 0);
  if (lane == 0) s_count[warp] = __popc(cuts);
  __syncthreads();
  int n_cut = 0, at = __popc(cuts & ((1u << lane) - 1u));
  for (int w = 0; w < WARPS; ++w) {
    if (w < warp) at += s_count[w];
    n_cut += s_count[w];
  }
  if (mine.q0 >= 0) s_cut[at] = mine;
  __syncthreads();
  const int hgroups = (pm + 31) / 32, per_row = hgroups * (kDV / 8 / kGroups);
  const int tasks = n_cut * per_row;
  for (int task = blockIdx.x; task < tasks; task += gridDim.x) {
    const CutRow c = s_cut[task / per_row];
    const int rest = task % per_row;
    const int h = rest % hgroups * 32 + lane, grp = rest / hgroups * kGroups + warp / SPLIT, sub = warp % SPLIT;
    float acc[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    float M = -INFINITY, l = 0.f;
    if (h < c.m) {
      for (int i0 = sub; i0 < c.count; i0 += SPLIT * kFlight) {
        uint4 o[kFlight][kVec];
        float m[kFlight], li[kFlight], sc[kFlight], top = M;
#pragma unroll
        for (int k = 0; k < kFlight; ++k) {
          const int i = i0 + SPLIT * k;
          m[k] = -INFINITY;
          li[k] = 0.f;
          sc[k] = F32 ? 1.f : 0.f;
#pragma unroll
          for (int v = 0; v < kVec; ++v) o[k][v] = make_uint4(0u, 0u, 0u, 0u);
          if (i < c.count) {
            // the first partial is its cluster's second, the others are their clusters' first
            const int64_t part = 2 * (int64_t)(c.first + i) + (i == 0 ? 1 : 0);
            m[k] = __ldg(part_ml + 2 * part * pm + h);
            li[k] = __ldg(part_ml + (2 * part + 1) * pm + h);
            if (!F32) sc[k] = __ldg(part_sc + (part * (kDV / 32) + grp / 4) * pm + h);
#pragma unroll
            for (int v = 0; v < kVec; ++v) o[k][v] = __ldg(part_o + (part * (kDV / 8) * kVec + grp * kVec + v) * pm + h);
          }
        }
#pragma unroll
        for (int k = 0; k < kFlight; ++k) top = fmaxf(top, m[k]);
        const float off = top == -INFINITY ? 0.f : top;
        const float a = exp2f(M - off);  // 0 at first
        M = top;
        l *= a;
#pragma unroll
        for (int e = 0; e < 8; ++e) acc[e] *= a;
#pragma unroll
        for (int k = 0; k < kFlight; ++k) {
          const float w = exp2f(m[k] - off), ws = w * sc[k];
          l = fmaf(w, li[k], l);
#pragma unroll
          for (int v = 0; v < kVec; ++v) {
            const uint32_t w4[4] = {o[k][v].x, o[k][v].y, o[k][v].z, o[k][v].w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              if (F32) {
                acc[4 * v + e] = fmaf(ws, __uint_as_float(w4[e]), acc[4 * v + e]);
              } else {
                const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w4[e]));
                acc[2 * e] = fmaf(ws, f.x, acc[2 * e]);
                acc[2 * e + 1] = fmaf(ws, f.y, acc[2 * e + 1]);
              }
            }
          }
        }
      }
    }
    if (SPLIT > 1) {
      __syncthreads();  // the sums of the task before are read
#pragma unroll
      for (int e = 0; e < 8; ++e) s_sum[warp][e][lane] = acc[e];
      s_sum[warp][8][lane] = l;
      s_sum[warp][9][lane] = M;
      __syncthreads();
      if (sub != 0) continue;
      float top = M;
#pragma unroll
      for (int u = 1; u < SPLIT; ++u) top = fmaxf(top, s_sum[warp + u][9][lane]);
      const float off = top == -INFINITY ? 0.f : top;
      l = 0.f;
#pragma unroll
      for (int e = 0; e < 8; ++e) acc[e] = 0.f;
#pragma unroll
      for (int u = 0; u < SPLIT; ++u) {
        const float w = exp2f(s_sum[warp + u][9][lane] - off);
        l = fmaf(w, s_sum[warp + u][8][lane], l);
#pragma unroll
        for (int e = 0; e < 8; ++e) acc[e] = fmaf(w, s_sum[warp + u][e][lane], acc[e]);
      }
      M = top;
    }
    if (h >= c.m) continue;
    const float inv = l == 0.f ? 0.f : 1.f / l;  // a NaN among the scores stays one
#pragma unroll
    for (int e = 0; e < 8; ++e) acc[e] *= inv;  // (as in a tile that nothing cuts: 0 * infinity is a NaN)
    const int64_t rh = (int64_t)c.q0 + h;
    if (out_bf16) {
      uint32_t w4[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const __nv_bfloat162 t2 = __floats2bfloat162_rn(acc[2 * e], acc[2 * e + 1]);
        w4[e] = *reinterpret_cast<const uint32_t*>(&t2);
      }
      reinterpret_cast<uint4*>(reinterpret_cast<__nv_bfloat16*>(out) + rh * kDV)[grp] = make_uint4(w4[0], w4[1], w4[2], w4[3]);
    } else {
      float4* const o4 = reinterpret_cast<float4*>(reinterpret_cast<float*>(out) + rh * kDV) + 2 * grp;
      o4[0] = make_float4(acc[0], acc[1], acc[2], acc[3]);
      o4[1] = make_float4(acc[4], acc[5], acc[6], acc[7]);
    }
    if (grp == 0 && lse) lse[rh] = l == 0.f ? -INFINITY : (M + log2f(l)) * 0.69314718055994531f;
  }
}

// Clusters of a launch: as many as the card runs at once.
int paged_clusters() {
  static PerDeviceOnce once;
  static int count[64] = {};
  int dev = 0;
  cudaGetDevice(&dev);
  const int half = std::max(1, std::min(device_info().sm_count / 2, kMaxWorkers));
  if (dev < 0 || dev >= 64) return half;
  const cudaError_t e = once.run([&] {
    cudaError_t e2 = cudaFuncSetAttribute(paged_mla_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemBytes);
    if (e2 != cudaSuccess) return e2;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(2 * half);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = kSmemBytes;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = 2;
    at[0].val.clusterDim.y = 1;
    at[0].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    int n = 0;
    e2 = cudaOccupancyMaxActiveClusters(&n, paged_mla_kernel, &cfg);
    if (e2 != cudaSuccess) return e2;
    count[dev] = std::max(1, std::min(n, half));
    return cudaSuccess;
  });
  return e == cudaSuccess ? count[dev] : half;
}

// Tokens whose (token, head) rows fit in one tile.
int tokens_per_tile(int T, int H) { return std::max(1, std::min(T, 128 / H)); }

// Tiles of up to 32 rows have a kernel of their own, one CTA per worker (128
// sequences of 500 to 4000 slots: 16 heads 74 us, 92 with the pair; 32 heads
// 82, 94; with 64 heads it took 109, the pair 100).
bool few_rows(int T, int H) { return tokens_per_tile(T, H) * H <= kFewRows; }
int paged_workers(int T, int H) { return few_rows(T, H) ? paged_few_workers() : paged_clusters(); }

size_t paged_workspace(int T, int H) {
  const size_t n = (size_t)paged_workers(T, H), m = (size_t)tokens_per_tile(T, H) * H;
  // (fp32 partials and no scales: more than fp16 ones with theirs)
  return n * sizeof(CutRow) + 2 * n * m * (2 + kDV) * sizeof(float);
}

}  // namespace
}  // namespace dsa

using namespace dsa;

extern "C" {

size_t dsa_paged_mla_workspace_size(int B, int T, int H) {
  if (B <= 0 || T <= 0 || (int64_t)B * T > (int64_t)1 << 24 || H < 1 || H > DSA_MAX_HEADS) return 0;
  return paged_workspace(T, H);
}

int dsa_paged_mla(const void* q, const void* kv_pages, const int32_t* page_table, int64_t ld_table, int max_pages,
                  const int32_t* lens, int B, int T, int H, int page_size, int64_t n_pages, float scale, void* out,
                  int out_dtype, float* lse, void* workspace, size_t ws_bytes, int32_t* dev_status, void* stream) {
  if (B <= 0 || T <= 0 || H < 1 || !q || !lens || !out) return DSA_ERR_INVALID_ARG;
  if ((int64_t)B * T > (int64_t)1 << 24 || H > DSA_MAX_HEADS) return DSA_ERR_UNSUPPORTED;
  if (int rc = check_pool(kv_pages, page_table, ld_table, max_pages, page_size, n_pages)) return rc;
  if (out_dtype != DSA_BF16 && out_dtype != DSA_F32) return DSA_ERR_INVALID_ARG;
  if (!(scale == scale) || !is_aligned16(q) || !is_aligned16(out) || !is_aligned4(lens, lse, dev_status))
    return DSA_ERR_INVALID_ARG;
  const size_t need = paged_workspace(T, H);
  if (!workspace || ws_bytes < need || !is_aligned16(workspace)) return DSA_ERR_WORKSPACE;
  MlaParams debug;
  take_attention_debug(debug);
  const int n = paged_workers(T, H);
  PagedMlaParams p;
  p.pool = PagePool{page_table, ld_table, n_pages, max_pages, page_size};
  p.lens = lens;
  p.T = T;
  p.H = H;
  p.tp = tokens_per_tile(T, H);
  p.tiles = (T + p.tp - 1) / p.tp;
  p.n_rows = B * p.tiles;
  p.n_workers = n;
  p.box = page_size % 64 == 0 ? 64 : page_size % 32 == 0 ? 32 : 16;
  p.scale_log2 = scale * 1.4426950408889634f;
  p.out = out;
  p.out_bf16 = out_dtype == DSA_BF16 ? 1 : 0;
  p.lse = lse;
  p.cut = reinterpret_cast<CutRow*>(workspace);
  const size_t pm = (size_t)p.tp * H;
  p.part_f32 = few_rows(T, H) || !p.out_bf16 ? 1 : 0;
  p.part_o = reinterpret_cast<uint4*>(p.cut + n);
  p.part_ml = reinterpret_cast<float*>(p.part_o + 2 * n * pm * (p.part_f32 ? kDV / 4 : kDV / 8));
  p.part_sc = p.part_ml + 2 * n * pm * 2;
  p.status = dev_status;
  p.debug_stall = debug.debug_stall;
  // A worker may write any number of empty tiles while its other warps wait for
  // it: 2 us each with one head, 5 with 128 (2^24 empty rows of one head: 0.23 s).
  p.wait_limit_ns = debug.wait_limit_ns + (debug.debug_stall ? 0 : 10000ull * (uint64_t)p.n_rows);
  const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const uint64_t rows = (uint64_t)n_pages * page_size;
  if (few_rows(T, H)) {
    if (launch_paged_mla_few(p, q, (uint64_t)B * T * H, kv_pages, rows, s) != cudaSuccess) return DSA_ERR_CUDA;
  } else {
    CUtensorMap tq, tk, tv;
    bool maps = make_tmap_2d(&tq, q, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, kDQK, (uint64_t)B * T * H, kDQK * 2, 64, 128,
                             CU_TENSOR_MAP_SWIZZLE_128B) &&
                make_tmap_2d(&tk, kv_pages, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, kDQK, rows, kDQK * 2, 64, (uint32_t)p.box,
                             CU_TENSOR_MAP_SWIZZLE_128B);
    tv = tk;
    if (p.box == 64) {  // a tile of V is one box: 64 rows of four column blocks
      const uint64_t dims[3] = {64, rows, kKB}, strides[2] = {kDQK * 2, 128};
      const uint32_t box_v[3] = {64, 64, 4};
      maps = maps &&
             make_tmap_3d(&tv, kv_pages, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, dims, strides, box_v, CU_TENSOR_MAP_SWIZZLE_128B);
    }
    if (!maps) return DSA_ERR_CUDA;
    if (launch_pdl(paged_mla_kernel, dim3(2 * (unsigned)n), dim3(kThreads), kSmemBytes, s, tq, tk, tv, p) != cudaSuccess)
      return DSA_ERR_CUDA;
  }
  if (n > 1) {
    // Warps that share a row's partials, by how many a tile of the batch has on
    // average (the lengths are known on the device only).  A batch of one long
    // row among empty or short ones therefore gets too few: one 32K row takes
    // 24.9 us alone and 35 to 41 among 63 others, with 16 heads 17.7 and 36.
    // With rows of like length: (one row of 32K: 30.9 us with eight, 33.0 with four, 37.0 with two; two rows
    // 30.9, 28.9, 30.8; eight rows 51.5, 47.5, 43.5 and 42.8 with one, because
    // the tasks then fill the card several times over).  A tile of few rows has
    // few tasks, more warps fit beside one another (16 heads, back to back: one
    // row of 32K 18.6 us with eight, 17.4 with sixteen, four rows 25.0 with four,
    // 23.8 with eight; 128 heads the other way round, 24.6 and 26.7).
    const int per_row = n / p.n_rows;
    const bool few = few_rows(T, H);
    const int split = per_row >= 64 ? (few ? 16 : 8) : few && per_row >= 32 ? 8 : per_row >= 16 ? 4 : 1;
    const int warps = std::max(split, 8), groups = warps / split;  // column groups per task
    const int64_t tasks = (int64_t)std::min(p.n_rows, n - 1) * (((int64_t)pm + 31) / 32) * (kDV / 8 / groups);
    const dim3 grid((unsigned)std::min<int64_t>(tasks, 8 * (int64_t)device_info().sm_count)), block(32 * warps);
    const auto pick = [split](auto f32) {
      constexpr bool kF32 = decltype(f32)::value;
      return split == 16  ? paged_mla_combine_kernel<16, 16, kF32>
             : split == 8 ? paged_mla_combine_kernel<8, 8, kF32>
             : split == 4 ? paged_mla_combine_kernel<4, 8, kF32>
                          : paged_mla_combine_kernel<1, 8, kF32>;
    };
    const auto kernel = p.part_f32 ? pick(std::true_type{}) : pick(std::false_type{});
    if (launch_pdl(kernel, grid, block, 0, s, (const CutRow*)p.cut, (const float*)p.part_ml, (const float*)p.part_sc, (const uint4*)p.part_o,
                   n, (int)pm, (int64_t)B * T * H, out, p.out_bf16, lse, dev_status) != cudaSuccess)
      return DSA_ERR_CUDA;
  }
  return DSA_OK;
}

}  // extern "C"
