// evict_plan.cu -- which slots of a paged cache survive a cut to `budget`
// slots, and the row moves that close the gaps.
//
// Per sequence of L > n = budget slots: every slot gets a 32-bit key (order-
// preserving in acc; all ones where the slot is protected, 0 for NaN), three
// digit passes (11, 11, 10 bits) over the keys find the n-th largest key tau
// and how many keys equal to tau stay (the lowest slots), and two prefix
// counts over the resulting bitmap rank the free slots below n and the
// survivors from n on: the i-th of one takes the i-th of the other.
// (Where the protected slots alone are more than n, the n-th key is all ones and
// a second search ranks them by their weight.)
//
// One thread-block cluster per sequence; CTA r owns the contiguous slots
// [r * S, (r + 1) * S).  The keys stay in shared memory as far as it goes, and
// acc and pos are then read once (HBM bounds a large plan at 8 bytes per slot).
// The bitmap has its place there too, a quarter byte per slot: all keys fit up
// to about 48600 slots per CTA (ld_slots 389000 with eight CTAs), of 786432
// slots (DSA_MAX_PLAN_SLOTS) 2600 do.  The others are made again from acc and
// pos where they are needed: these are read up to four times per search.
//
// B200: 32 sequences of 64K to 128K slots cut to 64K in 30 us (41 MB: 6.4 us of
// HBM), eight of 4097 slots in 10.8 us (ten calls in a graph).  What bounds it
// is instruction issue and about 30 barrier-separated steps: keys and first
// histogram 9 us, the digit passes 10, bitmap and ranks 5, lists 6.
#include <cooperative_groups.h>
#include <cuda_bf16.h>

#include <algorithm>

#include "paged.cuh"

namespace dsa {
namespace {

constexpr int kThreads = 1024, kWarps = kThreads / 32;
constexpr int kBins = 2048;
constexpr int kMaxCS = 8;
constexpr int kSmemMax = 227 * 1024;

struct alignas(16) PlanSmem {
  uint32_t hist[3][kBins];  // one per pass: no CTA clears what another still reads
  uint32_t warp_sum[3][kWarps];  // cluster-wide counts of each warp's bins, per pass
  alignas(16) uint64_t warp_tot[32];
  uint32_t cnt[2];          // this CTA's free slots below n, survivors from n on
  uint32_t base[2];         // those of the CTAs before it
  uint32_t total;           // moves of the sequence
  uint32_t digit, remaining, eq_before, bin_count;
};

static_assert((int64_t)sizeof(PlanSmem) + 8 * (DSA_MAX_PLAN_SLOTS / kMaxCS / 32 + 4) <= kSmemMax, "shared memory");

struct PlanArgs {
  const float* acc;
  const int32_t* pos;
  const int32_t* lens;
  const int32_t* end_pos;
  int64_t ld;
  int budget, recent;
  int32_t* new_lens;
  int32_t* n_moves;
  int32_t* dst;
  int32_t* src;
  int64_t ld_moves;
  int32_t* status;
};

// among: only the protected slots compete (0 for the others; -inf maps far
// above 1).
__device__ __forceinline__ uint32_t slot_key(float a, bool kept_always, bool among) {
  const uint32_t key = a != a ? 0u : float_order_key(a);
  if (among) return kept_always ? max(key, 1u) : 0u;
  return kept_always ? 0xffffffffu : key;
}

// Exclusive scan over the block of one value per thread; *total is the sum.
__device__ __noinline__ uint64_t scan_excl(uint64_t v, PlanSmem& sm, uint64_t* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  uint64_t* const warp_tot = sm.warp_tot;
  uint64_t inc = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint64_t u = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += u;
  }
  __syncthreads();  // warp_tot may still be read from the scan before
  if (lane == 31) warp_tot[warp] = inc;
  __syncthreads();
  const uint64_t w = lane < kWarps ? warp_tot[lane] : 0ull;
  uint64_t winc = w;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint64_t u = __shfl_up_sync(0xffffffffu, winc, o);
    if (lane >= o) winc += u;
  }
  *total = __shfl_sync(0xffffffffu, winc, 31);
  return inc - v + __shfl_sync(0xffffffffu, winc - w, warp);
}

__global__ void __launch_bounds__(kThreads, 1) evict_plan_kernel(const PlanArgs a, int key_cap) {
  namespace cg = cooperative_groups;
  extern __shared__ __align__(16) uint8_t smem_raw[];
  PlanSmem& sm = *reinterpret_cast<PlanSmem*>(smem_raw);
  uint32_t* const keys = reinterpret_cast<uint32_t*>(smem_raw + sizeof(PlanSmem));  // key_cap, then the bitmap
  uint32_t* const bitmap = keys + key_cap;
  cg::cluster_group cluster = cg::this_cluster();
  const int CS = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int b = blockIdx.x / CS;
  // a cluster barrier takes 1300 cycles even for one CTA
  auto meet = [&]() {
    if (CS > 1) cluster.sync();
    else __syncthreads();
  };

  grid_dependency_wait();  // acc and lens come from the previous kernel
  allow_dependents_launch();
  const int32_t L = a.lens[b];
  const int64_t protect_from = a.recent > 0 ? (int64_t)a.end_pos[b] - a.recent : 0;
  const bool bad = L < 0 || (int64_t)L > a.ld;
  const int32_t n = min(L, a.budget);
  int32_t* const dst = a.dst + (int64_t)b * a.ld_moves;
  int32_t* const src = a.src + (int64_t)b * a.ld_moves;
  auto pad_lists = [&](int64_t from) {
    for (int64_t i = from + (int64_t)rank * kThreads + threadIdx.x; i < a.ld_moves; i += (int64_t)CS * kThreads) {
      dst[i] = -1;
      src[i] = -1;
    }
  };
  if (bad || L <= a.budget) {  // nothing to evict (the same verdict in every CTA)
    if (rank == 0 && threadIdx.x == 0) {
      if (bad) report(a.status, DSA_ERR_BAD_OFFSETS);
      a.new_lens[b] = L;
      a.n_moves[b] = 0;
    }
    pad_lists(0);
    return;
  }
  const int S = ((L + CS - 1) / CS + 127) / 128 * 128;
  const int s_lo = min(rank * S, L), m = min(s_lo + S, L) - s_lo;  // this CTA's slots
  const float* const acc = a.acc + (int64_t)b * a.ld + s_lo;
  const int32_t* const pos = a.recent > 0 ? a.pos + (int64_t)b * a.ld + s_lo : nullptr;
  // More protected slots than the budget holds (positions that repeat, an
  // end_pos that lags): they compete among themselves, in a second search.
  bool among = false;
  auto make_key = [&](int i) { return slot_key(acc[i], pos && pos[i] >= protect_from, among); };

  // Adds four keys per lane to a histogram.  A warp whose keys are all alike
  // (fresh slots, say) adds once; otherwise the few lanes that share a bin are
  // served one after the other, which costs less than sorting them out.
  auto count4 = [&](uint32_t* hist, const uint32_t (&bin)[4], const bool (&on)[4]) {
    const uint32_t first = __shfl_sync(0xffffffffu, bin[0], 0);
    if (__all_sync(0xffffffffu, on[0] && on[1] && on[2] && on[3] && bin[0] == first && bin[1] == first && bin[2] == first &&
                                    bin[3] == first)) {
      if (lane == 0) atomicAdd(&hist[first], 128u);
      return;
    }
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (on[e]) atomicAdd(&hist[bin[e]], 1u);
  };
  // keys of the slots 4g .. 4g + 3 (those at or behind m are of no meaning)
  auto keys_of = [&](int g) -> uint4 {
    if (4 * g < key_cap) return *reinterpret_cast<const uint4*>(keys + 4 * g);
    uint4 k = make_uint4(0u, 0u, 0u, 0u);
    if (4 * g < m) k.x = make_key(4 * g);
    if (4 * g + 1 < m) k.y = make_key(4 * g + 1);
    if (4 * g + 2 < m) k.z = make_key(4 * g + 2);
    if (4 * g + 3 < m) k.w = make_key(4 * g + 3);
    return k;
  };
  auto key_of = [&](int i) { return i < key_cap ? keys[i] : make_key(i); };
  // ---- keys, four slots per thread at a time and kFlight such groups in
  // flight, and the histogram of their top 11 bits
  constexpr int kFlight = 2;
  const int m4 = (m + 3) / 4;
  uint32_t prefix, remaining;
#pragma unroll 1
  for (;;) {
    for (int i = threadIdx.x; i < 3 * kBins; i += kThreads) (&sm.hist[0][0])[i] = 0;
    __syncthreads();
    for (int g0 = 0; g0 < m4; g0 += kFlight * kThreads) {
      float4 av[kFlight];
      int4 pv[kFlight];
#pragma unroll
      for (int k = 0; k < kFlight; ++k) {
        const int g = g0 + k * kThreads + threadIdx.x;
        av[k] = make_float4(0.f, 0.f, 0.f, 0.f);
        pv[k] = make_int4(INT32_MIN, INT32_MIN, INT32_MIN, INT32_MIN);
        if (4 * g < m) {  // (whole groups: the rows' pitch is a multiple of 4)
          av[k] = __ldcs(reinterpret_cast<const float4*>(acc) + g);
          if (pos) pv[k] = __ldcs(reinterpret_cast<const int4*>(pos) + g);
        }
      }
#pragma unroll
      for (int k = 0; k < kFlight; ++k) {
        const int g = g0 + k * kThreads + threadIdx.x;
        if (__all_sync(0xffffffffu, 4 * g >= m)) break;
        const float a4[4] = {av[k].x, av[k].y, av[k].z, av[k].w};
        const int p4[4] = {pv[k].x, pv[k].y, pv[k].z, pv[k].w};
        uint32_t key[4], bin[4];
        bool on[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          key[e] = slot_key(a4[e], pos && p4[e] >= protect_from, among);
          bin[e] = key[e] >> 21;
          on[e] = 4 * g + e < m;
        }
        count4(sm.hist[0], bin, on);
        if (4 * g < key_cap) *reinterpret_cast<uint4*>(keys + 4 * g) = make_uint4(key[0], key[1], key[2], key[3]);
      }
    }
    __syncthreads();
    // ---- three digit passes: tau, and how many keys equal to it stay
    prefix = 0;
    remaining = (uint32_t)n;
#pragma unroll 1
    for (int pass = 0; pass < 3; ++pass) {
      const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0;
      const int bins = pass == 2 ? 1024 : 2048;
      if (pass > 0) {
        const int pshift = pass == 1 ? 21 : 10;
        for (int g0 = 0; g0 < m4; g0 += kThreads) {
          const int g = g0 + threadIdx.x;
          const uint4 k4 = g < m4 ? keys_of(g) : make_uint4(0u, 0u, 0u, 0u);
          const uint32_t key[4] = {k4.x, k4.y, k4.z, k4.w};
          bool on[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) on[e] = 4 * g + e < m && (key[e] >> pshift) == (prefix >> pshift);
          if (!__any_sync(0xffffffffu, on[0] || on[1] || on[2] || on[3])) continue;  // mostly: few keys share a prefix
          uint32_t bin[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) bin[e] = (key[e] >> shift) & (uint32_t)(bins - 1);
          count4(sm.hist[pass], bin, on);
        }
      }
      meet();
      // The bin, from the top, that holds the remaining-th largest key: lane l of
      // warp w has the bins bins-1 - 64 w - 2 l and the one below, summed over the
      // cluster.  The warps' sums say which warp has it, and that one looks
      // inside.
      const int hi = bins - 1 - 64 * warp - 2 * lane;
      uint32_t c0 = 0, c1 = 0;
      if (hi > 0) {
        for (int q = 0; q < CS; ++q) {
          const uint2 v = *reinterpret_cast<const uint2*>(cluster.map_shared_rank(&sm.hist[pass][0], q) + hi - 1);
          c0 += v.y;
          c1 += v.x;
        }
      }
      const uint32_t mine = __reduce_add_sync(0xffffffffu, c0 + c1);
      if (lane == 0) sm.warp_sum[pass][warp] = mine;
      __syncthreads();
      const uint32_t t = sm.warp_sum[pass][lane];
      uint32_t inc = t;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const uint32_t u = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += u;
      }
      uint32_t above = __shfl_sync(0xffffffffu, inc - t, warp);
      if (above < remaining && remaining <= above + mine) {
        inc = c0 + c1;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const uint32_t u = __shfl_up_sync(0xffffffffu, inc, o);
          if (lane >= o) inc += u;
        }
        above += inc - (c0 + c1);
        if (above < remaining && remaining <= above + c0 + c1) {
          const bool second = remaining > above + c0;
          sm.digit = (uint32_t)(second ? hi - 1 : hi);
          sm.remaining = remaining - above - (second ? c0 : 0u);
          sm.bin_count = second ? c1 : c0;
        }
      }
      __syncthreads();
      prefix |= sm.digit << shift;
      remaining = sm.remaining;
      if (pass < 2) __syncthreads();  // read before the next pass writes them
    }
    if (among || prefix != 0xffffffffu || sm.bin_count == remaining) break;  // (the same in every CTA)
    among = true;
    meet();  // the histograms are read
  }
  const uint32_t tau = prefix, need_eq = remaining;
  if (warp == 0) {  // keys equal to tau in the CTAs before this one
    uint32_t v = lane < rank ? cluster.map_shared_rank(&sm.hist[2][0], lane)[tau & 1023u] : 0u;
    v = __reduce_add_sync(0xffffffffu, v);
    if (lane == 0) sm.eq_before = v;
  }
  __syncthreads();
  // ---- which slots stay: a bitmap, one word per 32 slots; thread t owns a
  // contiguous run of words
  const int words = (m + 31) / 32;
  const int wpt = (words + kThreads - 1) / kThreads;
  for (int w = warp; w < words; w += kWarps) {
    const int i = 32 * w + lane;
    const uint32_t key = m <= key_cap ? keys[i] : i < m ? key_of(i) : 0u;  // (keys holds whole words)
    const uint32_t up = __ballot_sync(0xffffffffu, i < m && key > tau);
    const uint32_t eq = __ballot_sync(0xffffffffu, i < m && key == tau);
    if (lane == 0) {
      bitmap[2 * w] = up;
      bitmap[2 * w + 1] = eq;
    }
  }
  __syncthreads();
  const int w_lo = min((int)threadIdx.x * wpt, words), w_hi = min(w_lo + wpt, words);
  uint32_t eq_rank = 0;
  const bool all_eq = sm.bin_count == need_eq;  // every key equal to tau stays: no ranks are needed
  if (!all_eq) {
    uint32_t eqs = 0;
    uint64_t unused;
    for (int w = w_lo; w < w_hi; ++w) eqs += __popc(bitmap[2 * w + 1]);
    eq_rank = sm.eq_before + (uint32_t)scan_excl(eqs, sm, &unused);
  }
  // slots of word w below n
  auto below = [&](int w) -> uint32_t {
    const int k = n - (s_lo + 32 * w);
    return k >= 32 ? 0xffffffffu : k <= 0 ? 0u : (1u << k) - 1u;
  };
  auto held = [&](int w) -> uint32_t { return m - 32 * w >= 32 ? 0xffffffffu : (1u << (m - 32 * w)) - 1u; };
  uint32_t free_n = 0, surv_n = 0;
  for (int w = w_lo; w < w_hi; ++w) {
    uint32_t keep = bitmap[2 * w], eq = bitmap[2 * w + 1];
    if (all_eq) {
      keep |= eq;
      eq = 0;
    }
    while (eq && eq_rank < need_eq) {
      const uint32_t low = eq & (0u - eq);
      keep |= low;
      eq ^= low;
      ++eq_rank;
    }
    bitmap[2 * w] = keep;
    free_n += __popc(~keep & below(w) & held(w));
    surv_n += __popc(keep & ~below(w));
  }
  uint64_t both_all;
  const uint64_t both = scan_excl((uint64_t)surv_n << 32 | free_n, sm, &both_all);
  uint32_t fr = (uint32_t)both, sr = (uint32_t)(both >> 32);
  const uint32_t free_all = (uint32_t)both_all, surv_all = (uint32_t)(both_all >> 32);
  if (threadIdx.x == 0) {
    sm.cnt[0] = free_all;
    sm.cnt[1] = surv_all;
  }
  meet();
  if (warp == 0) {
    const uint32_t f = lane < CS ? cluster.map_shared_rank(&sm.cnt[0], lane)[0] : 0u;
    const uint32_t s = lane < rank ? cluster.map_shared_rank(&sm.cnt[0], lane)[1] : 0u;
    const uint32_t total = __reduce_add_sync(0xffffffffu, f);
    const uint32_t f_before = __reduce_add_sync(0xffffffffu, lane < rank ? f : 0u);
    const uint32_t s_before = __reduce_add_sync(0xffffffffu, s);
    if (lane == 0) {
      sm.total = total;
      sm.base[0] = f_before;
      sm.base[1] = s_before;
    }
  }
  meet();  // also: no CTA leaves while another reads its counts
  const uint32_t moves = sm.total;
  if ((int64_t)moves > a.ld_moves) {
    if (rank == 0 && threadIdx.x == 0) {
      report(a.status, DSA_ERR_BAD_OFFSETS);
      a.new_lens[b] = L;
      a.n_moves[b] = 0;
    }
    pad_lists(0);
    return;
  }
  // A word below n holds free slots, one from n on survivors; the word that n
  // cuts holds both, and its survivors are the first of all.  So one mask and
  // one rank per word say what is to be written, and the thread that owns the
  // cut word writes its survivors itself.
  fr += sm.base[0];
  sr += sm.base[1];
  for (int w = w_lo; w < w_hi; ++w) {
    const uint32_t keep = bitmap[2 * w], f = ~keep & below(w) & held(w), sv = keep & ~below(w);
    const bool low = s_lo + 32 * w < n;
    bitmap[2 * w] = low ? f : sv;
    bitmap[2 * w + 1] = low ? fr : sr;
    fr += __popc(f);
    sr += __popc(sv);
    if (low) {
      int at = 0;
      for (uint32_t x = sv; x; x &= x - 1) src[at++] = s_lo + 32 * w + __ffs((int)x) - 1;
    }
  }
  __syncthreads();
  // a warp writes a word's entries side by side
  const uint32_t lower = (1u << lane) - 1u;
#pragma unroll 2
  for (int w = warp; w < words; w += kWarps) {
    const uint2 v = *reinterpret_cast<const uint2*>(bitmap + 2 * w);
    const int slot = s_lo + 32 * w + lane;
    int32_t* const list = s_lo + 32 * w < n ? dst : src;
    if ((v.x >> lane) & 1u) list[v.y + __popc(v.x & lower)] = slot;
  }
  if (rank == 0 && threadIdx.x == 0) {
    a.new_lens[b] = n;
    a.n_moves[b] = (int32_t)moves;
  }
  pad_lists(moves);
}

}  // namespace
}  // namespace dsa

using namespace dsa;

extern "C" int dsa_evict_plan(const float* acc, const int32_t* pos, const int32_t* lens, const int32_t* end_pos, int B,
                              int64_t ld_slots, int budget, int recent, int32_t* new_lens, int32_t* n_moves,
                              int32_t* move_dst, int32_t* move_src, int64_t ld_moves, int32_t* dev_status,
                              void* stream) {
  if (B <= 0 || !acc || !lens || !new_lens || !n_moves || !move_dst || !move_src || ld_moves < 1)
    return DSA_ERR_INVALID_ARG;
  if (B > (1 << 24)) return DSA_ERR_UNSUPPORTED;
  if (budget < 1 || recent < 0 || recent > budget) return DSA_ERR_INVALID_ARG;
  if (recent > 0 && (!pos || !end_pos)) return DSA_ERR_INVALID_ARG;
  if (!is_aligned4(lens, end_pos, new_lens, n_moves, move_dst, move_src, dev_status)) return DSA_ERR_INVALID_ARG;
  if (int rc = check_slots(acc, pos, ld_slots)) return rc;
  if (ld_slots > DSA_MAX_PLAN_SLOTS) return DSA_ERR_UNSUPPORTED;
  // CTAs per sequence: one per 8192 slots, up to eight (a portable cluster);
  // fewer while the sequences make more than one wave of CTAs and the keys
  // still fit on chip (32 sequences of 131072 slots: 4 instead of 8).
  int cs = 1;
  while (cs < kMaxCS && ld_slots > (int64_t)8192 * cs) cs *= 2;
  while (cs > 1 && (int64_t)B * cs > device_info().sm_count && ld_slots <= (int64_t)40960 * (cs / 2)) cs /= 2;
  const int64_t slice = ((ld_slots + cs - 1) / cs + 127) / 128 * 128;
  const int64_t fixed = (int64_t)sizeof(PlanSmem) + 8 * ((slice + 31) / 32);
  const int key_cap = (int)std::min<int64_t>(slice, (kSmemMax - fixed) / 16 * 4);
  const int64_t smem = fixed + 4 * (int64_t)key_cap;
  static PerDeviceOnce attr;
  if (attr.run([] {
        return cudaFuncSetAttribute(evict_plan_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemMax);
      }) != cudaSuccess)
    return DSA_ERR_CUDA;
  const PlanArgs a{acc, pos, lens, end_pos, ld_slots, budget, recent, new_lens, n_moves, move_dst, move_src, ld_moves, dev_status};
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)B * (unsigned)cs);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = (size_t)smem;
  cfg.stream = reinterpret_cast<cudaStream_t>(stream);
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  at[1].id = cudaLaunchAttributeClusterDimension;
  at[1].val.clusterDim.x = (unsigned)cs;
  at[1].val.clusterDim.y = 1;
  at[1].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, evict_plan_kernel, a, key_cap) == cudaSuccess ? DSA_OK : DSA_ERR_CUDA;
}
