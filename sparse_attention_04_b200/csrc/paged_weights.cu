// paged_weights.cu -- the attention weight that every slot of a paged cache
// collects from the newest tokens' heads:
//   acc_out[b,s] = decay * acc[b,s] + sum_{t,h : s <= len-T+t} exp(scale q.k_s - lse)
//
// Plain form: one CTA per (sequence, 32 slots at a time), the rows staged in
// shared memory, lane = slot; each warp sums every eighth (t, h) in fp32, and
// the eight sums are joined in a fixed order.
#include <cuda_bf16.h>

#include <algorithm>

#include "paged.cuh"

namespace dsa {
namespace {

constexpr int kTile = 32, kRowPad = kDQK + 8;

__global__ void __launch_bounds__(256)
    paged_weights_kernel(const __nv_bfloat16* __restrict__ q, const __nv_bfloat16* __restrict__ kv, PagePool pool,
                         const int32_t* __restrict__ lens, const float* __restrict__ lse, int T, int H, float scale_log2,
                         float decay, const float* acc, float* acc_out, int64_t ld_slots, int32_t* status) {
  extern __shared__ __align__(16) uint8_t smem_raw[];
  __nv_bfloat16* tile = reinterpret_cast<__nv_bfloat16*>(smem_raw);
  float* sq = reinterpret_cast<float*>(smem_raw + kTile * kRowPad * 2);  // [8][576]
  __shared__ int s_ok[kTile];
  __shared__ float part[8][kTile];
  grid_dependency_wait();
  allow_dependents_launch();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int b = blockIdx.y;
  bool bad;
  const int32_t len = checked_len(lens[b], min(pool_capacity(pool), ld_slots), bad);
  if (bad && threadIdx.x == 0 && blockIdx.x == 0) report(status, DSA_ERR_BAD_OFFSETS);
  for (int64_t s0 = (int64_t)blockIdx.x * kTile; s0 < len; s0 += (int64_t)gridDim.x * kTile) {
    __syncthreads();
    for (int i = warp; i < kTile; i += 8) {
      const int64_t row = s0 + i < len ? pool_row(pool, b, (int32_t)(s0 + i)) : -1;
      if (lane == 0) {
        s_ok[i] = row >= 0;
        if (row < 0 && s0 + i < len) report(status, DSA_ERR_BAD_INDEX);
      }
      uint4* d = reinterpret_cast<uint4*>(tile + i * kRowPad);
      for (int c = lane; c < kDQK / 8; c += 32)
        d[c] = row >= 0 ? reinterpret_cast<const uint4*>(kv + row * kDQK)[c] : make_uint4(0, 0, 0, 0);
    }
    __syncthreads();
    float sum = 0.f;
    for (int th = warp; th < T * H; th += 8) {
      const int64_t row = (int64_t)b * T * H + th;
      const float ls = lse[row];
      __syncwarp();
      for (int c = lane; c < kDQK; c += 32) sq[warp * kDQK + c] = __bfloat162float(q[row * kDQK + c]);
      __syncwarp();
      float x = 0.f;
      const __nv_bfloat16* k = tile + lane * kRowPad;
      for (int c = 0; c < kDQK; c += 2) {
        const float2 kk = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(k + c));
        x = fmaf(kk.x, sq[warp * kDQK + c], x);
        x = fmaf(kk.y, sq[warp * kDQK + c + 1], x);
      }
      if (s0 + lane <= len - T + th / H && ls != -INFINITY) sum += exp2f(x * scale_log2 - ls * 1.4426950408889634f);
    }
    part[warp][lane] = sum;
    __syncthreads();
    if (warp == 0 && s0 + lane < len) {
      float v = 0.f;
      for (int w = 0; w < 8; ++w) v += part[w][lane];
      const int64_t o = (int64_t)b * ld_slots + s0 + lane;
      const float old = acc ? decay * acc[o] : 0.f;
      acc_out[o] = s_ok[lane] ? old + v : old;
    }
  }
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
  const PagePool pool{page_table, ld_table, n_pages, max_pages, page_size};
  constexpr int kSmem = kTile * kRowPad * 2 + 8 * kDQK * 4;
  static PerDeviceOnce attr;
  if (attr.run([] {
        return cudaFuncSetAttribute(paged_weights_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
      }) != cudaSuccess)
    return DSA_ERR_CUDA;
  if (B > 65535) return DSA_ERR_UNSUPPORTED;
  const int64_t x = std::min<int64_t>((std::min<int64_t>((int64_t)max_pages * page_size, ld_slots) + kTile - 1) / kTile, 1024);
  const cudaError_t e =
      launch_pdl(paged_weights_kernel, dim3((unsigned)x, (unsigned)B), dim3(256), kSmem,
                 reinterpret_cast<cudaStream_t>(stream), reinterpret_cast<const __nv_bfloat16*>(q),
                 reinterpret_cast<const __nv_bfloat16*>(kv_pages), pool, lens, lse, T, H, scale * 1.4426950408889634f, decay,
                 acc, acc_out, ld_slots, dev_status);
  return e == cudaSuccess ? DSA_OK : DSA_ERR_CUDA;
}
