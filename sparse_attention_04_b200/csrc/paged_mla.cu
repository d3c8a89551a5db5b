// paged_mla.cu -- absorbed MLA of the newest tokens over a whole paged cache.
//
// For query row (b, t) and head h, over the slots s <= lens[b] - T + t:
//   l_s = scale * q . kv_s[:576];  out = softmax(l) . kv[:, :512];  lse = log sum exp(l)
//
// Plain form: one CTA per (row, 8 heads), one warp per head; 32 slots at a
// time are staged in shared memory, each lane scores one of them, and the
// running maximum and sum of the softmax are kept in fp32.
#include <cuda_bf16.h>

#include "paged.cuh"

namespace dsa {
namespace {

constexpr int kHeads = 8, kTile = 32, kRowPad = kDQK + 8;

__global__ void __launch_bounds__(256)
    paged_mla_kernel(const __nv_bfloat16* __restrict__ q, const __nv_bfloat16* __restrict__ kv, PagePool pool,
                     const int32_t* __restrict__ lens, int T, int H, float scale_log2, void* out, int out_bf16, float* lse,
                     int32_t* status) {
  extern __shared__ __align__(16) uint8_t smem_raw[];
  __nv_bfloat16* tile = reinterpret_cast<__nv_bfloat16*>(smem_raw);      // [32][584]
  float* sq = reinterpret_cast<float*>(smem_raw + kTile * kRowPad * 2);  // [8][576]
  __shared__ int s_ok[kTile];
  grid_dependency_wait();
  allow_dependents_launch();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int groups = (H + kHeads - 1) / kHeads;
  const int r = blockIdx.x / groups, h = (blockIdx.x % groups) * kHeads + warp;
  const int b = r / T, t = r - b * T;
  bool bad;
  const int32_t len = checked_len(lens[b], pool_capacity(pool), bad);
  if (bad && threadIdx.x == 0) report(status, DSA_ERR_BAD_OFFSETS);
  const int L = max(0, len - T + t + 1);
  const int64_t rh = (int64_t)r * H + h;
  if (h < H)
    for (int c = lane; c < kDQK; c += 32) sq[warp * kDQK + c] = __bfloat162float(q[rh * kDQK + c]);
  float m = -INFINITY, l = 0.f, o[16];
  for (int c = 0; c < 16; ++c) o[c] = 0.f;
  for (int s0 = 0; s0 < L; s0 += kTile) {
    __syncthreads();
    for (int i = warp; i < kTile; i += 8) {
      const int64_t row = s0 + i < L ? pool_row(pool, b, s0 + i) : -1;
      if (lane == 0) {
        s_ok[i] = row >= 0;
        if (row < 0 && s0 + i < L) report(status, DSA_ERR_BAD_INDEX);
      }
      uint4* d = reinterpret_cast<uint4*>(tile + i * kRowPad);
      for (int c = lane; c < kDQK / 8; c += 32)
        d[c] = row >= 0 ? reinterpret_cast<const uint4*>(kv + row * kDQK)[c] : make_uint4(0, 0, 0, 0);
    }
    __syncthreads();
    float x = 0.f;
    const __nv_bfloat16* k = tile + lane * kRowPad;
    for (int c = 0; c < kDQK; c += 2) {
      const float2 kk = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(k + c));
      x = fmaf(kk.x, sq[warp * kDQK + c], x);
      x = fmaf(kk.y, sq[warp * kDQK + c + 1], x);
    }
    x = s_ok[lane] ? x * scale_log2 : -INFINITY;
    float mx = x;
    for (int d = 16; d; d >>= 1) mx = fmaxf(mx, __shfl_xor_sync(~0u, mx, d));
    const float m_new = fmaxf(m, mx), sub = m_new == -INFINITY ? 0.f : m_new;
    const float p = exp2f(x - sub), a = exp2f(m - sub);
    float ps = p;
    for (int d = 16; d; d >>= 1) ps += __shfl_xor_sync(~0u, ps, d);
    l = l * a + ps;
    m = m_new;
    for (int c = 0; c < 16; ++c) o[c] *= a;
    for (int j = 0; j < kTile; ++j) {
      const float pj = __shfl_sync(~0u, p, j);
      for (int c = 0; c < 16; ++c) o[c] = fmaf(pj, __bfloat162float(tile[j * kRowPad + 32 * c + lane]), o[c]);
    }
  }
  if (h >= H) return;
  const float inv = l == 0.f ? 0.f : 1.f / l;  // a NaN among the scores stays one
  for (int c = 0; c < 16; ++c) {
    if (out_bf16) reinterpret_cast<__nv_bfloat16*>(out)[rh * kDV + 32 * c + lane] = __float2bfloat16(o[c] * inv);
    else reinterpret_cast<float*>(out)[rh * kDV + 32 * c + lane] = o[c] * inv;
  }
  if (lse && lane == 0) lse[rh] = l == 0.f ? -INFINITY : (m + log2f(l)) * 0.69314718055994531f;
}

}  // namespace
}  // namespace dsa

using namespace dsa;

extern "C" {

size_t dsa_paged_mla_workspace_size(int B, int T, int H) {
  (void)B, (void)T, (void)H;
  return 0;
}

int dsa_paged_mla(const void* q, const void* kv_pages, const int32_t* page_table, int64_t ld_table, int max_pages,
                  const int32_t* lens, int B, int T, int H, int page_size, int64_t n_pages, float scale, void* out,
                  int out_dtype, float* lse, void* workspace, size_t ws_bytes, int32_t* dev_status, void* stream) {
  if (B <= 0 || T <= 0 || H < 1 || !q || !lens || !out) return DSA_ERR_INVALID_ARG;
  if ((int64_t)B * T > (int64_t)1 << 24 || H > DSA_MAX_HEADS) return DSA_ERR_UNSUPPORTED;
  if (int rc = check_pool(kv_pages, page_table, ld_table, max_pages, page_size, n_pages)) return rc;
  if (out_dtype != DSA_BF16 && out_dtype != DSA_F32) return DSA_ERR_INVALID_ARG;
  if (!(scale == scale) || !is_aligned16(q) || !is_aligned16(out)) return DSA_ERR_INVALID_ARG;
  const size_t need = dsa_paged_mla_workspace_size(B, T, H);
  if (need > 0 && (!workspace || ws_bytes < need || !is_aligned16(workspace))) return DSA_ERR_WORKSPACE;
  const PagePool pool{page_table, ld_table, n_pages, max_pages, page_size};
  constexpr int kSmem = kTile * kRowPad * 2 + kHeads * kDQK * 4;
  static PerDeviceOnce attr;
  if (attr.run([] {
        return cudaFuncSetAttribute(paged_mla_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
      }) != cudaSuccess)
    return DSA_ERR_CUDA;
  const unsigned grid = (unsigned)B * T * ((H + kHeads - 1) / kHeads);
  const cudaError_t e = launch_pdl(paged_mla_kernel, dim3(grid), dim3(256), kSmem, reinterpret_cast<cudaStream_t>(stream),
                                   reinterpret_cast<const __nv_bfloat16*>(q),
                                   reinterpret_cast<const __nv_bfloat16*>(kv_pages), pool, lens, T, H,
                                   scale * 1.4426950408889634f, out, out_dtype == DSA_BF16 ? 1 : 0, lse, dev_status);
  return e == cudaSuccess ? DSA_OK : DSA_ERR_CUDA;
}

}  // extern "C"
