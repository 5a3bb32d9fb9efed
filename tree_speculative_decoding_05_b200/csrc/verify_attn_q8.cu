// verify_attn_q8.cu — tree-verify MLA-absorb attention over the paged 8-bit cache.
//
// For request b with prefix P, node i, head h and cache rows j < P + Q (value
// c_j = scales[page(j)] * c_kv8[j], and k_j likewise):
//   s_j = softmax_scale * (q_lat . c_j + q_rope . k_j)   over visible j
//   out = sum_j softmax(s)_j c_j,   lse = ln sum_j exp(s_j)
//
// One CTA per (request, node): pages are widened to fp32 in shared memory one at a
// time and every thread keeps one latent column of all 64 heads' outputs.  Bound by
// fp32 arithmetic.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "ddt.h"
#include "ddt_internal.h"

namespace ddt {

namespace {

constexpr int kPage = DDT_PAGE_ROWS, kH = DDT_NUM_HEADS, kDL = DDT_D_LATENT;
constexpr int kD = DDT_D_LATENT + DDT_D_ROPE;
constexpr int kThreads = 512;
constexpr int kKeyPitch = kD + 1;  // floats; odd, so that a column's rows lie in all banks
constexpr int kSmemBytes = kPage * kKeyPitch * 4 + kH * kPage * 4 + 3 * kH * 4;

__global__ void __launch_bounds__(kThreads) verify_attn_q8_kernel(const ddt_attn_q8_args a) {
  extern __shared__ float smem[];
  float* key = smem;                      // [64][kKeyPitch]
  float* w = key + kPage * kKeyPitch;     // [64 heads][64 keys]
  float* row_max = w + kH * kPage;        // [64]
  float* row_sum = row_max + kH;
  float* row_fac = row_sum + kH;
  const int b = blockIdx.x / a.q_len, node = blockIdx.x % a.q_len, t = threadIdx.x;
  const ddt_q8_cache& c = a.cache;
  const int P = a.prefix_lens[b];
  const bool bad = P < 0 || static_cast<int64_t>(P) + a.q_len > static_cast<int64_t>(c.max_blocks) * kPage;
  const int T = P + a.q_len, n_blk = bad ? 0 : (T + kPage - 1) / kPage;
  const int32_t* table = c.block_table + static_cast<int64_t>(b) * c.max_blocks;
  int odd = 0;
  for (int k = t; k < n_blk; k += kThreads) odd |= table[k] < 0 || table[k] >= c.num_pages;
  odd = __syncthreads_or(odd);
  if (a.status && node == 0 && t == 0)
    a.status[b] = bad ? DDT_REQ_BAD_PREFIX : odd ? DDT_REQ_BAD_INDEX : DDT_REQ_OK;
  if (bad) return;
  const int64_t row0 = (static_cast<int64_t>(b) * a.q_len + node) * kH;
  const __nv_bfloat16* q_lat = static_cast<const __nv_bfloat16*>(a.q_lat) + row0 * kDL;
  const __nv_bfloat16* q_rope = static_cast<const __nv_bfloat16*>(a.q_rope) + row0 * DDT_D_ROPE;
  const int W = (a.q_len + 63) / 64;
  const uint64_t* mask = a.mask + (static_cast<int64_t>(b) * a.q_len + node) * W;
  float acc[kH];
#pragma unroll
  for (int h = 0; h < kH; ++h) acc[h] = 0.f;
  if (t < kH) {
    row_max[t] = -INFINITY;
    row_sum[t] = 0.f;
  }
  for (int blk = 0; blk < n_blk; ++blk) {
    const int page = table[blk];
    const int n = T - blk * kPage < kPage ? T - blk * kPage : kPage;
    const bool ok = page >= 0 && page < c.num_pages;
    const float scale = ok ? c.scales[page] : 0.f;
    __syncthreads();
    for (int idx = t; idx < kPage * kD; idx += kThreads) {
      const int r = idx / kD, d = idx % kD;
      float v = 0.f;
      if (ok && r < n) {
        const uint8_t* p = d < kDL ? static_cast<const uint8_t*>(c.c_kv) + page * c.ckv_page_stride +
                                         r * c.ckv_row_stride + d
                                   : static_cast<const uint8_t*>(c.k_rope) +
                                         page * c.kr_page_stride + r * c.kr_row_stride + d - kDL;
        v = __half2float(__half(__nv_cvt_fp8_to_halfraw(*p, __NV_E4M3))) * scale;
      }
      key[r * kKeyPitch + d] = v;
    }
    __syncthreads();
    // scores: thread -> key t % 64, heads t / 64 + 8 i
    const int j = t % kPage, pos = blk * kPage + j;
    const bool vis = pos < P || (pos < T && ((mask[(pos - P) / 64] >> ((pos - P) & 63)) & 1));
    for (int h = t / kPage; h < kH; h += kThreads / kPage) {
      float s = 0.f;
      for (int d = 0; d < kDL; ++d) s += __bfloat162float(q_lat[h * kDL + d]) * key[j * kKeyPitch + d];
      for (int d = 0; d < DDT_D_ROPE; ++d)
        s += __bfloat162float(q_rope[h * DDT_D_ROPE + d]) * key[j * kKeyPitch + kDL + d];
      w[h * kPage + j] = vis ? s * a.softmax_scale : -INFINITY;
    }
    __syncthreads();
    if (t < kH) {
      float top = row_max[t];
      for (int k = 0; k < kPage; ++k) top = fmaxf(top, w[t * kPage + k]);
      const float use = top == -INFINITY ? 0.f : top;
      const float fac = expf(row_max[t] - use);
      float sum = row_sum[t] * fac;
      for (int k = 0; k < kPage; ++k) {
        const float e = expf(w[t * kPage + k] - use);
        w[t * kPage + k] = e;
        sum += e;
      }
      row_max[t] = top;
      row_sum[t] = sum;
      row_fac[t] = fac;
    }
    __syncthreads();
#pragma unroll
    for (int h = 0; h < kH; ++h) {
      float o = acc[h] * row_fac[h];
      for (int k = 0; k < n; ++k) o += w[h * kPage + k] * key[k * kKeyPitch + t];
      acc[h] = o;
    }
  }
  __syncthreads();
  __nv_bfloat16* out = static_cast<__nv_bfloat16*>(a.out) + row0 * kDL;
#pragma unroll
  for (int h = 0; h < kH; ++h)
    out[h * kDL + t] = __float2bfloat16(row_sum[h] == 0.f ? 0.f : acc[h] / row_sum[h]);
  if (a.lse && t < kH) a.lse[row0 + t] = row_sum[t] == 0.f ? -INFINITY : row_max[t] + logf(row_sum[t]);
}

}  // namespace

ddt_status launch_verify_attn_q8(const ddt_attn_q8_args& a, int, float*, float*,
                                 cudaStream_t stream) {
  if (ensure_smem_limit(reinterpret_cast<const void*>(verify_attn_q8_kernel), kSmemBytes, 6) !=
      cudaSuccess)
    return DDT_ERR_CUDA;
  verify_attn_q8_kernel<<<a.B * a.q_len, kThreads, kSmemBytes, stream>>>(a);
  return cudaGetLastError() == cudaSuccess ? DDT_OK : DDT_ERR_CUDA;
}

}  // namespace ddt
