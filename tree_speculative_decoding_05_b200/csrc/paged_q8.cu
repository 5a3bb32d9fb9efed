// paged_q8.cu — the paged 8-bit latent cache: block tables and slot maps from the
// requests' lengths, the quantising write, and the compaction of accepted rows.
// (The attention over it is in verify_attn_q8.cu.)
//
// A page is 64 rows of 512 + 64 e4m3 values under one power-of-two fp32 scale.
// With a power of two, x / scale and a change of scale are exact shifts of the
// exponent, so the only rounding is the one to e4m3's three mantissa bits
// (relative 2^-4) or, below its normal range, to steps of 2^-9.
//
// Data-dependent errors go to the per-request status; no index read from device
// memory is followed before it has been checked.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include <climits>
#include <cstdint>

#include "ddt.h"
#include "ddt_internal.h"
#include "q8_common.cuh"

namespace ddt {

namespace {

constexpr int kPage = DDT_PAGE_ROWS;
constexpr int kMinExp = -40;                     // smallest exponent of a scale
constexpr int kLatVec8 = DDT_D_LATENT / 16;      // 16-byte vectors of an e4m3 latent row (32)
constexpr int kRowVec8 = kLatVec8 + DDT_D_ROPE / 16;  // and of a whole row (36)
constexpr int kLatVec16 = DDT_D_LATENT / 8;      // 16-byte vectors of a bf16 latent row (64)
constexpr int kRowVec16 = kLatVec16 + DDT_D_ROPE / 8;  // and of a whole row (72)

// A request's rows: how many there are to be, behind which prefix.
struct Span {
  int prefix, rows, status;
  int64_t first;  // index of its first row among all requests' rows
};

__device__ __forceinline__ Span load_span(const int32_t* prefix_lens, const int32_t* row_start,
                                          int b, int q_len, int max_blocks) {
  Span s;
  s.prefix = prefix_lens[b];
  s.first = row_start ? row_start[b] : static_cast<int64_t>(b) * q_len;
  const int64_t n = row_start ? static_cast<int64_t>(row_start[b + 1]) - s.first : q_len;
  s.status = DDT_REQ_OK;
  if (n < 0 || s.first < 0) s.status = DDT_REQ_BAD_LENGTH;
  else if (s.prefix < 0 || s.prefix + n > static_cast<int64_t>(max_blocks) * kPage)
    s.status = DDT_REQ_BAD_PREFIX;
  s.rows = s.status == DDT_REQ_OK ? static_cast<int>(n) : 0;
  return s;
}

__device__ __forceinline__ int cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return static_cast<int>(r);
}

// ---------------------------------------------------------------------------
// Page plan.  The state (tables, counts, the stack) is small and every request's
// place on the stack depends on all requests before it, so each CTA scans the
// requests for itself, 1024 at a time, and the CTAs of one cluster share the page
// numbers to be moved; nothing depends on the order in which threads run.
// Latency-bound: a handful of dependent loads, two block scans and the page numbers
// themselves (64 requests x 33 rows: 5 us; 1000 prompts of 1 to 2048 rows, 16000 pages
// and a million slots: 12.5 us a call, 24 us with one CTA).
// ---------------------------------------------------------------------------
constexpr int kPlanThreads = 1024;
constexpr int kPlanCtas = 8;  // of a large plan
constexpr int kSlotThreads = 256;
constexpr int kSlotRows = 4 * kSlotThreads;  // rows of one CTA at a time

// Inclusive scan over the CTA; `total` is the sum.  s_warp: 33 entries.
__device__ __forceinline__ int64_t block_scan(int64_t v, int64_t* s_warp, int64_t& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const int64_t u = __shfl_up_sync(0xffffffffu, v, off);
    if (lane >= off) v += u;
  }
  if (lane == 31) s_warp[warp] = v;
  __syncthreads();
  if (warp == 0) {
    int64_t w = s_warp[lane];
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const int64_t u = __shfl_up_sync(0xffffffffu, w, off);
      if (lane >= off) w += u;
    }
    s_warp[lane] = w;
  }
  __syncthreads();
  total = s_warp[31];
  if (warp > 0) v += s_warp[warp - 1];
  __syncthreads();  // s_warp may be written again
  return v;
}

// The slot of one row, or -1 where its request was not served or its page number
// is not one.
__device__ __forceinline__ int64_t slot_of(const Span& s, int64_t i, int n_blocks, int num_pages,
                                           int max_blocks, const int32_t* table_row) {
  const int64_t pos = s.prefix + i;
  const int64_t need = (static_cast<int64_t>(s.prefix) + s.rows + kPage - 1) / kPage;
  if (s.status != DDT_REQ_OK || n_blocks > max_blocks || need > n_blocks) return -1;
  const int page = table_row[pos / kPage];
  return page < 0 || page >= num_pages ? -1 : static_cast<int64_t>(page) * kPage + pos % kPage;
}

// Slots of rows [r0, r1) (all -1 with `refused`), row r0 + t + i * threads by thread t.
// A row's request is found by bisection, unless it is that of the thread's row before.
__device__ void write_slots(bool refused, const int32_t* prefix_lens, const int32_t* row_start,
                            int B, int q_len, int64_t r0, int64_t r1, int num_pages, int max_blocks,
                            const int32_t* block_table, const int32_t* n_blocks, int64_t* slots,
                            int t, int threads) {
  if (!row_start && q_len == 0) return;
  int b = 0;
  for (int64_t r = r0 + t; r < r1; r += threads) {
    if (row_start) {
      if (row_start[b + 1] <= r) {
        int hi = B;  // the last request with row_start[b] <= r
        while (hi - b > 1) {
          const int mid = (b + hi) >> 1;
          if (row_start[mid] <= r) b = mid;
          else hi = mid;
        }
      }
    } else {
      if (r >= static_cast<int64_t>(B) * q_len) return;
      b = r <= UINT_MAX ? static_cast<int>(static_cast<uint32_t>(r) / static_cast<uint32_t>(q_len))
                        : static_cast<int>(r / q_len);
    }
    const Span s = load_span(prefix_lens, row_start, b, q_len, max_blocks);
    const int64_t i = r - s.first;
    if (i < 0 || (row_start && r >= row_start[b + 1])) continue;  // no request's row
    slots[r] = refused ? -1
                       : slot_of(s, i, n_blocks[b], num_pages, max_blocks,
                                 block_table + static_cast<int64_t>(b) * max_blocks);
  }
}

// kCtas CTAs in one cluster (or one alone).  Every CTA derives the same plan from the
// state as it was; the state is changed only behind a cluster barrier.
template <int kCtas>
__global__ void __launch_bounds__(kPlanThreads) kv_pages_kernel(
    const int32_t* __restrict__ prefix_lens, const int32_t* __restrict__ row_start, int B,
    int q_len, int64_t slot_rows, int num_pages, int max_blocks, int32_t* block_table,
    int32_t* n_blocks, int32_t* free_pages, int32_t* n_free, int64_t* slots, int32_t* status) {
  __shared__ int64_t s_warp[32];
  __shared__ int64_t s_upto[kPlanThreads];  // pages of the chunk's requests up to and with each
  __shared__ int s_from[kPlanThreads];      // table entry at which a request's pages begin
  const int t = threadIdx.x;
  const int rank = kCtas > 1 ? cluster_rank() : 0;
  const bool one_chunk = B <= kPlanThreads;
  auto barrier = [] {  // all CTAs have come here; memory as the others left it
    if constexpr (kCtas > 1) {
      cluster_arrive();
      cluster_wait();
    } else {
      __syncthreads();
    }
  };

  struct Request {
    int held, need, status;
  } q = {0, 0, DDT_REQ_OK};
  auto load = [&](int b) {
    q = {0, 0, DDT_REQ_OK};
    if (b >= B) return;
    const Span s = load_span(prefix_lens, row_start, b, q_len, max_blocks);
    q.held = n_blocks[b];
    q.status = s.status;
    if (q.status == DDT_REQ_OK && (q.held < 0 || q.held > max_blocks)) q.status = DDT_REQ_BAD_INDEX;
    if (q.status != DDT_REQ_OK) q.held = 0;  // neither gives nor takes
    else q.need = (s.prefix + s.rows + kPage - 1) / kPage;
  };
  // Runs over the chunk's moving pages, the threads of all CTAs together: `amount`
  // pages of each thread's request, from table entry `from` on; f(request, table entry,
  // place).
  auto move_pages = [&](int b0, int amount, int from, auto f) -> int64_t {
    int64_t total;
    const int64_t upto = block_scan(amount, s_warp, total);
    if (total == 0) return 0;
    s_upto[t] = upto;
    s_from[t] = from;
    __syncthreads();
    for (int64_t k = static_cast<int64_t>(rank) * kPlanThreads + t; k < total;
         k += kCtas * kPlanThreads) {
      int lo = 0, hi = kPlanThreads - 1;  // first request with s_upto > k
      while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (s_upto[mid] > k) hi = mid;
        else lo = mid + 1;
      }
      const int64_t j = k - (lo ? s_upto[lo - 1] : 0);
      f(b0 + lo, s_from[lo] + static_cast<int>(j), k);
    }
    __syncthreads();
    return total;
  };

  const int free0 = *n_free;
  // 1. how many pages come back in all
  int64_t back = 0;
  for (int b0 = 0; b0 < B; b0 += kPlanThreads) {
    load(b0 + t);
    const int mine = q.held > q.need ? q.held - q.need : 0;
    if (__syncthreads_or(mine)) {
      int64_t total;
      block_scan(mine, s_warp, total);
      back += total;
    }
  }
  const int64_t free1 = free0 + back;
  const bool refused = free0 < 0 || free1 > num_pages;  // no such state: change nothing
  // 2. they go onto the stack, the first request's first page on top
  if (back > 0 && !refused) {
    int64_t done = 0;
    for (int b0 = 0; b0 < B; b0 += kPlanThreads) {
      if (!one_chunk) load(b0 + t);
      const int mine = q.held > q.need ? q.held - q.need : 0;
      done += move_pages(b0, mine, q.need, [&](int b, int entry, int64_t k) {
        int32_t* e = block_table + static_cast<int64_t>(b) * max_blocks + entry;
        free_pages[free1 - 1 - done - k] = *e;
        *e = -1;
      });
    }
    barrier();
  }
  // 3. pages are taken from the top, request by request
  int64_t wanted = 0, taken = 0;
  for (int b0 = 0; b0 < B; b0 += kPlanThreads) {
    if (!one_chunk) load(b0 + t);
    const int mine = q.need > q.held ? q.need - q.held : 0;
    int st = refused ? DDT_REQ_BAD_INDEX : q.status;
    if (__syncthreads_or(mine) && !refused) {
      int64_t total;
      const int64_t upto = wanted + block_scan(mine, s_warp, total);
      const bool served = upto <= free1;
      if (mine > 0 && !served) st = DDT_REQ_NO_PAGES;
      // the served ones are those before the first that is not, so their places
      // on the stack follow one another
      const int64_t base = wanted;
      taken += move_pages(b0, served ? mine : 0, q.held, [&](int b, int entry, int64_t k) {
        block_table[static_cast<int64_t>(b) * max_blocks + entry] = free_pages[free1 - 1 - base - k];
      });
      wanted += total;
    }
    if constexpr (kCtas > 1) barrier();  // every CTA has read this chunk's counts
    const int b = b0 + t;
    if (b < B && rank == 0) {
      if (st == DDT_REQ_OK && q.need != q.held) n_blocks[b] = q.need;
      if (status) status[b] = st;
    }
  }
  if (rank == 0 && t == 0 && !refused && free1 - taken != free0)
    *n_free = static_cast<int>(free1 - taken);
  // 4. not too many rows: their slots too
  if (slots && slot_rows > 0) {
    barrier();
    const int64_t per = (slot_rows + kCtas - 1) / kCtas, r0 = rank * per;
    write_slots(refused, prefix_lens, row_start, B, q_len, r0,
                r0 + per < slot_rows ? r0 + per : slot_rows, num_pages, max_blocks, block_table,
                n_blocks, slots, t, kPlanThreads);
  }
}

__global__ void __launch_bounds__(kSlotThreads) kv_slots_kernel(
    const int32_t* __restrict__ prefix_lens, const int32_t* __restrict__ row_start, int B,
    int q_len, int64_t n_rows, int num_pages, int max_blocks,
    const int32_t* __restrict__ block_table, const int32_t* __restrict__ n_blocks,
    const int32_t* __restrict__ n_free, int64_t* __restrict__ slots) {
  // After a plan no request holds more than it needs, and the stack's height is in
  // range; where that is not so, the plan refused the state as a whole.
  int refused = *n_free < 0 || *n_free > num_pages;
  for (int b = threadIdx.x; b < B; b += kSlotThreads) {
    const Span s = load_span(prefix_lens, row_start, b, q_len, max_blocks);
    const int held = n_blocks[b];
    refused |= s.status == DDT_REQ_OK && held <= max_blocks &&
               held > (s.prefix + s.rows + kPage - 1) / kPage;
  }
  refused = __syncthreads_or(refused);
  for (int64_t r0 = static_cast<int64_t>(blockIdx.x) * kSlotRows; r0 < n_rows;
       r0 += static_cast<int64_t>(gridDim.x) * kSlotRows)
    write_slots(refused, prefix_lens, row_start, B, q_len, r0,
                r0 + kSlotRows < n_rows ? r0 + kSlotRows : n_rows, num_pages, max_blocks,
                block_table, n_blocks, slots, threadIdx.x, kSlotThreads);
}

// ---------------------------------------------------------------------------
// e4m3
// ---------------------------------------------------------------------------
__device__ __forceinline__ bool scale_ok(float s) { return s > 0.f && s <= 3.402823466e38f; }

// Two floats to two e4m3 bytes (round to nearest even, saturating, NaN kept).
__device__ __forceinline__ uint32_t to_e4m3x2(float lo, float hi) {
  return __nv_cvt_float2_to_fp8x2(make_float2(lo, hi), __NV_SATFINITE, __NV_E4M3);
}

// Four e4m3 bytes times `ratio`, rounded again.
__device__ __forceinline__ uint32_t rescale4(uint32_t v, float ratio) {
  const float2 a = __half22float2(__half2(__nv_cvt_fp8x2_to_halfraw2(v & 0xffffu, __NV_E4M3)));
  const float2 b = __half22float2(__half2(__nv_cvt_fp8x2_to_halfraw2(v >> 16, __NV_E4M3)));
  return to_e4m3x2(a.x * ratio, a.y * ratio) | (to_e4m3x2(b.x * ratio, b.y * ratio) << 16);
}

__device__ __forceinline__ uint4 rescale16(uint4 v, float ratio) {
  return make_uint4(rescale4(v.x, ratio), rescale4(v.y, ratio), rescale4(v.z, ratio),
                    rescale4(v.w, ratio));
}

// Address of vector v (16 bytes; latent, then rope) of row 0 of a page, and the distance
// of the rows there (host-checked to fit).
__device__ __forceinline__ uint8_t* page_vec(const ddt_q8_cache& c, int64_t page, int v) {
  return v < kLatVec8 ? static_cast<uint8_t*>(c.c_kv) + page * c.ckv_page_stride + 16 * v
                      : static_cast<uint8_t*>(c.k_rope) + page * c.kr_page_stride +
                            16 * (v - kLatVec8);
}
__device__ __forceinline__ int row_step(const ddt_q8_cache& c, int v) {
  return static_cast<int>(v < kLatVec8 ? c.ckv_row_stride : c.kr_row_stride);
}

// ---------------------------------------------------------------------------
// Quantising write.  One CTA per page that a request's rows reach: it loads the
// page's new rows (at most 64 x 1152 bytes of bf16) into registers, all loads in
// flight together, takes their largest magnitude, and stores them at the scale
// that follows: one pass over the data, bound by memory for prompts and by the
// latency of load, reduction and store for a step's rows.  No page needs another's
// result.  Measured: 24 prompts of 1 to 4001 rows (83 MB) 22.3 us over data outside the
// L2, 3.7 TB/s = 0.57 of the measured HBM rate, the two pages that fit an SM's registers
// taking turns at loading, the maximum and storing; 17.3 us repeated on one set of
// buffers, which the L2 then holds (three pages staged in shared memory: 2 us slower
// there).  64 requests x 33 rows: 7.7 us with live rows rescaled, 5.1 without, 4.3
// repeated.
// ---------------------------------------------------------------------------
// The CTAs of a request that reaches few pages (kCluster, at most kMaxWriteCluster) are
// one cluster: the first one sets the status before the cluster's barrier, the others
// raise it behind it if they met a value that is not finite.  Those of a long prompt
// raise a status that was cleared before the launch.
constexpr int kWriteThreads = 512;
constexpr int kLatRows = kWriteThreads / kLatVec16;   // latent rows of one round (8)
constexpr int kLatPerThread = kPage / kLatRows;       // 8
constexpr int kVecPerThread = kLatPerThread + 1;
static_assert(kWriteThreads == kPage * (kRowVec16 - kLatVec16), "one rope vector per thread");
constexpr int kMaxWriteCluster = 4;

// Vectors of the page's new rows that a thread holds: eight of latent values, vector
// t % 64 of rows t / 64 + 8 i, so that a thread's addresses lie one distance apart, and
// one of rope values, vector t % 8 of row t / 8.
struct PageRows {
  uint4 x[kVecPerThread];
};

__device__ __forceinline__ void load_page_rows(PageRows& p, int64_t src, int n,
                                               const uint16_t* rows_ckv,
                                               const uint16_t* rows_krope) {
  const int t = threadIdx.x;
  const uint4* lat = reinterpret_cast<const uint4*>(rows_ckv) + src * kLatVec16 + t;
  const uint4* rope = reinterpret_cast<const uint4*>(rows_krope) + src * (kRowVec16 - kLatVec16) + t;
#pragma unroll
  for (int i = 0; i < kLatPerThread; ++i) {
    p.x[i] = make_uint4(0, 0, 0, 0);
    if (t / kLatVec16 + i * kLatRows < n) p.x[i] = lat[i * kWriteThreads];
  }
  p.x[kLatPerThread] = make_uint4(0, 0, 0, 0);
  if (t / (kRowVec16 - kLatVec16) < n) p.x[kLatPerThread] = *rope;
}

// The n rows to page rows off .. off + n - 1, by the whole CTA; returns whether a value
// was not finite.
__device__ __forceinline__ int write_page(const ddt_q8_cache& c, PageRows& rows, int page, int off,
                                          int n, uint32_t* s_max) {
  uint4 (&x)[kVecPerThread] = rows.x;
  const int t = threadIdx.x;
  const float old_scale = c.scales[page];
  // Largest magnitude as bf16 bits, two at a time (NaN when there is one).
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < kVecPerThread; ++i) {
    m = max_abs_bf16x2(m, x[i].x);
    m = max_abs_bf16x2(m, x[i].y);
    m = max_abs_bf16x2(m, x[i].z);
    m = max_abs_bf16x2(m, x[i].w);
  }
  uint32_t top = max_of_halves(m);
  // Not a finite value among them: NaN becomes 0, an infinity the largest finite
  // bf16 (which saturates), and the maximum is taken again over finite values.
  const bool odd = top >= 0x7f80u;
  if (odd) {
    top = 0;
    auto fix = [&](uint32_t h) -> uint32_t {
      const uint32_t mag = h & 0x7fffu;
      if (mag > 0x7f80u) return 0;
      if (mag == 0x7f80u) return (h & 0x8000u) | 0x7f7fu;
      top = max(top, mag);
      return h;
    };
#pragma unroll
    for (int i = 0; i < kVecPerThread; ++i) {
      uint32_t w[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
#pragma unroll
      for (int j = 0; j < 4; ++j) w[j] = fix(w[j] & 0xffffu) | (fix(w[j] >> 16) << 16);
      x[i] = make_uint4(w[0], w[1], w[2], w[3]);
    }
  }
  top = __reduce_max_sync(0xffffffffu, top);
  if ((t & 31) == 0) s_max[t >> 5] = top;
  const int any_odd = __syncthreads_or(odd);
#pragma unroll
  for (int i = 0; i < kWriteThreads / 32; ++i) top = max(top, s_max[i]);
  const int fit = e4m3_exponent(top), e = fit < kMinExp ? kMinExp : fit;
  float scale = pow2f(e), inv = pow2f(-e);
  if (off > 0 && scale_ok(old_scale) && old_scale >= scale) {
    scale = old_scale;
    inv = 1.f / old_scale;
  } else if (off > 0) {
    // The live rows before these move to the larger scale.
    const float ratio = scale_ok(old_scale) ? old_scale * inv : 0.f;
    for (int idx = t; idx < off * kRowVec8; idx += kWriteThreads) {
      const int r = idx / kRowVec8, v = idx - r * kRowVec8;
      uint4* p = reinterpret_cast<uint4*>(page_vec(c, page, v) + static_cast<int64_t>(r) * row_step(c, v));
      *p = rescale16(*p, ratio);
    }
  }
  // bf16 vector v holds half of e4m3 vector v / 2
  auto store = [&](const uint4& a, uint8_t* at) {
    const uint32_t w[4] = {a.x, a.y, a.z, a.w};
    uint32_t h[4];
#pragma unroll
    for (int j = 0; j < 4; ++j)
      h[j] = to_e4m3x2(__uint_as_float(w[j] << 16) * inv, __uint_as_float(w[j] & 0xffff0000u) * inv);
    *reinterpret_cast<uint2*>(at) = make_uint2(__byte_perm(h[0], h[1], 0x5410), __byte_perm(h[2], h[3], 0x5410));
  };
  const int lat_step = row_step(c, 0);
  uint8_t* lat = page_vec(c, page, 0) + 8 * (t % kLatVec16) +
                 static_cast<int64_t>(off + t / kLatVec16) * lat_step;
#pragma unroll
  for (int i = 0; i < kLatPerThread; ++i)
    if (t / kLatVec16 + i * kLatRows < n) store(x[i], lat + static_cast<int64_t>(i * kLatRows) * lat_step);
  constexpr int kRopeVec16 = kRowVec16 - kLatVec16;
  if (t / kRopeVec16 < n)
    store(x[kLatPerThread], page_vec(c, page, kLatVec8) + 8 * (t % kRopeVec16) +
                                static_cast<int64_t>(off + t / kRopeVec16) * row_step(c, kLatVec8));
  if (t == 0 && scale != old_scale) c.scales[page] = scale;
  return any_odd;
}

// The write starts while this runs and waits for its end before it touches a status, so
// the statuses are cleared behind the pages' loads (24 prompts, repeated: 20.4 us after a
// memset, 17.1 so; the plan's slots and the attention's merge gained nothing from it).
__global__ void kv_clear_status_kernel(int32_t* status, int B) {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int64_t b = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x;
  if (b < B) status[b] = DDT_REQ_OK;
}

__device__ __forceinline__ void await_clear() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

template <bool kCluster>
__global__ void __launch_bounds__(kWriteThreads, 1024 / kWriteThreads) kv_write_q8_kernel(
    const ddt_q8_cache c, const int32_t* __restrict__ prefix_lens,
    const int32_t* __restrict__ row_start, int q_len, int max_rows, int64_t n_rows,
    const uint16_t* __restrict__ rows_ckv, const uint16_t* __restrict__ rows_krope,
    int32_t* __restrict__ status, int pages_per_request) {
  __shared__ uint32_t s_max[kWriteThreads / 32];
  const int b = blockIdx.x / pages_per_request;
  const int k = blockIdx.x % pages_per_request;
  const int t = threadIdx.x;
  Span s = load_span(prefix_lens, row_start, b, q_len, c.max_blocks);
  if (s.status == DDT_REQ_OK && (s.rows > max_rows || s.first + s.rows > n_rows))
    s.status = DDT_REQ_BAD_LENGTH;
  const int blk0 = s.prefix / kPage;
  // This page's rows: cache rows [lo, hi).
  const int64_t page0 = static_cast<int64_t>(blk0 + k) * kPage;
  const int64_t lo = k == 0 ? s.prefix : page0;
  const int64_t end = static_cast<int64_t>(s.prefix) + s.rows;
  const int64_t hi = end < page0 + kPage ? end : page0 + kPage;
  if (!kCluster && k > 0 && lo >= hi) return;
  // The rows are on their way while the page numbers are looked at: every page of the
  // request's rows has to be one before any is written.
  PageRows rows;
  const int n = s.status == DDT_REQ_OK && lo < hi ? static_cast<int>(hi - lo) : 0;
  load_page_rows(rows, s.first + (lo - s.prefix), n, rows_ckv, rows_krope);
  const int32_t* table = c.block_table + static_cast<int64_t>(b) * c.max_blocks;
  int bad = 0;
  if (s.status == DDT_REQ_OK && s.rows > 0) {
    const int last = (s.prefix + s.rows - 1) / kPage;
    for (int blk = blk0 + t; blk <= last; blk += kWriteThreads) {
      const int page = table[blk];
      bad |= page < 0 || page >= c.num_pages;
    }
  }
  if (__syncthreads_or(bad)) s.status = DDT_REQ_BAD_INDEX;
  if (s.status != DDT_REQ_OK) {
    if (!kCluster) await_clear();
    if (k == 0 && t == 0 && status) status[b] = s.status;
    return;
  }
  int any_odd = 0;
  if (n > 0) any_odd = write_page(c, rows, table[blk0 + k], static_cast<int>(lo - page0), n, s_max);
  if (!kCluster) await_clear();
  if (!status) return;
  if (t == 0 && k == 0 && (kCluster || pages_per_request == 1))
    status[b] = any_odd ? DDT_REQ_NOT_FINITE : DDT_REQ_OK;
  if constexpr (kCluster) {
    cluster_arrive();
    cluster_wait();
  }
  if (t == 0 && k > 0 && any_odd) atomicMax(&status[b], DDT_REQ_NOT_FINITE);
  if (t == 0 && k == 0 && !kCluster && pages_per_request > 1 && any_odd)
    atomicMax(&status[b], DDT_REQ_NOT_FINITE);
}

// ---------------------------------------------------------------------------
// Compaction.  One CTA per request: the moving rows (576 bytes each, at most 72 KB) are
// all read into shared memory before any byte is written, so the gather is race-free
// for any path.  The scales of the at most three pages that rows move into are known
// from the pages' present scales alone, without a look at the values: a scale only ever
// rises, to the largest among the rows that come in.  Measured: 1024 requests, 62 rows
// moving in each (74 MB): 29 us over data outside the L2 where scales rise and the rest of
// those pages is rescaled, 21.6 us (3.4 TB/s = 0.52 of the measured HBM rate) where none
// does, 16.1 us repeated on one set of buffers, which the L2 then holds.  64 requests x 8
// rows: 9.7, 4.1 and 3.0 us (launch, then four dependent loads).  Three column slices of a
// request, clustered so that one may store the scales: 20 against 16 us, for the barriers'
// sake.
// ---------------------------------------------------------------------------
constexpr int kMoveThreads = 256;
constexpr int kMoveRows = kMoveThreads / kRowVec8;  // 7 rows at a time
constexpr int kMaxTreePages = (DDT_MAX_Q_LEN + 2 * (kPage - 1)) / kPage;  // 3
static_assert(DDT_MAX_Q_LEN <= kMoveThreads, "one thread per path entry");

__device__ __forceinline__ void copy16_async(void* smem_dst, const void* src) {
  const uint32_t d = static_cast<uint32_t>(__cvta_generic_to_shared(smem_dst));
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(d), "l"(src) : "memory");
}

__global__ void __launch_bounds__(kMoveThreads) kv_compact_q8_kernel(
    const ddt_q8_cache c, const int32_t* prefix_lens, const int32_t* __restrict__ path,
    const int32_t* __restrict__ accept_len, int q_len, int32_t* new_prefix_lens,
    int32_t* __restrict__ status) {
  extern __shared__ uint4 s_rows[];  // [q_len][kRowVec8]
  __shared__ int s_keep[DDT_MAX_Q_LEN];
  __shared__ int s_page[kMaxTreePages];
  __shared__ float s_old[kMaxTreePages];
  __shared__ int s_new[kMaxTreePages];  // bits of a positive float: ordered as integers
  const int b = blockIdx.x, t = threadIdx.x;
  const int P = prefix_lens[b];
  const int alen = accept_len[b];
  const int keep = t < q_len ? path[static_cast<int64_t>(b) * q_len + t] : 0;
  int st = DDT_REQ_OK;
  if (alen < 1 || alen > q_len) st = DDT_REQ_BAD_LENGTH;
  else if (P < 0 || static_cast<int64_t>(P) + q_len > static_cast<int64_t>(c.max_blocks) * kPage)
    st = DDT_REQ_BAD_PREFIX;
  int bad = 0;
  const int blk0 = P / kPage, o0 = P % kPage;
  if (st == DDT_REQ_OK) {
    const int n_blk = (o0 + q_len - 1) / kPage + 1;
    if (t < n_blk) {
      const int page = c.block_table[static_cast<int64_t>(b) * c.max_blocks + blk0 + t];
      bad = page < 0 || page >= c.num_pages;
      s_page[t] = page;
    }
    if (t < q_len) s_keep[t] = keep;
    bad |= t < alen && (keep < 0 || keep >= q_len);
  }
  if (__syncthreads_or(bad)) st = DDT_REQ_BAD_INDEX;
  if (st != DDT_REQ_OK) {
    if (t == 0) {
      if (status) status[b] = st;
      if (new_prefix_lens) new_prefix_lens[b] = P;
    }
    return;
  }
  // A thread has one vector of every kMoveRows-th row.
  const int v = t % kRowVec8;
  const int64_t step = row_step(c, v);
  uint8_t* at[kMaxTreePages];
#pragma unroll
  for (int g = 0; g < kMaxTreePages; ++g)
    at[g] = page_vec(c, g <= (o0 + q_len - 1) / kPage ? s_page[g] : 0, v);
  auto row = [&](int o) {  // of the tree block's pages
    uint8_t* p = o < kPage ? at[0] : o < 2 * kPage ? at[1] : at[2];
    return reinterpret_cast<uint4*>(p + (o % kPage) * step);
  };
  const int first = t < kMoveRows * kRowVec8 ? t / kRowVec8 : DDT_MAX_Q_LEN;  // no row
  // All moving rows into shared memory.
  for (int i = first; i < alen; i += kMoveRows) {
    const int from = s_keep[i];
    if (from != i) copy16_async(&s_rows[i * kRowVec8 + v], row(o0 + from));
  }
  if (t < (o0 + q_len - 1) / kPage + 1) {  // with the rows, the pages' scales
    const float sc = c.scales[s_page[t]];
    s_old[t] = scale_ok(sc) ? sc : 0.f;
    s_new[t] = __float_as_int(s_old[t]);
  }
  __syncthreads();
  if (t < alen)
    atomicMax(&s_new[(o0 + t) / kPage], __float_as_int(s_old[(o0 + keep) / kPage]));
  asm volatile("cp.async.wait_all;" ::: "memory");
  __syncthreads();
  // Pages whose scale rises: every row but those about to be written.
  const int last_blk = (o0 + alen - 1) / kPage;
  for (int g = 0; g <= last_blk; ++g) {
    const float now = __int_as_float(s_new[g]);
    if (now == s_old[g]) continue;
    const float ratio = s_old[g] / now;
    for (int r = first; r < kPage; r += kMoveRows) {
      const int i = g * kPage + r - o0;
      if (i >= 0 && i < alen && s_keep[i] != i) continue;
      uint4* p = row(g * kPage + r);
      *p = rescale16(*p, ratio);
    }
  }
  for (int i = first; i < alen; i += kMoveRows) {
    const int from = s_keep[i];
    if (from == i) continue;
    const float was = s_old[(o0 + from) / kPage], now = __int_as_float(s_new[(o0 + i) / kPage]);
    uint4 x = s_rows[i * kRowVec8 + v];
    if (was != now) x = rescale16(x, was / now);
    *row(o0 + i) = x;
  }
  if (t <= last_blk && __int_as_float(s_new[t]) != s_old[t])
    c.scales[s_page[t]] = __int_as_float(s_new[t]);
  if (t == 0) {
    if (status) status[b] = DDT_REQ_OK;
    if (new_prefix_lens) new_prefix_lens[b] = P + alen;
  }
}

}  // namespace

// ---------------------------------------------------------------------------
// Launchers
// ---------------------------------------------------------------------------
namespace {
// A launch in clusters of `cluster` CTAs, or (early) one that may start before the kernel
// ahead of it has ended, once that one's CTAs have said so.
template <typename... Params, typename... Args>
cudaError_t launch_with(void (*kernel)(Params...), unsigned ctas, int cluster, bool early,
                        int threads, cudaStream_t stream, Args... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(ctas);
  cfg.blockDim = dim3(threads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  cfg.attrs = attr;
  if (cluster > 1) {
    attr[cfg.numAttrs].id = cudaLaunchAttributeClusterDimension;
    attr[cfg.numAttrs].val.clusterDim.x = cluster;
    attr[cfg.numAttrs].val.clusterDim.y = 1;
    attr[cfg.numAttrs].val.clusterDim.z = 1;
    ++cfg.numAttrs;
  }
  if (early) {
    attr[cfg.numAttrs].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[cfg.numAttrs].val.programmaticStreamSerializationAllowed = 1;
    ++cfg.numAttrs;
  }
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, static_cast<Params>(args)...);
  return e != cudaSuccess ? e : cudaGetLastError();
}
}  // namespace

cudaError_t launch_kv_pages(const int32_t* prefix_lens, const int32_t* row_start, int B, int q_len,
                            int64_t n_rows, int num_pages, int max_blocks, int32_t* block_table,
                            int32_t* n_blocks, int32_t* free_pages, int32_t* n_free,
                            int64_t* slots, int32_t* status, cudaStream_t stream) {
  // Few rows: the planning CTAs write their slots; more get a launch of their own over
  // all SMs.  Few requests: one CTA plans.
  const bool fused = n_rows <= 4 * kPlanThreads;
  const int64_t slot_rows = fused ? n_rows : 0;
  cudaError_t e;
  if (B <= 256) {
    kv_pages_kernel<1><<<1, kPlanThreads, 0, stream>>>(
        prefix_lens, row_start, B, q_len, slot_rows, num_pages, max_blocks, block_table, n_blocks,
        free_pages, n_free, slots, status);
    e = cudaGetLastError();
  } else {
    e = launch_with(kv_pages_kernel<kPlanCtas>, kPlanCtas, kPlanCtas, false, kPlanThreads, stream,
                    prefix_lens, row_start, B, q_len, slot_rows, num_pages, max_blocks, block_table,
                    n_blocks, free_pages, n_free, slots, status);
  }
  if (e != cudaSuccess || !slots || fused) return e;
  const int64_t ctas = (n_rows + kSlotRows - 1) / kSlotRows;
  const int64_t most = 8ll * device_sm_count();
  kv_slots_kernel<<<static_cast<unsigned>(ctas < most ? ctas : most), kSlotThreads, 0, stream>>>(
      prefix_lens, row_start, B, q_len, n_rows, num_pages, max_blocks, block_table, n_blocks,
      n_free, slots);
  return cudaGetLastError();
}

cudaError_t launch_kv_write_q8(const ddt_q8_cache& c, const int32_t* prefix_lens,
                               const int32_t* row_start, int B, int q_len, int max_rows,
                               int64_t n_rows, const uint16_t* rows_ckv,
                               const uint16_t* rows_krope, int32_t* status, cudaStream_t stream) {
  // Rows of one request reach at most this many pages (one at least, so that the
  // status of an empty request is written).
  const int64_t pages = (static_cast<int64_t>(max_rows) + 2 * kPage - 2) / kPage;
  const int64_t per = pages > 0 ? pages : 1;
  const unsigned ctas = static_cast<unsigned>(per * B);
  if (per > 1 && per <= kMaxWriteCluster)
    return launch_with(kv_write_q8_kernel<true>, ctas, static_cast<int>(per), false, kWriteThreads,
                       stream, c, prefix_lens, row_start, q_len, max_rows, n_rows, rows_ckv,
                       rows_krope, status, static_cast<int>(per));
  // The statuses of long prompts start at OK; a page's CTA can only raise its request's.
  const bool cleared = status && per > 1;
  if (cleared) {
    kv_clear_status_kernel<<<static_cast<unsigned>((B + 255) / 256), 256, 0, stream>>>(status, B);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
  }
  return launch_with(kv_write_q8_kernel<false>, ctas, 1, cleared, kWriteThreads, stream, c,
                     prefix_lens, row_start, q_len, max_rows, n_rows, rows_ckv, rows_krope, status,
                     static_cast<int>(per));
}

cudaError_t launch_kv_compact_q8(const ddt_q8_cache& c, const int32_t* prefix_lens,
                                 const int32_t* path, const int32_t* accept_len, int B, int q_len,
                                 int32_t* new_prefix_lens, int32_t* status, cudaStream_t stream) {
  const int row = kRowVec8 * static_cast<int>(sizeof(uint4));
  const cudaError_t e = ensure_smem_limit(reinterpret_cast<const void*>(kv_compact_q8_kernel),
                                          DDT_MAX_Q_LEN * row, 5);
  if (e != cudaSuccess) return e;
  kv_compact_q8_kernel<<<B, kMoveThreads, static_cast<size_t>(q_len) * row, stream>>>(
      c, prefix_lens, path, accept_len, q_len, new_prefix_lens, status);
  return cudaGetLastError();
}

}  // namespace ddt
