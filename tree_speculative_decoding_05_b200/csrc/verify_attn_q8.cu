// verify_attn_q8.cu — tree-verify MLA-absorb attention over the paged 8-bit cache, on
// sm_100a tensor cores.
//
// For request b with prefix P, node i, head h and cache rows j < P + Q of pages with
// scale S_j, key (c_j, k_j) = S_j * (c8_j, k8_j) in e4m3:
//   s_j = softmax_scale * (q_lat . c_j + q_rope . k_j)   over visible j
//   out = sum_j softmax(s)_j c_j,   lse = ln sum_j exp(s_j)
//
// Mathematics.  The cache enters the tensor cores as it lies in memory, as e4m3, so no
// key is ever converted; the other operand of each product is split instead:
//   * q = 2^e (hi + lo) with e4m3 hi and lo, e from the row's largest magnitude.  bf16
//     has 8 significant bits, hi takes 4 of them and lo the rest, so the split is exact
//     down to 2^-19 of the row's maximum (e4m3's smallest step against 448).
//   * the weights w_j = S_j exp(s_j - m) likewise, hi + lo: relative error 2^-8 as a bf16
//     weight has.  S_j rides in the exponent (log2 S_j is added to the score), so a page's
//     scale costs nothing per key; the row sum takes sum(w_j of a page) / S_page.
//     Weights are held at 2^6 .. 2^8.75 for the largest one so far: steps of e4m3 below
//     its normal range are 2^-9, so the smallest weights keep 2^-16 of the largest.
// Two e4m3 passes cost what one bf16 pass does (twice the rate, half the bytes).  One
// pass would halve the tensor work and be 2.6 % off per weight, where a bf16 result
// allows 0.4 %.
//
// Layout (one CTA pair = one cluster of 2 on two SMs, as the bf16 kernel; shapes below
// are per pair unless said otherwise):
//   * 128 query rows: two tree nodes x 64 heads, 64 rows per CTA.  M = 128 with
//     cta_group::2 spreads a CTA's 64 rows over all 128 TMEM lanes: lanes 0-63 hold
//     columns [0, N/2), lanes 64-127 columns [N/2, N).
//   * a tile is 128 keys, two pages: each CTA stages one page for S = Q K^T (N = 128),
//     64 keys x 576 bytes in two slots (latent halves; rope rides with the first), and
//     for O += P V (N = 256, twice) its 128 columns of both pages, 8 KB per slot.  So
//     a page's rows are one TMA box, the thread that owns lanes of one half owns one
//     page, and its scale is one number per tile and thread.
//   * the last page of a request is loaded from row (valid rows - 64) on: TMA fills the
//     rows before the page's first with zeros and never reads those behind the sequence,
//     which may hold anything.
//   * TMEM per CTA: four S buffers (4 x 64 columns) + O (256 columns).
//   * warps 0-7 softmax and epilogue, two threads for each half row (32 keys each): with
//     one, its 64 exponentials and splits outlast the MMAs of a tile (64 requests x 33
//     nodes x 4096 rows: 1225 us, against 1098 us with two, back to back); 8 and 12 fill
//     the K rings of even and odd tiles, 10 the V ring; 9, 14 issue S of even and odd
//     tiles and 11 issues P V (on three sub-partitions); 13 checks a request's page
//     numbers for its status; 15-18 split the next item's queries while this one's last
//     tiles are at work.
//   * S runs up to three tiles ahead of the softmax; O is rescaled only when the running
//     maximum outgrows its reference by 2^2.75.
//   * long caches: splits write normalised partials, merged by the bf16 call's merge.
#include <cuda.h>
#include <cuda_runtime.h>

#include <climits>
#include <cmath>
#include <cstdint>

#include "ddt.h"
#include "ddt_internal.h"

namespace ddt {
static __device__ unsigned int ddt_fault_word = 0;  // this kernel's part, see ddt_fault_flags
}  // namespace ddt

#include "q8_common.cuh"
#include "sm100_ptx.cuh"
#include "verify_shared.cuh"

namespace ddt {

namespace vq {
constexpr int kPage = DDT_PAGE_ROWS;
constexpr int kTK = 2 * kPage;  // keys per tile
static_assert(kVerifyTileKeys % kTK == 0, "split ranges are whole tiles");
constexpr int kWarpKProd0 = 8, kWarpSIss0 = 9, kWarpVProd = 10, kWarpPVIss = 11, kWarpKProd1 = 12,
              kWarpStatus = 13, kWarpSIss1 = 14, kWarpQ0 = 15;
constexpr int kQWarps = 4;
constexpr int kThreads = 32 * (kWarpQ0 + kQWarps);
constexpr int kSoftmaxThreads = 256;
constexpr int kBox = 8192;  // 64 rows x 128 bytes
// Q: four latent chunks of 128 values hi, four lo, then rope hi and lo (64 x 64 bytes).
constexpr int kQLo = 4 * kBox, kQRope = 8 * kBox, kQRopeLo = kQRope + kBox / 2;
constexpr int kQBytes = 9 * kBox;
// K slot: two latent chunks, and in a tile's first slot the rope chunk behind them.
constexpr int kKSlots = 2;                     // per ring; a tile takes two
constexpr int kKRopeOff = 2 * kBox;
constexpr int kKSlotBytes = 2 * kBox + kBox / 2;
constexpr int kVSlots = 4;                     // 64 keys x 128 columns each
constexpr int kPBufBytes = 2 * kBox;           // 64 rows x 128 keys: hi, lo
constexpr int kPBufs = 2;
constexpr int kQSlots = 8;                     // row scales of up to 8 items, see below
constexpr int kMaxSortedB = 512;
constexpr int kOffQ = 0;
constexpr int kOffKRing = kOffQ + kQBytes;
constexpr int kOffVRing = kOffKRing + 2 * kKSlots * kKSlotBytes;
constexpr int kOffP = kOffVRing + kVSlots * kBox;
constexpr int kOffRedMax = kOffP + kPBufs * kPBufBytes;
constexpr int kOffRedL = kOffRedMax + 2 * 256 * 4;  // red_max: float[2][4][64]
constexpr int kOffQScale = kOffRedL + 256 * 4;  // float[kQSlots][64]
constexpr int kOffLen = kOffQScale + kQSlots * 64 * 4;
constexpr int kOffOrder = kOffLen + kMaxSortedB * 4;
constexpr int kOffBar = kOffOrder + kMaxSortedB * 4;
constexpr int kBarKFull = 0;  // ring g at g * kKSlots
constexpr int kBarKEmpty = kBarKFull + 2 * kKSlots;
constexpr int kBarVFull = kBarKEmpty + 2 * kKSlots;
constexpr int kBarVEmpty = kBarVFull + kVSlots;
constexpr int kBarQ = kBarVEmpty + kVSlots;  // queries of an item split, both CTAs
constexpr int kBarQFree = kBarQ + 1;         // both S issuers are done with them
constexpr int kBarQScale = kBarQFree + 1;    // this CTA's row scales of item i (i % kQSlots)
constexpr int kBarS = kBarQScale + kQSlots;
constexpr int kBarSFree = kBarS + 4;
constexpr int kBarP = kBarSFree + 4;
constexpr int kBarO = kBarP + kPBufs;        // four: P V of tile G done (G % 4)
constexpr int kBarQKDone = kBarO + 4;
constexpr int kBarPVDone = kBarQKDone + 2;
constexpr int kBarOFree = kBarPVDone + 1;
constexpr int kNumBars = kBarOFree + 1;
constexpr int kOffTmemPtr = kOffBar + kNumBars * 8;
constexpr int kOffAbort = kOffTmemPtr + 4;
constexpr int kSmemUsed = kOffAbort + 4;
constexpr int kSmemBytes = kSmemUsed + 1024;  // slack for 1024-byte alignment
static_assert(kSmemBytes <= 232448, "shared memory budget");
static_assert(kPBufs * kPBufBytes >= 64 * 256 * 2, "P buffers hold half an output tile");

constexpr int kTmemCols = 512, kTmemS = 0, kTmemO = 256;
constexpr uint32_t kIdescQK = idesc_e4m3_f32(128, kTK, false);
constexpr uint32_t kIdescPV = idesc_e4m3_f32(128, 256, true);
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
// The reference weight 2^kBase and the growth kSlack allowed before O is rescaled:
// 2^(6 + 2.75) = 431 <= 448.
constexpr float kBase = 6.0f, kSlack = 2.75f;
constexpr float kMinScale = 9.094947017729282e-13f;  // 2^-40

struct Params {
  const int32_t* prefix_lens;
  const int32_t* block_table;
  const float* scales;
  const uint16_t* q_lat;
  const uint16_t* q_rope;
  const uint64_t* mask;
  float* lse;
  float* part_lse;
  int32_t* status;
  int B, Q, num_pages, max_blocks, num_splits, n_pairs, write_partials;
  float scale_log2;  // softmax_scale * log2(e)
};

struct Item {
  int b, pair, split, P, T, t0, ntile;
  bool bad_prefix, valid;
};

__device__ __forceinline__ Item decode_item(const Params& p, int w, const int* order) {
  Item it;
  const int per_req = p.n_pairs * p.num_splits;
  const int slot = w / per_req;
  it.b = order ? order[slot] : slot;
  const int rem = w - slot * per_req;
  it.pair = rem / p.num_splits;
  it.split = rem - it.pair * p.num_splits;
  it.P = p.prefix_lens[it.b];
  it.bad_prefix = it.P < 0 || static_cast<int64_t>(it.P) + p.Q >
                                  static_cast<int64_t>(p.max_blocks) * kPage;
  it.T = it.P + p.Q;
  int t0 = 0, t1 = 0;
  if (!it.bad_prefix) {
    constexpr int kUnit = kVerifyTileKeys / kTK;
    split_range(it.T, p.num_splits, it.split, t0, t1);
    const int n = (it.T + kTK - 1) / kTK;
    t0 *= kUnit;
    t1 = t1 * kUnit < n ? t1 * kUnit : n;
  }
  it.t0 = t0;
  it.ntile = t1 - t0;
  it.valid = !it.bad_prefix && it.ntile > 0;
  return it;
}

// A block of the cache (64 rows): its page, -1 for none, and how many of its rows the
// request holds.
struct Block {
  int page, rows;
};
__device__ __forceinline__ Block load_block(const Params& p, const Item& it, int blk) {
  Block k;
  k.rows = it.T - kPage * blk;
  k.rows = k.rows < 0 ? 0 : k.rows > kPage ? kPage : k.rows;
  k.page = k.rows > 0 ? p.block_table[static_cast<int64_t>(it.b) * p.max_blocks + blk] : -1;
  return k;
}
// TMA coordinates of a block: its rows end the box; a block without rows, or whose page
// number is none, is a box of zeros.
__device__ __forceinline__ void block_coords(const Params& p, const Block& k, int& row, int& page) {
  const bool ok = k.page >= 0 && k.page < p.num_pages;
  row = ok ? k.rows - kPage : -kPage;
  page = ok ? k.page : 0;
}

// Two floats (lo in the low half) as the sum of two e4m3 pairs.  fp16 keeps 11 bits and
// the residual of the first rounding exactly; the values lie within 448.
__device__ __forceinline__ void split_e4m3x2(float lo, float hi, uint16_t& first,
                                             uint16_t& second) {
  asm("{\n\t.reg .b32 x, y, z;\n\t"
      "cvt.rn.f16x2.f32 x, %3, %2;\n\t"
      "cvt.rn.satfinite.e4m3x2.f16x2 %0, x;\n\t"
      "cvt.rn.f16x2.e4m3x2 y, %0;\n\t"
      "sub.rn.f16x2 z, x, y;\n\t"
      "cvt.rn.satfinite.e4m3x2.f16x2 %1, z;\n\t}"
      : "=h"(first), "=h"(second)
      : "f"(lo), "f"(hi));
}

__device__ __forceinline__ uint32_t pack16(uint16_t lo, uint16_t hi) {
  return static_cast<uint32_t>(lo) | (static_cast<uint32_t>(hi) << 16);
}

}  // namespace vq

// Persistent kernel: each CTA pair loops over work items (see work_index); rings,
// barriers and tensor memory live across items, and phases follow a count G of the tiles
// of all items that a CTA has seen.
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(vq::kThreads, 1)
    verify_attn_q8_kernel(const __grid_constant__ CUtensorMap tm_lat,
                          const __grid_constant__ CUtensorMap tm_rope,
                          const __grid_constant__ CUtensorMap tm_out, const vq::Params p) {
  using namespace vq;
  const uint32_t rank = cluster_ctarank();
  const int cluster = static_cast<int>(blockIdx.x >> 1);
  const int n_clusters = static_cast<int>(gridDim.x >> 1);
  const int n_items = p.B * p.n_pairs * p.num_splits;
  const int n_rounds = (n_items + n_clusters - 1) / n_clusters;
  const int Q = p.Q;

  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw_addr = smem_u32(smem_raw);
  const uint32_t base_addr = (raw_addr + 1023u) & ~1023u;
  uint8_t* base = smem_raw + (base_addr - raw_addr);
  const uint32_t sQ = base_addr + kOffQ;
  const uint32_t sVRing = base_addr + kOffVRing;
  const uint32_t sP = base_addr + kOffP;
  float* red_max = reinterpret_cast<float*>(base + kOffRedMax);
  float* red_l = reinterpret_cast<float*>(base + kOffRedL);
  float* q_scale = reinterpret_cast<float*>(base + kOffQScale);
  const uint32_t bars = base_addr + kOffBar;
  auto bar = [&](int i) -> uint32_t { return bars + 8u * static_cast<uint32_t>(i); };
  uint32_t* tmem_ptr_smem = reinterpret_cast<uint32_t*>(base + kOffTmemPtr);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(base + kOffAbort);
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    // Stage barriers: one arrival (the even CTA's producer, expecting both CTAs' bytes).
    for (int s = 0; s < 2 * kKSlots; ++s) {
      mbar_init(bar(kBarKFull + s), 1);
      mbar_init(bar(kBarKEmpty + s), 1);
    }
    for (int s = 0; s < kVSlots; ++s) {
      mbar_init(bar(kBarVFull + s), 1);
      mbar_init(bar(kBarVEmpty + s), 1);
    }
    mbar_init(bar(kBarQ), 2 * kQWarps);  // every converting warp of the pair
    mbar_init(bar(kBarQFree), 2);        // a commit of each S issuer
    for (int s = 0; s < kQSlots; ++s) mbar_init(bar(kBarQScale + s), kQWarps);
    for (int s = 0; s < 4; ++s) {
      mbar_init(bar(kBarS + s), 1);
      mbar_init(bar(kBarSFree + s), 2);  // one arrival per CTA
      mbar_init(bar(kBarO + s), 1);
    }
    for (int s = 0; s < kPBufs; ++s) mbar_init(bar(kBarP + s), 2);
    for (int g = 0; g < 2; ++g) mbar_init(bar(kBarQKDone + g), 1);
    mbar_init(bar(kBarPVDone), 1);
    mbar_init(bar(kBarOFree), 2);
    *abort_flag = 0;
    fence_mbar_init_cluster();
  }
  if (warp == kWarpSIss0) {
    tmem_alloc<2>(smem_u32(tmem_ptr_smem), kTmemCols);
    tmem_relinquish<2>();
  }
  // Requests by decreasing length (ties by index), found by every CTA for itself.
  int* len_smem = reinterpret_cast<int*>(base + kOffLen);
  int* order_smem = reinterpret_cast<int*>(base + kOffOrder);
  const bool sorted = p.B <= kMaxSortedB;
  if (sorted) {
    for (int b = threadIdx.x; b < p.B; b += kThreads) {
      const int P = p.prefix_lens[b];
      len_smem[b] = P < 0 || static_cast<int64_t>(P) + Q > static_cast<int64_t>(p.max_blocks) * kPage
                        ? 0 : P + Q;
    }
    __syncthreads();
    for (int bi = warp; bi < p.B; bi += kThreads / 32) {
      const int li = len_smem[bi];
      int before = 0;
      for (int bj = lane; bj < p.B; bj += 32) {
        const int lj = len_smem[bj];
        before += lj > li || (lj == li && bj < bi);
      }
      before = __reduce_add_sync(0xffffffffu, before);
      if (lane == 0) order_smem[before] = bi;
    }
  }
  tc_fence_before_sync();
  cluster_sync();
  tc_fence_after_sync();
  const uint32_t tmem = *tmem_ptr_smem;
  const int* order = sorted ? order_smem : nullptr;

  struct Ring {
    int stage = 0;
    uint32_t phase = 0;
    __device__ void advance(int n) {
      if (++stage == n) {
        stage = 0;
        phase ^= 1u;
      }
    }
  };
  const bool leader = rank == 0;
  const int ring_g = warp == kWarpKProd1 || warp == kWarpSIss1 ? 1 : 0;

  if (warp == kWarpKProd0 || warp == kWarpKProd1) {
    // ------------------------------------------------------ TMA: the K rings
    if (lane == 0) {
      const int g = ring_g;
      const int full0 = kBarKFull + g * kKSlots, empty0 = kBarKEmpty + g * kKSlots;
      const uint32_t ring = base_addr + kOffKRing + g * kKSlots * kKSlotBytes;
      Ring r;
      int64_t G = 0;
      for (int k = 0; k < n_rounds; ++k) {
        const int w = work_index(k, cluster, n_clusters, n_items);
        if (w < 0) continue;
        const Item it = decode_item(p, w, order);
        if (!it.valid) continue;
        // tiles of this ring, the page number of the next one loaded ahead of the wait
        int jj = static_cast<int>(G & 1) == g ? 0 : 1;
        Block next = load_block(p, it, 2 * (it.t0 + jj) + static_cast<int>(rank));
        for (; jj < it.ntile; jj += 2) {
          int row, page;
          block_coords(p, next, row, page);
          if (jj + 2 < it.ntile) next = load_block(p, it, 2 * (it.t0 + jj + 2) + static_cast<int>(rank));
          for (int half = 0; half < 2; ++half) {
            mbar_wait(bar(empty0 + r.stage), r.phase ^ 1u, abort_flag);
            const uint32_t bytes = 2 * (2 * kBox + (half == 0 ? kBox / 2 : 0));
            if (leader) mbar_arrive_expect_tx_local(bar(full0 + r.stage), bytes);
            const uint32_t fb = map_to_rank(bar(full0 + r.stage), 0);
            const uint32_t dst = ring + r.stage * kKSlotBytes;
            tma_load_3d_pair(dst, &tm_lat, fb, 256 * half, row, page);
            tma_load_3d_pair(dst + kBox, &tm_lat, fb, 256 * half + 128, row, page);
            if (half == 0) tma_load_3d_pair(dst + kKRopeOff, &tm_rope, fb, 0, row, page);
            r.advance(kKSlots);
          }
        }
        G += it.ntile;
      }
    }
    __syncwarp();
  } else if (warp == kWarpVProd) {
    // -------------------------------------------------------- TMA: the V ring
    if (lane == 0) {
      Ring r;
      for (int k = 0; k < n_rounds; ++k) {
        const int w = work_index(k, cluster, n_clusters, n_items);
        if (w < 0) continue;
        const Item it = decode_item(p, w, order);
        if (!it.valid) continue;
        const int blk0 = 2 * it.t0, n_blk = 2 * it.ntile;
        Block next = load_block(p, it, blk0);
        for (int i = 0; i < n_blk; ++i) {
          int row, page;
          block_coords(p, next, row, page);
          if (i + 1 < n_blk) next = load_block(p, it, blk0 + i + 1);
          for (int nh = 0; nh < 2; ++nh) {
            mbar_wait(bar(kBarVEmpty + r.stage), r.phase ^ 1u, abort_flag);
            if (leader) mbar_arrive_expect_tx_local(bar(kBarVFull + r.stage), 2 * kBox);
            const uint32_t fb = map_to_rank(bar(kBarVFull + r.stage), 0);
            tma_load_3d_pair(sVRing + r.stage * kBox, &tm_lat, fb,
                             256 * nh + 128 * static_cast<int>(rank), row, page);
            r.advance(kVSlots);
          }
        }
      }
    }
    __syncwarp();
  } else if (warp == kWarpSIss0 || warp == kWarpSIss1) {
    // -------------------------------------------------------- MMA: S = Q K^T
    // Issuer g takes tiles G with G % 2 == g; tile G goes to S buffer G % 4.
    if (leader && lane == 0) {
      const int g = ring_g;
      const int full0 = kBarKFull + g * kKSlots, empty0 = kBarKEmpty + g * kKSlots;
      const uint32_t ring = base_addr + kOffKRing + g * kKSlots * kKSlotBytes;
      Ring r;
      int iter = 0;
      int64_t G = 0;
      for (int k = 0; k < n_rounds; ++k) {
        const int w = work_index(k, cluster, n_clusters, n_items);
        if (w < 0) continue;
        const Item it = decode_item(p, w, order);
        if (!it.valid) continue;
        mbar_wait(bar(kBarQ), static_cast<uint32_t>(iter & 1), abort_flag);
        for (int jj = 0; jj < it.ntile; ++jj, ++G) {
          if (static_cast<int>(G & 1) != g) continue;
          const int sbuf = static_cast<int>(G & 3);
          if (G >= 4) {
            mbar_wait(bar(kBarSFree + sbuf), static_cast<uint32_t>(((G >> 2) - 1) & 1), abort_flag);
            tc_fence_after_sync();
          }
          const uint32_t d = tmem + kTmemS + 64u * static_cast<uint32_t>(sbuf);
          for (int half = 0; half < 2; ++half) {
            mbar_wait(bar(full0 + r.stage), r.phase, abort_flag);
            const uint32_t slot = ring + r.stage * kKSlotBytes;
            for (int u = 0; u < 2; ++u) {
              const uint32_t a0 = sQ + (2 * half + u) * kBox;
#pragma unroll
              for (int ks = 0; ks < 4; ++ks) {
                const uint64_t kd = smem_desc_sw128(slot + u * kBox + 32 * ks, 16, 1024);
                mma_f8_ss<2>(d, smem_desc_sw128(a0 + 32 * ks, 16, 1024), kd, kIdescQK,
                             (half | u | ks) != 0);
                mma_f8_ss<2>(d, smem_desc_sw128(a0 + kQLo + 32 * ks, 16, 1024), kd, kIdescQK, 1);
              }
            }
            if (half == 0) {
#pragma unroll
              for (int ks = 0; ks < 2; ++ks) {
                const uint64_t kd = smem_desc_sw64(slot + kKRopeOff + 32 * ks);
                mma_f8_ss<2>(d, smem_desc_sw64(sQ + kQRope + 32 * ks), kd, kIdescQK, 1);
                mma_f8_ss<2>(d, smem_desc_sw64(sQ + kQRopeLo + 32 * ks), kd, kIdescQK, 1);
              }
            }
            mma_commit<2>(bar(empty0 + r.stage), 0x3);
            r.advance(kKSlots);
          }
          mma_commit<2>(bar(kBarS + sbuf), 0x3);
        }
        mma_commit<2>(bar(kBarQFree), 0x3);  // this issuer no longer reads this item's Q
        ++iter;
      }
      mma_commit<2>(bar(kBarQKDone + g), 0x1);
      mbar_wait(bar(kBarQKDone + g), 0, abort_flag);
    }
    __syncwarp();
  } else if (warp == kWarpPVIss) {
    // ---------------------------------------------------------- MMA: O += P V
    if (leader && lane == 0) {
      Ring r;
      int iter = 0;
      int64_t G = 0;
      for (int k = 0; k < n_rounds; ++k) {
        const int w = work_index(k, cluster, n_clusters, n_items);
        if (w < 0) continue;
        const Item it = decode_item(p, w, order);
        if (!it.valid) continue;
        if (iter > 0) {  // both epilogues have read the previous item's O
          mbar_wait(bar(kBarOFree), static_cast<uint32_t>((iter - 1) & 1), abort_flag);
          tc_fence_after_sync();
        }
        for (int jj = 0; jj < it.ntile; ++jj, ++G) {
          const int pb = static_cast<int>(G % kPBufs);
          mbar_wait(bar(kBarP + pb), static_cast<uint32_t>((G / kPBufs) & 1), abort_flag);
          tc_fence_after_sync();
          for (int kb = 0; kb < 2; ++kb) {
            for (int nh = 0; nh < 2; ++nh) {
              mbar_wait(bar(kBarVFull + r.stage), r.phase, abort_flag);
              const uint32_t d = tmem + kTmemO + 128u * static_cast<uint32_t>(nh);
              const uint32_t a0 = sP + pb * kPBufBytes + kPage * kb;
              const uint32_t b0 = sVRing + r.stage * kBox;
#pragma unroll
              for (int ks = 0; ks < 2; ++ks) {
                const uint64_t vd = smem_desc_sw128(b0 + 4096 * ks, kBox, 1024);
                mma_f8_ss<2>(d, smem_desc_sw128(a0 + 32 * ks, 16, 1024), vd, kIdescPV,
                             !(jj == 0 && kb == 0 && ks == 0));
                mma_f8_ss<2>(d, smem_desc_sw128(a0 + kBox + 32 * ks, 16, 1024), vd, kIdescPV, 1);
              }
              mma_commit<2>(bar(kBarVEmpty + r.stage), 0x3);
              r.advance(kVSlots);
            }
          }
          mma_commit<2>(bar(kBarO + static_cast<int>(G & 3)), 0x3);
        }
        ++iter;
      }
      mma_commit<2>(bar(kBarPVDone), 0x1);
      mbar_wait(bar(kBarPVDone), 0, abort_flag);
    }
    __syncwarp();
  } else if (warp >= kWarpQ0) {
    // ------------------------------------------------- queries to e4m3 hi + lo
    // Warp u splits rows 16 u .. 16 u + 15 of this CTA's node.  A lane holds latent
    // values 16 lane .. + 15 and rope values 2 lane, 2 lane + 1 of a row; four rows are
    // loaded at a time, the first four before the wait for the previous item's S.
    const int u = warp - kWarpQ0;
    const uint32_t q_bar = map_to_rank(bar(kBarQ), 0);
    int iter = 0;
    for (int k = 0; k < n_rounds; ++k) {
      const int w = work_index(k, cluster, n_clusters, n_items);
      if (w < 0) continue;
      const Item it = decode_item(p, w, order);
      if (!it.valid) continue;
      const int node = 2 * it.pair + static_cast<int>(rank);
      const int64_t row0 = (static_cast<int64_t>(it.b) * Q + node) * 64 + 16 * u;
      const uint4* lat = reinterpret_cast<const uint4*>(p.q_lat) + row0 * 64 + 2 * lane;
      const uint32_t* rope = reinterpret_cast<const uint32_t*>(p.q_rope) + row0 * 32 + lane;
      const int slot = iter % kQSlots;
#pragma unroll 1
      for (int r0 = 0; r0 < 16; r0 += 4) {
        uint32_t x[4][9];
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          uint4 a = make_uint4(0, 0, 0, 0), c = a;
          x[r][8] = 0;
          if (node < Q) {
            a = lat[(r0 + r) * 64];
            c = lat[(r0 + r) * 64 + 1];
            x[r][8] = rope[(r0 + r) * 32];
          }
          x[r][0] = a.x, x[r][1] = a.y, x[r][2] = a.z, x[r][3] = a.w;
          x[r][4] = c.x, x[r][5] = c.y, x[r][6] = c.z, x[r][7] = c.w;
        }
        if (r0 == 0 && iter > 0)
          mbar_wait(bar(kBarQFree), static_cast<uint32_t>((iter - 1) & 1), abort_flag);
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          uint32_t m = 0;
#pragma unroll
          for (int j = 0; j < 9; ++j) m = max_abs_bf16x2(m, x[r][j]);
          const uint32_t top = __reduce_max_sync(0xffffffffu, max_of_halves(m));
          int e = e4m3_exponent(top);
          e = top == 0 ? 0 : e < -100 ? -100 : e;
          const float inv = pow2f(-e);
          const int row = 16 * u + r0 + r;
          uint32_t hi[4], lo[4];
          uint16_t f[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
#pragma unroll
            for (int v = 0; v < 2; ++v) {
              const uint32_t h = x[r][2 * j + v];
              split_e4m3x2(__uint_as_float(h << 16) * inv, __uint_as_float(h & 0xffff0000u) * inv,
                           f[v], f[2 + v]);
            }
            hi[j] = pack16(f[0], f[1]);
            lo[j] = pack16(f[2], f[3]);
          }
          uint8_t* at = base + kOffQ + (lane >> 3) * kBox + row * 128 + (((lane & 7) ^ (row & 7)) << 4);
          *reinterpret_cast<uint4*>(at) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
          *reinterpret_cast<uint4*>(at + kQLo) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
          const uint32_t h = x[r][8];
          split_e4m3x2(__uint_as_float(h << 16) * inv, __uint_as_float(h & 0xffff0000u) * inv, f[0],
                       f[1]);
          at = base + kOffQ + kQRope + row * 64 + (((lane >> 3) ^ ((row >> 1) & 3)) << 4) + 2 * (lane & 7);
          *reinterpret_cast<uint16_t*>(at) = f[0];
          *reinterpret_cast<uint16_t*>(at + kQRopeLo - kQRope) = f[1];
          // A row with NaN or an infinity gets NaN as its scale, and so NaN results.
          if (lane == 0)
            q_scale[slot * 64 + row] = top >= 0x7f80u ? __uint_as_float(0x7fc00000u) : pow2f(e);
        }
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive_local(bar(kBarQScale + slot));
        mbar_arrive_cluster(q_bar);
      }
      ++iter;
    }
  } else if (warp == kWarpStatus) {
    // A request's status, by the even CTA that has its first pair and split: whether
    // its prefix fits and all its page numbers are some.
    if (leader && p.status) {
      for (int k = 0; k < n_rounds; ++k) {
        const int w = work_index(k, cluster, n_clusters, n_items);
        if (w < 0) continue;
        const Item it = decode_item(p, w, order);
        if (it.pair != 0 || it.split != 0) continue;
        int st = it.bad_prefix ? DDT_REQ_BAD_PREFIX : DDT_REQ_OK;
        if (!it.bad_prefix) {
          bool bad = false;
          for (int blk = lane; blk * kPage < it.T; blk += 32) {
            const int page = p.block_table[static_cast<int64_t>(it.b) * p.max_blocks + blk];
            bad |= page < 0 || page >= p.num_pages;
          }
          if (__any_sync(0xffffffffu, bad)) st = DDT_REQ_BAD_INDEX;
        }
        if (lane == 0) p.status[it.b] = st;
      }
    }
  } else {
    // -------------------------------------------------------- softmax warps
    const int t = threadIdx.x;
    const int m = t & 63;         // row within this CTA (head)
    const int hf = (t >> 6) & 1;  // which page of the tile / which half of each O columns
    const int g = t >> 7;         // which 32 keys of the page, which half of O's chunks
    // warp w reads TMEM lanes 32 (w % 4) on
    const uint32_t lane_addr = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const int part_of = (2 * g + hf) * 64 + m;  // a row's four parts lie 64 apart
    const int W = (Q + 63) >> 6;
    const uint32_t p_full_leader0 = map_to_rank(bar(kBarP), 0);
    const uint32_t s_free_leader0 = map_to_rank(bar(kBarSFree), 0);
    const uint32_t o_free_leader = map_to_rank(bar(kBarOFree), 0);
    // P V completions, confirmed in tile order on four barriers; the softmax waits at
    // most for tile G - kPBufs while P V has finished at most tile G - 1.
    int64_t o_next = 0;
    auto wait_o_through = [&](int64_t last) {
      bool waited = false;
      while (o_next <= last) {
        mbar_wait(bar(kBarO + static_cast<int>(o_next & 3)), static_cast<uint32_t>((o_next >> 2) & 1),
                  abort_flag);
        ++o_next;
        waited = true;
      }
      if (waited) tc_fence_after_sync();
    };
    int64_t G = 0;
    int iter = 0;
    for (int k = 0; k < n_rounds; ++k) {
      const int w = work_index(k, cluster, n_clusters, n_items);
      if (w < 0) continue;
      const Item it = decode_item(p, w, order);
      if (!it.valid) continue;
      const int b = it.b, P = it.P, split = it.split;
      const int node = 2 * it.pair + static_cast<int>(rank);
      const bool node_valid = node < Q;
      uint64_t mw0 = 0, mw1 = 0;
      if (node_valid) {
        const uint64_t* mrow = p.mask + (static_cast<int64_t>(b) * Q + node) * W;
        mw0 = mrow[0];
        if (W > 1) mw1 = mrow[1];
      }
      // Page scales run two tiles ahead: the scale of the next tile's page is loaded
      // while the page number of the one after it is.  A page of scale 0 (never
      // written) and a block without a page count as the smallest scale.
      auto page_scale = [&](const Block& kb) {
        return kb.page >= 0 && kb.page < p.num_pages ? p.scales[kb.page] : 1.f;
      };
      const int blk0 = 2 * it.t0 + hf;
      Block cur = load_block(p, it, blk0), nxt = load_block(p, it, blk0 + 2);
      float ks_next = page_scale(cur);
      // The row scales of item i lie in slot i % 8: queries run at most five items
      // ahead (four S buffers), so a slot is read before it is written again.
      const int slot = iter % kQSlots;
      mbar_wait(bar(kBarQScale + slot), static_cast<uint32_t>((iter / kQSlots) & 1), abort_flag);
      const float row_scale = q_scale[slot * 64 + m] * p.scale_log2;
      ++iter;
      float m_ref = -INFINITY;  // log2 units, page scale included
      float l_sum = 0.f;
      float m_use = 0.f;
      for (int jj = 0; jj < it.ntile; ++jj, ++G) {
        const int sb = static_cast<int>(G & 1);
        const int pbuf = static_cast<int>(G % kPBufs);
        const int sbuf = static_cast<int>(G & 3);
        const int blk = blk0 + 2 * jj;
        float ks = ks_next;
        if (ks == 0.f) ks = kMinScale;
        const int rows = cur.rows;
        cur = nxt;
        ks_next = page_scale(cur);
        nxt = load_block(p, it, blk + 4);
        float sc = row_scale * ks;
        if (sc == 0.f) sc = 1.4e-45f;  // underflow: masked scores stay -inf
        const float lk = __log2f(ks);
        // Visible keys of the block's box: key of column c is key0 + c.
        const int key0 = kPage * blk + rows - kPage;
        uint64_t vis = ~0ull;
        if (rows < kPage || key0 + kPage > P) {
          const int np = P - key0;  // columns below np are prefix rows
          vis = np >= 64 ? ~0ull : np <= 0 ? 0ull : (1ull << np) - 1;
          // columns of tree rows: bit a = c - np of the node's words
          if (np >= 0) {
            if (np < 64) vis |= mw0 << np;
          } else {
            const int s = -np;
            vis |= s < 64 ? (mw0 >> s) | (mw1 << (64 - s)) : s < 128 ? mw1 >> (s - 64) : 0ull;
          }
          if (rows < kPage) vis = rows > 0 ? vis & (~0ull << (kPage - rows)) : 0ull;
        }
        mbar_wait(bar(kBarS + sbuf), static_cast<uint32_t>((G >> 2) & 1), abort_flag);
        tc_fence_after_sync();
        float x[32];
        {
          uint32_t r0[32];
          tmem_ld32(tmem + lane_addr + kTmemS + static_cast<uint32_t>(64 * sbuf + 32 * g), r0);
          tmem_wait_ld();
#pragma unroll
          for (int c = 0; c < 32; ++c) x[c] = __uint_as_float(r0[c]);
        }
        const uint32_t v32 = static_cast<uint32_t>(vis >> (32 * g));
        if (v32 != ~0u) {
#pragma unroll
          for (int c = 0; c < 32; ++c)
            if (!((v32 >> c) & 1u)) x[c] = -INFINITY;
        }
        float mx = x[0];
#pragma unroll
        for (int c = 1; c < 32; ++c) mx = fmaxf(mx, x[c]);
        tc_fence_before_sync();
        mx = fmaf(mx, sc, lk);  // a positive scale commutes with the maximum
        float* const red = red_max + sb * 256;
        red[part_of] = mx;
        named_barrier_sync(1, kSoftmaxThreads);
        // Every thread of this CTA has read S: release the buffer.
        if (t == 0) mbar_arrive_cluster(s_free_leader0 + 8u * sbuf);
        mx = fmaxf(fmaxf(red[m], red[64 + m]), fmaxf(red[128 + m], red[192 + m]));
        float factor = 1.f;
        bool rescale = false;
        if (m_ref == -INFINITY) {
          m_ref = mx;
        } else if (mx > m_ref + kSlack) {
          factor = fast_exp2(m_ref - mx);
          m_ref = mx;
          l_sum *= factor;
          rescale = true;
        }
        m_use = m_ref == -INFINITY ? 0.f : m_ref;
        const float shift = lk - m_use + kBase;
        uint32_t hi[8], lo[8];
        float part[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int c = 0; c < 8; ++c) {
          uint16_t f[4];
#pragma unroll
          for (int v = 0; v < 2; ++v) {
            const float e0 = fast_exp2(fmaf(x[4 * c + 2 * v], sc, shift));
            const float e1 = fast_exp2(fmaf(x[4 * c + 2 * v + 1], sc, shift));
            part[2 * v] += e0;
            part[2 * v + 1] += e1;
            split_e4m3x2(e0, e1, f[v], f[2 + v]);
          }
          hi[c] = pack16(f[0], f[1]);
          lo[c] = pack16(f[2], f[3]);
        }
        // the row sum counts keys, not keys times their page's scale
        l_sum += ((part[0] + part[1]) + (part[2] + part[3])) * (1.f / ks);
        // The P buffer of this tile was last read by the P V of tile G - kPBufs.
        wait_o_through(G - kPBufs);
        // P: K-major, 128-byte rows of 128 keys, swizzled; this thread's keys are a
        // quarter of the row.
        uint8_t* prow = base + kOffP + pbuf * kPBufBytes + m * 128;
#pragma unroll
        for (int v = 0; v < 2; ++v) {
          const int at = ((4 * hf + 2 * g + v) ^ (m & 7)) << 4;
          *reinterpret_cast<uint4*>(prow + at) =
              make_uint4(hi[4 * v], hi[4 * v + 1], hi[4 * v + 2], hi[4 * v + 3]);
          *reinterpret_cast<uint4*>(prow + kBox + at) =
              make_uint4(lo[4 * v], lo[4 * v + 1], lo[4 * v + 2], lo[4 * v + 3]);
        }
        if (jj > 0 && __any_sync(0xffffffffu, rescale)) {
          wait_o_through(G - 1);  // the P V of the previous tile is done
#pragma unroll 1
          for (int q = 4 * g; q < 4 * g + 4; ++q) {
            uint32_t o[32];
            const uint32_t addr = tmem + lane_addr + kTmemO + 32u * q;
            tmem_ld32(addr, o);
            tmem_wait_ld();
#pragma unroll
            for (int c = 0; c < 32; ++c) o[c] = __float_as_uint(__uint_as_float(o[c]) * factor);
            tmem_st32(addr, o);
          }
          tmem_wait_st();
        }
        fence_proxy_async_smem();
        tc_fence_before_sync();
        named_barrier_sync(2, kSoftmaxThreads);
        if (t == 0) mbar_arrive_cluster(p_full_leader0 + 8u * pbuf);
      }
      // ----------------------------------------------------------- epilogue
      wait_o_through(G - 1);
      red_l[part_of] = l_sum;
      named_barrier_sync(1, kSoftmaxThreads);
      const float l_row = (red_l[m] + red_l[64 + m]) + (red_l[128 + m] + red_l[192 + m]);
      const bool empty_row = l_row == 0.f;
      const float inv = empty_row ? 0.f : 1.f / l_row;
      const float lse_nat = empty_row ? -INFINITY : (m_use - kBase + __log2f(l_row)) * kLn2;
      uint8_t* stage = base + kOffP;
      const uint32_t stage_addr = base_addr + kOffP;
      if (!node_valid) {
        // A node past q_len (odd q_len): nothing to write; release O.
        tc_fence_before_sync();
        named_barrier_sync(2, kSoftmaxThreads);
        if (t == 0) mbar_arrive_cluster(o_free_leader);
      } else if (!p.write_partials) {
        const int row0 = (b * Q + node) * 64;
#pragma unroll 1
        for (int nh = 0; nh < 2; ++nh) {
#pragma unroll 1
          for (int q = 2 * g; q < 2 * g + 2; ++q) {
            uint32_t o[32];
            tmem_ld32(tmem + lane_addr + kTmemO + 128u * nh + 32u * q, o);
            tmem_wait_ld();
            // columns 256 nh + 128 hf + 32 q ..: 64-column box 2 hf + q / 2 of this half
            uint8_t* rowp = stage + (2 * hf + (q >> 1)) * kBox + m * 128;
#pragma unroll
            for (int v = 0; v < 4; ++v) {
              uint32_t y[4];
#pragma unroll
              for (int z = 0; z < 4; ++z)
                y[z] = pack_bf16x2(__uint_as_float(o[8 * v + 2 * z]) * inv,
                                   __uint_as_float(o[8 * v + 2 * z + 1]) * inv);
              *reinterpret_cast<uint4*>(rowp + (((4 * (q & 1) + v) ^ (m & 7)) << 4)) =
                  make_uint4(y[0], y[1], y[2], y[3]);
            }
          }
          if (nh == 1) tc_fence_before_sync();  // every read of O is done
          fence_proxy_async_smem();
          named_barrier_sync(2, kSoftmaxThreads);
          if (nh == 1 && t == 0) mbar_arrive_cluster(o_free_leader);
          if (t == 0) {
            for (int c = 0; c < 4; ++c)
              tma_store_3d(&tm_out, stage_addr + c * kBox, 256 * nh + 64 * c, row0, 0);
            bulk_commit_group();
            bulk_wait_group_read0();  // the staging buffer may be written again
          }
          named_barrier_sync(2, kSoftmaxThreads);
        }
        if (t < 64 && p.lse) p.lse[static_cast<int64_t>(row0) + m] = lse_nat;
      } else {
        // A split's normalised fp32 partial, in four rounds of 64 rows x 128 columns.
        const int64_t rows_total = static_cast<int64_t>(p.B) * Q * 64;
        const int64_t row0 = split * rows_total + (static_cast<int64_t>(b) * Q + node) * 64;
#pragma unroll 1
        for (int r = 0; r < 4; ++r) {
          uint32_t o[32];
          tmem_ld32(tmem + lane_addr + kTmemO + 128u * (r >> 1) + 32u * (2 * (r & 1) + g), o);
          tmem_wait_ld();
          uint8_t* rowp = stage + (2 * hf + g) * kBox + m * 128;
#pragma unroll
          for (int v = 0; v < 8; ++v)
            *reinterpret_cast<float4*>(rowp + ((v ^ (m & 7)) << 4)) =
                make_float4(__uint_as_float(o[4 * v]) * inv, __uint_as_float(o[4 * v + 1]) * inv,
                            __uint_as_float(o[4 * v + 2]) * inv, __uint_as_float(o[4 * v + 3]) * inv);
          if (r == 3) tc_fence_before_sync();
          fence_proxy_async_smem();
          named_barrier_sync(2, kSoftmaxThreads);
          if (r == 3 && t == 0) mbar_arrive_cluster(o_free_leader);
          if (t == 0) {
            for (int c = 0; c < 4; ++c)
              tma_store_3d(&tm_out, stage_addr + c * kBox,
                           256 * (r >> 1) + 128 * (c >> 1) + 64 * (r & 1) + 32 * (c & 1),
                           static_cast<int>(row0), 0);
            bulk_commit_group();
            bulk_wait_group_read0();
          }
          named_barrier_sync(2, kSoftmaxThreads);
        }
        if (t < 64) p.part_lse[row0 + m] = lse_nat;
      }
    }
    if (t == 0) bulk_wait_group0();  // this CTA's output stores have completed
  }

  // All MMAs of the pair are complete (the softmax warps waited for the last O, the
  // issuers for their final commits); release tensor memory.
  __syncwarp();
  tc_fence_before_sync();
  cluster_sync();
  if (warp == kWarpSIss0) {
    tc_fence_after_sync();
    tmem_dealloc<2>(tmem, kTmemCols);
  }
}

ddt_status launch_verify_attn_q8(const ddt_attn_q8_args& a, int num_splits, float* part_o,
                                 float* part_lse, cudaStream_t stream) {
  using namespace vq;
  const ddt_q8_cache& c = a.cache;
  const uint64_t pages = static_cast<uint64_t>(c.num_pages);
  const uint64_t rows = static_cast<uint64_t>(a.B) * a.q_len * 64;
  const bool partials = num_splits > 1;
  const uint64_t out_rows = partials ? rows * num_splits : rows;
  const int64_t items = static_cast<int64_t>(a.B) * ((a.q_len + 1) / 2) * num_splits;
  if (items > 0x3fffffffll || out_rows > INT_MAX) return DDT_ERR_UNSUPPORTED;
  // With one page its stride is never taken, but the map wants one.
  const uint64_t lat_page = c.num_pages > 1 ? c.ckv_page_stride : kPage * c.ckv_row_stride;
  const uint64_t rope_page = c.num_pages > 1 ? c.kr_page_stride : kPage * c.kr_row_stride;
  CUtensorMap m_lat, m_rope, m_out;
  bool ok = make_map(&m_lat, c.c_kv, DDT_D_LATENT, kPage, pages, c.ckv_row_stride, lat_page, kPage,
                     CU_TENSOR_MAP_DATA_TYPE_UINT8, 128) &&
            make_map(&m_rope, c.k_rope, DDT_D_ROPE, kPage, pages, c.kr_row_stride, rope_page, kPage,
                     CU_TENSOR_MAP_DATA_TYPE_UINT8, 64, CU_TENSOR_MAP_SWIZZLE_64B);
  ok = ok && (partials ? make_map(&m_out, part_o, 512, out_rows, 1, 512 * 4, out_rows * 512 * 4, 64,
                                  CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 32)
                       : make_map(&m_out, a.out, 512, out_rows, 1, 512 * 2, out_rows * 512 * 2, 64));
  if (!ok) return DDT_ERR_INVALID_ARG;
  if (ensure_smem_limit(reinterpret_cast<const void*>(verify_attn_q8_kernel), kSmemBytes, 6) !=
      cudaSuccess)
    return DDT_ERR_CUDA;
  Params p;
  p.prefix_lens = a.prefix_lens;
  p.block_table = c.block_table;
  p.scales = c.scales;
  p.q_lat = static_cast<const uint16_t*>(a.q_lat);
  p.q_rope = static_cast<const uint16_t*>(a.q_rope);
  p.mask = a.mask;
  p.lse = a.lse;
  p.part_lse = part_lse;
  p.status = a.status;
  p.B = a.B;
  p.Q = a.q_len;
  p.num_pages = c.num_pages;
  p.max_blocks = c.max_blocks;
  p.num_splits = num_splits;
  p.n_pairs = (a.q_len + 1) / 2;
  p.write_partials = partials;
  p.scale_log2 = a.softmax_scale * kLog2e;
  const int64_t slots = device_sm_count() / 2 > 0 ? device_sm_count() / 2 : 1;
  const int64_t grid = 2 * (items < slots ? items : slots);
  verify_attn_q8_kernel<<<static_cast<unsigned>(grid), kThreads, kSmemBytes, stream>>>(m_lat, m_rope,
                                                                                      m_out, p);
  if (cudaGetLastError() != cudaSuccess) return DDT_ERR_CUDA;
  if (!partials) return DDT_OK;
  ddt_attn_args merge = {};
  merge.B = a.B;
  merge.q_len = a.q_len;
  merge.capacity = c.max_blocks * kPage;
  merge.prefix_lens = a.prefix_lens;
  merge.out = a.out;
  merge.out_dtype = DDT_BF16;
  merge.lse = a.lse;
  return launch_verify_merge(merge, num_splits, 0, part_o, part_lse, stream);
}

cudaError_t q8_fault_flags(uint32_t* flags, bool reset) {
  unsigned int v = 0;
  cudaError_t e = cudaMemcpyFromSymbol(&v, ddt_fault_word, sizeof v);
  if (e != cudaSuccess) return e;
  *flags = v;
  const unsigned int zero = 0;
  return reset ? cudaMemcpyToSymbol(ddt_fault_word, &zero, sizeof zero) : cudaSuccess;
}

}  // namespace ddt
