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
//     down to half a step of e4m3's subnormals, 2^-17 of the row's maximum.
//   * the weights w_j = S_j exp(s_j - m) as hi (e4m3) + lo (e5m2, whose range is wider):
//     relative error 2^-8 as a bf16 weight has, and where hi runs out of range, below 2^-6,
//     at most 2^-14 absolute.  m follows the tiles' largest weights, up and down, so that
//     each tile's lies between 2^-4 and 2^8.75 (see kBase): small weights are kept however
//     many there are and whatever outweighs them.  S_j rides in the exponent (log2 S_j is
//     added to the score), so a page's scale costs nothing per key; the row sum takes
//     sum(w_j of a page) / S_page.  It adds the weights before they are rounded (adding
//     the rounded ones takes another conversion and two additions a pair): a row whose weights are
//     all off in one direction is off by as much, 2^-8 at most.  Scores, sums, the output
//     and the log-sum-exp stay in fp32.
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
//   * warps 0-7 softmax, two threads for each half row (32 keys each): with one, its 64
//     exponentials and splits outlast a tile's MMAs (64 requests x 33 nodes x 4096 rows:
//     1225 us back to back, 1098 us with two).  8 and 12 fill the K rings of even and odd
//     tiles, 10 the V ring; 9 and 14 issue S of even and odd tiles and 11 issues P V, each
//     as a whole warp with one lane elected: descriptors then stay in uniform registers
//     and an MMA goes out every 32 cycles, its own time, where a lone lane's loop manages
//     one in 68 (985 -> 912 us burst).  13 checks a request's page numbers for its status;
//     15-18 split the next item's queries while this one's last tiles are at work, and
//     then write this item's output while the softmax warps go on to the next.
//   * S runs up to four tiles ahead of the softmax; O is rescaled only when a tile's
//     maximum outgrows its reference by 2^4.75 (by 2^2.75: 918 us burst, so: 864) or falls
//     2^8 short of it.
//   * work items are chunks of a request's tiles for a pair of nodes.  The host knows only
//     a bound on the lengths, so the chunk is chosen on the device, by every CTA alike,
//     from the lengths themselves (plan_cost); a request of one chunk is written directly,
//     the others as normalised partials that a second kernel merges (64 single tokens over
//     caches of 1 to 4096 rows: 58 us uncut, 46 us).
//
// What bounds it.  64 x 33 x 4096: 865-895 us in a burst, 1.35-1.40 PFLOP/s = 0.82-0.85 of
// the measured bf16 GEMM burst; 1000-1035 us back to back under the 1 kW power cap, 0.85-0.88
// of the sustained GEMM.  A tile takes 2300-2400 cycles against 2176 of its MMAs (36 x 32 +
// 16 x 64): the softmax of the slower CTA of the pair sets the pace, and an item costs
// 5000-6000 cycles more (its queries are split only once S no longer reads the last ones).
// Short caches and few requests are bound by latency: 15 us for one request x 9 x 256,
// of which launch and plan 3, queries 5, a tile's chain of S, softmax and P V 3, output 2.
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
constexpr int kLSlots = 3;                     // row sums of up to 3 items, see below
constexpr int kQSlots = 6;                     // row scales of up to 6 items, see below
constexpr int kMaxSortedB = 512;                // requests that are put in order
constexpr int kMaxSplitB = 128;                 // requests among which chunks are chosen
constexpr int kOffQ = 0;
constexpr int kOffKRing = kOffQ + kQBytes;
constexpr int kOffVRing = kOffKRing + 2 * kKSlots * kKSlotBytes;
constexpr int kOffP = kOffVRing + kVSlots * kBox;
constexpr int kOffRedMax = kOffP + kPBufs * kPBufBytes;
constexpr int kOffRedL = kOffRedMax + 2 * 256 * 4;  // red_max: float[2][4][64]
constexpr int kRedL = 5 * 64;                       // red_l: four parts of each row sum, its maximum
constexpr int kOffQScale = kOffRedL + kLSlots * kRedL * 4;  // bf16[kQSlots][64]
constexpr int kOffOrder = kOffQScale + kQSlots * 64 * 2;  // uint16[2][kMaxSortedB], see Plan
constexpr int kOffStarts = kOffOrder + 2 * kMaxSortedB * 2;  // uint16[kMaxSortedB + 2]
constexpr int kOffPlan = kOffStarts + (kMaxSortedB + 2) * 2;  // int[4]
constexpr int kOffBar = (kOffPlan + 4 * 4 + 7) / 8 * 8;
constexpr int kOffTiles = kOffP;  // before the first tile: what the plan is made from
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
constexpr int kBarOFree = kBarPVDone + 1;      // both CTAs have read O
constexpr int kBarL = kBarOFree + 1;           // this CTA's row sums of item i (i % kLSlots)
constexpr int kNumBars = kBarL + kLSlots;
constexpr int kOffTmemPtr = kOffBar + kNumBars * 8;
constexpr int kOffAbort = kOffTmemPtr + 4;
constexpr int kSmemUsed = kOffAbort + 4;
constexpr int kSmemBytes = kSmemUsed + 1024;  // slack for 1024-byte alignment
static_assert(kSmemBytes <= 232448, "shared memory budget");
static_assert((2 * kMaxSortedB + 64 + kThreads / 32 * 2 * kMaxSplitB) * 4 <= kPBufs * kPBufBytes, "plan");

constexpr int kTmemCols = 512, kTmemS = 0, kTmemO = 256;
constexpr uint32_t kIdescQK = idesc_e4m3_f32(128, kTK, false);
constexpr uint32_t kIdescPVHi = idesc_e4m3_f32(128, 256, true);
constexpr uint32_t kIdescPVLo = kIdescPVHi | 1u << 7;  // A in e5m2 (format 1)
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
// A weight is held as a multiple of a unit of its row, 2^(m_ref - kBase), and is precise to
// 2^-8 from 2^-6 units on; below, steps are coarser and end at 2^-16.  The unit therefore
// follows the scores, both ways:
//   * up, when a tile's largest weight would pass 2^(kBase + kSlack) = 431 (of 448);
//   * down, when it would lie below 2^(kBase - kDrop) = 2^-4, as behind an attention sink,
//     whose weight may be 2^20 times one of the thousands that follow it and carry the
//     result.  O and the row sum then grow by that power, in fp32, which has room: the unit
//     stays within 2^-kDeep of the largest it was (|O| < 2^30 rows x 2^(kDeep + 9) x 448).
//     A tile of tree rows alone does not lower it: a node sees few of them, at 2^-14 each,
//     and would pay a pass over O at every item's end (1 x 9 x 256: 16.0 against 15.4 us,
//     64 x 33 x 4096 1 % slower);
//   * a tile whose largest weight is 2^kPeak times that of some other 32 of its keys puts it
//     at 2^8.5 units rather than 2^4, for the sake of the keys beside it.
// A change of unit costs a wait for P V and a pass over O, and any row of a warp's 32 causes
// it: for normally distributed scores (deviation 1.7) two rows in five outgrow 2^2.75 between
// the first tile and the 33rd, one in thirty 2^4.75, and falls by 2^8 are as rare.  Next to a
// unit that only rises and a lo in e4m3, which lost whole tails (a sink of 0.8 over 4096
// alike rows: the result 97 % off): 64 x 33 x 4096 881 -> 891 us, 64 x 65 over <= 8192 rows of
// uneven magnitude 1829 -> 1928, 1 x 9 x 256 15.2 -> 15.4.
constexpr float kBase = 4.0f, kSlack = 4.75f, kDrop = 8.0f, kDeep = 48.0f;
constexpr float kPeak = 8.0f, kPeakBase = 4.5f;
constexpr float kMinScale = 9.094947017729282e-13f;  // 2^-40

struct Params {
  const int32_t* prefix_lens;
  const int32_t* block_table;
  const float* scales;
  const uint16_t* q_lat;
  const uint16_t* q_rope;
  const uint64_t* mask;
  uint16_t* out;
  float* lse;
  float* part_o;    // [num_splits][B * Q * 64][512], see part_offset
  float* part_lse;  // [num_splits][B * Q * 64]
  int32_t* status;
  int32_t* chunk;   // the chunk chosen, for the merge
  int B, Q, num_pages, max_blocks, n_pairs;
  int max_splits;   // most chunks of a request that the partials have room for
  int forced;       // cut the longest request into max_splits chunks
  float scale_log2;  // softmax_scale * log2(e)
};

// The work list: first all whole chunks, requests by decreasing length (`order`; starts
// counts the chunks before a request's), then the remainders by decreasing size (order
// + kMaxSortedB).  Consecutive items are the node pairs of one chunk, which share its
// rows in the L2.
struct Plan {
  const uint16_t* order;  // null: requests as they come, one chunk each
  const uint16_t* starts;
  int chunk, full, n_items;  // tiles of a whole chunk; items that are whole chunks; all items
};

struct Item {
  int b, pair, split, P, T, t0, ntile;
  bool single, valid;  // single: the request's only chunk
};

// A request's tiles; 0 for one whose rows do not fit its table.
__device__ __forceinline__ int tiles_of(const Params& p, int P) {
  if (P < 0 || static_cast<int64_t>(P) + p.Q > static_cast<int64_t>(p.max_blocks) * kPage) return 0;
  return (P + p.Q + kTK - 1) / kTK;
}

__device__ __forceinline__ Item decode_item(const Params& p, int w, const Plan& plan) {
  Item it;
  const bool whole = w < plan.full;
  const int v = whole ? w : w - plan.full;
  const int u = v / p.n_pairs;
  it.pair = v - u * p.n_pairs;
  it.split = 0;
  if (!plan.order) {
    it.b = u;
  } else if (whole) {
    int lo = 0, hi = p.B;  // the last request with starts <= u
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (plan.starts[mid] <= u) lo = mid;
      else hi = mid;
    }
    it.b = plan.order[lo];
    it.split = u - plan.starts[lo];
  } else {
    it.b = plan.order[kMaxSortedB + u];
  }
  it.P = p.prefix_lens[it.b];
  it.T = it.P + p.Q;
  const int n = tiles_of(p, it.P);
  const int chunks = n / plan.chunk, rest = n - chunks * plan.chunk;
  if (!whole) it.split = chunks;
  it.t0 = it.split * plan.chunk;
  it.ntile = whole ? plan.chunk : rest;
  it.single = chunks + (rest > 0) == 1;
  it.valid = it.ntile > 0;
  return it;
}

// What a choice of chunk costs, in tiles: the longest of the pairs' shares under the
// schedule that work_index gives, each item counting kItemTiles on top of its tiles
// (queries, filling and draining the pipeline), and the merge.  By one warp, for requests
// of tiles[0 .. B); `sorted` has room for 2 kMaxSplitB numbers.  A request has at most 2^23
// tiles, so a remainder and an index fit into one.
constexpr float kItemTiles = 4.5f, kMergeTiles = 3.f;
__device__ float plan_cost(const int* tiles, int B, int n_pairs, int n_clusters, int chunk,
                           int* sorted) {
  const int lane = threadIdx.x & 31;
  int whole = 0, rests = 0;
  int* key = sorted + kMaxSplitB;  // rest and index in one, so that all differ
  for (int b = lane; b < B; b += 32) {
    const int n = tiles[b] / chunk, rest = tiles[b] - n * chunk;
    whole += n;
    rests += rest > 0;
    key[b] = rest * kMaxSplitB + b;
  }
  __syncwarp();
  for (int b = lane; b < B; b += 32) {
    const int mine = key[b];
    int rank = 0;
#pragma unroll 8
    for (int i = 0; i < B; ++i) rank += key[i] > mine;
    sorted[rank] = mine / kMaxSplitB;
  }
  whole = __reduce_add_sync(0xffffffffu, whole) * n_pairs;
  const int n = whole + __reduce_add_sync(0xffffffffu, rests) * n_pairs;
  __syncwarp();
  float most = 0.f;
  for (int j = lane; j < n_clusters; j += 32) {
    float share = 0.f;
    for (int k = 0; k * n_clusters < n; ++k) {
      const int w = work_index(k, j, n_clusters, n);
      if (w >= 0) share += kItemTiles + (w < whole ? chunk : sorted[n_pairs == 1 ? w - whole : (w - whole) / n_pairs]);
    }
    most = fmaxf(most, share);
  }
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, off));
  return most;
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

// Two floats (lo in the low half) as the sum of two pairs, the first e4m3, the second e4m3
// or e5m2.  fp16 keeps 11 bits and the residual of the first rounding exactly; the values
// lie within 448.
template <bool kWideSecond>
__device__ __forceinline__ void split_f8x2(float lo, float hi, uint16_t& first, uint16_t& second) {
  uint32_t z;
  asm("{\n\t.reg .b32 x, y;\n\t"
      "cvt.rn.f16x2.f32 x, %3, %2;\n\t"
      "cvt.rn.satfinite.e4m3x2.f16x2 %0, x;\n\t"
      "cvt.rn.f16x2.e4m3x2 y, %0;\n\t"
      "sub.rn.f16x2 %1, x, y;\n\t}"
      : "=h"(first), "=r"(z)
      : "f"(lo), "f"(hi));
  if constexpr (kWideSecond) asm("cvt.rn.satfinite.e5m2x2.f16x2 %0, %1;" : "=h"(second) : "r"(z));
  else asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(second) : "r"(z));
}

__device__ __forceinline__ uint32_t pack16(uint16_t lo, uint16_t hi) {
  return static_cast<uint32_t>(lo) | (static_cast<uint32_t>(hi) << 16);
}

__device__ __forceinline__ uint32_t mul_bf16x2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}

// One query row, by a warp: a lane has latent values 16 lane .. + 15 (x[0 .. 7]) and rope
// values 2 lane, 2 lane + 1 (x[8]).
__device__ __forceinline__ void split_row(const uint32_t (&x)[9], uint8_t* q, int row, int lane,
                                          uint16_t* scale) {
  uint32_t m = x[0];
#pragma unroll
  for (int j = 1; j < 9; ++j) m = max_abs_bf16x2(m, x[j]);
  const uint32_t top = __reduce_max_sync(0xffffffffu, max_of_halves(m));
  int e = e4m3_exponent(top);
  e = top == 0 ? 0 : e < -100 ? -100 : e;
  // a power of two: exact in bf16 (down to its subnormals, far below e4m3's steps)
  const uint32_t inv = static_cast<uint32_t>(127 - e) << 7 | static_cast<uint32_t>(127 - e) << 23;
  uint32_t hi[5], lo[5];
#pragma unroll
  for (int j = 0; j < 5; ++j) {
    uint16_t f[4] = {0, 0, 0, 0};
#pragma unroll
    for (int v = 0; v < (j < 4 ? 2 : 1); ++v) {
      const uint32_t h = mul_bf16x2(x[2 * j + v], inv);
      split_f8x2<false>(__uint_as_float(h << 16), __uint_as_float(h & 0xffff0000u), f[v], f[2 + v]);
    }
    hi[j] = pack16(f[0], f[1]);
    lo[j] = pack16(f[2], f[3]);
  }
  uint8_t* at = q + (lane >> 3) * kBox + row * 128 + (((lane & 7) ^ (row & 7)) << 4);
  *reinterpret_cast<uint4*>(at) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
  *reinterpret_cast<uint4*>(at + kQLo) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
  at = q + kQRope + row * 64 + (((lane >> 3) ^ ((row >> 1) & 3)) << 4) + 2 * (lane & 7);
  *reinterpret_cast<uint16_t*>(at) = static_cast<uint16_t>(hi[4]);
  *reinterpret_cast<uint16_t*>(at + kQRopeLo - kQRope) = static_cast<uint16_t>(lo[4]);
  // A row with NaN or an infinity gets NaN as its scale, and so NaN results.
  if (lane == 0) scale[row] = top >= 0x7f80u ? 0x7fc0 : static_cast<uint16_t>((e + 127) << 7);
}

// 32 bytes, aligned to a sector.
__device__ __forceinline__ void store_sector(void* at, const uint32_t (&y)[8]) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(at), "r"(y[0]), "r"(y[1]),
               "r"(y[2]), "r"(y[3]), "r"(y[4]), "r"(y[5]), "r"(y[6]), "r"(y[7])
               : "memory");
}

// 32 bytes of memory that the kernel does not write.
__device__ __forceinline__ void load_sector(const float* at, float (&y)[8]) {
  asm("ld.global.nc.v8.f32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
      : "=f"(y[0]), "=f"(y[1]), "=f"(y[2]), "=f"(y[3]), "=f"(y[4]), "=f"(y[5]), "=f"(y[6]),
        "=f"(y[7])
      : "l"(at));
}

// Place of columns col .. col + 7 of a row of the partials: a node's 64 heads side by side
// in each group of eight columns, so that a warp of lanes that hold a row each stores
// whole lines (a chunk's end 9000 -> 5600 cycles, 64 single tokens 48.1 -> 45.6 us).
__device__ __forceinline__ int64_t part_offset(int64_t row, int col) {
  return (row >> 6) * (64 * DDT_D_LATENT) + (col >> 3) * (64 * 8) + (row & 63) * 8;
}

__device__ __forceinline__ void prefetch_l2(const void* p) {
  asm volatile("prefetch.global.L2 [%0];" ::"l"(p));
}

}  // namespace vq

// Persistent kernel: each CTA pair loops over work items (see work_index); rings,
// barriers and tensor memory live across items, and phases follow a count G of the tiles
// of all items that a CTA has seen.
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(vq::kThreads, 1)
    verify_attn_q8_kernel(const __grid_constant__ CUtensorMap tm_lat,
                          const __grid_constant__ CUtensorMap tm_rope, const vq::Params p) {
  using namespace vq;
  const uint32_t rank = cluster_ctarank();
  const int cluster = static_cast<int>(blockIdx.x >> 1);
  const int n_clusters = static_cast<int>(gridDim.x >> 1);
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
  uint16_t* q_scale = reinterpret_cast<uint16_t*>(base + kOffQScale);  // as bf16, a power of two
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
    mbar_init(bar(kBarOFree), 2 * kQWarps);  // every writing warp of the pair
    for (int s = 0; s < kLSlots; ++s) mbar_init(bar(kBarL + s), kSoftmaxThreads);
    *abort_flag = 0;
    fence_mbar_init_cluster();
  }
  if (warp == kWarpSIss0) {
    tmem_alloc<2>(smem_u32(tmem_ptr_smem), kTmemCols);
    tmem_relinquish<2>();
  }
  __syncwarp();
  tc_fence_before_sync();
  cluster_arrive();  // barriers and tensor memory are ready
  // The plan, made by every CTA for itself.
  int* const plan_smem = reinterpret_cast<int*>(base + kOffPlan);  // longest, shortest, whole chunks
  Plan plan = {nullptr, nullptr, INT_MAX, 0, p.B * p.n_pairs};
  if (p.B <= kMaxSortedB) {
    int* tiles = reinterpret_cast<int*>(base + kOffTiles);
    int* rests = tiles + kMaxSortedB;
    float* costs = reinterpret_cast<float*>(rests + kMaxSortedB);  // [64]
    int* sorted = rests + kMaxSortedB + 64;                        // of each warp
    uint16_t* order = reinterpret_cast<uint16_t*>(base + kOffOrder);
    uint16_t* starts = reinterpret_cast<uint16_t*>(base + kOffStarts);
    plan.order = order;
    plan.starts = starts;
    const int mine = threadIdx.x < p.B ? tiles_of(p, p.prefix_lens[threadIdx.x]) : 0;
    if (threadIdx.x == 0) {
      plan_smem[0] = 1;
      plan_smem[1] = INT_MAX;
    }
    __syncthreads();
    if (threadIdx.x < p.B) {
      tiles[threadIdx.x] = mine;
      atomicMax(&plan_smem[0], mine);
      atomicMin(&plan_smem[1], mine);
    }
    __syncthreads();
    const int longest = plan_smem[0];
    const bool differs = plan_smem[1] != longest;
    plan.chunk = p.forced ? (longest + p.max_splits - 1) / p.max_splits : longest;
    if (p.max_splits > 1 && !p.forced) {
      // one warp prices one number of chunks for the longest request
      const int most = p.max_splits < longest ? p.max_splits : longest;
      for (int c = warp + 1; c <= most; c += kThreads / 32) {
        const float cost = plan_cost(tiles, p.B, p.n_pairs, n_clusters, (longest + c - 1) / c,
                                     sorted + warp * (2 * kMaxSplitB));
        if (lane == 0) costs[c - 1] = c > 1 ? cost + kMergeTiles : cost;
      }
      __syncthreads();
      int best = 1;
      for (int c = 2; c <= most; ++c)
        if (costs[c - 1] < costs[best - 1]) best = c;
      plan.chunk = (longest + best - 1) / best;
    }
    const int rest = mine % plan.chunk;
    if (threadIdx.x < p.B) rests[threadIdx.x] = rest;
    const int n_rests = __syncthreads_count(rest > 0);
    if (threadIdx.x < p.B) {
      int before = threadIdx.x, before_rest = threadIdx.x;
      if (differs) {
        before = before_rest = 0;
        const int i = threadIdx.x;
#pragma unroll 4
        for (int j = 0; j < p.B; ++j) {
          const int tj = tiles[j], rj = rests[j];
          before += tj > mine || (tj == mine && j < i);
          before_rest += rj > rest || (rj == rest && j < i);
        }
      }
      order[before] = static_cast<uint16_t>(threadIdx.x);
      order[kMaxSortedB + before_rest] = static_cast<uint16_t>(threadIdx.x);
    }
    __syncthreads();
    if (warp == 0) {
      int sum = 0;
      for (int r0 = 0; r0 < p.B; r0 += 32) {
        const int r = r0 + lane;
        const int whole = r < p.B ? tiles[order[r]] / plan.chunk : 0;
        int upto = whole;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
          const int o = __shfl_up_sync(0xffffffffu, upto, off);
          if (lane >= off) upto += o;
        }
        if (r < p.B) starts[r] = static_cast<uint16_t>(sum + upto - whole);
        sum += __shfl_sync(0xffffffffu, upto, 31);
      }
      if (lane == 0) plan_smem[2] = sum;
    }
    __syncthreads();
    plan.full = plan_smem[2] * p.n_pairs;
    plan.n_items = plan.full + n_rests * p.n_pairs;
    if (p.max_splits > 1 && blockIdx.x == 0 && threadIdx.x == 0) *p.chunk = plan.chunk;
  }
  const int n_items = plan.n_items;
  const int n_rounds = (n_items + n_clusters - 1) / n_clusters;
  __syncwarp();
  cluster_wait();
  tc_fence_after_sync();
  const uint32_t tmem = *tmem_ptr_smem;

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
  // Rows r .. r + 3 of this CTA's node of item `it`, split by one warp.
  auto split_rows = [&](const Item& it, int r, int iter) {
    const int node = 2 * it.pair + static_cast<int>(rank);
    const int64_t row0 = (static_cast<int64_t>(it.b) * Q + node) * 64 + r;
    const uint4* lat = reinterpret_cast<const uint4*>(p.q_lat) + row0 * 64 + 2 * lane;
    const uint32_t* rope = reinterpret_cast<const uint32_t*>(p.q_rope) + row0 * 32 + lane;
    uint32_t x[4][9];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      uint4 a = make_uint4(0, 0, 0, 0), c = a;
      x[i][8] = 0;
      if (node < Q) {
        a = lat[i * 64];
        c = lat[i * 64 + 1];
        x[i][8] = rope[i * 32];
      }
      x[i][0] = a.x, x[i][1] = a.y, x[i][2] = a.z, x[i][3] = a.w;
      x[i][4] = c.x, x[i][5] = c.y, x[i][6] = c.z, x[i][7] = c.w;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
      split_row(x[i], base + kOffQ, r + i, lane, q_scale + iter % kQSlots * 64);
  };
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
        const Item it = decode_item(p, w, plan);
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
        const Item it = decode_item(p, w, plan);
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
    // Issuer g takes tiles G with G % 2 == g; tile G goes to S buffer G % 4.  The whole
    // warp runs the loop and one lane issues: descriptors then stay in uniform registers
    // and an MMA goes out every 32 cycles, its own time, where a lone lane's loop manages
    // one in 68.
    if (leader) {
      const bool one = elect_one();
      const int g = ring_g;
      const int full0 = kBarKFull + g * kKSlots, empty0 = kBarKEmpty + g * kKSlots;
      const uint32_t ring = base_addr + kOffKRing + g * kKSlots * kKSlotBytes;
      const uint64_t q_desc = smem_desc_sw128(sQ, 16, 1024);
      const uint64_t rope_desc = smem_desc_sw64(sQ + kQRope);
      Ring r;
      int iter = 0;
      int64_t G = 0;
      for (int k = 0; k < n_rounds; ++k) {
        const int w = work_index(k, cluster, n_clusters, n_items);
        if (w < 0) continue;
        const Item it = decode_item(p, w, plan);
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
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            mbar_wait(bar(full0 + r.stage), r.phase, abort_flag);
            const uint32_t slot = ring + r.stage * kKSlotBytes;
            const uint64_t k_desc = smem_desc_sw128(slot, 16, 1024);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const uint64_t kd = k_desc + (((i >> 2) * kBox + 32 * (i & 3)) >> 4);
              const uint64_t qd = q_desc + (((2 * half + (i >> 2)) * kBox + 32 * (i & 3)) >> 4);
              if (one) mma_f8_ss<2>(d, qd, kd, kIdescQK, half + i != 0);
              if (one) mma_f8_ss<2>(d, qd + (kQLo >> 4), kd, kIdescQK, 1);
            }
            if (half == 0) {
              const uint64_t r_desc = smem_desc_sw64(slot + kKRopeOff);
#pragma unroll
              for (int ks = 0; ks < 2; ++ks) {
                if (one) mma_f8_ss<2>(d, rope_desc + 2 * ks, r_desc + 2 * ks, kIdescQK, 1);
                if (one)
                  mma_f8_ss<2>(d, rope_desc + ((kQRopeLo - kQRope) >> 4) + 2 * ks, r_desc + 2 * ks,
                               kIdescQK, 1);
              }
            }
            if (one) mma_commit<2>(bar(empty0 + r.stage), 0x3);
            r.advance(kKSlots);
          }
          if (one) mma_commit<2>(bar(kBarS + sbuf), 0x3);
        }
        if (one) mma_commit<2>(bar(kBarQFree), 0x3);  // this issuer no longer reads this item's Q
        ++iter;
      }
      if (one) mma_commit<2>(bar(kBarQKDone + g), 0x1);
      __syncwarp();
      mbar_wait(bar(kBarQKDone + g), 0, abort_flag);
    }
    __syncwarp();
  } else if (warp == kWarpPVIss) {
    // ---------------------------------------------------------- MMA: O += P V
    if (leader) {
      const bool one = elect_one();
      Ring r;
      int iter = 0;
      int64_t G = 0;
      for (int k = 0; k < n_rounds; ++k) {
        const int w = work_index(k, cluster, n_clusters, n_items);
        if (w < 0) continue;
        const Item it = decode_item(p, w, plan);
        if (!it.valid) continue;
        if (iter > 0) {  // both CTAs' output warps have read the previous item's O
          mbar_wait(bar(kBarOFree), static_cast<uint32_t>((iter - 1) & 1), abort_flag);
          tc_fence_after_sync();
        }
        for (int jj = 0; jj < it.ntile; ++jj, ++G) {
          const int pb = static_cast<int>(G % kPBufs);
          mbar_wait(bar(kBarP + pb), static_cast<uint32_t>((G / kPBufs) & 1), abort_flag);
          tc_fence_after_sync();
          const uint64_t p_desc = smem_desc_sw128(sP + pb * kPBufBytes, 16, 1024);
#pragma unroll
          for (int i = 0; i < 4; ++i) {  // page i / 2, column half i % 2
            mbar_wait(bar(kBarVFull + r.stage), r.phase, abort_flag);
            const uint32_t d = tmem + kTmemO + 128u * (i & 1);
            const uint64_t v_desc = smem_desc_sw128(sVRing + r.stage * kBox, kBox, 1024);
#pragma unroll
            for (int ks = 0; ks < 2; ++ks) {
              const uint64_t pd = p_desc + ((kPage * (i >> 1) + 32 * ks) >> 4);
              const uint64_t vd = v_desc + ((4096 * ks) >> 4);
              if (one) mma_f8_ss<2>(d, pd, vd, kIdescPVHi, jj > 0 || i >= 2 || ks > 0);
              if (one) mma_f8_ss<2>(d, pd + (kBox >> 4), vd, kIdescPVLo, 1);
            }
            if (one) mma_commit<2>(bar(kBarVEmpty + r.stage), 0x3);
            r.advance(kVSlots);
          }
          if (one) mma_commit<2>(bar(kBarO + static_cast<int>(G & 3)), 0x3);
        }
        ++iter;
      }
      if (one) mma_commit<2>(bar(kBarPVDone), 0x1);
      __syncwarp();
      mbar_wait(bar(kBarPVDone), 0, abort_flag);
    }
    __syncwarp();
  } else if (warp >= kWarpQ0) {
    // ----------------------- queries to e4m3 hi + lo, and outputs to memory
    const int u = warp - kWarpQ0;
    const uint32_t q_bar = map_to_rank(bar(kBarQ), 0);
    const uint32_t o_free_leader = map_to_rank(bar(kBarOFree), 0);
    // Rows 16 u .. 16 u + 15 of this CTA's node of item `it`, the iter-th one.
    auto split_queries = [&](const Item& it, int iter) {
      const int node = 2 * it.pair + static_cast<int>(rank);
      const int64_t row0 = (static_cast<int64_t>(it.b) * Q + node) * 64 + 16 * u;
      if (node < Q) {  // rows of 1024 and of 128 bytes, one line a lane
#pragma unroll
        for (int i = 0; i < 4; ++i) prefetch_l2(p.q_lat + row0 * 512 + (32 * i + lane) * 64);
        if (lane < 16) prefetch_l2(p.q_rope + row0 * 64 + lane * 64);
      }
      if (iter > 0)
        mbar_wait(bar(kBarQFree), static_cast<uint32_t>((iter - 1) & 1), abort_flag);
#pragma unroll 1
      for (int r = 16 * u; r < 16 * u + 16; r += 4) split_rows(it, r, iter);
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive_local(bar(kBarQScale + iter % kQSlots));
        mbar_arrive_cluster(q_bar);
      }
    };
    int k = 0;
    auto next_item = [&](Item& it) {
      for (; k < n_rounds; ++k) {
        const int w = work_index(k, cluster, n_clusters, n_items);
        if (w < 0) continue;
        it = decode_item(p, w, plan);
        if (it.valid) {
          ++k;
          return true;
        }
      }
      return false;
    };
    Item cur, nxt;
    bool have = next_item(cur);
    if (have) split_queries(cur, 0);
    int64_t G = 0;
    const int t = (warp & 3) * 32 + lane;  // TMEM lane
    const int m = t & 63, hf = t >> 6;
    const uint32_t lane_addr = static_cast<uint32_t>((warp & 3) * 32) << 16;
    for (int iter = 0; have; ++iter) {
      const bool more = next_item(nxt);
      if (more) split_queries(nxt, iter + 1);
      // The row sums of item i lie in slot i % 3: the softmax of item j is done only once
      // the output of item j - 3 is (two P buffers, and the P V of an item waits for the
      // output of the one before).
      G += cur.ntile;
      const float* red = red_l + iter % kLSlots * kRedL;
      mbar_wait(bar(kBarL + iter % kLSlots), static_cast<uint32_t>((iter / kLSlots) & 1), abort_flag);
      const float l_row = (red[m] + red[64 + m]) + (red[128 + m] + red[192 + m]);
      const float m_use = red[256 + m];
      const bool empty_row = l_row == 0.f;
      const float inv = empty_row ? 0.f : 1.f / l_row;
      const float lse_nat = empty_row ? -INFINITY : (m_use - kBase + __log2f(l_row)) * kLn2;
      const int node = 2 * cur.pair + static_cast<int>(rank);
      const int64_t row = (static_cast<int64_t>(cur.b) * Q + node) * 64 + m;
      mbar_wait(bar(kBarO + static_cast<int>((G - 1) & 3)), static_cast<uint32_t>(((G - 1) >> 2) & 1),
                abort_flag);
      tc_fence_after_sync();
      // Lane t has columns 256 nh + 128 hf + 0 .. 127 of its row; 32 at a time, in runs
      // of whole 32-byte sectors.
      if (node < Q) {
        const int64_t prow = cur.split * static_cast<int64_t>(p.B) * Q * 64 + row;
        uint16_t* out = p.out + row * DDT_D_LATENT + 128 * hf;
        float* part = p.part_o + part_offset(prow, 128 * hf);
#pragma unroll 1
        for (int q = 0; q < 8; ++q) {
          uint32_t o[32];
          tmem_ld32(tmem + lane_addr + kTmemO + 32u * q, o);
          tmem_wait_ld();
          if (q == 7) {
            tc_fence_before_sync();
            __syncwarp();
            if (lane == 0) mbar_arrive_cluster(o_free_leader);
          }
          const int col = 256 * (q >> 2) + 32 * (q & 3);
          if (cur.single) {
#pragma unroll
            for (int v = 0; v < 2; ++v) {
              uint32_t y[8];
#pragma unroll
              for (int z = 0; z < 8; ++z)
                y[z] = pack_bf16x2(__uint_as_float(o[16 * v + 2 * z]) * inv,
                                   __uint_as_float(o[16 * v + 2 * z + 1]) * inv);
              store_sector(out + col + 16 * v, y);
            }
          } else {  // a chunk's normalised fp32 partial
#pragma unroll
            for (int v = 0; v < 4; ++v) {
              uint32_t y[8];
#pragma unroll
              for (int z = 0; z < 8; ++z) y[z] = __float_as_uint(__uint_as_float(o[8 * v + z]) * inv);
              store_sector(part + part_offset(0, col + 8 * v), y);
            }
          }
        }
        if (hf == 0) {
          if (!cur.single) p.part_lse[prow] = lse_nat;
          else if (p.lse) p.lse[row] = lse_nat;
        }
      } else {  // a node past q_len (odd q_len): nothing to write
        tc_fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive_cluster(o_free_leader);
      }
      cur = nxt;
      have = more;
    }
  } else if (warp == kWarpStatus) {
    // Every request's status, by one even CTA: whether its prefix fits and all its page
    // numbers are some.
    if (leader && p.status) {
      for (int b = cluster; b < p.B; b += n_clusters) {
        const int P = p.prefix_lens[b];
        int st = DDT_REQ_OK;
        if (tiles_of(p, P) == 0) {
          st = DDT_REQ_BAD_PREFIX;
        } else {
          bool bad = false;
          for (int blk = lane; blk * kPage < P + Q; blk += 32) {
            const int page = p.block_table[static_cast<int64_t>(b) * p.max_blocks + blk];
            bad |= page < 0 || page >= p.num_pages;
          }
          if (__any_sync(0xffffffffu, bad)) st = DDT_REQ_BAD_INDEX;
        }
        if (lane == 0) p.status[b] = st;
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
      const Item it = decode_item(p, w, plan);
      if (!it.valid) continue;
      const int b = it.b, P = it.P;
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
      // The row scales of item i lie in slot i % 6: queries run at most five items ahead
      // (four S buffers), so a slot is read before it is written again.
      const int slot = iter % kQSlots;
      mbar_wait(bar(kBarQScale + slot), static_cast<uint32_t>((iter / kQSlots) & 1), abort_flag);
      const float row_scale =
          __uint_as_float(static_cast<uint32_t>(q_scale[slot * 64 + m]) << 16) * p.scale_log2;
      ++iter;
      float m_ref = -INFINITY;  // log2 units, page scale included
      float m_low = -INFINITY;  // the reference falls no further
      float l_sum = 0.f;
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
        // mx - m_ref outside [-kDrop, kSlack] (false where both are -inf)
        if (fabsf(mx - m_ref + 0.5f * (kDrop - kSlack)) > 0.5f * (kDrop + kSlack)) {
          const float least = fminf(fminf(red[m], red[64 + m]), fminf(red[128 + m], red[192 + m]));
          float next = mx - least > kPeak ? mx - kPeakBase : mx;
          if (mx < m_ref)  // not for a tile of tree rows alone, nor one that shows no key
            next = kPage * (blk - hf) >= P || mx == -INFINITY ? m_ref : fmaxf(next, m_low);
          if (m_ref != -INFINITY && next != m_ref) {
            factor = fast_exp2(m_ref - next);
            l_sum *= factor;
            rescale = true;
          }
          m_ref = next;
          m_low = fmaxf(m_low, m_ref - kDeep);
        }
        const float shift = lk - (m_ref == -INFINITY ? 0.f : m_ref) + kBase;
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
            split_f8x2<true>(e0, e1, f[v], f[2 + v]);
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
      // The row sums and their reference go to the output warps.
      float* red = red_l + (iter - 1) % kLSlots * kRedL;
      red[part_of] = l_sum;
      if (t < 64) red[256 + m] = m_ref == -INFINITY ? 0.f : m_ref;
      mbar_arrive_local(bar(kBarL + (iter - 1) % kLSlots));
    }
  }

  // All MMAs of the pair are complete (the output warps waited for the last O,
  // the issuers for their final commits); release tensor memory.
  __syncwarp();
  tc_fence_before_sync();
  cluster_sync();
  if (warp == kWarpSIss0) {
    tc_fence_after_sync();
    tmem_dealloc<2>(tmem, kTmemCols);
  }
}

// lse = ln sum_s exp(lse_s), out = sum_s exp(lse_s - lse) out_s over the chunks of a request
// that has several; the others have been written.  A CTA has eight heads of a node; a warp
// has 64 columns of them, eight lanes (of eight columns each) for each of four heads at a
// time; neighbouring lanes have neighbouring heads, whose partials are one line (with
// neighbouring columns instead: 6.3 against 4.9 us for 64 single tokens).
__global__ void __launch_bounds__(256, 3) verify_merge_q8_kernel(
    const float* __restrict__ part_o, const float* __restrict__ part_lse,
    const int32_t* __restrict__ chunk, const int32_t* __restrict__ prefix_lens,
    uint16_t* __restrict__ out, float* __restrict__ lse, int B, int Q, int max_blocks) {
  const int64_t rows_total = static_cast<int64_t>(B) * Q * 64;
  const int lane = threadIdx.x & 31, sub = lane >> 2;
  const int64_t row0 = static_cast<int64_t>(blockIdx.x) * 8 + (lane & 3);  // and row0 + 4
  const int col = 64 * (threadIdx.x >> 5) + 8 * sub;
  const int c = *chunk;
  const int P = prefix_lens[blockIdx.x / (8 * static_cast<unsigned>(Q))];
  if (P < 0 || static_cast<int64_t>(P) + Q > static_cast<int64_t>(max_blocks) * vq::kPage) return;
  const int n = ((P + Q + vq::kTK - 1) / vq::kTK + c - 1) / c;  // at most 64
  if (n <= 1) return;
  // Two chunks of two heads in flight, the first ones while the weights are found.
  float v[2][2][8];
  const float* at = part_o + vq::part_offset(row0, col);
  auto fetch = [&](int s0) {
#pragma unroll
    for (int u = 0; u < 2; ++u)
      if (s0 + u < n)
#pragma unroll
        for (int h = 0; h < 2; ++h)
          vq::load_sector(at + (s0 + u) * rows_total * DDT_D_LATENT + 4 * h * 8, v[u][h]);
  };
  fetch(0);
  // A head's eight lanes share its chunks' log-sum-exps.
  float first[2], top[2], w[2], sum[2], acc[2][8] = {};
#pragma unroll
  for (int h = 0; h < 2; ++h)
    first[h] = top[h] = sub < n ? part_lse[sub * rows_total + row0 + 4 * h] : -INFINITY;
  for (int s = sub + 8; s < n; s += 8)
#pragma unroll
    for (int h = 0; h < 2; ++h) top[h] = fmaxf(top[h], part_lse[s * rows_total + row0 + 4 * h]);
#pragma unroll
  for (int h = 0; h < 2; ++h) {
#pragma unroll
    for (int off = 4; off < 32; off <<= 1) top[h] = fmaxf(top[h], __shfl_xor_sync(0xffffffffu, top[h], off));
    // NaN stays NaN; a row that sees no key in any chunk has sum 0
    if (top[h] == -INFINITY) top[h] = 0.f;
    sum[h] = 0.f;
  }
  for (int s0 = 0; s0 < n; s0 += 2) {
    if ((s0 & 7) == 0) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        float l = first[h];
        if (s0 > 0) l = s0 + sub < n ? part_lse[(s0 + sub) * rows_total + row0 + 4 * h] : -INFINITY;
        w[h] = l == -INFINITY ? 0.f : fast_exp2((l - top[h]) * vq::kLog2e);
        sum[h] += w[h];
      }
    }
#pragma unroll
    for (int u = 0; u < 2; ++u)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const float wu = __shfl_sync(0xffffffffu, w[h], 4 * ((s0 & 6) + u) + (lane & 3));  // 0 past the last
        if (wu != 0.f) {
#pragma unroll
          for (int k = 0; k < 8; ++k) acc[h][k] += wu * v[u][h][k];
        }
      }
    fetch(s0 + 2);
  }
#pragma unroll
  for (int h = 0; h < 2; ++h) {
#pragma unroll
    for (int off = 4; off < 32; off <<= 1) sum[h] += __shfl_xor_sync(0xffffffffu, sum[h], off);
    const float inv = sum[h] == 0.f ? 0.f : 1.f / sum[h];
    const float(&a)[8] = acc[h];
    const int64_t row = row0 + 4 * h;
    *reinterpret_cast<uint4*>(out + row * DDT_D_LATENT + col) =
        make_uint4(pack_bf16x2(a[0] * inv, a[1] * inv), pack_bf16x2(a[2] * inv, a[3] * inv),
                   pack_bf16x2(a[4] * inv, a[5] * inv), pack_bf16x2(a[6] * inv, a[7] * inv));
    if (lse && col == 0) lse[row] = sum[h] == 0.f ? -INFINITY : top[h] + __logf(sum[h]);
  }
}

// Most chunks of a request that a call may use: one past kMaxSortedB requests (the work list
// is then none), where the items fill the CTA pairs anyhow or the caches are short (partials
// and their merge cost about as much as three tiles), else enough to fill them a few times
// over, within the tiles.  Items that fill the pairs are balanced by their order alone where
// lengths are alike; one request much longer than its batch is not cut there and runs on by
// itself (128 single tokens, one over 32768 rows and the others over 1024: 261 tiles on one
// pair against 27 on the average, by plan_cost), since partials are laid out for all rows
// times all chunks.
int q8_max_splits(const ddt_attn_q8_args& a, int sm_count) {
  if (a.B > vq::kMaxSortedB) return 1;
  if (a.num_splits > 0) return a.num_splits;
  const int64_t slots = sm_count / 2 > 0 ? sm_count / 2 : 1;
  const int64_t items = static_cast<int64_t>(a.B) * ((a.q_len + 1) / 2);
  const int64_t tiles = (static_cast<int64_t>(a.max_prefix) + a.q_len + vq::kTK - 1) / vq::kTK;
  if (items >= slots || a.B > vq::kMaxSplitB || tiles < 8) return 1;
  const int64_t most = 4 * slots / items + 1 < tiles ? 4 * slots / items + 1 : tiles;
  return static_cast<int>(most < 32 ? most : 32);
}

size_t q8_workspace_bytes(const ddt_attn_q8_args& a, int max_splits) {
  if (max_splits <= 1) return 0;
  const size_t rows = static_cast<size_t>(a.B) * a.q_len * 64;
  return 256 + static_cast<size_t>(max_splits) * rows * (DDT_D_LATENT + 1) * sizeof(float);
}

ddt_status launch_verify_attn_q8(const ddt_attn_q8_args& a, int max_splits, void* workspace,
                                 cudaStream_t stream) {
  using namespace vq;
  const ddt_q8_cache& c = a.cache;
  const uint64_t pages = static_cast<uint64_t>(c.num_pages);
  const int64_t rows = static_cast<int64_t>(a.B) * a.q_len * 64;
  const int64_t items = static_cast<int64_t>(a.B) * ((a.q_len + 1) / 2) * max_splits;
  if (items > 0x3fffffffll || rows / 8 > INT_MAX) return DDT_ERR_UNSUPPORTED;
  // With one page its stride is never taken, but the map wants one.
  const uint64_t lat_page = c.num_pages > 1 ? c.ckv_page_stride : kPage * c.ckv_row_stride;
  const uint64_t rope_page = c.num_pages > 1 ? c.kr_page_stride : kPage * c.kr_row_stride;
  CUtensorMap m_lat, m_rope;
  const bool ok = make_map(&m_lat, c.c_kv, DDT_D_LATENT, kPage, pages, c.ckv_row_stride, lat_page, kPage,
                           CU_TENSOR_MAP_DATA_TYPE_UINT8, 128) &&
                  make_map(&m_rope, c.k_rope, DDT_D_ROPE, kPage, pages, c.kr_row_stride, rope_page, kPage,
                           CU_TENSOR_MAP_DATA_TYPE_UINT8, 64, CU_TENSOR_MAP_SWIZZLE_64B);
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
  p.out = static_cast<uint16_t*>(a.out);
  p.lse = a.lse;
  p.chunk = static_cast<int32_t*>(workspace);
  p.part_o = max_splits > 1 ? reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + 256) : nullptr;
  p.part_lse = max_splits > 1 ? p.part_o + max_splits * rows * DDT_D_LATENT : nullptr;
  p.status = a.status;
  p.B = a.B;
  p.Q = a.q_len;
  p.num_pages = c.num_pages;
  p.max_blocks = c.max_blocks;
  p.n_pairs = (a.q_len + 1) / 2;
  p.max_splits = max_splits;
  p.forced = a.num_splits > 0;
  p.scale_log2 = a.softmax_scale * kLog2e;
  const int64_t slots = device_sm_count() / 2 > 0 ? device_sm_count() / 2 : 1;
  const int64_t grid = 2 * (items < slots ? items : slots);
  verify_attn_q8_kernel<<<static_cast<unsigned>(grid), kThreads, kSmemBytes, stream>>>(m_lat, m_rope, p);
  if (cudaGetLastError() != cudaSuccess) return DDT_ERR_CUDA;
  if (max_splits <= 1) return DDT_OK;
  verify_merge_q8_kernel<<<static_cast<unsigned>(rows / 8), 256, 0, stream>>>(
      p.part_o, p.part_lse, p.chunk, a.prefix_lens, p.out, a.lse, a.B, a.q_len, c.max_blocks);
  return cudaGetLastError() == cudaSuccess ? DDT_OK : DDT_ERR_CUDA;
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
