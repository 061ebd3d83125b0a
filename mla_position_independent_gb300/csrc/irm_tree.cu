// Attention of a tree of drafted tokens over the paged cache (absorbed MLA), sm_103a.
//
// Per query row (node i, head h) of a request with ctx committed rows and n drafts:
//   s_t = scale * (q_lat . cKV_t + q_rope . k_r,t) over the rows t < ctx and the drafts' rows
//   ctx + k whose bit k is set in node i's mask;  O = softmax(s) . cKV, lse = ln sum exp(s).
//
// Work unit: 128 query rows (of a request's n H rows, node-major) x a run of pages, on a pair
// of CTAs (a cluster of 2, one CTA per SM); a page (64 rows) is one tile.
//   - The contraction of Q K^T and the columns of O are split over the pair: CTA r loads, with
//     TMA, cKV columns [256 r, 256 r + 256) and k_r columns [32 r, 32 r + 32) of each page, so
//     each row is read once by the pair, and 32 KiB a tile leave room for five tiles in flight.
//     128 rows x 512 fp32 columns of O alone would fill one SM's TMEM.
//   - The softmax is split by rows: CTA r owns query rows [64 r, 64 r + 64).  Each CTA sends the
//     other its fp32 partial scores of the other's rows (16 KiB a tile, st.async from registers),
//     adds what it receives to its own partials, and after the exponentials writes its rows of P
//     for its own P V and copies them to the other's (8 KiB a tile, one bulk copy a warp).
//     Nothing is computed twice, and no partial score is rounded on the way.
//   - O accumulates in TMEM (256 columns), P V reads P and the page's cKV from shared memory;
//     Q K^T reads Q's cKV columns from TMEM (128 columns) into one of two score buffers (64 each).
//   - Two sets of four warps take even and odd tiles, a thread a row: of each set the two warps
//     of the CTA's own rows run the softmax, the other two ship scores.  While one set is in its
//     exponentials the other is in its exchange; all that passes from tile to tile is the running
//     maximum (in shared memory, one mbarrier per 32 rows).
//   - The maximum moves only when a tile exceeds it by 2^8 (P stays <= 256, and the final sum uses
//     the same maximum, so the result is exact); then the owner's factor per row, which travels
//     with P, rescales O in both CTAs.  l is summed in fp32 before P is rounded to bf16 for
//     the tensor cores (the rounding of P, half a step of bf16 a key, is of the output's own size).
//   - Rows that no node of the unit sees (masked drafts, rows behind the last one) may hold NaN.
//     Their scores are replaced whatever they are; a warp clears their cKV columns in shared memory,
//     beside Q K^T, before P V reads them.
// Warps: 0-7 scores, 8 TMA, 9 Q K^T issue and TMEM, 10 P V issue, 11 Q and the clearing (8-bit: Q and k_r),
// and over an 8-bit cache 12-15 the conversion.
//
// 8-bit cache (tree_attn_kernel<true>; rows of 512 e4m3 codes, a scale for 128 columns, and k_r in bf16).  The
// same kernel, but TMA brings codes (16 KiB a page and CTA, two pages in flight), and four warps turn them into
// the bf16 tile that the tensor core reads, a thread a row of 128 columns: with a power of two as scale that
// is exact (down to bf16's least step, 2^-133), so scores, probabilities and O are rounded nowhere else than over a bf16 cache.  The tensor core's
// own 8-bit form was not taken: it would need P in 8 bits, whose 2^-9 to 448 lose the many small probabilities
// next to one large one.  A code takes 4 instructions with its loads, stores and waits; unseen rows are
// converted with scale 0, which clears them.  Pages wait as codes, so four pages of bf16 do.
//
// Long contexts are cut into pieces of equal length (the rest last, so that the short ones fill the
// gaps); their normalised fp32 partials are merged by a second kernel.
// Every wait is bounded (2 s) and reports a timeout in the status word.
//
// What bounds it.  64 requests x 32768 rows, 128 heads, two nodes: 850 to 866 us by replay, 1.36 PFLOP/s, 0.70 of
// the measured bf16 rate (before the waits in fewer instructions 866 to 872, and 940 once under the power cap at 1.77
// GHz); a tile takes 0.94 us in the units' own time, ~1800 cycles.  Two limits are near it:
//   - Issue of MMAs: at N = 64 one takes 44.5 cycles, not 32, so that Q K^T (18) and P V (4 of 128
//     cycles) keep the tensor core for 1313 cycles a tile.  N = 128 runs at the full rate, but two
//     pages at once start both sets at once: 1066 us.
//   - The tiles in flight: a page is held from its TMA until its P V, ~8000 cycles, in which a softmax
//     warp waits ~1070 cycles for the other CTA's scores.  With four pages in flight 975 us (855 with
//     five), although the received scores then have a buffer for each set.  So everything else makes
//     room for the fifth: one buffer for received scores (their senders keep them in registers until it
//     is free), k_r in a ring of two.
// Measured and not taken (64 x 32768, when the kernel stood at the figure in brackets): P by st.async of
// 16 bytes 1115 (988 with bulk copies); scores by bulk copies 1049 (991); by plain remote stores and a
// release 1193 (988); tiles of 32 rows, four sets 1381 (988); pages of 64 rows with four sets of 32
// keys 1010 (988); softmax split by keys 1.09 times the time; a second warp for each row 1.18 times.
// Few rows (16 heads, one node, 76 requests) stream 0.88 us a further page, 6.3 TB/s, 0.93 of the
// measured copy rate.  One short request (512 rows, 16 heads) takes 12.1 us, of which one tile alone
// (63 rows) is 8.4: it is set-up, the chain of one tile and the way out.
// The 8-bit cache: 64 x 32768 rows, 128 heads, two nodes 1057 us (1.10 PFLOP/s, 0.57 of the measured rate).  It holds
// 0.57 of the bytes, but at every shape measured it is slower than a bf16 cache on the same GPU: these 1057 against 850 to 866,
// 8 x 8192 with 16 heads 26.2 against 23.9, 64 x 8192 130 against 118, 16 x 32768 122 against 117, 152 x 2048 82
// against 79, one request of 512 rows 12.9 against 12.4.  The conversion is as many
// instructions again as all other warps execute (ncu: 40.3 to 19.3 million for 38 x 8192 rows of 128 heads), and the
// tile's chain has four pages to hide in, not five.  What it spent its time on first was fetching instructions: with the conversion
// unrolled (1880 us) 3.5 warps waited for one at each issue, the SM's instruction cache hit 82% and the next
// level ran at 82% of its rate.  A short loop 1320, half a page's columns handed over early and two pages of
// codes with four of bf16 1186, waits in fewer instructions 1108, one hand-over 1062.  Not taken: eight converting
// warps with registers moved to the score warps 1400; the converting warps on the schedulers of the warps
// that only ship scores 1280; idle score warps that convert where there are few rows, with a third page of
// codes in flight, 140 instead of 132 us (64 x 8192, 16 heads).
#include <cuda.h>
#include <cuda_runtime.h>
#include <algorithm>
#include <cmath>
#include <cstdint>
#include <cstring>
#include <mutex>

#include "irm_common.cuh"
#include "irm_host_util.h"
#include "irm_pipeline.cuh"
#include "irm_tma.cuh"

namespace irm {
namespace {

constexpr int kBatch = 256;  // requests per launch (their lengths travel in the parameters)
constexpr int kBM = 128;     // query rows of a unit
constexpr int kHalf = 64;    // of which a CTA owns
constexpr int kScoreWarps = 8;
constexpr int kTmaWarp = 8, kSWarp = 9, kPvWarp = 10, kClearWarp = 11;
constexpr int kConvWarp = 12, kConvWarps = 4;  // of an 8-bit cache
constexpr uint32_t kFull = 0xffffffffu;
constexpr float kLn2 = 0.6931471805599453f;

// Shared memory: barriers and small arrays, then 1024-byte aligned tiles.
constexpr uint32_t kSlab = 64 * 128;                  // 64 rows x 64 columns
constexpr uint32_t kStage = 4 * kSlab;                // the cKV columns of a page
constexpr uint32_t kCodes = 64 * 256;                 // and their codes, two boxes of 128 columns
constexpr uint32_t kKr = 64 * 64;                     // and its 32 k_r columns, which only Q K^T needs
constexpr uint32_t kXBytes = kHalf * kPage * 4;       // received scores of one tile
constexpr uint32_t kPBytes = kBM * 128;               // P of one tile
constexpr uint32_t kOffBars = 0;
constexpr uint32_t kOffTmem = 416;
constexpr uint32_t kOffAbort = 420;
constexpr uint32_t kOffFlag = 432;                    // int [2 sets][2 warps]: some factor is not 1
constexpr uint32_t kOffMax = 512;                     // float [64]: running maximum of the own rows
constexpr uint32_t kOffCorr = kOffMax + 64 * 4;       // float [4 tiles][64]: the peer rows' factors
constexpr uint32_t kPrBytes = kPBytes / 4 + 128 + 4;  // what a warp sends of P: 32 rows, factors, flag
constexpr uint32_t kOffQr = 2048;                     // 128 rows x 64 B (swizzled)
constexpr uint32_t kOffSum = kOffQr;                  // at the end: float2 [2][64], (maximum, sum) of each set
constexpr uint32_t kOffInv = kOffSum + 2 * 64 * 8;    // and float [128], 1 / l of every row
constexpr uint32_t kOffX = kOffQr + 128 * 64;         // 16-byte words [16][64 rows]
constexpr uint32_t kOffKr = kOffX + kXBytes;          // [2]
constexpr uint32_t kOffP = kOffKr + 2 * kKr;
constexpr uint32_t kOffKv = kOffP + 2 * kPBytes;
static_assert(kOffCorr + 4 * 64 * 4 <= kOffQr && kOffQr % 1024 == 0 && kOffKr % 1024 == 0 && kOffP % 1024 == 0, "layout");

enum : int {
  BAR_S_FULL = 0,                    // [2] Q K^T done
  BAR_S_FREE = BAR_S_FULL + 2,       // [2] the set's live warps read the score buffer
  BAR_X_FULL = BAR_S_FREE + 2,       // [2][32 rows] the peer's partial scores arrived, keys 32 to 63 (1 + tx)
  BAR_X_FREE = BAR_X_FULL + 4,       // [2][32 rows] the peer's warp has read what was sent
  BAR_PR_FULL = BAR_X_FREE + 4,      // [2] the peer's rows of P and factors arrived (its live warps + tx)
  BAR_P_FREE = BAR_PR_FULL + 2,      // [2] P V of the buffer done in both CTAs (2)
  BAR_GO = BAR_P_FREE + 2,           // [2] the own rows' P written and O rescaled: live warps
  BAR_RESC = BAR_GO + 2,             // [2] O rescaled for 32 of the peer's rows (only where a factor is not 1)
  BAR_PV = BAR_RESC + 2,             // P V of a tile done in this CTA
  BAR_MAX = BAR_PV + 1,              // [2] running maximum of 32 own rows published
  BAR_QIN = BAR_MAX + 2,             // Q's TMA bytes (1 + tx)
  BAR_Q = BAR_QIN + 1,               // Q's cKV columns copied to TMEM (8 warps)
  BAR_INV = BAR_Q + 1,               // the peer rows' 1 / l arrived (1 + tx)
  BAR_DRAIN = BAR_INV + 1,           // [2] all UMMAs of an issuer done
  BAR_X_HALF = BAR_DRAIN + 2,        // [2][32 rows] the peer's partial scores, keys 0 to 31 (1 + tx)
  BAR_LANDED = BAR_X_HALF + 4,       // [stage] TMA bytes of the page (1 + tx); 8-bit: its cKV is there as bf16 (4 warps)
};

// What depends on the cache's type: pages in shared memory, and the barriers of their ring.
template <bool kCodes8>
struct Layout {
  static constexpr int kThreads = (kCodes8 ? 16 : 12) * 32;
  static constexpr int kStages = kCodes8 ? 4 : 5;  // pages of bf16
  static constexpr int kRaw = kCodes8 ? 2 : 0;     // pages of codes
  static constexpr uint32_t kRing = kStages * kSlab;  // pages in turn, for each 64 columns
  static constexpr int kQStage = kCodes8 ? 1 : 2;     // 4 slabs of Q's cKV columns at the start, in this stage and the next
  static constexpr uint32_t kOffQl = kOffKv + kQStage * kSlab;
  static constexpr uint32_t kOffRaw = kOffKv + kStages * kStage;
  static constexpr uint32_t kSmem = kOffRaw + kRaw * kCodes + 1024;  // room to align the base
  static constexpr int BAR_FREE = BAR_LANDED + kStages;    // [stage] P V of the page done; bf16: and the clearing warp past it (2)
  static constexpr int BAR_CLEAR = BAR_FREE + kStages;     // bf16: [stage] unseen rows cleared for P V (pages with drafts only)
  static constexpr int BAR_RAW_FULL = BAR_FREE + kStages;  // 8-bit: [raw] TMA bytes of the codes (1 + tx)
  static constexpr int BAR_RAW_FREE = BAR_RAW_FULL + kRaw; // [raw] codes read (4 warps)
  static constexpr int BAR_KR = BAR_RAW_FREE + kRaw;       // [2] TMA bytes of k_r (1 + tx)
  static constexpr int kBars = kCodes8 ? BAR_KR + 2 : BAR_CLEAR + kStages;
  static_assert(kBM * 128 <= 2 * kSlab && kStages >= kQStage + 2, "Q's place");
  static_assert(kSmem <= 232448, "shared memory");
  static_assert(kBars * 8 <= kOffTmem, "barrier area");
};

constexpr uint32_t kTmemO = 0, kTmemQ = 256, kTmemS = 384, kTmemCols = 512;
constexpr uint32_t kIdescS = idesc_bf16_f32(kBM, kPage, 0, 0);
constexpr uint32_t kIdescPV = idesc_bf16_f32(kBM, 256, 0, 1);

// A request: its first node (of the batch's T) and nodes, its rows before them, and how many units of
// full pieces, units of rests and partials come before its own.
struct Request {
  int32_t first, n, ctx, long_base, rest_base, part_base, pad[2];
};

struct TreeArgs {
  // pages [rows, 576]: boxes of 64 x 64, and of 64 rows x 32 columns; 8-bit [rows, 656 bytes]: of 64 rows x 128
  // bytes, and of 64 rows x 32 columns of k_r
  CUtensorMap map_lat, map_rope;
  CUtensorMap map_ql, map_qr;     // queries [T H, 512] and [T H, 64]: boxes of 32 rows x 64, and x 32 columns
  const int32_t* page_table;
  const uint32_t* mask;
  const uint8_t* kv8;  // 8-bit: the pages, for their scales
  int64_t n_pages;
  int B, b0, H, max_pages, mask_words;
  int piece;   // pages of a piece
  uint32_t zero;  // 0, which the compiler does not know
  int n_long;  // units of full pieces; the requests' rests follow
  float scale_log2;
  __nv_bfloat16* out;
  float* lse;
  float* opart;    // fp32 [partial][128][512]
  float* lsepart;  // fp32 [partial][128], log2 units
  int* status;
  Request req[kBatch];
};
static_assert(sizeof(TreeArgs) <= 32764, "kernel parameter block");

__host__ __device__ inline int row_tiles(int n, int H) { return (n * H + kBM - 1) / kBM; }
__host__ __device__ inline int page_count(int ctx, int n) { return n > 0 ? (ctx + n + kPage - 1) / kPage : 0; }

// Last b in [0, B) with req[b].*base <= u: the owner of u among requests with a positive share.
template <int32_t Request::*base>
__device__ __forceinline__ int owner_of(const TreeArgs& a, int u) {
  int lo = 0, hi = a.B;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (a.req[mid].*base <= u) lo = mid; else hi = mid;
  }
  return lo;
}

// 64 mask bits from bit `first` (>= 0) of a node's mask on; bits from n on are clear.
__device__ __forceinline__ uint64_t mask_window(const uint32_t* mask, int words, int first, int n) {
  if (first >= n) return 0;
  const int w = first >> 5, s = first & 31;
  const uint64_t lo = mask[w], mid = w + 1 < words ? mask[w + 1] : 0u, hi = w + 2 < words ? mask[w + 2] : 0u;
  uint64_t v = (lo | mid << 32) >> s;
  if (s != 0) v |= hi << (64 - s);
  return n - first < 64 ? v & ((1ull << (n - first)) - 1) : v;
}

// Which of the rows T .. T + 63 of its request a node sees.
__device__ __forceinline__ uint64_t seen_rows(const uint32_t* mask, int words, int T, int ctx, int n) {
  const int off = T - ctx;
  if (off >= 0) return mask_window(mask, words, off, n);
  if (off <= -64) return ~0ull;
  return ((1ull << -off) - 1) | mask_window(mask, words, 0, n) << -off;
}

// Paired fp32 arithmetic of sm_100 and later; each half rounds as the scalar form.
__device__ __forceinline__ uint64_t f2_pack(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float2 f2_unpack(uint64_t v) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
  return r;
}
__device__ __forceinline__ uint64_t f2_fma(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t f2_add(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// O columns of this warp's 32 lanes times each lane's factor.
__device__ __forceinline__ void rescale_o(uint32_t tO, float corr) {
#pragma unroll 1
  for (int c = 0; c < 256; c += 32) {
    uint32_t r[32];
    tmem_ld32(tO + c, r);
    tmem_ld_wait();
#pragma unroll
    for (int i = 0; i < 32; ++i) r[i] = __float_as_uint(__uint_as_float(r[i]) * corr);
    tmem_st32(tO + c, r);
  }
  tmem_st_wait();
}

// Four e4m3 codes as bf16 times the scale (a pair of bf16, 2^120 times the scale of the codes): a code's
// sign and 7 bits, put where bf16 has sign, low exponent bits and first mantissa bits, are its value
// times 2^-120, denormals included.  The codes come as (0, 2) and (1, 3), which saves moving bytes: Q's
// columns are put in the same order, and O's back.
__device__ __forceinline__ uint2 codes_to_bf16(uint32_t w, __nv_bfloat162 scale) {
  const uint32_t e = (w << 4 & 0x07f007f0u) | (w << 8 & 0x80008000u), o = (w >> 4 & 0x07f007f0u) | (w & 0x80008000u);
  const __nv_bfloat162 x = __hmul2(*reinterpret_cast<const __nv_bfloat162*>(&e), scale);
  const __nv_bfloat162 y = __hmul2(*reinterpret_cast<const __nv_bfloat162*>(&o), scale);
  return make_uint2(*reinterpret_cast<const uint32_t*>(&x), *reinterpret_cast<const uint32_t*>(&y));
}

template <bool kCodes8>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(Layout<kCodes8>::kThreads, 1)
    tree_attn_kernel(const __grid_constant__ TreeArgs a) {
  using L = Layout<kCodes8>;
  constexpr int kStages = L::kStages, kRaw = kCodes8 ? L::kRaw : 1, BAR_FREE = L::BAR_FREE;
  constexpr uint32_t kRing = L::kRing, kOffQl = L::kOffQl;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);  // alike in both CTAs
  const uint32_t sb = smem_u32(smem);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int rank = (int)cluster_ctarank();
  const uint32_t peer = (uint32_t)rank ^ 1u;

  // ---- the unit -------------------------------------------------------------------------
  const int unit = (int)(blockIdx.x >> 1);
  const bool is_rest = unit >= a.n_long;
  const int at = is_rest ? unit - a.n_long : unit;
  const int b = is_rest ? owner_of<&Request::rest_base>(a, at) : owner_of<&Request::long_base>(a, at);
  const Request req = a.req[b];
  const int first_node = req.first, n = req.n, ctx = req.ctx;
  const int mtiles = row_tiles(n, a.H), tiles_all = page_count(ctx, n);
  const int in_b = at - (is_rest ? req.rest_base : req.long_base);
  const int piece = is_rest ? tiles_all / a.piece : in_b / mtiles;
  const int mtile = is_rest ? in_b : in_b % mtiles;
  const int kb = piece * a.piece;
  const int ntiles = min(a.piece, tiles_all - kb);
  const int pieces = (tiles_all + a.piece - 1) / a.piece;
  const int row0 = mtile * kBM, rows_valid = min(kBM, n * a.H - row0);
  const int64_t grow0 = (int64_t)first_node * a.H + row0;  // row of the batch's T H
  const int tail = max(0, ctx / kPage - kb);               // first tile of the unit with drafts

  auto bar = [&](int i) -> uint32_t { return sb + kOffBars + 8u * (uint32_t)i; };
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + kOffAbort);
  // quadrants of 32 rows that hold valid rows, of the own and of the peer's 64
  auto live_of = [&](int r) -> int { return max(0, min(2, (rows_valid - kHalf * r + 31) / 32)); };
  const int live_own = live_of(rank), live_peer = live_of((int)peer);

  if (tid == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(bar(BAR_LANDED + s), kCodes8 ? kConvWarps : 1);
      mbar_init(bar(BAR_FREE + s), kCodes8 ? 1 : 2);
      if (!kCodes8) mbar_init(bar(L::BAR_CLEAR + s), 1);
    }
    if (kCodes8) {
      for (int s = 0; s < kRaw; ++s) {
        mbar_init(bar(L::BAR_RAW_FULL + s), 1);
        mbar_init(bar(L::BAR_RAW_FREE + s), kConvWarps);
      }
      for (int s = 0; s < 2; ++s) mbar_init(bar(L::BAR_KR + s), 1);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(bar(BAR_S_FULL + s), 1);
      mbar_init(bar(BAR_S_FREE + s), live_own + live_peer);
      for (int h = 0; h < 2; ++h) {
        mbar_init(bar(BAR_X_FULL + 2 * s + h), 1);
        mbar_init(bar(BAR_X_HALF + 2 * s + h), 1);
        mbar_init(bar(BAR_X_FREE + 2 * s + h), 1);
      }
      mbar_init(bar(BAR_PR_FULL + s), max(1, live_peer));
      mbar_init(bar(BAR_P_FREE + s), 2);
      mbar_init(bar(BAR_GO + s), max(1, live_own));
      mbar_init(bar(BAR_RESC + s), 1);
      mbar_init(bar(BAR_MAX + s), 1);
      mbar_init(bar(BAR_DRAIN + s), 1);
      // the first two tiles' bytes (a barrier that nothing is sent to is not waited for either)
      for (int h = 0; h < live_own; ++h) {
        mbar_arrive_expect_tx(bar(BAR_X_FULL + 2 * s + h), kXBytes / 4);
        mbar_arrive_expect_tx(bar(BAR_X_HALF + 2 * s + h), kXBytes / 4);
      }
      for (int k = 0; k < live_peer; ++k) mbar_arrive_expect_tx(bar(BAR_PR_FULL + s), kPrBytes);
    }
    mbar_init(bar(BAR_PV), 1);
    mbar_init(bar(BAR_QIN), 1);
    mbar_init(bar(BAR_Q), kScoreWarps);
    mbar_init(bar(BAR_INV), 1);
    if (live_peer) mbar_arrive_expect_tx(bar(BAR_INV), (uint32_t)live_peer * 128u);
    *abort_flag = 0;
    fence_mbar_init_cluster();
  }
  // what the first copies need, on its way during the set-up
  const int32_t* ptab = a.page_table + (int64_t)(a.b0 + b) * a.max_pages + kb;
  int page0 = 0;
  if (warp == kTmaWarp || (kCodes8 && warp == kClearWarp)) {
    if (lane < ntiles) page0 = ptab[lane];
  }
  if (warp == kTmaWarp) {
    if (lane == 0) {
      tma_prefetch_map(&a.map_lat);
      tma_prefetch_map(&a.map_rope);
    }
  } else if (warp == kClearWarp && lane == 0) {
    tma_prefetch_map(&a.map_ql);
    tma_prefetch_map(&a.map_qr);
  }
  if (warp == kSWarp) {
    tmem_alloc(sb + kOffTmem, kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  cluster_arrive();  // every warp waits for it before its first remote access, or at its end
  const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(smem + kOffTmem);
  bool ok = true;
  float2 state = make_float2(-INFINITY, 0.f);  // of the own rows' warps: maximum and sum of their tiles

  if (warp < kScoreWarps) {
    const int set = warp >> 2, quad = warp & 3;
    const bool own = (quad >> 1) == rank;
    const bool live = quad * 32 < rows_valid;
    const int m = quad * 32 + lane;   // row of the unit = TMEM lane
    const int mh = m & (kHalf - 1);   // and of its owner's half
    const uint32_t lanes = (uint32_t)(quad * 32) << 16;
    const uint32_t tS = tmem + kTmemS + 64u * (uint32_t)set + lanes;
    const uint32_t tO = tmem + kTmemO + lanes;
    const bool valid = m < rows_valid;
    // ---- Q, this CTA's cKV columns: from shared memory (where TMA put it) to TMEM; set h takes
    //      slabs 2h, 2h + 1
    ok = warp_wait_compact<false>(bar(BAR_QIN), 0, abort_flag);
    if (live && ok) {
#pragma unroll
      for (int slab = 2 * set; slab < 2 * set + 2; ++slab) {
        uint32_t r[32];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          uint4 v = *reinterpret_cast<const uint4*>(smem + kOffQl + slab * kRing + sw128_offset((uint32_t)m, (uint32_t)i));
          if (kCodes8)  // columns 0, 2, 1, 3 of each four
            v = make_uint4(__byte_perm(v.x, v.y, 0x5410), __byte_perm(v.x, v.y, 0x7632), __byte_perm(v.z, v.w, 0x5410),
                           __byte_perm(v.z, v.w, 0x7632));
          r[4 * i] = v.x;
          r[4 * i + 1] = v.y;
          r[4 * i + 2] = v.z;
          r[4 * i + 3] = v.w;
        }
        tmem_st32(tmem + kTmemQ + 32u * (uint32_t)slab + lanes, r);
      }
      tmem_st_wait();
    }
    tc_fence_before();
    __syncwarp();
    if (lane == 0) mbar_arrive(bar(BAR_Q));
    __syncwarp();
    cluster_wait();
    const uint32_t buf = (uint32_t)set;  // a set's tiles all use the buffers of its number
    const uint32_t remX = mapa_shared(sb + kOffX, peer);
    const int xq = 2 * set + (quad & 1);
    const uint32_t remXfull = mapa_shared(bar(BAR_X_FULL + xq), peer);
    const uint32_t remXhalf = mapa_shared(bar(BAR_X_HALF + xq), peer);
    const uint32_t remXfree = mapa_shared(bar(BAR_X_FREE + xq), peer);
    const uint32_t remP = mapa_shared(sb + kOffP + buf * kPBytes, peer);
    const uint32_t remPfull = mapa_shared(bar(BAR_PR_FULL + set), peer);
    const uint32_t remCorr = mapa_shared(sb + kOffCorr + 4u * (uint32_t)mh, peer);
    const uint32_t remFlag = mapa_shared(sb + kOffFlag + 8u * buf + 4u * (uint32_t)(quad & 1), peer);
    const uint4* X = reinterpret_cast<const uint4*>(smem + kOffX);
    float* max_sh = reinterpret_cast<float*>(smem + kOffMax);
    const float* corr_sh = reinterpret_cast<const float*>(smem + kOffCorr);
    const uint32_t* mask = a.mask + (int64_t)(first_node + (row0 + (valid ? m : 0)) / a.H) * a.mask_words;
    float m_l = -INFINITY, l = 0.f;  // this set's sum, relative to m_l

    // The factors of the peer's rows at tile t, after its P has arrived.  A sender looks at them one
    // turn late, after it has shipped the scores of tile t + 2, so that the peer never waits for it;
    // P V waits for this only where a factor is not 1.
    auto take_factors = [&](int t) -> bool {
      if (!warp_wait_compact<true>(bar(BAR_PR_FULL + set), (uint32_t)(t >> 1) & 1u, abort_flag)) return false;
      if (lane == 0 && t + 2 < ntiles) mbar_arrive_expect_tx(bar(BAR_PR_FULL + set), kPrBytes);
      const float corr = corr_sh[(t & 3) * kHalf + mh];
      if (t > 0 && __any_sync(kFull, corr != 1.f)) {
        if (!warp_wait_compact<false>(bar(BAR_PV), (uint32_t)(t - 1) & 1u, abort_flag)) return false;
        tc_fence_after();
        rescale_o(tO, corr);
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(BAR_RESC + (quad & 1)));
      }
      return true;
    };

    int j = set;
    for (; live && ok && j < ntiles; j += 2) {  // warps without valid rows have no part in it
      const uint32_t ph = (uint32_t)(j >> 1) & 1u;
      uint32_t s[64];
      uint64_t see = 0;  // read before the waits
      if (own && j >= tail && valid) see = seen_rows(mask, a.mask_words, (kb + j) * kPage, ctx, n);
      if (!(ok = warp_wait_compact<false>(bar(BAR_S_FULL + set), ph, abort_flag))) break;
      tc_fence_after();
      tmem_ld32(tS, reinterpret_cast<uint32_t(&)[32]>(s[0]));
      tmem_ld32(tS + 32u, reinterpret_cast<uint32_t(&)[32]>(s[32]));
      tmem_ld_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(BAR_S_FREE + set));
      if (own) {
        float corr = 1.f;
        // ================= softmax of a row =================
        // the maximum is taken over each half of the scores as it comes
        float v[64];
        if (!(ok = warp_wait_compact<true>(bar(BAR_X_HALF + xq), ph, abort_flag))) break;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const uint4 x = X[i * kHalf + mh];
          v[4 * i] = __uint_as_float(s[4 * i]) + __uint_as_float(x.x);
          v[4 * i + 1] = __uint_as_float(s[4 * i + 1]) + __uint_as_float(x.y);
          v[4 * i + 2] = __uint_as_float(s[4 * i + 2]) + __uint_as_float(x.z);
          v[4 * i + 3] = __uint_as_float(s[4 * i + 3]) + __uint_as_float(x.w);
        }
        if (j >= tail) {
#pragma unroll
          for (int i = 0; i < 32; ++i)
            if (!(see >> i & 1)) v[i] = -INFINITY;
        }
        float u[11];
#pragma unroll
        for (int i = 0; i < 10; ++i) u[i] = fmax3(v[3 * i], v[3 * i + 1], v[3 * i + 2]);
        u[10] = fmaxf(v[30], v[31]);
        const float low = fmax3(fmax3(fmax3(u[0], u[1], u[2]), fmax3(u[3], u[4], u[5]), fmax3(u[6], u[7], u[8])), u[9], u[10]);
        if (!(ok = warp_wait_compact<true>(bar(BAR_X_FULL + xq), ph, abort_flag))) break;
#pragma unroll
        for (int i = 8; i < 16; ++i) {
          const uint4 x = X[i * kHalf + mh];
          v[4 * i] = __uint_as_float(s[4 * i]) + __uint_as_float(x.x);
          v[4 * i + 1] = __uint_as_float(s[4 * i + 1]) + __uint_as_float(x.y);
          v[4 * i + 2] = __uint_as_float(s[4 * i + 2]) + __uint_as_float(x.z);
          v[4 * i + 3] = __uint_as_float(s[4 * i + 3]) + __uint_as_float(x.w);
        }
        if (j >= tail) {
#pragma unroll
          for (int i = 32; i < 64; ++i)
            if (!(see >> i & 1)) v[i] = -INFINITY;
        }
        float t[11];
#pragma unroll
        for (int i = 0; i < 10; ++i) t[i] = fmax3(v[32 + 3 * i], v[33 + 3 * i], v[34 + 3 * i]);
        t[10] = fmaxf(v[62], v[63]);
        const float raw = fmax3(fmax3(fmax3(t[0], t[1], t[2]), fmax3(t[3], t[4], t[5]), fmax3(t[6], t[7], t[8])), fmax3(t[9], t[10], low), low);
        const float top = raw * a.scale_log2;
        // The peer may overwrite the received scores once they have been read, so the arrival that says so
        // takes its address through a vote of the warp on the maximum of all that it read: it cannot be
        // made before every lane's loads have returned.  (Without the vote the loads could still be under
        // way: 64 x 32768 rows 855 instead of 873 us.)  A release at cluster scope costs far more, 1260 us
        // from here, where it also waits for the st.async under way, and 1500 from a warp that has none.
        const uint32_t vote = __ballot_sync(kFull, raw > 0.f);
        if (lane == 0) {
          if (j + 2 < ntiles) {
            mbar_arrive_expect_tx(bar(BAR_X_FULL + xq), kXBytes / 4);
            mbar_arrive_expect_tx(bar(BAR_X_HALF + xq), kXBytes / 4);
          }
          mbar_arrive_remote_relaxed(remXfree + (vote & a.zero));
        }
        if (j > 0 && !(ok = warp_wait_compact<false>(bar(BAR_MAX + (quad & 1)), (uint32_t)(j - 1) & 1u, abort_flag))) break;
        const float before = j > 0 ? max_sh[mh] : -INFINITY;
        const bool up = top > before + 8.f;
        const float now = up ? top : before;
        max_sh[mh] = now;
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(BAR_MAX + (quad & 1)));
        if (up) corr = fast_exp2(before - now);
        if (now != m_l) l *= fast_exp2(m_l - now);  // m_l = -inf: l is 0
        m_l = now;
        const float use = now == -INFINITY ? 0.f : now;
        const uint64_t c2 = f2_pack(a.scale_log2, a.scale_log2), m2 = f2_pack(-use, -use);
        uint64_t sum[2] = {0ull, 0ull};
        uint32_t pk[32];
#pragma unroll
        for (int i = 0; i < 32; ++i) {
          const float2 x = f2_unpack(f2_fma(f2_pack(v[2 * i], v[2 * i + 1]), c2, m2));
          const float p0 = fast_exp2(x.x), p1 = fast_exp2(x.y);
          sum[i & 1] = f2_add(sum[i & 1], f2_pack(p0, p1));
          pk[i] = pack_bf16(p0, p1);
        }
        const float2 part = f2_unpack(f2_add(sum[0], sum[1]));
        l += part.x + part.y;
        if (j >= 2 && !(ok = warp_wait_compact<true>(bar(BAR_P_FREE + set), ph ^ 1u, abort_flag))) break;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const uint4 w = make_uint4(pk[4 * i], pk[4 * i + 1], pk[4 * i + 2], pk[4 * i + 3]);
          const uint32_t off = sw128_offset((uint32_t)m, (uint32_t)i);
          st_shared_v4(sb + kOffP + buf * kPBytes + off, w);
        }
        st_async_b32(remCorr + (uint32_t)(j & 3) * (kHalf * 4u), __float_as_uint(corr), remPfull);
        fence_proxy_async_smem();  // P is read by the copy and by the tensor core
        __syncwarp();
        if (lane == 0) bulk_to_peer(remP + (uint32_t)quad * 4096u, sb + kOffP + buf * kPBytes + (uint32_t)quad * 4096u, 4096u, remPfull);
        const bool moved = __any_sync(kFull, corr != 1.f);
        if (lane == 0) st_async_b32(remFlag, moved ? 1u : 0u, remPfull);
        if (j > 0 && moved) {
          if (!(ok = warp_wait_compact<false>(bar(BAR_PV), (uint32_t)(j - 1) & 1u, abort_flag))) break;
          tc_fence_after();
          rescale_o(tO, corr);
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(BAR_GO + set));
      } else {
        // ================= partial scores of the peer's rows =================
        if (j >= 1 && !(ok = warp_wait_compact<true>(bar(BAR_X_FREE + (xq ^ 2)), (uint32_t)((j - 1) >> 1) & 1u, abort_flag))) break;
#pragma unroll
        for (int i = 0; i < 16; ++i)
          st_async_v4_b32(remX + (uint32_t)(i * kHalf + mh) * 16u, make_uint4(s[4 * i], s[4 * i + 1], s[4 * i + 2], s[4 * i + 3]),
                          i < 8 ? remXhalf : remXfull);
        if (j >= 2 && !(ok = take_factors(j - 2))) break;
      }
    }
    if (ok && live && !own && j > set) ok = take_factors(j - 2);
    if (own) state = make_float2(m_l, l);
  } else if (warp == kTmaWarp) {
    // ================= pages in =================
    int page = 0, sent = 0;
    for (int j = 0; j < ntiles; ++j) {
      if ((j & 31) == 0) {
        page = j == 0 ? page0 : j + lane < ntiles ? ptab[j + lane] : 0;
        if (page < 0 || page >= a.n_pages) {
          set_status(a.status, kDevErrBounds);
          page = (int)a.n_pages;  // behind the tensor: zeros
        }
      }
      const int y = __shfl_sync(kFull, page, j & 31) * kPage;
      if constexpr (kCodes8) {
        const int r = j % kRaw;
        if (j >= kRaw && !(ok = warp_wait_compact<false>(bar(L::BAR_RAW_FREE + r), ((uint32_t)(j / kRaw) & 1u) ^ 1u, abort_flag))) break;
        if (lane == 0) {
          mbar_arrive_expect_tx(bar(L::BAR_RAW_FULL + r), kCodes);
#pragma unroll
          for (int c = 0; c < 2; ++c)
            tma_load_2d(sb + L::kOffRaw + (uint32_t)r * kCodes + c * kSlab, &a.map_lat, 256 * rank + 128 * c, y, bar(L::BAR_RAW_FULL + r));
        }
        sent = j + 1;
        continue;
      }
      const int s = j % kStages;
      // stages 2 and 3 hold Q until it is in TMEM
      if (j == 2 && !(ok = warp_wait_compact<false>(bar(BAR_Q), 0, abort_flag))) break;
      if (j >= kStages && !(ok = warp_wait_compact<false>(bar(BAR_FREE + s), ((uint32_t)(j / kStages) & 1u) ^ 1u, abort_flag))) break;
      if (lane == 0) {
        const uint32_t st = sb + kOffKv + (uint32_t)s * kSlab;
        mbar_arrive_expect_tx(bar(BAR_LANDED + s), kStage + kKr);
#pragma unroll
        for (int c = 0; c < 4; ++c) tma_load_2d(st + c * kRing, &a.map_lat, 256 * rank + 64 * c, y, bar(BAR_LANDED + s));
      }
      sent = j + 1;
      // the k_r buffer's last page has been through Q K^T
      if (j >= 2 && !(ok = warp_wait_compact<false>(bar(BAR_S_FULL + (j & 1)), ((uint32_t)(j >> 1) & 1u) ^ 1u, abort_flag))) break;
      if (lane == 0) tma_load_2d(sb + kOffKr + (uint32_t)(j & 1) * kKr, &a.map_rope, kDLat + 32 * rank, y, bar(BAR_LANDED + s));
    }
    // the copies in flight land before the CTA ends, whatever became of the others
    ok = warp_wait_compact<false>(bar(BAR_QIN), 0, nullptr) && ok;
    constexpr int kFlight = kCodes8 ? kRaw : kStages, kBar = kCodes8 ? L::BAR_RAW_FULL : BAR_LANDED;
    for (int j = max(0, sent - kFlight); j < sent; ++j)
      ok = warp_wait_compact<false>(bar(kBar + j % kFlight), (uint32_t)(j / kFlight) & 1u, nullptr) && ok;
    __syncwarp();
    cluster_wait();
  } else if (warp == kSWarp) {
    // ================= Q K^T (one thread) =================
    if (lane == 0) {
      ok = mbar_wait_compact<false>(bar(BAR_QIN), 0, abort_flag) && mbar_wait_compact<false>(bar(BAR_Q), 0, abort_flag);
      tc_fence_after();
      const uint64_t aq = sdesc_sw64(sb + kOffQr, 512);
      for (int j = 0; j < ntiles && ok; ++j) {
        const int s = j % kStages, set = j & 1;
        if (!kCodes8 && !(ok = mbar_wait_compact<false>(bar(BAR_LANDED + s), (uint32_t)(j / kStages) & 1u, abort_flag))) break;
        if (kCodes8 && !(ok = mbar_wait_compact<false>(bar(L::BAR_KR + set), (uint32_t)(j >> 1) & 1u, abort_flag))) break;
        if (j >= 2 && !(ok = mbar_wait_compact<false>(bar(BAR_S_FREE + set), ((uint32_t)(j >> 1) & 1u) ^ 1u, abort_flag))) break;
        tc_fence_after();
        const uint32_t st = sb + kOffKv + (uint32_t)s * kSlab;
        const uint64_t bd = sdesc_sw128(st, 16, 1024), bk = sdesc_sw64(sb + kOffKr + (uint32_t)set * kKr, 512);
        const uint32_t d = tmem + kTmemS + 64u * (uint32_t)set;
        auto rope = [&](uint32_t first) {
#pragma unroll
          for (int kk = 0; kk < 2; ++kk) umma_bf16(d, sdesc_add(aq, kk * 32), sdesc_add(bk, kk * 32), kIdescS, kk == 0 ? first : 1u);
        };
        auto slab = [&](int c, uint32_t first) {
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)
            umma_bf16_ts(d, tmem + kTmemQ + 32u * c + 8u * kk, sdesc_add(bd, c * kRing + kk * 32), kIdescS, kk == 0 ? first : 1u);
        };
        if constexpr (kCodes8) {  // in the order in which they come
          rope(0u);
          if (!(ok = mbar_wait_compact<false>(bar(BAR_LANDED + s), (uint32_t)(j / kStages) & 1u, abort_flag))) break;
          tc_fence_after();
          slab(0, 1u);
          slab(1, 1u);
          slab(2, 1u);
          slab(3, 1u);
        } else {
          slab(0, 0u);
          slab(1, 1u);
          slab(2, 1u);
          slab(3, 1u);
          rope(1u);
        }
        umma_commit(bar(BAR_S_FULL + set));
      }
      umma_commit(bar(BAR_DRAIN));
      ok = mbar_wait_compact<false>(bar(BAR_DRAIN), 0, nullptr) && ok;
    }
    __syncwarp();
    cluster_wait();
  } else if (warp == kPvWarp) {
    // ================= P V (one thread) =================
    if (lane == 0) {
      uint32_t resc = 0;  // parities of the next rescalings of the peer's rows
      for (int j = 0; j < ntiles && ok; ++j) {
        const int s = j % kStages, set = j & 1;
        const uint32_t ph = (uint32_t)(j >> 1) & 1u;
        if (!kCodes8 && j >= tail) {
          if (!(ok = mbar_wait_compact<false>(bar(L::BAR_CLEAR + s), (uint32_t)((j - tail) / kStages) & 1u, abort_flag))) break;
          fence_proxy_async_smem();  // the cleared rows' plain stores
        }
        if (live_own && !(ok = mbar_wait_compact<false>(bar(BAR_GO + set), ph, abort_flag))) break;
        if (live_peer) {
          if (!(ok = mbar_wait_compact<true>(bar(BAR_PR_FULL + set), ph, abort_flag))) break;
          uint32_t f0, f1;
          asm volatile("ld.volatile.shared.v2.u32 {%0, %1}, [%2];" : "=r"(f0), "=r"(f1) : "r"(sb + kOffFlag + 8u * (uint32_t)set) : "memory");
          // a rescaling waits for P V of the tile before, so these phases are passed one by one
          const uint32_t moved = j > 0 ? f0 | (live_peer > 1 ? 2u * f1 : 0u) : 0u;
          if (moved != 0) {
            if (moved & 1u) ok = mbar_wait_compact<false>(bar(BAR_RESC), resc & 1u, abort_flag);
            if (ok && moved & 2u) ok = mbar_wait_compact<false>(bar(BAR_RESC + 1), resc >> 1, abort_flag);
            resc ^= moved;
            if (!ok) break;
          }
        }
        tc_fence_after();
        const uint64_t ad = sdesc_sw128(sb + kOffP + (uint32_t)set * kPBytes, 16, 1024);
        const uint64_t bd = sdesc_sw128(sb + kOffKv + (uint32_t)s * kSlab, kRing, 1024);
#pragma unroll
        for (int kk = 0; kk < 4; ++kk)
          umma_bf16(tmem + kTmemO, sdesc_add(ad, kk * 32), sdesc_add(bd, kk * 2048), kIdescPV, (j | kk) ? 1u : 0u);
        umma_commit(bar(BAR_FREE + s));
        umma_commit(bar(BAR_PV));
        umma_commit_multicast(bar(BAR_P_FREE + set), (uint16_t)3);
      }
      umma_commit(bar(BAR_DRAIN + 1));
      ok = mbar_wait_compact<false>(bar(BAR_DRAIN + 1), 0, nullptr) && ok;
    }
    __syncwarp();
    cluster_wait();
  } else if (kCodes8 && warp >= kConvWarp) {
    // ================= codes to bf16: a thread a row of 128 columns =================
    const int r = (warp & 1) * 32 + lane, box = (warp - kConvWarp) >> 1;
    const int node0 = row0 / a.H, node1 = (row0 + rows_valid - 1) / a.H;
    const uint8_t* scales = a.kv8 + (int64_t)r * IRM_ROW_BYTES8 + IRM_ROW8_SCALES + 4 * (2 * rank + box);
    // a page's scale is read one page ahead, its index two (a page outside the cache reads as zeros)
    auto page_at = [&](int j) -> int {
      int v = -1;
      if (j < ntiles) asm volatile("ld.global.nc.b32 %0, [%1];" : "=r"(v) : "l"(ptab + j));
      return v;
    };
    auto scale_of = [&](int page) -> uint32_t {
      uint32_t v = 0;  // volatile: it is not put off to where it is used
      if (page >= 0 && page < a.n_pages)
        asm volatile("ld.global.nc.b32 %0, [%1];" : "=r"(v) : "l"(scales + (int64_t)page * (kPage * IRM_ROW_BYTES8)));
      return v;
    };
    uint32_t next = scale_of(page_at(0));
    int page = page_at(1);
    for (int j = 0; j < ntiles; ++j) {
      const int raw = j % kRaw, s = j % kStages;
      const uint32_t scale = next;
      next = scale_of(page);
      page = page_at(j + 2);
      bool seen = true;
      if (j >= tail) {  // rows that no node of the unit sees become zeros
        uint64_t see = 0;
        for (int i = node0 + lane; i <= node1; i += 32)
          see |= seen_rows(a.mask + (int64_t)(first_node + i) * a.mask_words, a.mask_words, (kb + j) * kPage, ctx, n);
        const uint32_t lo = __reduce_or_sync(kFull, (uint32_t)see), hi = __reduce_or_sync(kFull, (uint32_t)(see >> 32));
        seen = ((warp & 1 ? hi : lo) >> lane & 1u) != 0;
      }
      if (!(ok = warp_wait_compact<false>(bar(L::BAR_RAW_FULL + raw), (uint32_t)(j / kRaw) & 1u, abort_flag))) break;
      // the second and third page's places hold Q until it is in TMEM
      if (j == L::kQStage && !(ok = warp_wait_compact<false>(bar(BAR_Q), 0, abort_flag))) break;
      if (j >= kStages && !(ok = warp_wait_compact<false>(bar(BAR_FREE + s), ((uint32_t)(j / kStages) & 1u) ^ 1u, abort_flag))) break;
      // zeros for an unseen row (a code's bits are a finite number, whatever it is)
      const __nv_bfloat162 m = __float2bfloat162_rn(seen ? __uint_as_float(scale & 0xffff0000u) * 0x1p120f : 0.f);
      const uint32_t from = sb + L::kOffRaw + (uint32_t)raw * kCodes + (uint32_t)box * kSlab + (uint32_t)r * 128u;
      const uint32_t to = sb + kOffKv + (uint32_t)(2 * box) * kRing + (uint32_t)s * kSlab + (uint32_t)r * 128u;
      uint4 v = ld_shared_v4(from + ((uint32_t)(r & 7) << 4));
      // a loop: unrolled, the warps' different code does not fit the instruction caches
#pragma unroll 2
      for (uint32_t i = 0; i < 8; ++i) {
        const uint4 w = v;
        v = ld_shared_v4(from + (((i + 1u & 7u) ^ (uint32_t)(r & 7)) << 4));
        const uint2 a0 = codes_to_bf16(w.x, m), a1 = codes_to_bf16(w.y, m), a2 = codes_to_bf16(w.z, m), a3 = codes_to_bf16(w.w, m);
        const uint32_t at = to + (i >> 2) * kRing + ((2u * i & 7u ^ (uint32_t)(r & 7)) << 4);
        st_shared_v4(at, make_uint4(a0.x, a0.y, a1.x, a1.y));
        st_shared_v4(at ^ 16u, make_uint4(a2.x, a2.y, a3.x, a3.y));
      }
      // The copy of a later page may overwrite the codes once they have been read: as with the received scores, the
      // arrival that says so depends on what was read last (without that, loads were still under way in a full SM
      // and read the later page's codes).
      const uint32_t vote = __ballot_sync(kFull, v.x != 0u);
      if (lane == 0) mbar_arrive(bar(L::BAR_RAW_FREE + raw) + (vote & a.zero));
      fence_proxy_async_smem();  // read by the tensor core
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(BAR_LANDED + s));
    }
    __syncwarp();
    cluster_wait();
  } else if (warp == kClearWarp) {
    // ================= Q in =================
    if (lane == 0) {
      const int quads = (rows_valid + 31) / 32;
      mbar_arrive_expect_tx(bar(BAR_QIN), (uint32_t)quads * 32u * (512u + 64u));
      for (int q = 0; q < quads; ++q) {  // rows behind the request's last (another's, or zeros) are never looked at
        const int y = (int)grow0 + 32 * q;
#pragma unroll
        for (int c = 0; c < 4; ++c)
          tma_load_2d(sb + kOffQl + c * kRing + q * 4096, &a.map_ql, 256 * rank + 64 * c, y, bar(BAR_QIN));
        tma_load_2d(sb + kOffQr + q * 2048, &a.map_qr, 32 * rank, y, bar(BAR_QIN));
      }
    }
    __syncwarp();
    if constexpr (kCodes8) {
      // ================= k_r in =================
      int page = 0, sent = 0;
      for (int j = 0; j < ntiles; ++j) {
        if ((j & 31) == 0) {
          page = j == 0 ? page0 : j + lane < ntiles ? ptab[j + lane] : 0;
          if (page < 0 || page >= a.n_pages) page = (int)a.n_pages;  // recorded by the other copying warp
        }
        const int y = __shfl_sync(kFull, page, j & 31) * kPage;
        // the buffer's last page has been through Q K^T
        if (j >= 2 && !(ok = warp_wait_compact<false>(bar(BAR_S_FULL + (j & 1)), ((uint32_t)(j >> 1) & 1u) ^ 1u, abort_flag))) break;
        if (lane == 0) {
          mbar_arrive_expect_tx(bar(L::BAR_KR + (j & 1)), kKr);
          tma_load_2d(sb + kOffKr + (uint32_t)(j & 1) * kKr, &a.map_rope, IRM_ROW8_ROPE / 2 + 32 * rank, y, bar(L::BAR_KR + (j & 1)));
        }
        sent = j + 1;
      }
      for (int j = max(0, sent - 2); j < sent; ++j) ok = warp_wait_compact<false>(bar(L::BAR_KR + (j & 1)), (uint32_t)(j >> 1) & 1u, nullptr) && ok;
    } else {
    // ================= rows that no node of the unit sees become zeros =================
    const int node0 = row0 / a.H, node1 = (row0 + rows_valid - 1) / a.H;
    for (int j = 0; j < ntiles; ++j) {
      const int s = j % kStages;
      uint32_t lo = 0, hi = 0;
      if (j >= tail) {
        uint64_t see = 0;
        for (int i = node0 + lane; i <= node1; i += 32)
          see |= seen_rows(a.mask + (int64_t)(first_node + i) * a.mask_words, a.mask_words, (kb + j) * kPage, ctx, n);
        lo = __reduce_or_sync(kFull, (uint32_t)see);
        hi = __reduce_or_sync(kFull, (uint32_t)(see >> 32));
      }
      if (!(ok = warp_wait_compact<false>(bar(BAR_LANDED + s), (uint32_t)(j / kStages) & 1u, abort_flag))) break;
      if (j >= tail) {
        const uint32_t st = sb + kOffKv + (uint32_t)s * kSlab;
        const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
        const uint64_t gone = ~((uint64_t)hi << 32 | lo);
#pragma unroll 8
        for (uint32_t r = 0; r < 64; ++r) {
          if (gone >> r & 1) st_shared_v4(st + (uint32_t)(lane >> 3) * kRing + sw128_offset(r, (uint32_t)lane & 7u), zero);
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(L::BAR_CLEAR + s));
      }
      // every page is waited for, and given back, so that no phase is missed
      if (lane == 0) mbar_arrive(bar(BAR_FREE + s));
    }
    }
    __syncwarp();
    cluster_wait();
  }
  if (!ok) {
    *abort_flag = 1;
    set_status(a.status, kDevErrTimeout);
  }
  // ---- sums of the rows, to both CTAs ----------------------------------------------------
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp < kScoreWarps && (warp >> 1 & 1) == rank)
    reinterpret_cast<float2*>(smem + kOffSum)[(warp >> 2) * kHalf + (warp & 1) * 32 + lane] = state;
  __syncthreads();
  const bool split = pieces > 1;
  if (split) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");  // the merge waits for the rest of it
  const int64_t part = split ? (int64_t)req.part_base + (int64_t)mtile * pieces + piece : 0;
  float* inv_sh = reinterpret_cast<float*>(smem + kOffInv);
  if (tid < kHalf) {
    const int m = kHalf * rank + tid;
    // both sets' sums are relative to the last maximum they saw; O to the last one of all, the larger
    const float2 x = reinterpret_cast<const float2*>(smem + kOffSum)[tid];
    const float2 y = reinterpret_cast<const float2*>(smem + kOffSum)[kHalf + tid];
    const float mx = fmaxf(x.x, y.x), use = mx == -INFINITY ? 0.f : mx;
    float l = x.y * fast_exp2(x.x - use) + y.y * fast_exp2(y.x - use);
    // No key seen: maximum -inf and sum 0, and then alone O = 0 and lse = -inf.  Any other sum that is not a
    // positive number comes from scores that are NaN, infinite or beyond 2^30, and stays visible.
    const bool none = m >= rows_valid || *abort_flag != 0 || (mx == -INFINITY && l == 0.f);
    if (!(l > 0.f && l < INFINITY)) l = NAN;
    const float inv = none ? 0.f : 1.f / l, lse2 = none ? -INFINITY : mx + __log2f(l);
    inv_sh[m] = inv;
    if (tid < 32 * live_own)
      st_async_b32(mapa_shared(sb + kOffInv + 4u * (uint32_t)m, peer), __float_as_uint(inv), mapa_shared(bar(BAR_INV), peer));
    if (m < rows_valid) {
      if (split) a.lsepart[part * kBM + m] = lse2;
      else if (a.lse != nullptr) a.lse[grow0 + m] = lse2 * kLn2;
    }
  }
  __syncthreads();
  cluster_arrive();  // waited for at the end: until then the peer may still send here
  // ---- O / l: a warp takes 64 columns of its 32 rows at a time, through shared memory, so that
  //      its stores are whole 128-byte lines --------------------------------------------------
  if (warp < kScoreWarps) {
    const int quad = warp & 3, m = quad * 32 + lane;
    if (quad * 32 < rows_valid) {
      if ((quad >> 1) != rank && !warp_wait_compact<true>(bar(BAR_INV), 0, abort_flag)) set_status(a.status, kDevErrTimeout);
      const float inv = inv_sh[m];
      uint8_t* stage = smem + kOffKv + warp * 8192;
      for (int c = 128 * (warp >> 2); c < 128 * (warp >> 2) + 128; c += 64) {
        uint32_t r[64];
        const uint32_t tO = tmem + kTmemO + ((uint32_t)(quad * 32) << 16) + (uint32_t)c;
        tmem_ld32(tO, reinterpret_cast<uint32_t(&)[32]>(r[0]));
        tmem_ld32(tO + 32u, reinterpret_cast<uint32_t(&)[32]>(r[32]));
        tmem_ld_wait();
#pragma unroll
        for (int i = 0; i < 64; ++i) r[i] = inv != 0.f ? __float_as_uint(__uint_as_float(r[i]) * inv) : 0u;
        if (kCodes8) {  // columns 0, 2, 1, 3 of each four
#pragma unroll
          for (int i = 0; i < 64; i += 4) {
            const uint32_t x = r[i + 1];
            r[i + 1] = r[i + 2];
            r[i + 2] = x;
          }
        }
        const int col = 256 * rank + c;
        __syncwarp();
        if (split) {  // rows of 256 bytes, 16-byte pieces XOR-ed with the row
#pragma unroll
          for (int i = 0; i < 16; ++i)
            *reinterpret_cast<uint4*>(stage + lane * 256 + ((i ^ (lane & 7)) << 4)) =
                make_uint4(r[4 * i], r[4 * i + 1], r[4 * i + 2], r[4 * i + 3]);
          __syncwarp();
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            const int row = 2 * i + (lane >> 4), q = lane & 15;
            if (quad * 32 + row < rows_valid)
              *reinterpret_cast<uint4*>(a.opart + (part * kBM + quad * 32 + row) * kDLat + col + 4 * q) =
                  *reinterpret_cast<const uint4*>(stage + row * 256 + ((q ^ (row & 7)) << 4));
          }
        } else {
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            uint32_t w[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) w[k] = pack_bf16(__uint_as_float(r[8 * i + 2 * k]), __uint_as_float(r[8 * i + 2 * k + 1]));
            *reinterpret_cast<uint4*>(stage + sw128_offset((uint32_t)lane, (uint32_t)i)) = make_uint4(w[0], w[1], w[2], w[3]);
          }
          __syncwarp();
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const int row = 4 * i + (lane >> 3), q = lane & 7;
            if (quad * 32 + row < rows_valid)
              *reinterpret_cast<uint4*>(a.out + (grow0 + quad * 32 + row) * kDLat + col + 8 * q) =
                  *reinterpret_cast<const uint4*>(stage + sw128_offset((uint32_t)row, (uint32_t)q));
          }
        }
      }
    }
  }
  __syncwarp();
  cluster_wait();
  tc_fence_before();
  __syncthreads();
  if (warp == kSWarp) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
}

// Rows whose context was cut into pieces: O = sum 2^(lse_p - max) O_p / sum 2^(lse_p - max).  Rows
// of uncut requests have nothing to do.  A piece of which a row sees nothing (lse -inf) weighs 0; a NaN
// among the lse, which the maximum passes over, makes the row's sum NaN.
//
// Few pieces (and so, as a rule, many rows): a warp a row, 16 columns a lane, no barrier.
constexpr int kMergeFew = 8;
constexpr int kMergeRows = 4;  // rows of a block
__global__ void __launch_bounds__(32 * kMergeRows) tree_merge_few_kernel(const __grid_constant__ TreeArgs a, int64_t rows) {
  const int64_t r = (int64_t)blockIdx.x * kMergeRows + (threadIdx.x >> 5);
  if (r >= rows) return;
  const int lane = threadIdx.x & 31;
  const int node = a.req[0].first + (int)(r / a.H);
  const Request req = a.req[owner_of<&Request::first>(a, node)];
  const int tiles = page_count(req.ctx, req.n), pieces = (tiles + a.piece - 1) / a.piece;
  if (pieces <= 1) return;
  const int row = (node - req.first) * a.H + (int)(r % a.H);
  const int64_t part = (int64_t)req.part_base + (int64_t)(row / kBM) * pieces;
  asm volatile("griddepcontrol.wait;" ::: "memory");  // launched before the units' kernel has ended
  const float* lse = a.lsepart + part * kBM + row % kBM;
  const float4* o = reinterpret_cast<const float4*>(a.opart + (part * kBM + row % kBM) * kDLat) + lane;
  const float mine = lane < pieces ? lse[(int64_t)lane * kBM] : -INFINITY;
  float mx = mine;
#pragma unroll
  for (int k = 4; k > 0; k >>= 1) mx = fmaxf(mx, __shfl_xor_sync(kFull, mx, k));  // kMergeFew lanes
  mx = __shfl_sync(kFull, mx, 0);
  const float w = mine == -INFINITY ? 0.f : fast_exp2(mine - mx);
  float4 acc[4] = {};
  float sum = 0.f;
#pragma unroll 2
  for (int p = 0; p < pieces; ++p) {
    const float wp = __shfl_sync(kFull, w, p);
    sum += wp;
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      const float4 v = __ldcs(o + (int64_t)p * kBM * (kDLat / 4) + 32 * c);
      acc[c].x += wp * v.x;
      acc[c].y += wp * v.y;
      acc[c].z += wp * v.z;
      acc[c].w += wp * v.w;
    }
  }
  const float inv = sum != 0.f ? 1.f / sum : 0.f;
  const int64_t grow = (int64_t)req.first * a.H + row;
#pragma unroll
  for (int c = 0; c < 4; ++c)
    *reinterpret_cast<uint2*>(a.out + grow * kDLat + 128 * c + 4 * lane) =
        make_uint2(pack_bf16(acc[c].x * inv, acc[c].y * inv), pack_bf16(acc[c].z * inv, acc[c].w * inv));
  if (a.lse != nullptr && lane == 0) a.lse[grow] = sum != 0.f ? (mx + __log2f(sum)) * kLn2 : -INFINITY;
}

// Many pieces (few rows): a block a row; groups of 128 threads (4 columns a thread) share the row's
// pieces, eight loads of a thread in flight, and add up in shared memory.
constexpr int kMergeGroup = kDLat / 4;
constexpr int kMergeGroups = 4;
constexpr int kMergeWeights = 128;

__global__ void __launch_bounds__(kMergeGroup * kMergeGroups) tree_merge_kernel(const __grid_constant__ TreeArgs a) {
  __shared__ float weight[kMergeWeights], top[16];
  __shared__ float4 sums[kMergeGroups][kMergeGroup];
  const int tid = threadIdx.x, group = tid / kMergeGroup;
  constexpr int groups = kMergeGroups;
  const int node = a.req[0].first + (int)(blockIdx.x / a.H);
  const Request req = a.req[owner_of<&Request::first>(a, node)];
  const int tiles = page_count(req.ctx, req.n), pieces = (tiles + a.piece - 1) / a.piece;
  if (pieces <= 1) return;
  const int row = (node - req.first) * a.H + (int)(blockIdx.x % a.H);
  const int64_t part = (int64_t)req.part_base + (int64_t)(row / kBM) * pieces;
  asm volatile("griddepcontrol.wait;" ::: "memory");  // launched before the units' kernel has ended
  const float* lse = a.lsepart + part * kBM + row % kBM;
  const float* o = a.opart + (part * kBM + row % kBM) * kDLat + 4 * (tid % kMergeGroup);
  float mx = -INFINITY;
  for (int p = tid; p < pieces; p += blockDim.x) mx = fmaxf(mx, lse[(int64_t)p * kBM]);
#pragma unroll
  for (int k = 16; k > 0; k >>= 1) mx = fmaxf(mx, __shfl_xor_sync(kFull, mx, k));
  if ((tid & 31) == 0) top[tid >> 5] = mx;
  __syncthreads();
  for (int w = 0; w < (int)blockDim.x / 32; ++w) mx = fmaxf(mx, top[w]);
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  float sum = 0.f;
  for (int p0 = 0; p0 < pieces; p0 += kMergeWeights) {
    const int n = min(kMergeWeights, pieces - p0);
    if (tid < n) {
      const float x = lse[(int64_t)(p0 + tid) * kBM];
      weight[tid] = x == -INFINITY ? 0.f : fast_exp2(x - mx);
    }
    __syncthreads();
    for (int k = 0; k < n; ++k) sum += weight[k];
    constexpr int kUnroll = 8;
    for (int k0 = group; k0 < n; k0 += kUnroll * groups) {
      float4 v[kUnroll];
#pragma unroll
      for (int u = 0; u < kUnroll; ++u)
        if (k0 + u * groups < n) v[u] = __ldcs(reinterpret_cast<const float4*>(o + (int64_t)(p0 + k0 + u * groups) * kBM * kDLat));
#pragma unroll
      for (int u = 0; u < kUnroll; ++u)
        if (k0 + u * groups < n) {
          const float w = weight[k0 + u * groups];
          acc.x += w * v[u].x;
          acc.y += w * v[u].y;
          acc.z += w * v[u].z;
          acc.w += w * v[u].w;
        }
    }
    __syncthreads();
  }
  sums[group][tid % kMergeGroup] = acc;
  __syncthreads();
  if (group > 0) return;
  for (int g = 1; g < groups; ++g) {
    const float4 v = sums[g][tid];
    acc.x += v.x;
    acc.y += v.y;
    acc.z += v.z;
    acc.w += v.w;
  }
  const float inv = sum != 0.f ? 1.f / sum : 0.f;
  const int64_t grow = (int64_t)req.first * a.H + row;
  *reinterpret_cast<uint2*>(a.out + grow * kDLat + 4 * tid) =
      make_uint2(pack_bf16(acc.x * inv, acc.y * inv), pack_bf16(acc.z * inv, acc.w * inv));
  if (a.lse != nullptr && tid == 0) a.lse[grow] = sum != 0.f ? (mx + __log2f(sum)) * kLn2 : -INFINITY;
}

// ---------------------------------------------------------------------------------- host

// Cut of a batch's contexts: pages of a piece, and what follows from it.
struct Plan {
  int piece;
  int64_t n_long, n_rest;
  int64_t parts;  // partial results (units of cut requests)
};
// Bounds of a cut; without one a batch has at most kBatch * 1024 units and no partials.
constexpr int64_t kMaxUnits = int64_t(1) << 29;
constexpr int64_t kMaxParts = 8192;  // 2.1 GB of workspace; 100 x 131072 rows, 512 query rows each, take 1200

// Time until the last of a batch's units ends, in tile times: n_long units of `piece` pages each and
// then n_rest of `rest` (their mean), each with a start and end of `unit` tiles, are taken in this
// order by `pairs` pairs of SMs as they come free.
double makespan(int64_t n_long, double piece, int64_t n_rest, double rest, double unit, int pairs) {
  const double tl = piece + unit, tr = rest + unit;
  const int64_t waves = n_long / pairs, over = n_long % pairs;  // `over` pairs run one long unit more
  const double t0 = (double)waves * tl, t1 = t0 + tl;
  if (n_rest == 0) return over ? t1 : t0;
  // k rests on each of the pairs that come free first, until the others come free too
  const int64_t early = over ? pairs - over : 0;
  const int64_t fit = (int64_t)((t1 - t0) / tr + 0.999) * early;  // those started before t1
  if (over && n_rest <= fit) return std::max(t1, t0 + std::ceil((double)n_rest / (double)early) * tr);
  const double from = over ? t1 : t0;
  const int64_t left = over ? n_rest - (int64_t)((t1 - t0) / tr) * early : n_rest;
  return from + std::ceil((double)left / pairs) * tr;
}

// The cut with the least estimated time.  In tile times, measured: a unit's start and end take ~10 (12
// where units have at most 64 rows), a cut batch's merge 5 and a tenth for each partial.  With 8 for
// many rows 23 x 5000 ragged rows, 13 nodes of 24 heads, take 33.4 instead of 31.8 us; with a
// twentieth for a partial 16 x 2000, 5 nodes of 32 heads, 22.7 instead of 19.1 us; with 6 and 0.15 for
// the merge 4 x 1000, 4 nodes of 128 heads, is not cut: 24.6 instead of 19.3 us.
constexpr double kMergeCost = 5.0, kPartCost = 0.1;
Plan plan_batch(const int32_t* ctx, const int32_t* indptr, int B, int H, int pairs) {
  struct Like {
    int tiles, mt, count;  // neighbouring requests alike count as one
  } like[kBatch];
  int kinds = 0, most = 1, rows = 0;
  for (int b = 0; b < B; ++b) {
    const int n = indptr[b + 1] - indptr[b], tiles = page_count(ctx[b], n), mt = row_tiles(n, H);
    if (n == 0) continue;
    most = std::max(most, tiles);
    rows = std::max(rows, n * H);
    if (kinds > 0 && like[kinds - 1].tiles == tiles && like[kinds - 1].mt == mt) ++like[kinds - 1].count;
    else like[kinds++] = Like{tiles, mt, 1};
  }
  Plan best{most, 0, 0, 0};
  double best_cost = 1e300;
  // pieces from the longest context down, by steps of a few percent (fewer steps where every
  // request is of another length)
  const double unit = rows <= kHalf ? 12.0 : 10.0;
  const double step = kinds <= 8 ? 0.97 : 0.88;
  int last = 0;
  for (double f = 1.0;; f *= step) {
    const int piece = std::max(1, (int)std::ceil((double)most * f));
    if (piece != last) {
      Plan p{piece, 0, 0, 0};
      double rests = 0.0;
      for (int k = 0; k < kinds; ++k) {
        const Like& g = like[k];
        const int full = g.tiles / piece, rest = g.tiles - full * piece;
        const int64_t units = (int64_t)g.mt * g.count;
        p.n_long += units * full;
        if (rest) p.n_rest += units;
        rests += (double)units * rest;
        if (full + (rest ? 1 : 0) > 1) p.parts += (int64_t)units * (full + (rest ? 1 : 0));
      }
      const double cost = makespan(p.n_long, piece, p.n_rest, p.n_rest ? rests / p.n_rest : 0.0, unit, pairs) +
                          (p.parts ? kMergeCost + kPartCost * (double)p.parts : 0.0);
      if (p.n_long + p.n_rest > kMaxUnits) break;  // shorter pieces make more of them
      if (p.parts <= kMaxParts && cost < best_cost - 1e-9) {
        best_cost = cost;
        best = p;
      }
      last = piece;
    }
    if (piece == 1 || f * most < 3.0) break;
  }
  return best;
}

int sm_pairs() {
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) {
    (void)cudaGetLastError();
    sms = 152;
  }
  return std::max(1, sms / 2);
}

size_t opart_bytes(int64_t parts) { return align_up((size_t)parts * kBM * kDLat * sizeof(float), 256); }
size_t lsepart_bytes(int64_t parts) { return align_up((size_t)parts * kBM * sizeof(float), 256); }

irm_status check_lengths(const int32_t* ctx, const int32_t* indptr, int B, int H, int* most_nodes, int64_t* most_rows) {
  irm_status st = check_trees(indptr, B, most_nodes);
  if (st != IRM_OK) return st;
  if (H < 1 || H > IRM_MAX_HEADS) return fail(IRM_ERR_UNSUPPORTED, "H=%d outside [1, %d]", H, IRM_MAX_HEADS);
  if (ctx == nullptr) return fail(IRM_ERR_INVALID_ARG, "null context lengths");
  *most_rows = 0;
  for (int b = 0; b < B; ++b) {
    if (ctx[b] < 0) return fail(IRM_ERR_INVALID_ARG, "request %d: context length %d is negative", b, ctx[b]);
    const int64_t rows = (int64_t)ctx[b] + (indptr[b + 1] - indptr[b]);
    if (rows > INT32_MAX - kPage) return fail(IRM_ERR_UNSUPPORTED, "request %d: context exceeds int32", b);
    if (indptr[b + 1] > indptr[b] && rows > *most_rows) *most_rows = rows;
  }
  return IRM_OK;
}

// Scratch of the largest launch (the launches follow one another on the stream), and the first one's plan.
size_t scratch_bytes(const int32_t* ctx, const int32_t* indptr, int B, int H, int pairs, Plan* first) {
  *first = plan_batch(ctx, indptr, std::min(kBatch, B), H, pairs);
  int64_t parts = first->parts;
  for (int b0 = kBatch; b0 < B; b0 += kBatch)
    parts = std::max(parts, plan_batch(ctx + b0, indptr + b0, std::min(kBatch, B - b0), H, pairs).parts);
  return opart_bytes(parts) + lsepart_bytes(parts);
}

// cuTensorMapEncodeTiled, looked up through the runtime (a host-only function of the driver).
using EncodeFn = decltype(&cuTensorMapEncodeTiled);
EncodeFn encode_fn() {
  static const EncodeFn fn = [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess) {
      (void)cudaGetLastError();
      p = nullptr;
    }
    return reinterpret_cast<EncodeFn>(p);
  }();
  return fn;
}

// Map of `rows` rows of `width` elements: boxes of box_rows x box_cols, as wide as the swizzle.
template <class T>
irm_status encode_map(CUtensorMap* m, const void* base, int64_t rows, int width, uint32_t box_rows, uint32_t box_cols) {
  constexpr bool kBytes = sizeof(T) == 1;
  const EncodeFn fn = encode_fn();
  if (fn == nullptr) return fail(IRM_ERR_CUDA, "cuTensorMapEncodeTiled is not available");
  const cuuint64_t dims[2] = {(cuuint64_t)width, (cuuint64_t)rows}, strides[1] = {(cuuint64_t)width * sizeof(T)};
  const cuuint32_t box[2] = {box_cols, box_rows}, step[2] = {1, 1};
  const CUresult r = fn(m, kBytes ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(base), dims, strides, box, step,
                        CU_TENSOR_MAP_INTERLEAVE_NONE, box_cols * sizeof(T) == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
                        CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? IRM_OK : fail(IRM_ERR_CUDA, "cuTensorMapEncodeTiled failed (%d)", (int)r);
}

// The kernel's dynamic shared memory limit belongs to the device: raised once on each.
template <bool kCodes8>
cudaError_t raise_smem_limit() {
  static std::mutex mu;
  static bool done[128];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  std::lock_guard<std::mutex> lk(mu);
  if (dev >= 0 && dev < 128 && done[dev]) return cudaSuccess;
  e = cudaFuncSetAttribute(tree_attn_kernel<kCodes8>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)Layout<kCodes8>::kSmem);
  if (e == cudaSuccess && dev >= 0 && dev < 128) done[dev] = true;
  return e;
}

template <bool kCodes8>
irm_status attend(const void* q_lat, const void* q_rope, int B, int H, const int32_t* ctx_host,
                  const int32_t* q_indptr_host, const void* paged_kv, int64_t n_pages,
                  const int32_t* page_table, int max_pages, const uint32_t* tree_mask, int mask_words,
                  float softmax_scale, void* out, float* lse, void* workspace, size_t workspace_bytes,
                  cudaStream_t stream) {
  int nodes = 0;
  int64_t rows = 0;
  irm_status st = check_lengths(ctx_host, q_indptr_host, B, H, &nodes, &rows);
  if (st != IRM_OK) return st;
  if (n_pages < 1 || n_pages >= (int64_t(1) << 25)) return fail(IRM_ERR_UNSUPPORTED, "n_pages %lld outside [1, 2^25)", (long long)n_pages);
  if (max_pages < 1) return fail(IRM_ERR_INVALID_ARG, "max_pages must be positive");
  if ((rows + kPage - 1) / kPage > max_pages)
    return fail(IRM_ERR_INVALID_ARG, "a request of %lld rows needs more than max_pages=%d pages", (long long)rows, max_pages);
  if (mask_words < 1 || (int64_t)mask_words * 32 < nodes)
    return fail(IRM_ERR_INVALID_ARG, "mask_words=%d does not cover %d nodes", mask_words, nodes);
  if (!std::isfinite(softmax_scale * 1.4426950408889634f) || softmax_scale <= 0.f)
    return fail(IRM_ERR_INVALID_ARG, "softmax_scale must be finite and positive");
  if ((int64_t)q_indptr_host[B] * H >= INT32_MAX) return fail(IRM_ERR_UNSUPPORTED, "too many query rows");
  if (!q_lat || !q_rope || !paged_kv || !page_table || !tree_mask || !out) return fail(IRM_ERR_INVALID_ARG, "null device pointer");
  if (!aligned(q_lat, 16) || !aligned(q_rope, 16) || !aligned(paged_kv, 16) || !aligned(out, 16))
    return fail(IRM_ERR_INVALID_ARG, "q_lat, q_rope, paged_kv and out must be 16-byte aligned");
  if (!aligned(page_table, 4) || !aligned(tree_mask, 4) || !aligned(lse, 4))
    return fail(IRM_ERR_INVALID_ARG, "misaligned device pointer");
  const int pairs = sm_pairs();
  Plan first;
  const size_t need = IRM_WORKSPACE_HEADER + scratch_bytes(ctx_host, q_indptr_host, B, H, pairs, &first);
  if (!workspace || !aligned(workspace, 256) || workspace_bytes < need)
    return fail(IRM_ERR_WORKSPACE, "workspace must be 256-byte aligned and hold %zu bytes (got %zu)", need, workspace_bytes);
  if (q_indptr_host[B] == 0) return IRM_OK;
  TreeArgs a{};
  const int64_t q_rows = (int64_t)q_indptr_host[B] * H;
  const int64_t kv_rows = n_pages * kPage;
  if (kCodes8) {
    st = encode_map<uint8_t>(&a.map_lat, paged_kv, kv_rows, IRM_ROW_BYTES8, kPage, 128);
    if (st == IRM_OK) st = encode_map<uint16_t>(&a.map_rope, paged_kv, kv_rows, IRM_ROW_BYTES8 / 2, kPage, 32);
    a.kv8 = static_cast<const uint8_t*>(paged_kv);
  } else {
    st = encode_map<uint16_t>(&a.map_lat, paged_kv, kv_rows, kDRow, kPage, 64);
    if (st == IRM_OK) st = encode_map<uint16_t>(&a.map_rope, paged_kv, kv_rows, kDRow, kPage, 32);
  }
  if (st != IRM_OK) return st;
  if ((st = encode_map<uint16_t>(&a.map_ql, q_lat, q_rows, kDLat, 32, 64)) != IRM_OK) return st;
  if ((st = encode_map<uint16_t>(&a.map_qr, q_rope, q_rows, kDRope, 32, 32)) != IRM_OK) return st;
  cudaError_t e = raise_smem_limit<kCodes8>();
  if (e != cudaSuccess) return cuda_fail(e, "tree attention set-up");
  a.page_table = page_table;
  a.mask = tree_mask;
  a.n_pages = n_pages;
  a.H = H;
  a.max_pages = max_pages;
  a.mask_words = mask_words;
  a.scale_log2 = softmax_scale * 1.4426950408889634f;
  a.out = static_cast<__nv_bfloat16*>(out);
  a.lse = lse;
  a.status = static_cast<int*>(workspace);
  for (int b0 = 0; b0 < B; b0 += kBatch) {
    a.b0 = b0;
    a.B = std::min(kBatch, B - b0);
    const int32_t *ctx = ctx_host + b0, *indptr = q_indptr_host + b0;
    const Plan p = b0 == 0 ? first : plan_batch(ctx, indptr, a.B, H, pairs);
    const int units = (int)(p.n_long + p.n_rest);
    if (units == 0) continue;
    a.piece = p.piece;
    a.n_long = (int)p.n_long;
    int nl = 0, nr = 0, most_pieces = 0;
    int64_t np = 0;
    for (int b = 0; b < a.B; ++b) {
      const int n = indptr[b + 1] - indptr[b], tiles = page_count(ctx[b], n), mt = row_tiles(n, H);
      const int full = tiles / p.piece, rest = tiles % p.piece ? 1 : 0;
      a.req[b] = Request{indptr[b], n, ctx[b], nl, nr, (int32_t)np, {0, 0}};
      nl += mt * full;
      nr += mt * rest;
      most_pieces = std::max(most_pieces, full + rest);
      if (full + rest > 1) np += (int64_t)mt * (full + rest);
    }
    uint8_t* ws = static_cast<uint8_t*>(workspace) + IRM_WORKSPACE_HEADER;
    a.opart = reinterpret_cast<float*>(ws);
    a.lsepart = reinterpret_cast<float*>(ws + opart_bytes(p.parts));
    tree_attn_kernel<kCodes8><<<2 * units, Layout<kCodes8>::kThreads, Layout<kCodes8>::kSmem, stream>>>(a);
    if ((e = cudaGetLastError()) != cudaSuccess) return cuda_fail(e, "tree attention launch");
    if (p.parts) {
      cudaLaunchConfig_t cfg = {};
      const int64_t merge_rows = (int64_t)(indptr[a.B] - indptr[0]) * H;
      const bool few = most_pieces <= kMergeFew;
      cfg.gridDim = dim3((unsigned)(few ? (merge_rows + kMergeRows - 1) / kMergeRows : merge_rows));
      cfg.blockDim = dim3(few ? 32 * kMergeRows : kMergeGroup * kMergeGroups);
      cfg.stream = stream;
      cudaLaunchAttribute early[1];
      early[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
      early[0].val.programmaticStreamSerializationAllowed = 1;
      cfg.attrs = early;
      cfg.numAttrs = 1;
      e = few ? cudaLaunchKernelEx(&cfg, tree_merge_few_kernel, a, merge_rows) : cudaLaunchKernelEx(&cfg, tree_merge_kernel, a);
      if (e != cudaSuccess) return cuda_fail(e, "tree attention merge launch");
    }
  }
  return IRM_OK;
}

}  // namespace
}  // namespace irm

extern "C" {

irm_status irm_mla_attn_tree_workspace_size(const int32_t* ctx_host, const int32_t* q_indptr_host, int B, int H,
                                            size_t* bytes) {
  using namespace irm;
  if (bytes == nullptr) return fail(IRM_ERR_INVALID_ARG, "bytes is null");
  int nodes = 0;
  int64_t rows = 0;
  const irm_status st = check_lengths(ctx_host, q_indptr_host, B, H, &nodes, &rows);
  if (st != IRM_OK) return st;
  Plan first;
  *bytes = IRM_WORKSPACE_HEADER + scratch_bytes(ctx_host, q_indptr_host, B, H, sm_pairs(), &first);
  return IRM_OK;
}

irm_status irm_mla_attn_tree(const void* q_lat, const void* q_rope, int B, int H, const int32_t* ctx_host,
                             const int32_t* q_indptr_host, const void* paged_kv, int64_t n_pages,
                             const int32_t* page_table, int max_pages, const uint32_t* tree_mask, int mask_words,
                             float softmax_scale, void* out, float* lse, void* workspace, size_t workspace_bytes,
                             cudaStream_t stream) {
  return irm::attend<false>(q_lat, q_rope, B, H, ctx_host, q_indptr_host, paged_kv, n_pages, page_table, max_pages, tree_mask, mask_words,
                             softmax_scale, out, lse, workspace, workspace_bytes, stream);
}

irm_status irm_mla_attn_tree8(const void* q_lat, const void* q_rope, int B, int H, const int32_t* ctx_host,
                              const int32_t* q_indptr_host, const void* paged_kv, int64_t n_pages,
                              const int32_t* page_table, int max_pages, const uint32_t* tree_mask, int mask_words,
                              float softmax_scale, void* out, float* lse, void* workspace, size_t workspace_bytes,
                              cudaStream_t stream) {
  return irm::attend<true>(q_lat, q_rope, B, H, ctx_host, q_indptr_host, paged_kv, n_pages, page_table, max_pages, tree_mask, mask_words,
                            softmax_scale, out, lse, workspace, workspace_bytes, stream);
}

}  // extern "C"
