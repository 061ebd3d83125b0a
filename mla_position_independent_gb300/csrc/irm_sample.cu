// Sampling from logits with temperature, top-k, top-p and min-p, from given uniform numbers: the token,
// the probabilities left (what the draft verification takes), or both.
//
// Per row, candidates in the order of their logits (ties: lowest index first):
//   w_v = exp((l_v - max) / T);  top-k keeps the first k;  top-p of those the shortest run whose w reach p
//   of their sum;  min-p of those the ones with w >= min_p;  token = lowest v with
//   cumsum(w)(v) > r sum(w) in index order over what is left.
// What is kept is a run of the order from its start, so it is described by its last element, a cut
// (logit, index), and no row is sorted: a histogram of the logits' distance from the maximum (1023 bins, 23
// an octave of w) finds the bin that holds the cut.  Up to 128 elements that may be kept are ranked among
// themselves and the row finished from them.  Else the candidates, up to a few bins behind the cut, are listed
// where shared memory holds them, and the cut's bin ranked, after a second histogram inside the bin if it has more
// than 256.  A top-p cut: some 96 elements are ranked around a guess from the histogram and each bin's middle
// weight, with the exact sum before them, which confirms the guess or moves it.  p of the sum of all weights is
// known by bounds: the candidates' exactly, the others' in fp32 with what rounding may have done to it; where an
// element's running weight lies between the bounds (one row in a hundred), or bins are so full that
// passes repeat, that sum too is made exact.  The draw is an inverse of the sums of 128 elements each, then
// of one group.  More than 256 in a bin's 1024th part are mostly equal logits, of which a count finds the last.
//
// Arithmetic.  Which token comes out must not depend on the split or the order of addition, and a flat
// row of 100k entries has cumulative sums 1e-5 apart, so weights are integers in units of 2^-43 and
// their sums are exact.  fp32 exponentials (2^-23) would move 100k boundaries by 1e-7 each, so that one
// draw in a hundred came out wrong; here a weight is good to 2^-37 of the largest and 2^-33 of itself: the distance from the
// maximum and its product with 1 / T in two fp32 parts, 32 table values and a polynomial of degree 5, some
// 70 instructions.  fp64 runs at 1 / 64 of the fp32 rate on this GPU.  Thresholds (p of a sum, r of a sum) are
// exact products of 24 and 64 bits.  Probabilities are fp32 exponentials (2^-21) over the exact
// sum.
//
// A cluster of 1 to 8 CTAs shares a row, which stays in shared memory from its one read, in the type in which it
// came, where a CTA's part fits (some 53600 logits of fp32, 65536 of bf16); longer rows are read again by each pass.
//
// What bounds it.  One row: latency, 14.7 us for 102400 logits with top-k 50 and top-p 0.9, of which the row and its
// maximum take 2.6, the histogram and its exchange 4, the list and its exchange 4, the ranks 3.  Many rows:
// instructions and what a CTA does whatever its part's length (scans, exchanges, ranks), which is why few CTAs
// a row are best: 384 bf16 rows with top-p and probabilities 209 us (35 by their bytes), 111 instructions a warp and
// 32 logits at 0.58 a clock and scheduler, two CTAs of 512 threads on an SM.  Steps that were, for these 384 rows: a pass
// over all elements, and one over those near the cut, for each sum 635; the candidates listed with their weights
// 475; one element a lane, ranks by four lanes an element 409; fewer neighbours and shorter lists 390; bf16 rows held as
// bf16 by clusters of 4 instead of 8 285, of 3 279; four logits a lane and lists by masks 270, rows finished from
// lists of 128 instead of 448 elements 262; the sum of what is not listed by bounds, and a missed window
// moved, 217 (fp32 302 -> 268, 64 rows with some flat distributions 56 -> 57), a candidate in one word 206 to 213.
// Not taken: all of the sum by bounds, which decide too seldom (440 instead of 409); lists sorted by a bitonic
// network instead of ranked (270 instead of 259); bounds also where the cut's bin has more than 256 (64 rows with
// flat ones 62).
#include <cuda_runtime.h>
#include <algorithm>
#include <cmath>
#include <cstdint>
#include <mutex>
#include <type_traits>

#include "irm_common.cuh"
#include "irm_host_util.h"
#include "irm_pipeline.cuh"

namespace irm {
namespace {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxCluster = 8;
constexpr int kMaxVocab = 1 << 20;
constexpr int kBins = 1024;         // the last one holds what has no weight
constexpr int kList = 256;          // elements that are ranked among themselves
constexpr int kFew = 128;           // elements from which a row is finished at once (each is compared with each, twice)
constexpr int kNear = 96;           // elements around its guess that a top-p cut ranks at once
constexpr int kGroup = 128;         // elements that a warp looks at at once
constexpr int kGroups = 512;        // sums of a CTA's logits that are kept, of 128 each (in rows that do not stay in shared memory 256)
constexpr uint32_t kFull = 0xffffffffu;
constexpr float kOctaves = 43.9f;   // below 2^-43.9 a weight rounds to nothing
constexpr float kBinScale = (kBins - 1) / kOctaves;
constexpr uint64_t kOne = 1ull << 43;
static_assert(kList <= kThreads && 2 * kThreads == kBins, "a thread an element, two bins a thread");

struct SampleArgs {
  const void* logits;
  int64_t ld;
  int V, seg;    // logits of a row, and of a CTA's part of it (a multiple of 4)
  int cap, cap_bare;  // candidates that a CTA can hold in shared memory with their weights, and without
  const float *temperature, *top_p, *min_p, *uniforms;
  const int32_t* top_k;
  int32_t* token;
  float* probs;
  int64_t probs_ld;
  int* status;
  int vec_in, vec_out;  // whole vectors of logits, of probabilities
};

struct __align__(16) Item {
  float l;
  int32_t idx;
  uint64_t w;
};

// 2^(i / 32): four more than its first 21 bits, and the rest
__constant__ float kPow[2][32] = {
    {0x1.4p+2f, 0x1.4166c4p+2f, 0x1.42d562p+2f, 0x1.444c08p+2f,
     0x1.45caep+2f, 0x1.47521cp+2f, 0x1.48e1eap+2f, 0x1.4a7a78p+2f,
     0x1.4c1bf8p+2f, 0x1.4dc69cp+2f, 0x1.4f7a9ap+2f, 0x1.513822p+2f,
     0x1.52ff6cp+2f, 0x1.54d0aep+2f, 0x1.56ac2p+2f, 0x1.5891fap+2f,
     0x1.5a827ap+2f, 0x1.5c7dd8p+2f, 0x1.5e8452p+2f, 0x1.609626p+2f,
     0x1.62b396p+2f, 0x1.64dcdep+2f, 0x1.671246p+2f, 0x1.69540ep+2f,
     0x1.6ba27ep+2f, 0x1.6dfddcp+2f, 0x1.70667p+2f, 0x1.72dc84p+2f,
     0x1.756064p+2f, 0x1.77f25cp+2f, 0x1.7a92bep+2f, 0x1.7d41dap+2f},
    {0x0p+0f, -0x1.6753d4p-23f, -0x1.30677p-24f, -0x1.7f6d26p-23f,
     0x1.e3ea8cp-23f, 0x1.8b45cep-23f, -0x1.18a9dcp-24f, -0x1.5c0424p-25f,
     0x1.4636e2p-25f, 0x1.b9d54ep-23f, -0x1.9f6e5ep-23f, -0x1.f9e76ep-24f,
     -0x1.564eaep-23f, -0x1.4b1584p-23f, -0x1.15bd5ep-23f, 0x1.81d2acp-23f,
     -0x1.980c44p-24f, -0x1.713a08p-24f, -0x1.829fdp-25f, 0x1.94cce2p-24f,
     -0x1.eeaafap-23f, 0x1.866e3p-23f, 0x1.51f848p-27f, 0x1.91f12ap-23f,
     0x1.95ad3ap-24f, -0x1.a09438p-25f, -0x1.13d56cp-23f, -0x1.18837cp-23f,
     -0x1.1822dcp-23f, 0x1.9bdcdap-23f, 0x1.152486p-23f, -0x1.248dd6p-23f}};

struct Shared {
  uint64_t part[kWarps][4];
  uint64_t tot[2][kMaxCluster][4];
  union {
    uint32_t hist[kBins];
    uint64_t gsum[kGroups];
  } u;
  Item list[kList], own[kList];  // what is ranked: of the whole row, and what this CTA has of it
  float th4[32], tl[32];  // kPow: read at an index of each lane's own
  uint32_t n_own, scan[kWarps];
  float fscan[kWarps], mass;
  // 1 / (h T) in two parts, and log2(e) / (h T).  h is 1; 2^-24 for a temperature so high that differences of
  // logits that overflow still count, and that 1 / T may be denormal; 2^24 for one so low that differences of denormal
  // logits count
  float ih, il, ch, h, m;
  float ch_off;  // what ch is off by, so that exp2(t) has to be changed by ch_off |t| of itself
  int bin, cut_idx;
  uint32_t bin_count, bin_above, near_lo, near_hi;
  float cut_l;
  uint64_t sum;
};

__device__ __forceinline__ uint64_t warp_sum64(uint64_t v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(kFull, v, o);
  return v;
}
// floor(f x) for 0 <= f <= 1, and the same rounded up: the product of 24 and 64 bits.
__device__ __forceinline__ uint64_t part_of_sum(float f, uint64_t x, bool up) {
  const uint32_t b = __float_as_uint(f), e = b >> 23;  // f = m 2^(e - 150)
  if (e == 0) return up && b != 0 && x != 0 ? 1ull : 0ull;  // a denormal times less than 2^64
  const uint64_t m = (b & 0x7fffffu) | 0x800000u, lo = m * x, hi = __umul64hi(m, x);
  const uint32_t k = 150u - e;  // 23 .. 149
  if (k >= 128) return up && (hi | lo) != 0 ? 1ull : 0ull;
  const uint64_t whole = k >= 64 ? hi >> (k - 64) : lo >> k | hi << (64 - k);
  const bool rest = k >= 64 ? (lo | (k > 64 ? hi << (128 - k) : 0ull)) != 0 : lo << (64 - k) != 0;
  return whole + (up && rest ? 1ull : 0ull);
}
__device__ __forceinline__ uint64_t warp_max64(uint64_t v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const uint64_t x = __shfl_xor_sync(kFull, v, o);
    v = x > v ? x : v;
  }
  return v;
}
__device__ __forceinline__ void st_peer_u64(uint32_t addr, uint64_t v) {
  asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(addr), "l"(v) : "memory");
}
__device__ __forceinline__ uint32_t ld_peer_u32(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ uint2 ld_peer_v2(uint32_t addr) {
  uint2 v;
  asm volatile("ld.shared::cluster.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ uint4 ld_peer_v4(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared::cluster.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr) : "memory");
  return v;
}

// Order-preserving integer of a logit (no NaN, no -0), and back.
__device__ __forceinline__ uint32_t order_key(float l) {
  const uint32_t b = __float_as_uint(l);
  return b >> 31 ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float key_logit(uint32_t k) { return __uint_as_float(k >> 31 ? k & 0x7fffffffu : ~k); }
// NaN as -infinity, -0 as 0
__device__ __forceinline__ float clean(float l) { return l == l ? l + 0.f : -INFINITY; }

// Distance of a logit from the maximum in octaves of weight (<= 0; NaN or below -kOctaves: no weight).  h m overflows
// where neighbouring logits are far more octaves apart than a weight has: the distance is then infinite, and negative
// for a negative maximum too.
__device__ __forceinline__ float octaves(float l, float m, float h, float ch) { return l == m ? 0.f : -fabsf(fmaf(l, h, -h * m)) * ch; }
__device__ __forceinline__ int bin_of(float t) { return t > -kOctaves ? min(kBins - 2, (int)__float2uint_rz(-t * kBinScale)) : kBins - 1; }
// The same inside a bin: its elements spread over kBins again.  Every pass has to place an element alike, so the product
// and the difference are rounded one by one (fused by some passes and not by others they would differ by up to 1 / 32 of a part).
__device__ __forceinline__ int fine_of(float t, int bin) {
  return min(kBins - 1, max(0, (int)(__fsub_rn(__fmul_rn(-t, kBinScale), (float)bin) * (float)kBins)));
}

// exp((l - m) / T) in units of 2^-43, for a logit with a weight (octaves > -kOctaves).
__device__ __forceinline__ uint64_t weight(float l, float m, const Shared& sh) {
  if (l == m) return kOne;
  const float hl = sh.h * l, hm = sh.h * m, d = hl - hm;
  const bool low = fabsf(l) > fabsf(m);
  const float big = low ? hl : -hm, small = low ? -hm : hl;
  const float dl = small - (d - big);  // what the difference lost
  const float th = d * sh.ih;
  const float te = fmaf(dl, sh.ih, fmaf(d, sh.il, fmaf(d, sh.ih, -th)));
  // th + te = k ln2 / 32 + x: ln2 / 32 in 12 bits, whose products with k are exact, and the rest
  constexpr float kLn2Hi = 0x1.62ep-6f, kLn2Lo = 0x1.0bfbe8p-20f;
  const float shifted = fmaf(th, 46.16624130844683f, 0x1.8p23f);  // to the nearest whole number
  const float kf = shifted - 0x1.8p23f;
  const float x0 = fmaf(kf, -kLn2Hi, th), x1 = fmaf(kf, -kLn2Lo, te);
  const float xh = x0 + x1, xl = x1 - (xh - x0);
  const int k = __float_as_int(shifted) - __float_as_int(0x1.8p23f), i = k & 31, n = -(k >> 5);
  // e^x - 1 = x + x^2 (1/2 + x/6 + x^2/24 + x^3/120), |x| < 0.011
  const float s = xh * xh;
  const float q = fmaf(xh, fmaf(xh, fmaf(xh, 1.f / 120.f, 1.f / 24.f), 1.f / 6.f), 0.5f);
  const float yh = fmaf(s, q, xh);
  const float yl = fmaf(s, q, xh - yh) + fmaf(xl, xh, xl);
  const float t4 = sh.th4[i], tl = sh.tl[i], t = t4 - 4.f;
  const float ph = __fmul_rn(t, yh), pl = fmaf(t, yh, -ph);
  const float a = t4 + ph;  // in [4, 8): multiples of 2^-21 (ph is the rounded product: what it lost is in pl)
  const float rest = fmaf(tl, yh, fmaf(t, yl, pl)) + (ph - (a - t4)) + tl;
  const float b = rest + 0x1.8p-19f;  // |rest| <= 2^-21 and a little: multiples of 2^-42
  const int64_t v = ((int64_t)(__float_as_int(a) - 0x40800000) << 21) + (__float_as_int(b) - __float_as_int(0x1.8p-19f));
  return (((uint64_t)v << 2 >> n) + 1) >> 1;
}

// The same, called: where few elements need it, so that the code of a row's one pass stays in the instruction caches.
__device__ __noinline__ uint64_t weight_of(float l, float m, const Shared& sh) { return weight(l, m, sh); }

// exp((l - m) / T) in fp32, to 2^-21 of itself: the exponent in two parts, since 44 octaves times a rounding or two of
// it would be 2^-17.
__device__ __forceinline__ float share(float l, float m, const Shared& sh) {
  if (l == m) return 1.f;
  const float hl = sh.h * l, hm = sh.h * m, d = hl - hm;
  const bool low = fabsf(l) > fabsf(m);
  const float big = low ? hl : -hm, small = low ? -hm : hl;
  const float dl = small - (d - big);
  const float th = d * sh.ih, te = fmaf(dl, sh.ih, fmaf(d, sh.il, fmaf(d, sh.ih, -th)));
  constexpr float kLog2e = 1.4426950408889634f, kLog2eLo = (float)(1.4426950408889634 - (double)kLog2e);
  const float y = th * kLog2e, rest = fmaf(th, kLog2e, -y) + fmaf(th, kLog2eLo, te * kLog2e);
  const float w = fast_exp2(y);
  return fmaf(w, rest * 0.6931472f, w);
}

template <bool BF16, bool RES>
__global__ void __launch_bounds__(kThreads, 2) sample_kernel(const __grid_constant__ SampleArgs a) {
  extern __shared__ __align__(16) uint8_t row_bytes[];
  using Held = typename std::conditional<BF16, uint16_t, float>::type;
  Held* row_sh = reinterpret_cast<Held*>(row_bytes);  // the CTA's logits, in the type in which they came
  __shared__ Shared sh;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  uint32_t C;
  asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(C));
  const uint32_t rank = cluster_ctarank();
  const int64_t b = (int64_t)(blockIdx.x / C);
  const int v0 = min(a.V, (int)rank * a.seg), n_own = min(a.V, v0 + a.seg) - v0;
  const float* f32 = static_cast<const float*>(a.logits) + b * a.ld + v0;
  const __nv_bfloat16* b16 = static_cast<const __nv_bfloat16*>(a.logits) + b * a.ld + v0;
  cluster_arrive();  // waited for before the first store into a peer's shared memory

  auto one = [&](int i) -> float {
    if (!RES) return clean(BF16 ? __bfloat162float(b16[i]) : f32[i]);
    return BF16 ? __uint_as_float((uint32_t)row_sh[i] << 16) : (float)row_sh[i];
  };
  // A warp looks at a contiguous part of the CTA's logits, a group (four neighbours a lane) at a time.
  const int wseg = (n_own + kWarps * kGroup - 1) / (kWarps * kGroup) * kGroup;
  const int w0 = min(n_own, warp * wseg), w1 = min(n_own, w0 + wseg);
  // f(logit, index, weight()) for the CTA's logits, or for the candidates once they are listed (in index order)
  // Candidates: the weight (44 bits) and behind it the place in the CTA's part; too many for that: the places alone.
  uint64_t* cand = reinterpret_cast<uint64_t*>(row_sh + (RES ? a.seg : 0));
  uint16_t* cand_at = reinterpret_cast<uint16_t*>(cand);
  int n_cand = -1;
  bool weighed = true;
  auto place = [&](int i) -> int { return weighed ? (int)(cand[i] & 0xffffu) : cand_at[i]; };
  auto each = [&](auto f) {
    if (n_cand >= 0 && weighed) {
      for (int i = tid; i < n_cand; i += kThreads) {
        const uint64_t x = cand[i];
        const int at = (int)(x & 0xffffu);
        f(one(at), v0 + at, [&] { return x >> 16; });
      }
      return;
    }
    const bool bare = n_cand >= 0;
    for (int i = bare ? tid : w0 + lane; i < (bare ? n_cand : w1); i += bare ? kThreads : 32) {
      const int at = bare ? cand_at[i] : i;
      const float l = one(at);
      f(l, v0 + at, [&] { return weight_of(l, sh.m, sh); });
    }
  };
  // The same for the passes that most rows take: four neighbours a lane at a time.
  auto each4 = [&](auto f) {
    if (n_cand >= 0 || !RES) {
      each(f);
      return;
    }
    for (int i = w0 + 4 * lane; i < w1; i += kGroup) {
      float x[4];
      if (BF16) {
        const uint2 w = *reinterpret_cast<const uint2*>(row_sh + i);
        x[0] = __uint_as_float(w.x << 16), x[1] = __uint_as_float(w.x & 0xffff0000u);
        x[2] = __uint_as_float(w.y << 16), x[3] = __uint_as_float(w.y & 0xffff0000u);
      } else {
        const float4 w = *reinterpret_cast<const float4*>(row_sh + i);
        x[0] = w.x, x[1] = w.y, x[2] = w.z, x[3] = w.w;
      }
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (i + e < w1) f(x[e], v0 + i + e, [&] { return weight_of(x[e], sh.m, sh); });
    }
  };

  auto cluster_sync = [&] {
    __syncwarp();  // the barrier's instruction is a whole warp's
    cluster_arrive();
    cluster_wait();
  };
  int slot = 0;
  // sums over the cluster of N values a thread; `before`: of v[0], what the CTAs before this one have
  uint64_t before = 0;
  auto cluster_sum = [&](auto& v, bool take_max = false) {
    constexpr int N = sizeof(v) / sizeof(v[0]);
#pragma unroll
    for (int k = 0; k < N; ++k) {
      const uint64_t x = take_max ? warp_max64(v[k]) : warp_sum64(v[k]);
      if (lane == 0) sh.part[warp][k] = x;
    }
    __syncthreads();
    if (warp == 0) {
#pragma unroll
      for (int k = 0; k < N; ++k) {
        const uint64_t mine = lane < kWarps ? sh.part[lane][k] : 0ull;
        const uint64_t x = take_max ? warp_max64(mine) : warp_sum64(mine);
        if (lane < (int)C) st_peer_u64(mapa_shared(smem_u32(&sh.tot[slot][rank][k]), (uint32_t)lane), x);
      }
    }
    __syncwarp();
    cluster_arrive();
    cluster_wait();
#pragma unroll
    for (int k = 0; k < N; ++k) {
      uint64_t t = 0;
      for (int c = 0; c < (int)C; ++c) {
        if (k == 0 && c == (int)rank) before = t;
        const uint64_t x = sh.tot[slot][c][k];
        t = take_max ? (x > t ? x : t) : t + x;
      }
      v[k] = t;
    }
    slot ^= 1;
  };

  // ---- the row's settings ----------------------------------------------------------------
  const float temp = a.temperature ? a.temperature[b] : 1.f, top_p = a.top_p ? a.top_p[b] : 1.f;
  const float min_p = a.min_p ? a.min_p[b] : 0.f;
  const int top_k = a.top_k ? a.top_k[b] : 0;
  const float uniform = a.token ? a.uniforms[b] : 0.f, rf = fminf(fmaxf(uniform, 0.f), 1.f);
  if (rank == 0 && tid == 0 && !(uniform >= 0.f && uniform < 1.f)) set_status(a.status, kDevErrBounds);
  const bool first_alone = !(temp > 0.f) || top_k == 1 || top_p <= 0.f || min_p > 1.f;
  if (tid < 32) {
    sh.th4[tid] = kPow[0][tid];
    sh.tl[tid] = kPow[1][tid];
  } else if (tid == 32) {
    const float h = temp > 0x1p100f ? 0x1p-24f : temp < 0x1p-100f ? 0x1p24f : 1.f;
    const float ht = h * temp, inv = 1.f / ht;  // h T is exact
    sh.h = h;
    sh.ih = inv;
    sh.il = inv > 0.f ? fmaf(-inv, ht, 1.f) * inv : 0.f;  // T may be infinite
    constexpr float kLog2e = 1.4426950408889634f, kLog2eLo = (float)(1.4426950408889634 - (double)kLog2e);
    sh.ch = inv * kLog2e;
    const float lost = fmaf(inv, kLog2e, -sh.ch) + fmaf(inv, kLog2eLo, sh.il * kLog2e);
    sh.ch_off = sh.ch > 0.f ? -0.6931472f * lost / sh.ch : 0.f;
  }
  // ---- the row, and its maximum ------------------------------------------------------------
  auto hold = [&](int i, float x) {
    if (BF16) reinterpret_cast<uint16_t*>(row_bytes)[i] = (uint16_t)(__float_as_uint(x) >> 16);
    else reinterpret_cast<float*>(row_bytes)[i] = x;
  };
  float best = -INFINITY;
  if (RES && a.vec_in) {
    constexpr int kAhead = 4;
    const int whole = w0 + (w1 - w0) / 4 * 4;  // w0 is a multiple of 4
    for (int i = w0 + 4 * lane; i < whole; i += kAhead * kGroup) {
      float4 x[kAhead];
#pragma unroll
      for (int u = 0; u < kAhead; ++u) {
        const int at = min(i + u * kGroup, whole - 4);  // the last one again: neither stored nor counted amiss
        if (BF16) {
          const uint2 w = *reinterpret_cast<const uint2*>(b16 + at);
          x[u] = make_float4(__uint_as_float(w.x << 16), __uint_as_float(w.x & 0xffff0000u), __uint_as_float(w.y << 16),
                             __uint_as_float(w.y & 0xffff0000u));
        } else {
          x[u] = *reinterpret_cast<const float4*>(f32 + at);
        }
      }
#pragma unroll
      for (int u = 0; u < kAhead; ++u) {
        x[u] = make_float4(clean(x[u].x), clean(x[u].y), clean(x[u].z), clean(x[u].w));
        Held* to = row_sh + min(i + u * kGroup, whole - 4);
        if (BF16)
          *reinterpret_cast<uint2*>(to) = make_uint2(__byte_perm(__float_as_uint(x[u].x), __float_as_uint(x[u].y), 0x7632),
                                                     __byte_perm(__float_as_uint(x[u].z), __float_as_uint(x[u].w), 0x7632));
        else
          *reinterpret_cast<float4*>(to) = x[u];
        best = fmaxf(best, fmaxf(fmaxf(x[u].x, x[u].y), fmaxf(x[u].z, x[u].w)));
      }
    }
    if (lane < w1 - whole) {
      const float x = clean(BF16 ? __bfloat162float(b16[whole + lane]) : f32[whole + lane]);
      hold(whole + lane, x);
      best = fmaxf(best, x);
    }
  } else {
#pragma unroll 4
    for (int i = w0 + lane; i < w1; i += 32) {
      const float x = clean(BF16 ? __bfloat162float(b16[i]) : f32[i]);
      if (RES) hold(i, x);
      best = fmaxf(best, x);
    }
  }
  __syncwarp();  // a warp reads what its own lanes have stored
  cluster_wait();
  uint64_t top[1] = {order_key(best)};
  cluster_sum(top, true);
  const float m = key_logit((uint32_t)top[0]);
  if (tid == 0) sh.m = m;
  __syncthreads();
  float* probs = a.probs ? a.probs + b * a.probs_ld + v0 : nullptr;
  auto zero_probs = [&] {
    const int whole = a.vec_out ? w0 + (w1 - w0) / 4 * 4 : w0;
    for (int i = w0 + 4 * lane; i < whole; i += kGroup) *reinterpret_cast<float4*>(probs + i) = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int i = whole + lane; i < w1; i += 32) probs[i] = 0.f;
  };

  const bool none = m == -INFINITY;
  if (none || first_alone) {  // the same in every CTA of the cluster
    int first = -1;
    if (!none) {
      uint64_t at[1] = {0};  // the lowest index, as the largest complement
      each([&](float l, int idx, auto) {
        if (l == m) at[0] = max(at[0], (unsigned long)(uint32_t)~idx);
      });
      cluster_sum(at, true);
      first = (int)~(uint32_t)at[0];
    }
    if (probs != nullptr) {
      zero_probs();
      __syncthreads();
      if (tid == 0 && first >= v0 && first < v0 + n_own) probs[first - v0] = 1.f;
    }
    if (a.token != nullptr && rank == 0 && tid == 0) a.token[b] = first;
    cluster_sync();  // no CTA ends while another may still store into it
    return;
  }
  const float ch = sh.ch, half = sh.h;

  // ---- what is kept: everything before, and up to, (cut_l, cut_idx) in the order -----------------
  float cut_l = -INFINITY;
  int cut_idx = INT_MAX;
  auto kept = [&](float l, int idx) { return l > cut_l || (l == cut_l && idx <= cut_idx); };

  // Counts of the bins over the cluster, of what is kept; with `bin` >= 0 those inside that bin.  Each thread
  // gets its two bins' sums.
  auto clear_bins = [&] {
    __syncthreads();
    for (int i = tid; i < kBins; i += kThreads) sh.u.hist[i] = 0;
    __syncthreads();
  };
  auto cluster_bins = [&]() -> uint2 {  // behind a cluster barrier
    uint2 sum = make_uint2(0u, 0u), x[kMaxCluster];
    const uint32_t mine = smem_u32(&sh.u.hist[2 * tid]);
#pragma unroll
    for (uint32_t c = 0; c < kMaxCluster; ++c) x[c] = c < C ? ld_peer_v2(mapa_shared(mine, c)) : sum;
#pragma unroll
    for (uint32_t c = 0; c < kMaxCluster; ++c) {
      sum.x += x[c].x;
      sum.y += x[c].y;
    }
    return sum;
  };
  auto histogram = [&](int bin) -> uint2 {
    clear_bins();
    each4([&](float l, int idx, auto) {
      const float t = octaves(l, m, half, ch);
      const int x = bin_of(t);
      if (x < kBins - 1 && (bin < 0 || x == bin) && kept(l, idx)) atomicAdd(&sh.u.hist[bin < 0 ? x : fine_of(t, bin)], 1u);
    });
    cluster_sync();
    return cluster_bins();
  };
  // Of a thread's two bins the one where the running sum from `from` on reaches k, and the sum before it.
  auto bin_at = [&](uint2 h, uint32_t from, uint32_t k) {
    const bool second = from + h.x < k;
    sh.bin = 2 * tid + (second ? 1 : 0);
    sh.bin_count = second ? h.y : h.x;
    sh.bin_above = from + (second ? h.x : 0u);
  };
  // Inclusive block scan of a thread's value.
  auto scan_u32 = [&](uint32_t v) -> uint32_t {
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t x = __shfl_up_sync(kFull, v, o);
      if (lane >= o) v += x;
    }
    __syncthreads();
    if (lane == 31) sh.scan[warp] = v;
    __syncthreads();
    for (int w = 0; w < warp; ++w) v += sh.scan[w];
    return v;
  };
  auto scan_f32 = [&](float v) -> float {
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const float x = __shfl_up_sync(kFull, v, o);
      if (lane >= o) v += x;
    }
    __syncthreads();
    if (lane == 31) sh.fscan[warp] = v;
    __syncthreads();
    for (int w = 0; w < warp; ++w) v += sh.fscan[w];
    return v;
  };
  // Up to bin `last`, which has everything with a weight where it is the last one of those: a comparison.
  auto edge_of = [](int last) -> float { return last < kBins - 2 ? (float)(last + 1) : (float)(2 * kBins); };
  auto before_edge = [&](float l, float edge) -> bool {
    const float t = octaves(l, m, half, ch);
    return t > -kOctaves && -t * kBinScale < edge;  // bin_of(t) <= last
  };
  // The elements for which pick(t) holds (kList of the cluster at most): each CTA collects its own, and behind a
  // cluster barrier all read all.
  auto collect = [&](auto pick) {
    __syncthreads();
    if (tid == 0) sh.n_own = 0;
    __syncthreads();
    each([&](float l, int idx, auto w) {
      const float t = octaves(l, m, half, ch);
      if (t > -kOctaves && pick(t) && kept(l, idx)) {
        const uint32_t at = atomicAdd(&sh.n_own, 1u);
        if (at < (uint32_t)kList) sh.own[at] = Item{l, idx, w()};
      }
    });
  };
  auto collect_to = [&](int last) {
    __syncthreads();
    if (tid == 0) sh.n_own = 0;
    __syncthreads();
    const float edge = edge_of(last);
    each4([&](float l, int idx, auto w) {
      if (before_edge(l, edge) && kept(l, idx)) {
        const uint32_t at = atomicAdd(&sh.n_own, 1u);
        if (at < (uint32_t)kList) sh.own[at] = Item{l, idx, w()};
      }
    });
    cluster_sync();
  };
  auto read_all = [&] {
    uint32_t n[kMaxCluster], at = 0;
#pragma unroll
    for (uint32_t c = 0; c < kMaxCluster; ++c) n[c] = c < C ? min(ld_peer_u32(mapa_shared(smem_u32(&sh.n_own), c)), (uint32_t)kList) : 0u;
#pragma unroll
    for (uint32_t c = 0; c < kMaxCluster; ++c) {
      if (c < C && (uint32_t)tid < n[c] && at + tid < (uint32_t)kList)
        *reinterpret_cast<uint4*>(&sh.list[at + tid]) = ld_peer_v4(mapa_shared(smem_u32(&sh.own[tid]), c));
      at += n[c];
    }
    __syncthreads();
  };
  auto gather = [&](auto pick) {
    collect(pick);
    cluster_sync();
    read_all();
  };
  // Lists the CTA's candidates, those up to bin `last`, in index order with their weights; where they are too many
  // without them (64 rows with some flat distributions 150 us when those went on with the whole row, 83 so), and where
  // they are too many for that as well the row stays what is looked at.
  // `others`: of what is not listed its sum, and what that may be off by (not meant where nothing is listed).
  auto list_candidates = [&](int last, auto sum_others, uint64_t (&others)[2]) {
    if (!RES || n_cand >= 0) return;
    const float edge = edge_of(last);
    // which of 32 neighbours are: lane j keeps the mask of the warp's j-th 32, of the (32 + j)-th, ...
    constexpr int kMasks = (1 << 16) / kWarps / 1024;
    uint32_t masks[kMasks] = {}, n = 0;
#pragma unroll
    for (int c = 0; c < kMasks; ++c) {
      const int to = min(w1, w0 + 1024 * (c + 1));
      float rest[4] = {}, slope = 0.f;
      for (int i = w0 + 1024 * c; i < to; i += 128) {
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          const int at = i + 32 * u + lane;
          const float t = at < w1 ? octaves(one(at), m, half, ch) : -INFINITY;
          const bool counts = t > -kOctaves, in = counts && -t * kBinScale < edge;  // bin_of(t) <= last
          const uint32_t mask = __ballot_sync(kFull, in);
          if (lane == ((i - w0) >> 5 & 31) + u) masks[c] = mask;
          if (decltype(sum_others)::value) {
            const float w = counts && !in ? fast_exp2(t) : 0.f;
            rest[u] += w;
            slope = fmaf(w, counts ? -t : 0.f, slope);
          }
        }
      }
      if (decltype(sum_others)::value) {
        // What rounding took from 1 / T goes by the octaves.  Else off by at most: an exponential 2^-22 of itself, its
        // exponent two roundings; ten additions, each 2^-24; an exact weight 2^-33 of itself and half a unit.
        const float raw = (rest[0] + rest[1]) + (rest[2] + rest[3]), all = fmaf(slope, sh.ch_off, raw);
        const float off = 1.01f * (raw * (0x1p-22f + 12.f * 0x1p-24f) + slope * (0.6931472f * 2.f * 0x1p-24f));
        others[0] += (uint64_t)(all * (float)kOne);
        others[1] += (uint64_t)(off * (float)kOne) + 18u;
      }
      n += __popc(masks[c]);
    }
    n = __reduce_add_sync(kFull, n);
    __syncthreads();
    if (lane == 0) sh.scan[warp] = n;
    __syncthreads();
    uint32_t at = 0, all = 0;
    for (int w = 0; w < kWarps; ++w) {
      if (w < warp) at += sh.scan[w];
      all += sh.scan[w];
    }
    if (all > (uint32_t)a.cap_bare) return;
    weighed = all <= (uint32_t)a.cap;
    const uint32_t first = at;
#pragma unroll
    for (int c = 0; c < kMasks; ++c) {
      uint32_t mask = masks[c], incl = __popc(mask);
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const uint32_t x = __shfl_up_sync(kFull, incl, o);
        if (lane >= o) incl += x;
      }
      for (uint32_t to = at + incl - __popc(mask); mask != 0; mask &= mask - 1) {
        const uint32_t x = w0 + 1024 * c + 32 * lane + __ffs(mask) - 1;
        if (weighed) cand[to++] = x;
        else cand_at[to++] = (uint16_t)x;
      }
      at += __shfl_sync(kFull, incl, 31);
    }
    __syncwarp();
    for (uint32_t i = weighed ? first + lane : at; i < at; i += 32) cand[i] |= weight_of(one((int)cand[i]), m, sh) << 16;
    n_cand = (int)all;
    __syncthreads();
  };
  // Everything that may be kept is in the list (kFew at most): the rest of the work is four lanes an element.  Of
  // the list's order the first k stay; top-p of `total` (0: of what stays).
  // The running weight that has to be reached is given by its bounds (0: top-p of what stays); false where they
  // do not decide.
  auto finish_list = [&](int n, int k, uint64_t target, uint64_t target_hi) -> bool {
    constexpr int lanes = kThreads / kFew;
    const int me_at = tid / lanes, part = tid % lanes;
    const bool in = me_at < n;
    const Item me = sh.list[in ? me_at : 0];
    auto of_lanes = [&](uint64_t x) -> uint64_t {
#pragma unroll
      for (int o = 1; o < lanes; o <<= 1) x += __shfl_xor_sync(kFull, x, o);
      return x;
    };
    // its rank, and the weight before it
    uint32_t r = 0;
    uint64_t wb = 0;
#pragma unroll 2
    for (int j = in ? part : n; j < n; j += lanes) {
      const Item x = sh.list[j];
      if (x.l > me.l || (x.l == me.l && x.idx < me.idx)) {
        ++r;
        wb += x.w;
      }
    }
    wb = of_lanes(wb);
    r = (uint32_t)of_lanes(r);
    // behind this barrier no warp reads the list's weights, or sh.part, as they were
    if (target == 0 && in && (int)r == min(k, n) - 1) sh.sum = wb + me.w;  // all lanes of the one element
    if (__syncthreads_or(in && r > 0 && wb >= target && wb < target_hi)) return false;  // never where the bounds are equal
    if (target == 0) target = top_p < 1.f ? part_of_sum(top_p, sh.sum, true) : ~0ull;
    const uint64_t least = min_p > 0.f ? part_of_sum(min_p, kOne, true) : 0ull;
    const bool stay = in && (int)r < k && (r == 0 || (wb < target && me.w >= least));
    uint64_t s = stay ? wb + me.w : 0ull;  // the last that stays has them all
    s = warp_max64(s);
    if (lane == 0) sh.part[warp][0] = s;
    if (in && !stay) sh.list[me_at].w = 0;
    __syncthreads();
    for (int w = 0; w < kWarps; ++w) s = sh.part[w][0] > s ? sh.part[w][0] : s;
    if (probs != nullptr) {
      zero_probs();
      __syncthreads();
      if (stay && part == 0 && me.idx >= v0 && me.idx < v0 + n_own)
        probs[me.idx - v0] = share(me.l, m, sh) * ((float)kOne / (float)s);
    }
    if (a.token != nullptr && rank == 0) {
      uint64_t at = part_of_sum(rf, s, false);
      if (at >= s) at = s - 1;
      uint64_t x = 0;
#pragma unroll 2
      for (int j = stay ? part : n; j < n; j += lanes) x += sh.list[j].idx < me.idx ? sh.list[j].w : 0ull;
      x = of_lanes(x);
      if (stay && at >= x && at < x + me.w) a.token[b] = me.idx;
    }
    cluster_sync();
    return true;
  };

  // The cut at the list's element where the running value (1 an element, or its weight), from `above` on, reaches
  // the target, of which bounds are given; false where none does for both.
  auto cut_in_list = [&](bool weights, uint64_t target, uint64_t target_hi, uint64_t above, uint32_t n) -> bool {
    bool here = false;
    constexpr uint32_t kLanes = 4;  // of an element
    for (uint32_t e0 = 0; e0 < n; e0 += kThreads / kLanes) {
      const uint32_t e = e0 + tid / kLanes;
      const Item me = sh.list[e < n ? e : 0];
      uint64_t x = 0;
#pragma unroll 2
      for (uint32_t j = tid % kLanes; j < n; j += kLanes) {
        const Item y = sh.list[j];
        if (y.l > me.l || (y.l == me.l && y.idx < me.idx)) x += weights ? y.w : 1ull;
      }
      x += __shfl_xor_sync(kFull, x, 1);
      x += __shfl_xor_sync(kFull, x, 2) + above;
      if (e < n && x < target && x + (weights ? me.w : 1ull) >= target_hi) {
        here = true;
        sh.cut_l = me.l;  // all lanes of the one element
        sh.cut_idx = me.idx;
      }
    }
    if (!__syncthreads_or(here)) return false;
    cut_l = sh.cut_l;
    cut_idx = sh.cut_idx;
    return true;
  };
  // The same in a bin (or its part `fine`) of `count` elements, before which the bins have `above`.
  auto cut_in_bin = [&](bool weights, uint64_t target, uint64_t above, uint32_t count, int bin, int fine) {
    auto inside = [&](float t) { return bin_of(t) == bin && (fine < 0 || fine_of(t, bin) == fine); };
    if (count <= (uint32_t)kList) {
      gather(inside);
      cut_in_list(weights, target, target, above, count);
      return;
    }
    // Too many: the largest key from which on the values reach the target, bit by bit where the bin's keys differ (few,
    // or none).
    auto in_bin = [&](float l, int idx) -> bool {
      const float t = octaves(l, m, half, ch);
      return t > -kOctaves && inside(t) && kept(l, idx);
    };
    auto reach = [&](uint32_t from) -> uint64_t {
      uint64_t s[1] = {0};
      each([&](float l, int idx, auto w) {
        if (in_bin(l, idx) && order_key(l) >= from) s[0] += weights ? w() : 1ull;
      });
      cluster_sum(s);
      return above + s[0];
    };
    uint64_t ends[2] = {0, 0};
    each([&](float l, int idx, auto) {
      if (!in_bin(l, idx)) return;
      ends[0] = max(ends[0], (unsigned long)order_key(l));
      ends[1] = max(ends[1], (unsigned long)~order_key(l));
    });
    cluster_sum(ends, true);
    uint32_t key = (uint32_t)ends[0];
    int bits = 32 - __clz(key ^ ~(uint32_t)ends[1]);
    for (int bit = bits - 1; bit >= 0; --bit) key &= ~(1u << bit);
    const bool differ = bits > 0;
    while (--bits >= 0) {
      const uint32_t want = key | 1u << bits;
      if (reach(want) >= target) key = want;
    }
    // of those with this key the first in index order that reach it: a count
    const uint64_t base = differ ? reach(key + 1) : above;
    const uint64_t each_has = weights ? weight_of(key_logit(key), m, sh) : 1ull, nth = (target - base + each_has - 1) / each_has;
    const int items = n_cand >= 0 ? n_cand : n_own, part = (items + kThreads - 1) / kThreads * 32;
    const int i0 = min(items, warp * part), i1 = min(items, i0 + part);
    auto index_of = [&](int i) -> int {  // of an item that is one of them; else -1
      if (i >= i1) return -1;
      const int at = n_cand >= 0 ? place(i) : i;
      const float l = one(at);
      return order_key(l) == key && kept(l, v0 + at) ? v0 + at : -1;
    };
    uint32_t mine = 0;
    for (int i = i0; i < i1; i += 32) mine += __popc(__ballot_sync(kFull, index_of(i + lane) >= 0));
    __syncthreads();
    if (lane == 0) sh.scan[warp] = mine;
    uint64_t c[1] = {lane == 0 ? mine : 0u};
    cluster_sum(c);
    uint64_t run = before;
    for (int w = 0; w < warp; ++w) run += sh.scan[w];
    uint64_t found[1] = {0};
    if (nth > run && nth <= run + mine) {
      for (int i = i0; i < i1; i += 32) {
        const int idx = index_of(i + lane);
        const uint32_t mask = __ballot_sync(kFull, idx >= 0);
        if (idx >= 0 && run + __popc(mask & ((1u << lane) - 1u)) + 1 == nth) found[0] = (uint64_t)idx;
        run += __popc(mask);
      }
    }
    cluster_sum(found);
    cut_l = key_logit(key);
    cut_idx = (int)found[0];
  };
  // ---- top-k ------------------------------------------------------------------------------
  if (top_k > 0 && top_k < a.V) {
    const uint32_t k = (uint32_t)top_k;
    uint2 h = histogram(-1);
    uint32_t incl = scan_u32((h.x + h.y)), excl = incl - (h.x + h.y);
    if (tid == 0) sh.bin = -1;
    __syncthreads();
    if (excl < k && k <= incl) bin_at(h, excl, k);
    __syncthreads();
    const int bin = sh.bin;  // -1: those with a weight are fewer than k
    uint32_t count = sh.bin_count, above = sh.bin_above;
    if (bin < 0) {
      cluster_sync();  // the counts have been read
    } else {
      if (above + count <= (uint32_t)kFew) {
        collect_to(bin);
        read_all();
        finish_list((int)(above + count), (int)k, 0, 0);
        return;
      }
      uint64_t unused[2];
      list_candidates(bin, std::false_type(), unused);
      int fine = -1;
      if (count > (uint32_t)kList) {
        cluster_sync();  // the counts have been read
        h = histogram(bin);
        incl = scan_u32((h.x + h.y)) + above;
        excl = incl - (h.x + h.y);
        if (excl < k && k <= incl) bin_at(h, excl, k);
        __syncthreads();
        fine = sh.bin;
        count = sh.bin_count;
        above = sh.bin_above;
      }
      cut_in_bin(false, k, above, count, bin, fine);
    }
  }
  // ---- top-p ------------------------------------------------------------------------------
  if (top_p < 1.f) {
    // The sum of all weights: of rows that stay in shared memory, and from which top-k has taken nothing, exactly
    // that of the candidates, once they are listed, and bounds of what the others add, which nearly always decide;
    // else (and where they do not) exactly.
    uint64_t target = 0, target_hi = 0;
    const bool bounded = RES && n_cand < 0 && cut_idx == INT_MAX;
    clear_bins();
    if (bounded) {
      each4([&](float l, int, auto) {
        const int x = bin_of(octaves(l, m, half, ch));
        if (x < kBins - 1) atomicAdd(&sh.u.hist[x], 1u);
      });
      cluster_sync();
    } else {
      uint64_t z[1] = {0};
      auto add = [&](float l, int idx, auto w) {
        const int x = bin_of(octaves(l, m, half, ch));
        if (x < kBins - 1 && kept(l, idx)) {
          atomicAdd(&sh.u.hist[x], 1u);
          z[0] += w();
        }
      };
      if (n_cand >= 0) {
        each(add);
      } else {
#pragma unroll 2
        for (int i = w0 + lane; i < w1; i += 32) {
          const float l = one(i);
          add(l, v0 + i, [&] { return weight(l, m, sh); });
        }
      }
      cluster_sum(z);
      target = target_hi = part_of_sum(top_p, z[0], true);
    }
    int bin = -1, fine = -1;
    uint64_t above = 0;
    uint32_t count = 0;
    bool done = false;
    for (int level = 0; level < 2; ++level) {
      const uint2 h = level == 0 ? cluster_bins() : histogram(bin);
      // the guess: counts times the weight at the bin's middle
      const float width = level ? 1.f / kBins : 1.f, mid = fast_exp2(-((level ? (float)bin : 0.f) + (2.f * tid + 0.5f) * width) / kBinScale);
      const float mid1 = mid * fast_exp2(-width / kBinScale);
      const float mass0 = mid * (float)h.x, mass1 = mid1 * (float)h.y;
      const float incl = scan_f32(mass0 + mass1);
      if (tid == kThreads - 1) sh.mass = incl;
      const uint32_t c_incl = scan_u32(h.x + h.y), c_mid = c_incl - h.y, c_excl = c_mid - h.x;
      if (tid == 0) sh.bin = kBins - 1;
      __syncthreads();
      // in whole rows the share of the same sum, so that what the middles are off by cancels
      const float at = level == 0 ? top_p * sh.mass : (float)(target - above) * (1.f / (float)kOne);
      if (at <= incl) atomicMin(&sh.bin, 2 * tid + (incl - mass1 < at ? 1 : 0));  // the first: the same in every CTA
      __syncthreads();
      int guess = min(sh.bin, kBins - 2);
      if (level == 0) {
        // a few bins behind the guess for its error; few enough up to there: they are the list, if they do reach
        // the target
        const int last = min(guess + 12 | 1, kBins - 1);
        if (tid == last >> 1) sh.bin_above = c_incl;
        // elements before and up to a bin, told by the thread that has it
        auto tell_before = [&](int of) {
          if (tid == of >> 1) sh.near_lo = of & 1 ? c_mid : c_excl;
        };
        auto tell_upto = [&](int of) {
          if (tid == of >> 1) sh.near_hi = of & 1 ? c_incl : c_mid;
        };
        if (tid == guess >> 1) sh.bin_count = guess & 1 ? h.y : h.x;
        __syncthreads();
        const uint32_t n = sh.bin_above;
        bool exactly = bounded && sh.bin_count > (uint32_t)kList;
        uint64_t z[2] = {0, 0};
        list_candidates(last, std::true_type(), z);
        if (bounded && !exactly) {
          // where they do not fit, all of them
          if (n_cand < 0) z[0] = z[1] = 0;
          each([&](float l, int, auto w) {
            if (octaves(l, m, half, ch) > -kOctaves) z[0] += w();
          });
          cluster_sum(z);
          target = part_of_sum(top_p, z[0] - z[1], true);
          target_hi = part_of_sum(top_p, z[0] + z[1], true);
        }
        // the sum of the list's weights
        auto listed_sum = [&](uint32_t n) -> uint64_t {
          uint64_t s = warp_sum64(tid < (int)n ? sh.list[tid].w : 0ull);
          if (lane == 0) sh.part[warp][0] = s;
          __syncthreads();
          s = 0;
          for (int w = 0; w < kWarps; ++w) s += sh.part[w][0];
          __syncthreads();  // the next sum's values are not among these
          return s;
        };
        int tries = 0;
        for (bool few = n <= (uint32_t)kFew;;) {
          if (exactly) {  // the bounds do not decide, or are not worth it
            uint64_t z[1] = {0};
#pragma unroll 2
            for (int i = w0 + lane; i < w1; i += 32) {
              const float l = one(i);
              if (octaves(l, m, half, ch) > -kOctaves) z[0] += weight(l, m, sh);
            }
            cluster_sum(z);
            target = target_hi = part_of_sum(top_p, z[0], true);
            exactly = false;
          }
          if (few) {
            collect_to(last);
            read_all();
            if (listed_sum(n) < target_hi) {  // the row may reach it behind them
              few = false;
              cluster_sync();  // nothing else is collected before all have read
              continue;
            }
            if (finish_list((int)n, INT_MAX, target, target_hi)) return;
          } else {
            // the bins around the guess, as many as fit, are ranked at once, and what lies before them summed
            tell_before(guess);
            tell_upto(guess);
            __syncthreads();
            const uint32_t lo_c = sh.near_lo, hi_c = sh.near_hi, wing = kNear > hi_c - lo_c ? (kNear - (hi_c - lo_c)) / 2 : 0u;
            __syncthreads();
            if (tid == 0) {
              sh.bin = kBins;
              sh.bin_count = 0;
            }
            __syncthreads();
            if (c_mid + wing >= lo_c) atomicMin(&sh.bin, c_excl + wing >= lo_c ? 2 * tid : 2 * tid + 1);
            if (c_mid <= hi_c + wing) atomicMax(&sh.bin_count, (uint32_t)(c_incl <= hi_c + wing ? 2 * tid + 1 : 2 * tid));
            __syncthreads();
            const int near_first = min(sh.bin, guess), near_last = max(guess, min((int)sh.bin_count, last));
            tell_before(near_first);
            tell_upto(near_last);
            if (tid == near_first >> 1) sh.mass = incl - mass1 - (near_first & 1 ? 0.f : mass0);
            __syncthreads();
            const uint32_t near = sh.near_hi - sh.near_lo;
            if (near <= (uint32_t)kList) {
              uint64_t s[1] = {0};
              collect([&](float t) {
                const int x = bin_of(t);
                return x >= near_first && x <= near_last;
              });
              each([&](float l, int idx, auto w) {
                const float t = octaves(l, m, half, ch);
                if (t > -kOctaves && bin_of(t) < near_first && kept(l, idx)) s[0] += w();
              });
              cluster_sum(s);
              read_all();
              if (cut_in_list(true, target, target_hi, s[0], near)) {
                done = true;
                break;
              }
              const uint64_t end = s[0] + listed_sum(near);
              cluster_sync();
              if (tries++ < 2 && (target_hi <= s[0] || target > end)) {  // outside: from the exact sum on, by the histogram
                if (tid == 0) sh.bin = kBins - 1;
                __syncthreads();
                const float from = sh.mass + (float)(int64_t)(target - s[0]) * (1.f / (float)kOne);
                if (from <= incl) atomicMin(&sh.bin, 2 * tid + (incl - mass1 < from ? 1 : 0));
                __syncthreads();
                const int moved = sh.bin;
                if (moved <= last && moved < kBins - 1 && moved != guess) {
                  guess = moved;
                  continue;
                }
              }
            }
            if (target == target_hi) break;
          }
          exactly = true;
        }
        if (done) break;
      }
      // the exact sums around the guess
      auto part_of = [&](float t) -> int {  // -1: before the bin that is looked into; kBins: behind
        const int x = bin_of(t);
        return level == 0 ? x : x < bin ? -1 : x > bin ? kBins : fine_of(t, bin);
      };
      uint64_t base = 0;
      for (int guard = 0; guard < kBins; ++guard) {
        // the bins next to it that have something: equal logits leave most of them empty
        __syncthreads();
        if (tid == 0) {
          sh.bin = -1;
          sh.bin_count = kBins;
        }
        __syncthreads();
        if (h.x != 0 && 2 * tid < guess) atomicMax(&sh.bin, 2 * tid);
        if (h.y != 0 && 2 * tid + 1 < guess) atomicMax(&sh.bin, 2 * tid + 1);
        if (h.x != 0 && 2 * tid > guess) atomicMin(&sh.bin_count, 2u * tid);
        if (h.y != 0 && 2 * tid + 1 > guess) atomicMin(&sh.bin_count, 2u * tid + 1u);
        __syncthreads();
        const int prev = sh.bin, next = (int)sh.bin_count;
        uint64_t s[4] = {0, 0, 0, 0};
        each([&](float l, int idx, auto w) {
          const float t = octaves(l, m, half, ch);
          const int x = t > -kOctaves ? part_of(t) : kBins;
          if (x <= next && x < kBins && kept(l, idx)) {
            const uint64_t y = w();
            if (x < prev) s[0] += y;
            else if (x == prev) s[1] += y;
            else if (x == guess) s[2] += y;
            else s[x < guess ? 0 : 3] += y;
          }
        });
        cluster_sum(s);
        if (target <= s[0]) {
          guess = prev;
        } else if (target <= s[0] + s[1]) {
          guess = prev;
          base = s[0];
          break;
        } else if (target <= s[0] + s[1] + s[2]) {
          base = s[0] + s[1];
          break;
        } else if (target <= s[0] + s[1] + s[2] + s[3]) {
          guess = next;
          base = s[0] + s[1] + s[2];
          break;
        } else {
          guess = next;
          if (level == 0) n_cand = -1;  // the candidates may end before it: the row has them all
        }
      }
      above = base;
      if (tid == guess >> 1) sh.bin_count = guess & 1 ? h.y : h.x;
      __syncthreads();
      count = sh.bin_count;
      if (level == 0) bin = guess; else fine = guess;
      if (count <= (uint32_t)kList) break;
    }
    if (!done) cut_in_bin(true, target, above, count, bin, fine);
  }
  // ---- the sum of what is left, by groups of a warp's elements ------------------------------------
  const uint64_t least = min_p > 0.f ? part_of_sum(min_p, kOne, true) : 0ull;
  const bool listed = n_cand >= 0;
  constexpr int kSummed = RES ? kGroup : 2 * kGroup;
  static_assert(kGroups * kSummed >= (RES ? 1 << 16 : kMaxVocab / kMaxCluster), "a sum for every group");
  const int n_left = listed ? n_cand : n_own, groups = (n_left + kSummed - 1) / kSummed;
  // the weight left of element i of what is looked at (behind its end: none)
  auto left = [&](int i, auto weigh) -> uint64_t {
    if (i >= n_left) return 0ull;
    if (listed && weighed) {
      const uint64_t x = cand[i];
      const int at = (int)(x & 0xffffu);
      return kept(one(at), v0 + at) && x >> 16 >= least ? x >> 16 : 0ull;
    }
    const int at = listed ? cand_at[i] : i;
    const float l = one(at);
    if (!(octaves(l, m, half, ch) > -kOctaves) || !kept(l, v0 + at)) return 0ull;
    const uint64_t w = weigh(l);
    return w >= least ? w : 0ull;
  };
  auto called = [&](float l) -> uint64_t { return weight_of(l, m, sh); };
  __syncthreads();
  uint64_t s[1] = {0};
  for (int g = warp; g < groups; g += kWarps) {
    uint64_t w = 0;
#pragma unroll 2
    for (int e = 0; e < kSummed; e += 32) w += left(g * kSummed + e + lane, [&](float l) -> uint64_t { return weight(l, m, sh); });
    s[0] += w;
    w = __any_sync(kFull, w != 0) ? warp_sum64(w) : 0ull;
    if (lane == 0) sh.u.gsum[g] = w;
  }
  cluster_sum(s);
  const uint64_t total = s[0], start = before;
  if (probs != nullptr) {
    const float inv = (float)kOne / (float)total;
    if (listed) {
      zero_probs();
      __syncthreads();
      for (int i = tid; i < n_cand; i += kThreads) {
        const int at = place(i);
        const float l = one(at);
        if (kept(l, v0 + at) && (least == 0 || left(i, called) != 0)) probs[at] = share(l, m, sh) * inv;
      }
    } else {
      // min-p in octaves: what is right at it goes by the weight itself
      const float edge = min_p > 0.f ? log2f(min_p) : -INFINITY;
      auto p = [&](int i) -> float {
        const float l = one(i), t = octaves(l, m, half, ch);
        bool stay = t > -kOctaves && kept(l, v0 + i) && t >= edge - 0.001f;
        if (stay && t < edge + 0.001f) stay = left(i, called) != 0;
        return stay ? share(l, m, sh) * inv : 0.f;
      };
#pragma unroll 4
      for (int i = w0 + lane; i < w1; i += 32) probs[i] = p(i);
    }
  }
  // ---- the token: the group, then the element, where the running sum passes r of the total ---------------
  if (a.token != nullptr && warp == 0) {
    uint64_t at = part_of_sum(rf, total, false);
    if (at >= total) at = total - 1;
    uint64_t run = start;
    // inclusive sums over the warp's lanes; true where the one that `at` falls to is among them
    auto scan = [&](uint64_t w, uint64_t& incl) -> bool {
      incl = w;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const uint64_t x = __shfl_up_sync(kFull, incl, o);
        if (lane >= o) incl += x;
      }
      const uint64_t all = __shfl_sync(kFull, incl, 31);
      if (at >= run && at < run + all) return true;
      run += all;
      return false;
    };
    for (int g0 = 0; g0 < groups; g0 += 32) {
      const uint64_t w = g0 + lane < groups ? sh.u.gsum[g0 + lane] : 0ull;
      uint64_t incl;
      if (!scan(w, incl)) continue;
      const int src = __ffs((int)__ballot_sync(kFull, at >= run + incl - w && at < run + incl)) - 1;
      run += __shfl_sync(kFull, incl - w, src);
      for (int e = 0; e < kSummed; e += 32) {
        const int i = (g0 + src) * kSummed + e + lane;
        const uint64_t x = left(i, called);
        if (!scan(x, incl)) continue;
        if (at >= run + incl - x && at < run + incl) a.token[b] = v0 + (listed ? place(i) : i);
        break;
      }
      break;
    }
  }
  cluster_sync();
}

using Kernel = void (*)(SampleArgs);

constexpr size_t kSmemTwo = 233472 / 2 - 1024, kSmemOne = 232448;  // of a CTA, with another one on the SM and alone
constexpr size_t kCand = sizeof(uint64_t);  // a candidate's bytes
constexpr int kCandLeast = 512;  // candidates that a CTA has room for where two share an SM

// What a device has room for at once, clusters of 1 to 8 CTAs with two CTAs on an SM and with one (clusters do
// not cross the SM groups, so it is less than the SMs divided), and whether the kernels' limits are raised.
struct Device {
  bool ready;
  int two[kMaxCluster + 1], one[kMaxCluster + 1];
};
Kernel kernel_of(bool half, bool resident) {
  return resident ? (half ? sample_kernel<true, true> : sample_kernel<false, true>)
                  : (half ? sample_kernel<true, false> : sample_kernel<false, false>);
}
cudaError_t device_of(Device& out) {
  static std::mutex mu;
  static Device known[128];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  std::lock_guard<std::mutex> lk(mu);
  const bool keep = dev >= 0 && dev < 128;
  if (keep && known[dev].ready) {
    out = known[dev];
    return cudaSuccess;
  }
  for (const bool half : {false, true}) {
    e = cudaFuncSetAttribute(kernel_of(half, true), cudaFuncAttributeMaxDynamicSharedMemorySize, (int)(kSmemOne - sizeof(Shared)));
    if (e != cudaSuccess) return e;
  }
  for (int C = 1; C <= kMaxCluster; ++C) {
    for (const bool two : {false, true}) {
      cudaLaunchConfig_t cfg = {};
      cfg.gridDim = dim3(C);
      cfg.blockDim = dim3(kThreads);
      cfg.dynamicSmemBytes = (two ? kSmemTwo : kSmemOne) - sizeof(Shared);
      cudaLaunchAttribute attr[1];
      attr[0].id = cudaLaunchAttributeClusterDimension;
      attr[0].val.clusterDim = {(unsigned)C, 1, 1};
      cfg.attrs = attr;
      cfg.numAttrs = 1;
      e = cudaOccupancyMaxActiveClusters(two ? &out.two[C] : &out.one[C], kernel_of(true, true), &cfg);
      if (e != cudaSuccess) return e;
    }
  }
  out.ready = true;
  if (keep) known[dev] = out;
  return cudaSuccess;
}

int part_of_row(int V, int C) { return ((V + C - 1) / C + 3) / 4 * 4; }

// CTAs of a row.  Many rows: as few as let two CTAs share an SM (what a CTA does beside its part of the row
// is the larger half: 384 rows of 102400 fp32 logits, top-p with probabilities, 263 us with 5, 345 with 8; bf16
// 215 with 3, 227 with 4, 339 with 8).  Few rows: more, as long as each CTA has an SM (one row 26 us with 8, 29
// with 5; 20 rows with top-k 17.1 with 6, 19.5 with 8, which share SMs, but with top-p 41 and 38); then as many as let
// the batch be worked on at once (44 rows 45 with 6, 57 with 8), or 8 if fewer do not save a turn (64 rows 58 with 8 and
// 63 with 5 where some of the rows have flat distributions, which take longest, 66 and 64 where all are alike; 128
// rows 85 and 67, 126 and 106).
int cluster_size(int64_t rows, int V, size_t bytes, const Device& dev) {
  int least = 1;
  while (least < kMaxCluster && part_of_row(V, least) * bytes + kCandLeast * kCand + sizeof(Shared) > kSmemTwo) ++least;
  const int most = std::max(least, std::min(kMaxCluster, V / 1024));
  for (int C = most; C >= std::max(least, 5); --C)
    if (rows <= dev.one[C]) return C;
  for (int C = most; C > least; --C)
    if (rows <= dev.two[C]) return C;
  auto turns = [&](int C) -> int64_t { return (rows + dev.two[C] - 1) / std::max(1, dev.two[C]); };
  return turns(most) <= turns(least) ? most : least;
}

// Whether rows of `a` bytes at p share a byte with rows of `b` bytes at q: not where their spans lie apart, nor where
// both are columns of rows of the same stride.
bool rows_overlap(const void* p, int64_t p_stride, int64_t a, const void* q, int64_t q_stride, int64_t b, int64_t rows) {
  using wide = __int128;
  const wide x = (wide)(uintptr_t)p, y = (wide)(uintptr_t)q;
  if (x + (wide)p_stride * (rows - 1) + a <= y || y + (wide)q_stride * (rows - 1) + b <= x) return false;
  if (rows == 1 || p_stride != q_stride) return true;
  const wide d = ((y - x) % p_stride + p_stride) % p_stride;
  return d < a || d + b > p_stride;
}

}  // namespace
}  // namespace irm

extern "C" irm_status irm_sample(const void* logits, int logits_type, int64_t row_stride, int64_t n_rows, int32_t vocab,
                                 const float* temperature, const int32_t* top_k, const float* top_p, const float* min_p,
                                 const float* uniforms, int32_t* token, float* probs, int64_t probs_stride,
                                 void* workspace, size_t workspace_bytes, cudaStream_t stream) {
  using namespace irm;
  if (logits_type != IRM_FP32 && logits_type != IRM_BF16)
    return fail(IRM_ERR_UNSUPPORTED, "logits_type %d is neither IRM_FP32 nor IRM_BF16", logits_type);
  if (vocab < 1 || vocab > kMaxVocab) return fail(IRM_ERR_UNSUPPORTED, "vocab %d outside [1, 2^20]", vocab);
  if (n_rows < 0 || n_rows > (INT32_MAX >> 3)) return fail(IRM_ERR_INVALID_ARG, "n_rows %lld outside [0, 2^28)", (long long)n_rows);
  if (row_stride < vocab) return fail(IRM_ERR_INVALID_ARG, "row_stride is smaller than vocab");
  if (probs != nullptr && probs_stride < vocab) return fail(IRM_ERR_INVALID_ARG, "probs_stride is smaller than vocab");
  if (token == nullptr && probs == nullptr) return fail(IRM_ERR_INVALID_ARG, "neither token nor probs is wanted");
  if (n_rows > 0 && (!logits || (token != nullptr && !uniforms))) return fail(IRM_ERR_INVALID_ARG, "null device pointer");
  const bool half = logits_type == IRM_BF16;
  if (!aligned(logits, half ? 2 : 4)) return fail(IRM_ERR_INVALID_ARG, "misaligned device pointer");
  for (const void* p : {(const void*)temperature, (const void*)top_k, (const void*)top_p, (const void*)min_p, (const void*)uniforms,
                        (const void*)token, (const void*)probs})
    if (!aligned(p, 4)) return fail(IRM_ERR_INVALID_ARG, "misaligned device pointer");
  if (!workspace || !aligned(workspace, 256) || workspace_bytes < IRM_WORKSPACE_HEADER)
    return fail(IRM_ERR_WORKSPACE, "workspace must be 256-byte aligned and hold %d bytes", IRM_WORKSPACE_HEADER);
  if (n_rows == 0) return IRM_OK;
  const int64_t each = half ? 2 : 4;
  if (row_stride > INT64_MAX / 8 || probs_stride > INT64_MAX / 8) return fail(IRM_ERR_INVALID_ARG, "rows are too far apart");
  if (probs != nullptr && rows_overlap(logits, row_stride * each, vocab * each, probs, probs_stride * 4, vocab * int64_t(4), n_rows))
    return fail(IRM_ERR_INVALID_ARG, "logits and probs overlap");
  Device dev{};
  cudaError_t e = device_of(dev);
  if (e != cudaSuccess) return cuda_fail(e, "sampling set-up");
  const int C = cluster_size(n_rows, vocab, each, dev);
  SampleArgs a{};
  a.logits = logits;
  a.ld = row_stride;
  a.V = vocab;
  a.seg = part_of_row(vocab, C);
  a.temperature = temperature;
  a.top_k = top_k;
  a.top_p = top_p;
  a.min_p = min_p;
  a.uniforms = uniforms;
  a.token = token;
  a.probs = probs;
  a.probs_ld = probs_stride;
  a.status = static_cast<int*>(workspace);
  a.vec_in = row_stride % 4 == 0 && aligned(logits, half ? 8 : 16);
  a.vec_out = probs_stride % 4 == 0 && aligned(probs, 16);
  // in shared memory, where a place in the part has 16 bits
  const size_t row = (size_t)a.seg * each;
  const bool resident = a.seg <= 1 << 16 && row + kCandLeast * kCand + sizeof(Shared) <= kSmemOne;
  const Kernel kernel = kernel_of(half, resident);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(n_rows * C));
  cfg.blockDim = dim3(kThreads);
  if (resident) {
    const bool two = row + kCandLeast * kCand + sizeof(Shared) <= kSmemTwo;
    const size_t room = (two ? kSmemTwo : kSmemOne) - sizeof(Shared) - row;
    a.cap = (int)std::min<size_t>((size_t)a.seg, room / kCand);
    a.cap_bare = (int)std::min<size_t>((size_t)a.seg, a.cap * kCand / sizeof(uint16_t));
    cfg.dynamicSmemBytes = row + a.cap * kCand;
  }
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = (unsigned)C;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, kernel, a);
  return e == cudaSuccess ? IRM_OK : cuda_fail(e, "sampling launch");
}
