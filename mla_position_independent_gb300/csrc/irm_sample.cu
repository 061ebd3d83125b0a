// Sampling from logits with temperature, top-k, top-p and min-p, from given uniform numbers: the token,
// the probabilities left (what the draft verification takes), or both.
//
// Per row, candidates in the order of their logits (ties: lowest index first):
//   w_v = exp((l_v - max) / T);  top-k keeps the first k;  top-p of those the shortest run whose w reach p
//   of their sum;  min-p of those the ones with w >= min_p;  token = lowest v with
//   cumsum(w)(v) > r sum(w) in index order over what is left.
// What is kept is a run of the order from its start, so it is described by its last element, a cut
// (logit, index), and no row is sorted: a histogram of the logits' distance from the maximum (1023 bins of
// 1 / 23 octave of w) finds the bin that holds the cut, and the few hundred elements of that bin are
// ranked among themselves.
//
// Arithmetic.  Which token comes out must not depend on the split or the order of addition, and a flat
// row of 100k entries has cumulative sums 1e-5 apart, so weights are integers in units of 2^-43 and
// their sums are exact.  fp32 exponentials (2^-23) would move 100k boundaries by 1e-7 each, so that one
// draw in a hundred came out wrong; here a weight is good to 2^-37 of the largest: the distance from the
// maximum and its product with 1 / T in two fp32 parts, 32 table values and a polynomial of degree 5.
// fp64 runs at 1 / 64 of the fp32 rate on this GPU.  The histogram only guesses the bin of a top-p cut; the exact
// sums above and inside decide, and move the guess where it was off.
//
// A cluster of CTAs shares a row, which stays in shared memory as fp32 from its one read where it fits (51200
// logits a CTA); longer rows are read again by each pass.
#include <cuda_runtime.h>
#include <cmath>
#include <cstdint>
#include <mutex>

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
constexpr int kList = 448;          // elements that are ranked among themselves, a thread each (two CTAs' memory fits an SM)
constexpr int kGroup = 128;         // elements that a warp looks at at once
constexpr int kGroups = kMaxVocab / kMaxCluster / kGroup;
constexpr uint32_t kFull = 0xffffffffu;
constexpr float kOctaves = 43.9f;   // below 2^-43.9 a weight rounds to nothing
constexpr float kBinScale = (kBins - 1) / kOctaves;
constexpr uint64_t kOne = 1ull << 43;
static_assert(kList <= kThreads && 2 * kThreads == kBins, "a thread an element, two bins a thread");

struct SampleArgs {
  const void* logits;
  int64_t ld;
  int V, seg;  // logits of a row, and of a CTA's part of it (a multiple of 4)
  const float *temperature, *top_p, *min_p, *uniforms;
  const int32_t* top_k;
  int32_t* token;
  float* probs;
  int64_t probs_ld;
  int vec_in, vec_out;  // whole vectors of logits, of probabilities
};

struct __align__(16) Item {
  float l;
  int32_t idx;
  uint64_t w;
};

struct Shared {
  uint64_t part[kWarps][4];
  uint64_t tot[2][kMaxCluster][4];
  union {
    struct {
      uint32_t hist[kBins];
      Item list[kList];
    } s;
    uint64_t gsum[kGroups];
  } u;
  float th4[32], tl[32];  // 2^(i / 32): four more than its 21 bits, and the rest
  uint32_t n_list, scan[kWarps];
  float fscan[kWarps];
  // 1 / (h T) in two parts, and log2(e) / (h T).  h is 1; 1/2 for a temperature so high that differences of
  // logits that overflow still count; 2^24 for one so low that differences of denormal logits do
  float ih, il, ch, h;
  int bin, cut_idx;
  uint32_t bin_count, bin_above;
  float cut_l;
  uint64_t sum;
};

__device__ __forceinline__ uint64_t warp_sum64(uint64_t v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(kFull, v, o);
  return v;
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
__device__ __forceinline__ void st_peer_v4(uint32_t addr, uint4 v) {
  asm volatile("st.shared::cluster.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}
__device__ __forceinline__ uint64_t ld_peer_u64(uint32_t addr) {
  uint64_t v;
  asm volatile("ld.shared::cluster.u64 %0, [%1];" : "=l"(v) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ uint32_t add_peer_u32(uint32_t addr, uint32_t v) {
  uint32_t r;
  asm volatile("atom.relaxed.cluster.shared::cluster.add.u32 %0, [%1], %2;" : "=r"(r) : "r"(addr), "r"(v) : "memory");
  return r;
}

// Order-preserving integer of a logit (no NaN, no -0), and back.
__device__ __forceinline__ uint32_t order_key(float l) {
  const uint32_t b = __float_as_uint(l);
  return b >> 31 ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float key_logit(uint32_t k) { return __uint_as_float(k >> 31 ? k & 0x7fffffffu : ~k); }
// NaN as -infinity, -0 as 0
__device__ __forceinline__ float clean(float l) { return l == l ? l + 0.f : -INFINITY; }

// Distance of a logit from the maximum in octaves of weight (<= 0; NaN or below -kOctaves: no weight).
__device__ __forceinline__ float octaves(float l, float m, float h, float ch) { return l == m ? 0.f : fmaf(l, h, -h * m) * ch; }
__device__ __forceinline__ int bin_of(float t) { return t > -kOctaves ? min(kBins - 2, (int)(-t * kBinScale)) : kBins - 1; }
// The same inside a bin: its elements spread over kBins again.
__device__ __forceinline__ int fine_of(float t, int bin) {
  return min(kBins - 1, max(0, (int)((-t * kBinScale - (float)bin) * (float)kBins)));
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
  const float kf = rintf(th * 46.16624130844683f);
  const float x0 = fmaf(kf, -kLn2Hi, th), x1 = fmaf(kf, -kLn2Lo, te);
  const float xh = x0 + x1, xl = x1 - (xh - x0);
  const int k = (int)kf, i = k & 31, n = -(k >> 5);
  // e^x - 1 = x + x^2 (1/2 + x/6 + x^2/24 + x^3/120), |x| < 0.011
  const float s = xh * xh;
  const float q = fmaf(xh, fmaf(xh, fmaf(xh, 1.f / 120.f, 1.f / 24.f), 1.f / 6.f), 0.5f);
  const float yh = fmaf(s, q, xh);
  const float yl = fmaf(s, q, xh - yh) + fmaf(xl, xh, xl);
  const float t4 = sh.th4[i], tl = sh.tl[i], t = t4 - 4.f;
  const float ph = t * yh, pl = fmaf(t, yh, -ph);
  const float a = t4 + ph;  // in [4, 8): multiples of 2^-21
  const float rest = fmaf(tl, yh, fmaf(t, yl, pl)) + (ph - (a - t4)) + tl;
  const float b = rest + 0x1.8p-19f;  // |rest| <= 2^-21 and a little: multiples of 2^-42
  const int64_t v = ((int64_t)(__float_as_int(a) - 0x40800000) << 21) + (__float_as_int(b) - __float_as_int(0x1.8p-19f));
  return (((uint64_t)v << 2 >> n) + 1) >> 1;
}

template <bool BF16, bool RES>
__global__ void __launch_bounds__(kThreads, 2) sample_kernel(const __grid_constant__ SampleArgs a) {
  extern __shared__ __align__(16) float row_sh[];
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

  // four consecutive logits of the CTA's part (behind its end: -infinity)
  auto fetch = [&](int i) -> float4 {
    float x[4];
    if (a.vec_in && i + 4 <= n_own) {
      if (BF16) {
        const uint2 w = *reinterpret_cast<const uint2*>(b16 + i);
        x[0] = __uint_as_float(w.x << 16);
        x[1] = __uint_as_float(w.x & 0xffff0000u);
        x[2] = __uint_as_float(w.y << 16);
        x[3] = __uint_as_float(w.y & 0xffff0000u);
      } else {
        const float4 w = *reinterpret_cast<const float4*>(f32 + i);
        x[0] = w.x;
        x[1] = w.y;
        x[2] = w.z;
        x[3] = w.w;
      }
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e) x[e] = i + e < n_own ? (BF16 ? __bfloat162float(b16[i + e]) : f32[i + e]) : -INFINITY;
    }
    return make_float4(clean(x[0]), clean(x[1]), clean(x[2]), clean(x[3]));
  };
  auto four = [&](int i) -> float4 { return RES ? *reinterpret_cast<const float4*>(row_sh + i) : fetch(i); };
  // f(logit, index) for the CTA's logits, four neighbours a lane; one that is behind the end is -infinity
  auto each = [&](auto f) {
    for (int i = 4 * tid; i < n_own; i += 4 * kThreads) {
      const float4 x = four(i);
      f(x.x, v0 + i);
      f(x.y, v0 + i + 1);
      f(x.z, v0 + i + 2);
      f(x.w, v0 + i + 3);
    }
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
  const float rf = a.uniforms ? fminf(fmaxf(a.uniforms[b], 0.f), 1.f) : 0.f;
  const bool first_alone = !(temp > 0.f) || top_k == 1 || top_p <= 0.f || min_p > 1.f;
  if (tid < 32) {
    const double t = exp2((double)tid / 32.0);
    const float hi = rintf((float)t * 0x1p21f) * 0x1p-21f;
    sh.th4[tid] = hi + 4.f;
    sh.tl[tid] = (float)(t - (double)hi);
  } else if (tid == 32) {
    const float h = temp > 0x1p100f ? 0.5f : temp < 0x1p-100f ? 0x1p24f : 1.f;
    const double inv = 1.0 / ((double)h * (double)temp);
    sh.h = h;
    sh.ih = (float)inv;
    sh.il = (float)(inv - (double)sh.ih);
    sh.ch = (float)(inv * 1.4426950408889634);
  }
  // ---- the row, and its maximum ------------------------------------------------------------
  uint64_t top[1] = {0};
  for (int i = 4 * tid; i < n_own; i += 4 * kThreads) {
    const float4 x = fetch(i);
    if (RES) *reinterpret_cast<float4*>(row_sh + i) = x;
    const float y[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (i + e < n_own) {
        const uint64_t k = (uint64_t)order_key(y[e]) << 32 | (uint32_t)~(v0 + i + e);
        top[0] = k > top[0] ? k : top[0];
      }
  }
  cluster_wait();
  cluster_sum(top, true);
  const float m = key_logit((uint32_t)(top[0] >> 32));
  const int first = (int)~(uint32_t)top[0];
  float* probs = a.probs ? a.probs + b * a.probs_ld + v0 : nullptr;
  // p(i) for the CTA's probabilities, four neighbours at a time
  auto write_probs = [&](auto p) {
    for (int i = 4 * tid; i < n_own; i += 4 * kThreads) {
      const float4 y = p(i);
      if (a.vec_out && i + 4 <= n_own) {
        *reinterpret_cast<float4*>(probs + i) = y;
      } else {
        const float z[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (i + e < n_own) probs[i + e] = z[e];
      }
    }
  };
  auto zero_probs = [&] { write_probs([](int) { return make_float4(0.f, 0.f, 0.f, 0.f); }); };

  const bool none = m == -INFINITY;
  if (none || first_alone) {  // the same in every CTA of the cluster
    if (probs != nullptr) {
      zero_probs();
      __syncthreads();
      if (tid == 0 && !none && first >= v0 && first < v0 + n_own) probs[first - v0] = 1.f;
    }
    if (a.token != nullptr && rank == 0 && tid == 0) a.token[b] = none ? -1 : first;
    cluster_arrive();  // no CTA ends while another may still store into it
    cluster_wait();
    return;
  }
  const float ch = sh.ch, half = sh.h;

  // ---- what is kept: everything before, and up to, (cut_l, cut_idx) in the order -----------------
  float cut_l = -INFINITY;
  int cut_idx = INT_MAX;
  auto kept = [&](float l, int idx) { return l > cut_l || (l == cut_l && idx <= cut_idx); };

  // Counts of the bins over the cluster, of what is kept; with `bin` >= 0 those inside that bin.  Each thread
  // gets its two bins' sums.
  auto histogram = [&](int bin) -> uint2 {
    __syncthreads();
    for (int i = tid; i < kBins; i += kThreads) sh.u.s.hist[i] = 0;
    if (tid == 0) sh.n_list = 0;
    __syncthreads();
    each([&](float l, int idx) {
      const float t = octaves(l, m, half, ch);
      const int x = bin_of(t);
      if (x < kBins - 1 && (bin < 0 || x == bin) && kept(l, idx)) atomicAdd(&sh.u.s.hist[bin < 0 ? x : fine_of(t, bin)], 1u);
    });
    __syncthreads();
    cluster_arrive();
    cluster_wait();
    uint2 sum = make_uint2(0u, 0u);
    const uint32_t mine = smem_u32(&sh.u.s.hist[2 * tid]);
    for (uint32_t c = 0; c < C; ++c) {
      const uint64_t x = ld_peer_u64(mapa_shared(mine, c));
      sum.x += (uint32_t)x;
      sum.y += (uint32_t)(x >> 32);
    }
    return sum;
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
  // The elements for which pick(t) holds, to every CTA's list.
  auto gather = [&](auto pick) {
    each([&](float l, int idx) {
      const float t = octaves(l, m, half, ch);
      if (t > -kOctaves && pick(t) && kept(l, idx)) {
        const uint64_t w = weight(l, m, sh);
        const uint32_t at = add_peer_u32(mapa_shared(smem_u32(&sh.n_list), 0), 1u);
        const uint4 v = make_uint4(__float_as_uint(l), (uint32_t)idx, (uint32_t)w, (uint32_t)(w >> 32));
        if (at < (uint32_t)kList)
          for (uint32_t c = 0; c < C; ++c) st_peer_v4(mapa_shared(smem_u32(&sh.u.s.list[at]), c), v);
      }
    });
    cluster_arrive();
    cluster_wait();
  };
  // Rank of the thread's element among the list's first n, and the weight before it.
  auto rank_in_list = [&](int n, uint64_t& w_before) -> int {
    int r = 0;
    w_before = 0;
    if (tid < n) {
      const Item me = sh.u.s.list[tid];
      for (int j = 0; j < n; ++j) {
        const Item x = sh.u.s.list[j];
        if (x.l > me.l || (x.l == me.l && x.idx < me.idx)) {
          ++r;
          w_before += x.w;
        }
      }
    }
    return r;
  };

  // Everything that may be kept is in the list: the rest of the work is a thread an element.  Of the list's
  // order the first k stay; top-p of `total` (0: of what stays).
  auto finish_list = [&](int n, int k, uint64_t total) {
    uint64_t wb;
    const int r = rank_in_list(n, wb);
    const Item me = sh.u.s.list[tid < n ? tid : 0];
    if (tid < n && r == min(k, n) - 1) sh.sum = wb + me.w;
    __syncthreads();
    if (total == 0) total = sh.sum;
    const uint64_t target = top_p < 1.f ? (uint64_t)ceil((double)top_p * (double)total) : ~0ull;
    const uint64_t least = min_p > 0.f ? (uint64_t)ceil((double)min_p * (double)kOne) : 0ull;
    const bool stay = tid < n && r < k && (r == 0 || (wb < target && me.w >= least));
    uint64_t s = stay ? wb + me.w : 0ull;  // the last that stays has them all
    s = warp_max64(s);
    __syncthreads();
    if (lane == 0) sh.part[warp][0] = s;
    if (tid < n && !stay) sh.u.s.list[tid].w = 0;
    __syncthreads();
    for (int w = 0; w < kWarps; ++w) s = sh.part[w][0] > s ? sh.part[w][0] : s;
    if (probs != nullptr) {
      zero_probs();
      __syncthreads();
      if (stay && me.idx >= v0 && me.idx < v0 + n_own) probs[me.idx - v0] = (float)((double)me.w / (double)s);
    }
    if (a.token != nullptr && rank == 0) {
      uint64_t at = (uint64_t)((double)rf * (double)s);
      if (at >= s) at = s - 1;
      uint64_t x = 0;
      if (stay)
        for (int j = 0; j < n; ++j) x += sh.u.s.list[j].idx < me.idx ? sh.u.s.list[j].w : 0ull;
      if (stay && at >= x && at < x + me.w) a.token[b] = me.idx;
    }
    cluster_arrive();
    cluster_wait();
  };

  // The cut at the element where the order's running value (1 an element, or its weight) reaches `target`, from
  // what the bins before `bin` (and before its part `fine`) have, `above`.  Values: counts or weights.
  auto value = [&](bool weights, float l) -> uint64_t { return weights ? weight(l, m, sh) : 1ull; };
  auto cut_in_bin = [&](bool weights, uint64_t target, uint64_t above, uint32_t count, int bin, int fine) {
    auto inside = [&](float t) { return bin_of(t) == bin && (fine < 0 || fine_of(t, bin) == fine); };
    if (count <= (uint32_t)kList) {
      gather(inside);
      uint64_t wb;
      const int n = (int)count, r = rank_in_list(n, wb);
      if (tid < n) {
        const Item me = sh.u.s.list[tid];
        const uint64_t x = above + (weights ? wb : (uint64_t)r);
        if (x < target && x + (weights ? me.w : 1ull) >= target) {
          sh.cut_l = me.l;
          sh.cut_idx = me.idx;
        }
      }
      __syncthreads();
      cut_l = sh.cut_l;
      cut_idx = sh.cut_idx;
      return;
    }
    // Too many alike: bit by bit, the largest key from which on the values reach the target, then the index.
    auto reach = [&](auto pick) -> uint64_t {
      uint64_t s[1] = {0};
      each([&](float l, int idx) {
        const float t = octaves(l, m, half, ch);
        if (t > -kOctaves && inside(t) && kept(l, idx) && pick(order_key(l), idx)) s[0] += value(weights, l);
      });
      cluster_sum(s);
      return above + s[0];
    };
    uint32_t key = 0;
    for (int bit = 31; bit >= 0; --bit) {
      const uint32_t want = key | 1u << bit;
      if (reach([&](uint32_t k, int) { return k >= want; }) >= target) key = want;
    }
    int idx = -1;  // the largest index up to which the target is not reached
    for (int bit = 20; bit >= 0; --bit) {
      const int want = idx + (1 << bit);
      if (want < a.V && reach([&](uint32_t k, int i) { return k > key || (k == key && i <= want); }) < target) idx = want;
    }
    cut_l = key_logit(key);
    cut_idx = idx + 1;
  };
  // The thread that holds the first bin for which reached(its running sum) says where the cut is.
  auto publish = [&](int bin, uint32_t count, uint32_t above) {
    sh.bin = bin;
    sh.bin_count = count;
    sh.bin_above = above;
  };

  // ---- top-k ------------------------------------------------------------------------------
  if (top_k > 0 && top_k < a.V) {
    const uint32_t k = (uint32_t)top_k;
    uint2 h = histogram(-1);
    uint32_t incl = scan_u32(h.x + h.y), excl = incl - h.x - h.y;
    if (tid == 0) publish(-1, 0, 0);
    __syncthreads();
    if (excl < k && k <= incl) k <= excl + h.x ? publish(2 * tid, h.x, excl) : publish(2 * tid + 1, h.y, excl + h.x);
    __syncthreads();
    int bin = sh.bin;  // -1: those with a weight are fewer than k
    uint32_t count = sh.bin_count, above = sh.bin_above;
    if (bin >= 0) {
      if (above + count <= (uint32_t)kList) {
        gather([&](float t) { return bin_of(t) <= bin; });
        finish_list((int)(above + count), (int)k, 0);
        return;
      }
      int fine = -1;
      if (count > (uint32_t)kList) {
        cluster_arrive();  // the counts have been read
        cluster_wait();
        h = histogram(bin);
        incl = scan_u32(h.x + h.y) + above;
        excl = incl - h.x - h.y;
        __syncthreads();
        if (excl < k && k <= incl) k <= excl + h.x ? publish(2 * tid, h.x, excl) : publish(2 * tid + 1, h.y, excl + h.x);
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
    uint64_t z[1] = {0};
    each([&](float l, int idx) {
      if (octaves(l, m, half, ch) > -kOctaves && kept(l, idx)) z[0] += weight(l, m, sh);
    });
    cluster_sum(z);
    const uint64_t target = (uint64_t)ceil((double)top_p * (double)z[0]);
    int bin = -1, fine = -1;
    uint64_t above = 0;
    uint32_t count = 0;
    for (int level = 0; level < 2; ++level) {
      const uint2 h = histogram(bin);
      // the guess: counts times the weight at the bin's middle (inside one bin: of the bin)
      const float w0 = exp2f(-((float)(level ? bin : 2 * tid) + 0.5f) / kBinScale);
      const float w1 = level ? w0 : exp2f(-((float)(2 * tid + 1) + 0.5f) / kBinScale);
      const float mass0 = w0 * (float)h.x, mass1 = w1 * (float)h.y;
      const float at = (float)(target - above) * (1.f / (float)kOne);
      const float incl = scan_f32(mass0 + mass1), excl = incl - mass0 - mass1;
      const uint32_t c_incl = scan_u32(h.x + h.y);
      if (tid == 0) sh.bin = kBins - 1;
      __syncthreads();
      if (at <= incl) atomicMin(&sh.bin, at <= excl + mass0 ? 2 * tid : 2 * tid + 1);  // the same in every CTA
      __syncthreads();
      int guess = min(sh.bin, kBins - 2);
      if (level == 0 && sh.bin < kBins - 4) {
        // few enough up to the bins behind the guess: they are the list, if they do reach the target
        if (tid == (guess + 2) >> 1) sh.bin_above = c_incl;
        __syncthreads();
        const uint32_t n = sh.bin_above;
        if (n <= (uint32_t)kList) {
          const int last = ((guess + 2) | 1);
          gather([&](float t) { return bin_of(t) <= last; });
          uint64_t s = tid < (int)n ? sh.u.s.list[tid].w : 0ull;
          s = warp_sum64(s);
          __syncthreads();
          if (lane == 0) sh.part[warp][0] = s;
          __syncthreads();
          s = 0;
          for (int w = 0; w < kWarps; ++w) s += sh.part[w][0];
          if (s >= target) {
            finish_list((int)n, INT_MAX, z[0]);
            return;
          }
          if (tid == 0) sh.n_list = 0;  // stored into again behind the next exchange
          __syncthreads();
        }
      }
      // the exact sums around the guess
      auto part_of = [&](float t) -> int {  // -1: before the bin that is looked into; kBins: behind
        const int x = bin_of(t);
        return level == 0 ? x : x < bin ? -1 : x > bin ? kBins : fine_of(t, bin);
      };
      uint64_t base = 0;
      for (int guard = 0; guard < kBins; ++guard) {
        uint64_t s[4] = {0, 0, 0, 0};
        each([&](float l, int idx) {
          const float t = octaves(l, m, half, ch);
          const int x = t > -kOctaves ? part_of(t) : kBins;
          if (x <= guess + 1 && x < kBins && kept(l, idx)) {
            const uint64_t w = weight(l, m, sh);
            if (x < guess - 1) s[0] += w;
            else if (x == guess - 1) s[1] += w;
            else if (x == guess) s[2] += w;
            else s[3] += w;
          }
        });
        cluster_sum(s);
        if (target <= s[0]) {
          guess -= 2;
        } else if (target <= s[0] + s[1]) {
          guess -= 1;
          base = s[0];
          break;
        } else if (target <= s[0] + s[1] + s[2]) {
          base = s[0] + s[1];
          break;
        } else if (target <= s[0] + s[1] + s[2] + s[3]) {
          guess += 1;
          base = s[0] + s[1] + s[2];
          break;
        } else {
          guess += 2;
        }
      }
      above = base;
      if (tid == (guess >> 1)) sh.bin_count = guess & 1 ? h.y : h.x;
      __syncthreads();
      count = sh.bin_count;
      if (level == 0) bin = guess; else fine = guess;
      if (count <= (uint32_t)kList) break;
    }
    cut_in_bin(true, target, above, count, bin, fine);
  }
  // ---- the sum of what is left, by groups of a warp's elements ------------------------------------
  const uint64_t least = min_p > 0.f ? (uint64_t)ceil((double)min_p * (double)kOne) : 0ull;
  auto left = [&](float l, int idx) -> uint64_t {
    if (!(octaves(l, m, half, ch) > -kOctaves) || !kept(l, idx)) return 0ull;
    const uint64_t w = weight(l, m, sh);
    return w >= least ? w : 0ull;
  };
  __syncthreads();
  uint64_t s[1] = {0}, lowest[1] = {0};
  for (int i = 4 * tid, g = warp; i - 4 * lane < n_own; i += 4 * kThreads, g += kWarps) {
    uint64_t w = 0;
    if (i < n_own) {
      const float4 x = four(i);
      const float y[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const uint64_t z = left(y[e], v0 + i + e);
        w += z;
        if (z != 0) lowest[0] = max(lowest[0], (unsigned long)~order_key(y[e]));
      }
    }
    s[0] += w;
    w = __any_sync(kFull, w != 0) ? warp_sum64(w) : 0ull;
    if (lane == 0) sh.u.gsum[g] = w;
  }
  cluster_sum(s);
  const uint64_t total = s[0], start = before;
  if (probs != nullptr) {
    cluster_sum(lowest, true);
    const float last = key_logit(~(uint32_t)lowest[0]);  // min-p may have kept less than the cut
    const float inv = (float)((double)kOne / (double)total);
    write_probs([&](int i) {
      const float4 x = four(i);
      auto p = [&](float l, int idx) {
        const float t = octaves(l, m, half, ch);
        return t > -kOctaves && l >= last && kept(l, idx) ? fast_exp2(t) * inv : 0.f;
      };
      return make_float4(p(x.x, v0 + i), p(x.y, v0 + i + 1), p(x.z, v0 + i + 2), p(x.w, v0 + i + 3));
    });
  }
  // ---- the token: the group, then the element, where the running sum passes r of the total ---------------
  if (a.token != nullptr && warp == 0) {
    uint64_t at = (uint64_t)((double)rf * (double)total);
    if (at >= total) at = total - 1;
    uint64_t run = start;
    const int groups = (n_own + kGroup - 1) / kGroup;
    for (int g0 = 0; g0 < groups; g0 += 32) {
      const uint64_t w = g0 + lane < groups ? sh.u.gsum[g0 + lane] : 0ull;
      const uint64_t all = warp_sum64(w);
      if (at < run || at >= run + all) {
        run += all;
        continue;
      }
      uint64_t incl = w;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const uint64_t x = __shfl_up_sync(kFull, incl, o);
        if (lane >= o) incl += x;
      }
      const unsigned hit = __ballot_sync(kFull, at >= run + incl - w && at < run + incl);
      const int g = g0 + __ffs((int)hit) - 1;
      run += __shfl_sync(kFull, incl - w, __ffs((int)hit) - 1);
      const int i = g * kGroup + 4 * lane;
      uint64_t x[4] = {0, 0, 0, 0};
      if (i < n_own) {
        const float4 y = four(i);
        x[0] = left(y.x, v0 + i);
        x[1] = left(y.y, v0 + i + 1);
        x[2] = left(y.z, v0 + i + 2);
        x[3] = left(y.w, v0 + i + 3);
      }
      const uint64_t mine = x[0] + x[1] + x[2] + x[3];
      incl = mine;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const uint64_t z = __shfl_up_sync(kFull, incl, o);
        if (lane >= o) incl += z;
      }
      uint64_t z = run + incl - mine;
      if (at >= z && at < z + mine) {
        int e = 0;
        while (at >= z + x[e]) z += x[e++];
        a.token[b] = v0 + i + e;
      }
      break;
    }
  }
  cluster_arrive();
  cluster_wait();
}

using Kernel = void (*)(SampleArgs);

// CTAs of a row: as many as a row's parts need to stay in shared memory with two CTAs on an SM (25600 logits
// each), more where the batch leaves SMs empty.
constexpr int kPart = 25600, kPartMost = 51200;
int cluster_size(int64_t rows, int V) {
  int C = 1;
  while (C < kMaxCluster && (int64_t)C * kPart < V) C *= 2;
  while (C < kMaxCluster && rows * C * 2 <= 2 * 152 && V > C * 1024) C *= 2;
  return C;
}

// A kernel's dynamic shared memory limit belongs to the device: raised once on each.
cudaError_t raise_smem_limit(Kernel k, int which) {
  static std::mutex mu;
  static bool done[2][128];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  std::lock_guard<std::mutex> lk(mu);
  if (dev >= 0 && dev < 128 && done[which][dev]) return cudaSuccess;
  e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, kPartMost * (int)sizeof(float));
  if (e == cudaSuccess && dev >= 0 && dev < 128) done[which][dev] = true;
  return e;
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
  const int C = cluster_size(n_rows, vocab);
  SampleArgs a{};
  a.logits = logits;
  a.ld = row_stride;
  a.V = vocab;
  a.seg = ((vocab + C - 1) / C + 3) / 4 * 4;
  a.temperature = temperature;
  a.top_k = top_k;
  a.top_p = top_p;
  a.min_p = min_p;
  a.uniforms = uniforms;
  a.token = token;
  a.probs = probs;
  a.probs_ld = probs_stride;
  a.vec_in = row_stride % 4 == 0 && aligned(logits, half ? 8 : 16);
  a.vec_out = probs_stride % 4 == 0 && aligned(probs, 16);
  const bool resident = a.seg <= kPartMost;
  const Kernel kernel = resident ? (half ? sample_kernel<true, true> : sample_kernel<false, true>)
                                 : (half ? sample_kernel<true, false> : sample_kernel<false, false>);
  cudaError_t e = resident ? raise_smem_limit(kernel, half) : cudaSuccess;
  if (e != cudaSuccess) return cuda_fail(e, "sampling set-up");
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(n_rows * C));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = resident ? (size_t)a.seg * sizeof(float) : 0;
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
