// Verification of drafted tokens against the target model's probabilities, from given uniform
// numbers (speculative sampling over a tree; the emitted tokens follow the target's
// distribution exactly, whatever was drafted).
//
// Per request, with node 0 the last committed token, p_u the target's and q_u the draft
// model's row at node u, and w, S the residual distribution (unnormalised) and its sum:
//   u = 0, w = p_0, S = 1.  For the children i of u in index order, x = token_i:
//     accept when r_i q_u(x) S < w(x): u = i, w = p_i, S = 1;
//     else w <- max(w - S q_u, 0), S <- sum w.
//   When no child is left: next token = the lowest v with cumsum(w)(v) > r_0 sum(w).
// All children of a node were drawn from the same row, so after k rejections
//   w = max(p_u - A q_u, 0) with A = S_0 + .. + S_(k-1):
// what a rejection takes off is never negative, so the clips at zero are one clip at the end, and an
// entry costs the same after one rejection as after ten (with the subtractions one by one, 16
// requests x 24 nodes x 102400 entries took 53.1 us, now 32.4).
// Without draft probabilities the drafts are taken as chosen without chance (q one-hot at the
// child's token): a rejection takes w(x) out of w and S.
// A node's children come after it, so one pass over the nodes in index order is the walk.
//
// Arithmetic.  Sums over the vocabulary decide which token comes out, so they must not depend
// on the order of addition or on the split: every probability becomes a 44-bit fixed-point
// integer (resolution 5.7e-14) and sums are 64-bit integers, exact in any order (below 2^20
// entries of 1.0 fit).  fp32 sums would shift the boundaries of a flat 100k-entry row by more
// than some of its entries are wide; fp64 sums depend on their order in the last bits.
// The acceptance tests run in fp64 on the fp32 inputs, in the order written above.
//
// What bounds it: latency.  One row of V fp32 (two with draft probabilities) per request is read for
// the final draw, 0.06 us of memory time at one request of 102400 entries and 3.9 us at 64, but
// the chain of launch, gather, walk, sum, cluster exchange and locating the token takes 11.2 and
// 18.1 us.  So a cluster of C CTAs shares a request's row in contiguous warp segments; the CTA
// totals travel through distributed shared memory, and what is located is one group of one
// warp's loads, from group sums kept during the sum.  The children's probabilities are gathered in
// one round of loads, all nodes at once, before the walk, which then runs in shared memory.
// With draft probabilities each rejection that another child follows is one more pass over two
// rows (16 requests, 24 nodes, 102400 entries: 32.4 us).
#include <cuda_runtime.h>
#include <cmath>
#include <cstdint>
#include <cstring>

#include "irm_common.cuh"
#include "irm_host_util.h"

namespace irm {
namespace {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxCluster = 8;
constexpr int kMaxVocab = 1 << 20;
constexpr int kMaxGroups = 64;  // groups of a warp's segment
constexpr int kBatch = 1024;  // requests per launch (their offsets travel in the parameters)
constexpr uint32_t kFull = 0xffffffffu;

struct VerifyArgs {
  const float* target;
  const float* draft;
  int64_t ld;  // elements between rows
  int V, b0, max_path;
  const int32_t* tokens;
  const int32_t* parents;
  const float* uniforms;
  int32_t* n_accept;
  int32_t* path;
  int32_t* next_token;
  int* status;
  int32_t indptr[kBatch + 1];
};
static_assert(sizeof(VerifyArgs) <= 32764, "kernel parameter block");

// Probability in units of 2^-44, rounded to the nearest; NaN and negative values are 0, values above 1
// are 1.  The mantissa is shifted to its place: the conversion instruction to 64 bits runs at about
// the fp64 rate, ~1 a clock on an SM, which made it the bound (63 us for one row on one SM).
__device__ __forceinline__ uint32_t unit_bits(float p) { return __float_as_uint(fminf(fmaxf(p, 0.f), 1.f)); }
__device__ __forceinline__ uint64_t fixed44(float p) {
  const uint32_t b = unit_bits(p), e = b >> 23;  // 127 for 1.0; a denormal counts as 2^-126, which the shift drops
  const uint64_t wide = (uint64_t)((b & 0x7fffffu) | 0x800000u) << 22;  // 2^45 at e = 127
  return ((wide >> min(127u - e, 63u)) + 1u) >> 1;
}
// q A in units of 2^-44, rounded down, for a probability q and A in those units (A < 2^55; it is at most
// IRM_MAX_TREE): 24 x 55 bits as two products of 32 x 32.
__device__ __forceinline__ uint64_t times44(float q, uint64_t A) {
  const uint32_t b = unit_bits(q), e = b >> 23, m = (b & 0x7fffffu) | 0x800000u;
  const uint64_t t = (uint64_t)m * (uint32_t)(A >> 23) + (((uint64_t)m * (uint32_t)(A & 0x7fffffu)) >> 23);
  return t >> min(127u - e, 63u);
}
__device__ __forceinline__ double from44(uint64_t s) { return (double)s * 0x1p-44; }

struct Shared {
  int32_t par[IRM_MAX_TREE], tok[IRM_MAX_TREE], path[IRM_MAX_TREE];
  float r[IRM_MAX_TREE], p[IRM_MAX_TREE], q[IRM_MAX_TREE];
  int32_t rej[IRM_MAX_TREE];  // without draft probabilities: the distinct tokens rejected at the current node
  uint64_t S, A;              // with: S at the current node, and the sum of the S that were rejected with
  uint64_t wsum[kWarps], gsum[kWarps][kMaxGroups];  // sums of the warps' segments, and of each group of their loads
  uint64_t ctot[2][kMaxCluster];
  int32_t u, k, next_i, depth, need_sum;
};

// Residual of one vocabulary entry, in fixed point.
__device__ __forceinline__ uint64_t residual(float p, float q, uint64_t A) {
  const uint64_t w = fixed44(p), sub = times44(q, A);
  return w > sub ? w - sub : 0ull;
}

__device__ __forceinline__ uint64_t warp_sum(uint64_t v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(kFull, v, o);
  return v;
}

__device__ __forceinline__ void st_cluster_u64(uint32_t addr, uint64_t v) {
  asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(addr), "l"(v) : "memory");
}

// Four consecutive entries of a row (zero past the end).
template <bool VEC>
__device__ __forceinline__ float4 load4(const float* p, int v, int end) {
  if (VEC) return v < end ? __ldg(reinterpret_cast<const float4*>(p + v)) : make_float4(0.f, 0.f, 0.f, 0.f);
  float4 a;
  a.x = v < end ? __ldg(p + v) : 0.f;  // whole vectors are only sure where rows and segments are
  a.y = v + 1 < end ? __ldg(p + v + 1) : 0.f;
  a.z = v + 2 < end ? __ldg(p + v + 2) : 0.f;
  a.w = v + 3 < end ? __ldg(p + v + 3) : 0.f;
  return a;
}

template <bool VEC, bool DRAFT>
__global__ void __launch_bounds__(kThreads, 2) tree_verify_kernel(const __grid_constant__ VerifyArgs a) {
  __shared__ Shared sh;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  uint32_t C;
  asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(C));
  const uint32_t rank = cluster_ctarank();
  const int b = (int)(blockIdx.x / C);
  const int lo = a.indptr[b], n = a.indptr[b + 1] - lo;
  const int64_t gb = (int64_t)a.b0 + b;
  if (n == 0) {  // the same in every CTA of the cluster
    if (rank == 0) {
      for (int k = tid; k < a.max_path; k += kThreads) a.path[gb * a.max_path + k] = -1;
      if (tid == 0) {
        a.n_accept[gb] = 0;
        a.next_token[gb] = -1;
      }
    }
    return;
  }
  cluster_arrive();  // waited for before the first store into a peer's shared memory
  // ---- the tree and its tokens' probabilities at their parents, one round of loads ------
  bool bad = false;
  for (int i = tid; i < n; i += kThreads) {
    const int par = a.parents[lo + i], tok = a.tokens[lo + i];
    const bool child = i > 0 && par >= 0 && par < i, in = tok >= 0 && tok < a.V;
    float p = 0.f, q = 0.f;
    if (child && in) {
      p = __ldg(a.target + (int64_t)(lo + par) * a.ld + tok);
      if (DRAFT) q = __ldg(a.draft + (int64_t)(lo + par) * a.ld + tok);
    }
    bad |= i > 0 && !(child && in);
    sh.par[i] = child ? par : -1;
    sh.tok[i] = in ? tok : -1;
    sh.p[i] = fminf(fmaxf(p, 0.f), 1.f);
    sh.q[i] = fminf(fmaxf(q, 0.f), 1.f);
    sh.r[i] = a.uniforms[lo + i];
  }
  if (bad && rank == 0) set_status(a.status, kDevErrBounds);
  if (tid == 0) {
    sh.u = 0;
    sh.k = 0;
    sh.next_i = 1;
    sh.depth = 1;
    sh.path[0] = 0;
    sh.S = 1ull << 44;
    sh.A = 0;
  }
  __syncthreads();
  cluster_wait();

  const int segs = (int)C * kWarps;
  const int seg = ((a.V + segs - 1) / segs + 3) / 4 * 4;
  const int v0 = min(a.V, ((int)rank * kWarps + warp) * seg), v1 = min(a.V, v0 + seg);

  // Sum over the vocabulary of the residual after k rejections at node u, and the part of it that lies
  // before this CTA's slice; sh.wsum and sh.gsum keep this CTA's warp and group sums.  A group is
  // what a warp has in flight at once: 4 vectors a lane (2 of each row with draft probabilities).
  constexpr int kAhead = DRAFT ? 2 : 4, kGroup = 128 * kAhead;
  int pass = 0;
  auto vocab_sum = [&](int u, int k, uint64_t& before) -> uint64_t {
    const float* p = a.target + (int64_t)(lo + u) * a.ld;
    const float* q = DRAFT && k > 0 ? a.draft + (int64_t)(lo + u) * a.ld : nullptr;
    const uint64_t A = sh.A;
    uint64_t s = 0;
    for (int g = 0; v0 + g * kGroup < v1; ++g) {
      float4 x[kAhead], y[kAhead];
#pragma unroll
      for (int e = 0; e < kAhead; ++e) {
        x[e] = load4<VEC>(p, v0 + g * kGroup + 128 * e + 4 * lane, v1);
        if (DRAFT && q != nullptr) y[e] = load4<VEC>(q, v0 + g * kGroup + 128 * e + 4 * lane, v1);
      }
      uint64_t sg = 0;
#pragma unroll
      for (int e = 0; e < kAhead; ++e) {
        const float xs[4] = {x[e].x, x[e].y, x[e].z, x[e].w};
        const float ys[4] = {y[e].x, y[e].y, y[e].z, y[e].w};
#pragma unroll
        for (int f = 0; f < 4; ++f) sg += DRAFT && q != nullptr ? residual(xs[f], ys[f], A) : fixed44(xs[f]);
      }
      sg = warp_sum(sg);
      if (lane == 0) sh.gsum[warp][g] = sg;
      s += sg;
    }
    if (lane == 0) sh.wsum[warp] = s;
    __syncthreads();
    if (!DRAFT && k > 0) {  // the rejected tokens leave the row
      for (int t = tid; t < k; t += kThreads) {
        const int x = sh.rej[t], w = x / seg - (int)rank * kWarps;
        if (w >= 0 && w < kWarps) {
          const unsigned long long gone = 0ull - fixed44(__ldg(p + x));
          atomicAdd(reinterpret_cast<unsigned long long*>(&sh.wsum[w]), gone);
          atomicAdd(reinterpret_cast<unsigned long long*>(&sh.gsum[w][(x - (x / seg) * seg) / kGroup]), gone);
        }
      }
      __syncthreads();
    }
    const int slot = pass++ & 1;
    if (warp == 0) {
      const uint64_t mine = warp_sum(lane < kWarps ? sh.wsum[lane] : 0ull);
      if (lane < (int)C) st_cluster_u64(mapa_shared(smem_u32(&sh.ctot[slot][rank]), (uint32_t)lane), mine);
    }
    __syncwarp();
    cluster_arrive();
    cluster_wait();
    uint64_t t = 0;
    for (int c = 0; c < (int)C; ++c) {
      if (c == (int)rank) before = t;
      t += sh.ctot[slot][c];
    }
    return t;
  };

  // ---- the walk: warp 0 until a residual sum is needed (draft probabilities) or no child is left ----
  uint64_t before = 0;
  for (;;) {
    if (warp == 0) {
      int u = sh.u, k = sh.k, i = sh.next_i, depth = sh.depth, need = 0;
      uint64_t S44 = sh.S, A44 = sh.A;
      double S = DRAFT ? from44(S44) : 1.0;
      while (depth < a.max_path) {
        // next child of u, 32 nodes at a time
        int found = -1;
        for (int base = i; base < n; base += 32) {
          const unsigned m = __ballot_sync(kFull, base + lane < n && sh.par[base + lane] == u);
          if (m) {
            found = base + __ffs((int)m) - 1;
            break;
          }
        }
        if (found < 0) break;
        i = found + 1;
        const int x = sh.tok[found];
        const double p = (double)sh.p[found], r = (double)sh.r[found];
        double w = p;
        bool take;
        if (DRAFT) {
          const double q = (double)sh.q[found];
          w = fmax(w - q * from44(A44), 0.0);
          take = x >= 0 && r * q * S < w;
        } else {
          bool again = false;  // already rejected at this node
          for (int t = lane; t < k; t += 32) again |= sh.rej[t] == x;
          if (__any_sync(kFull, again)) w = 0.0;
          take = x >= 0 && r * S < w;
        }
        if (take) {
          u = found;
          k = 0;
          S = 1.0;
          S44 = 1ull << 44;
          A44 = 0;
          if (lane == 0) sh.path[depth] = found;
          ++depth;
        } else if (x >= 0) {
          if (DRAFT) {
            ++k;
            A44 += S44;
            // the new sum only matters when another child is left to test
            bool more = false;
            for (int t = i + lane; t < n; t += 32) more |= sh.par[t] == u;
            need = __any_sync(kFull, more) ? 1 : 0;
            if (need) break;
          } else if (w > 0.0) {
            if (lane == 0) sh.rej[k] = x;
            __syncwarp();
            ++k;
            S -= w;
          }
        }
      }
      if (lane == 0) {
        sh.u = u;
        sh.k = k;
        sh.next_i = i;
        sh.depth = depth;
        sh.need_sum = need;
        sh.S = S44;
        sh.A = A44;
      }
    }
    __syncthreads();
    if (!DRAFT || !sh.need_sum) break;
    const uint64_t t = vocab_sum(sh.u, sh.k, before);
    if (tid == 0) sh.S = t;
    __syncthreads();
  }

  // ---- the next token: inverse of the residual's running sum --------------------------
  const int u = sh.u;
  int k = sh.k;
  uint64_t total = vocab_sum(u, k, before);
  if (total == 0 && k > 0) {  // nothing is left but rounding: draw from the target's row
    k = 0;
    __syncthreads();
    total = vocab_sum(u, 0, before);
  }
  if (rank == 0) {
    for (int t = tid; t < a.max_path; t += kThreads) a.path[gb * a.max_path + t] = t < sh.depth ? sh.path[t] : -1;
    if (tid == 0) a.n_accept[gb] = sh.depth;
    if (tid == 0 && total == 0) a.next_token[gb] = -1;
  }
  if (total == 0) return;
  const double rf = (double)fminf(fmaxf(sh.r[0], 0.f), 1.f);
  uint64_t thr = (uint64_t)(rf * (double)total);
  if (thr >= total) thr = total - 1;
  // the warp whose segment holds the threshold
  for (int w = 0; w < warp; ++w) before += sh.wsum[w];
  if (thr < before || thr >= before + sh.wsum[warp]) return;
  // its group, then its vector, then its entry
  int g = 0;
  while (thr >= before + sh.gsum[warp][g]) before += sh.gsum[warp][g++];
  const float* p = a.target + (int64_t)(lo + u) * a.ld;
  const float* q = DRAFT && k > 0 ? a.draft + (int64_t)(lo + u) * a.ld : nullptr;
  float4 x[kAhead], y[kAhead];
#pragma unroll
  for (int e = 0; e < kAhead; ++e) {
    x[e] = load4<VEC>(p, v0 + g * kGroup + 128 * e + 4 * lane, v1);
    if (DRAFT && q != nullptr) y[e] = load4<VEC>(q, v0 + g * kGroup + 128 * e + 4 * lane, v1);
  }
#pragma unroll
  for (int e = 0; e < kAhead; ++e) {
    const int v = v0 + g * kGroup + 128 * e + 4 * lane;
    const float xs[4] = {x[e].x, x[e].y, x[e].z, x[e].w};
    const float ys[4] = {y[e].x, y[e].y, y[e].z, y[e].w};
    uint64_t w4[4], mine = 0;
#pragma unroll
    for (int f = 0; f < 4; ++f) {
      uint64_t w = DRAFT && q != nullptr ? residual(xs[f], ys[f], sh.A) : fixed44(xs[f]);
      if (!DRAFT)
        for (int t = 0; t < k; ++t)
          if (sh.rej[t] == v + f) w = 0;
      w4[f] = w;
      mine += w;
    }
    const uint64_t all = warp_sum(mine);
    if (thr >= before + all) {
      before += all;
      continue;
    }
    uint64_t incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint64_t t = __shfl_up_sync(kFull, incl, o);
      if (lane >= o) incl += t;
    }
    uint64_t at = before + incl - mine;
    if (thr >= at && thr < at + mine) {
      int f = 0;
      if (thr >= at + w4[0]) {
        at += w4[0];
        f = 1;
        if (thr >= at + w4[1]) {
          at += w4[1];
          f = thr >= at + w4[2] ? 3 : 2;
        }
      }
      a.next_token[gb] = v + f;
    }
    return;
  }
}

// CTAs a request's vocabulary is spread over: as many as keep the batch on the GPU at once (two CTAs
// an SM).  Measured, vocabulary 102400: 1 request 20.8 / 17.7 / 11.3 us with 2 / 4 / 8; 64 requests
// 36.3 / 24.6 / 27.0 us.  A large vocabulary needs enough of them for its groups
// (of 256 entries at least).
int cluster_size(int B, int vocab) {
  const int fit = 2 * 152 / B;
  int C = fit >= 8 ? 8 : fit >= 4 ? 4 : fit >= 2 ? 2 : 1;
  while (C < kMaxCluster && vocab > C * kWarps * (kMaxGroups - 1) * 256) C *= 2;
  return C;
}

using Kernel = void (*)(VerifyArgs);

}  // namespace
}  // namespace irm

extern "C" irm_status irm_tree_verify(const float* target_probs, const float* draft_probs, int64_t row_stride,
                                      int32_t vocab, const int32_t* tokens, const int32_t* parents,
                                      const float* uniforms, const int32_t* q_indptr_host, int B, int max_path,
                                      int32_t* n_accept, int32_t* path, int32_t* next_token, void* workspace,
                                      size_t workspace_bytes, cudaStream_t stream) {
  using namespace irm;
  int most = 0;
  irm_status st = check_trees(q_indptr_host, B, &most);
  if (st != IRM_OK) return st;
  if (vocab < 1 || vocab > kMaxVocab) return fail(IRM_ERR_UNSUPPORTED, "vocab %d outside [1, 2^20]", vocab);
  if (row_stride < vocab) return fail(IRM_ERR_INVALID_ARG, "row_stride is smaller than vocab");
  if (max_path < 1) return fail(IRM_ERR_INVALID_ARG, "max_path must be positive");
  if (!n_accept || !path || !next_token || (most > 0 && (!target_probs || !tokens || !parents || !uniforms)))
    return fail(IRM_ERR_INVALID_ARG, "null device pointer");
  for (const void* p : {(const void*)target_probs, (const void*)draft_probs, (const void*)tokens, (const void*)parents,
                        (const void*)uniforms, (const void*)n_accept, (const void*)path, (const void*)next_token})
    if (!aligned(p, 4)) return fail(IRM_ERR_INVALID_ARG, "misaligned device pointer");
  if (!workspace || !aligned(workspace, 256) || workspace_bytes < IRM_WORKSPACE_HEADER)
    return fail(IRM_ERR_WORKSPACE, "workspace must be 256-byte aligned and hold %d bytes", IRM_WORKSPACE_HEADER);
  VerifyArgs a{};
  a.target = target_probs;
  a.draft = draft_probs;
  a.ld = row_stride;
  a.V = vocab;
  a.max_path = max_path;
  a.tokens = tokens;
  a.parents = parents;
  a.uniforms = uniforms;
  a.n_accept = n_accept;
  a.path = path;
  a.next_token = next_token;
  a.status = static_cast<int*>(workspace);
  const bool vec = vocab % 4 == 0 && row_stride % 4 == 0 && aligned(target_probs, 16) && aligned(draft_probs, 16);
  for (int b0 = 0; b0 < B; b0 += kBatch) {
    const int nb = B - b0 < kBatch ? B - b0 : kBatch;
    a.b0 = b0;
    std::memcpy(a.indptr, q_indptr_host + b0, (size_t)(nb + 1) * sizeof(int32_t));
    cudaLaunchConfig_t cfg = {};
    const int C = cluster_size(nb, vocab);
    cfg.gridDim = dim3((unsigned)(nb * C));
    cfg.blockDim = dim3(kThreads);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)C;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const Kernel kernel = draft_probs != nullptr ? (vec ? tree_verify_kernel<true, true> : tree_verify_kernel<false, true>)
                                                 : (vec ? tree_verify_kernel<true, false> : tree_verify_kernel<false, false>);
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, a);
    if (e != cudaSuccess) return cuda_fail(e, "tree verification launch");
  }
  return IRM_OK;
}
