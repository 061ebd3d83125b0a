// Attention of a tree of drafted tokens over the paged cache (absorbed MLA), sm_103a.
//
// Per query row (node i, head h) of a request with ctx committed rows and n drafts:
//   s_t = scale * (q_lat . cKV_t + q_rope . k_r,t) over the rows t < ctx and the drafts' rows
//   ctx + k whose bit k is set in node i's mask;  O = softmax(s) . cKV, lse = ln sum exp(s).
//
// One block per query row: a warp computes one key's score at a time, the block keeps a
// running maximum and sum over tiles of 64 keys (one page) and four output columns a thread.
#include <cuda_runtime.h>
#include <cmath>
#include <cstdint>
#include <cstring>

#include "irm_common.cuh"
#include "irm_host_util.h"

namespace irm {
namespace {

constexpr int kBatch = 1024;  // requests per launch (their lengths travel in the parameters)
constexpr int kThreads = 128;
constexpr uint32_t kFull = 0xffffffffu;

struct TreeArgs {
  const __nv_bfloat16* q_lat;
  const __nv_bfloat16* q_rope;
  const __nv_bfloat16* kv;
  const int32_t* page_table;
  const uint32_t* mask;
  int64_t n_pages;
  int B, b0, H, max_pages, mask_words;
  float scale;
  __nv_bfloat16* out;
  float* lse;
  int* status;
  int32_t ctx[kBatch], indptr[kBatch + 1];
};
static_assert(sizeof(TreeArgs) <= 32764, "kernel parameter block");

__global__ void __launch_bounds__(kThreads) tree_attn_kernel(const __grid_constant__ TreeArgs a) {
  __shared__ float score[kPage];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int64_t row = (int64_t)blockIdx.x;  // node of this launch * H + head
  const int node = (int)(row / a.H) + a.indptr[0];
  int lo = 0, hi = a.B;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (a.indptr[mid] <= node) lo = mid; else hi = mid;
  }
  const int b = lo, ctx = a.ctx[b], n = a.indptr[b + 1] - a.indptr[b];
  const int64_t grow = (int64_t)a.indptr[0] * a.H + row;
  const uint32_t* mask = a.mask + (int64_t)node * a.mask_words;
  const int32_t* ptab = a.page_table + (int64_t)(a.b0 + b) * a.max_pages;
  float q[18];
#pragma unroll
  for (int e = 0; e < 16; ++e) q[e] = __bfloat162float(a.q_lat[grow * kDLat + 32 * e + lane]);
#pragma unroll
  for (int e = 0; e < 2; ++e) q[16 + e] = __bfloat162float(a.q_rope[grow * kDRope + 32 * e + lane]);
  float m = -INFINITY, l = 0.f, acc[4] = {0.f, 0.f, 0.f, 0.f};
  for (int T = 0; T < ctx + n; T += kPage) {
    const int page = ptab[T / kPage];
    const bool in = page >= 0 && page < a.n_pages;
    if (!in && tid == 0) set_status(a.status, kDevErrBounds);
    const __nv_bfloat16* rows = a.kv + (int64_t)(in ? page : 0) * kPage * kDRow;
    for (int r = warp; r < kPage; r += kThreads / 32) {
      const int t = T + r, k = t - ctx;
      const bool see = t < ctx || (k < n && (mask[k >> 5] >> (k & 31) & 1u));
      float s = 0.f;
      if (see && in) {
#pragma unroll
        for (int e = 0; e < 18; ++e) s += q[e] * __bfloat162float(rows[r * kDRow + 32 * e + lane]);
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(kFull, s, o);
      if (lane == 0) score[r] = see ? s * a.scale : -INFINITY;
    }
    __syncthreads();
    float mx = m;
    for (int r = 0; r < kPage; ++r) mx = fmaxf(mx, score[r]);
    if (mx != -INFINITY) {
      const float corr = expf(m - mx);
      m = mx;
      l *= corr;
#pragma unroll
      for (int e = 0; e < 4; ++e) acc[e] *= corr;
      for (int r = 0; r < kPage; ++r) {
        if (score[r] == -INFINITY) continue;
        const float p = expf(score[r] - mx);
        l += p;
        if (in) {
#pragma unroll
          for (int e = 0; e < 4; ++e) acc[e] += p * __bfloat162float(rows[r * kDRow + 128 * e + tid]);
        }
      }
    }
    __syncthreads();
  }
  const float inv = l > 0.f ? 1.f / l : 0.f;
#pragma unroll
  for (int e = 0; e < 4; ++e) a.out[grow * kDLat + 128 * e + tid] = __float2bfloat16_rn(acc[e] * inv);
  if (a.lse != nullptr && tid == 0) a.lse[grow] = l > 0.f ? m + logf(l) : -INFINITY;
}

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
  *bytes = IRM_WORKSPACE_HEADER;
  return IRM_OK;
}

irm_status irm_mla_attn_tree(const void* q_lat, const void* q_rope, int B, int H, const int32_t* ctx_host,
                             const int32_t* q_indptr_host, const void* paged_kv, int64_t n_pages,
                             const int32_t* page_table, int max_pages, const uint32_t* tree_mask, int mask_words,
                             float softmax_scale, void* out, float* lse, void* workspace, size_t workspace_bytes,
                             cudaStream_t stream) {
  using namespace irm;
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
  if (!std::isfinite(softmax_scale) || softmax_scale <= 0.f)
    return fail(IRM_ERR_INVALID_ARG, "softmax_scale must be finite and positive");
  if (!q_lat || !q_rope || !paged_kv || !page_table || !tree_mask || !out) return fail(IRM_ERR_INVALID_ARG, "null device pointer");
  if (!aligned(q_lat, 16) || !aligned(q_rope, 16) || !aligned(paged_kv, 16) || !aligned(out, 16))
    return fail(IRM_ERR_INVALID_ARG, "q_lat, q_rope, paged_kv and out must be 16-byte aligned");
  if (!aligned(page_table, 4) || !aligned(tree_mask, 4) || !aligned(lse, 4))
    return fail(IRM_ERR_INVALID_ARG, "misaligned device pointer");
  if (!workspace || !aligned(workspace, 256) || workspace_bytes < IRM_WORKSPACE_HEADER)
    return fail(IRM_ERR_WORKSPACE, "workspace must be 256-byte aligned and hold %d bytes", IRM_WORKSPACE_HEADER);
  if (q_indptr_host[B] == 0) return IRM_OK;
  TreeArgs a{};
  a.q_lat = static_cast<const __nv_bfloat16*>(q_lat);
  a.q_rope = static_cast<const __nv_bfloat16*>(q_rope);
  a.kv = static_cast<const __nv_bfloat16*>(paged_kv);
  a.page_table = page_table;
  a.mask = tree_mask;
  a.n_pages = n_pages;
  a.H = H;
  a.max_pages = max_pages;
  a.mask_words = mask_words;
  a.scale = softmax_scale;
  a.out = static_cast<__nv_bfloat16*>(out);
  a.lse = lse;
  a.status = static_cast<int*>(workspace);
  for (int b0 = 0; b0 < B; b0 += kBatch) {
    a.b0 = b0;
    a.B = B - b0 < kBatch ? B - b0 : kBatch;
    std::memcpy(a.ctx, ctx_host + b0, (size_t)a.B * sizeof(int32_t));
    std::memcpy(a.indptr, q_indptr_host + b0, (size_t)(a.B + 1) * sizeof(int32_t));
    const int64_t blocks = (int64_t)(a.indptr[a.B] - a.indptr[0]) * H;
    if (blocks == 0) continue;
    tree_attn_kernel<<<(unsigned)blocks, kThreads, 0, stream>>>(a);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return cuda_fail(e, "tree attention launch");
  }
  return IRM_OK;
}

}  // extern "C"
