// Pages of the paged cache, kept on the device: resize (allocate, trim, free), fork, compact
// the rows of an accepted draft path, copy pages.
//
// Bookkeeping (resize, fork) is one CTA: its state is a few bytes per page, and one CTA orders
// its phases with block barriers instead of further launches.  The only state of a page is
// its holder count (0 = free); the free pages handed out are the lowest ones, found by a scan
// of the counts in index order, so nothing depends on the order in which atomics land (they
// only add to counts whose sum is read after a barrier).
// Moving rows (fork's partial pages, compact, copy) is pure bandwidth: 16-byte vectors, every
// layer in one launch.
#include <cuda_runtime.h>
#include <cstdint>
#include <cstring>
#include <exception>
#include <mutex>
#include <vector>

#include "irm_common.cuh"
#include "irm_host_util.h"

namespace irm {
namespace {

constexpr int kDevErrNoPages = 4;
constexpr int kDevErrShared = 8;

constexpr int kThreads = 1024;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxSlots = 8192;
constexpr int kMaxForks = 1024;
constexpr int64_t kMaxEntries = int64_t(1) << 30;  // of a page table: all requests' pages are counted in int32
constexpr uint32_t kFull = 0xffffffffu;
constexpr int kRowVec = kDRow * 2 / 16;        // 16-byte vectors of a row: 72
constexpr int kPageVec = kRowVec * kPage;      // and of a page: 4608
constexpr int kScanPages = 16;                 // counts one thread looks at per round of the scan

__device__ __forceinline__ int pages_of(int rows) { return (rows + kPage - 1) / kPage; }

// Exclusive prefix sum of one value per thread over the block; *total gets the sum.
__device__ __forceinline__ int block_exclusive(int v, int* part, int* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(kFull, x, o);
    if (lane >= o) x += y;
  }
  __syncthreads();  // part may still be read from the call before
  if (lane == 31) part[warp] = x;
  __syncthreads();
  if (warp == 0) {
    int w = part[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(kFull, w, o);
      if (lane >= o) w += y;
    }
    part[lane] = w;
  }
  __syncthreads();
  *total = part[kWarps - 1];
  return (warp ? part[warp - 1] : 0) + x - v;
}

// Bits of the free pages among the kScanPages counts from page p on.
__device__ __forceinline__ unsigned free_bits(const int32_t* refcount, int64_t p, int64_t n_pages, bool vec) {
  unsigned m = 0;
  if (vec && p + kScanPages <= n_pages) {
    int4 v[kScanPages / 4];
#pragma unroll
    for (int e = 0; e < kScanPages / 4; ++e) v[e] = *reinterpret_cast<const int4*>(refcount + p + 4 * e);
#pragma unroll
    for (int e = 0; e < kScanPages / 4; ++e)
      m |= ((v[e].x == 0 ? 1u : 0u) | (v[e].y == 0 ? 2u : 0u) | (v[e].z == 0 ? 4u : 0u) | (v[e].w == 0 ? 8u : 0u)) << (4 * e);
  } else {
    for (int e = 0; e < kScanPages; ++e)
      if (p + e < n_pages && refcount[p + e] == 0) m |= 1u << e;
  }
  return m;
}

// The lowest `want` free pages, in index order: take(rank, page) for each.  Returns false, having
// taken none, when there are fewer.  Called by the whole block; a thread's ranks increase.
template <class Take>
__device__ __forceinline__ bool take_free(const int32_t* refcount, int64_t n_pages, int want, int* part, Take take) {
  if (want == 0) return true;
  const bool vec = (reinterpret_cast<uintptr_t>(refcount) & 15u) == 0;
  constexpr int64_t kRound = (int64_t)kThreads * kScanPages;
  int found = 0, n = 0, rank = 0, rounds = 0;
  unsigned m = 0;
  for (int64_t p0 = 0; p0 < n_pages && found < want; p0 += kRound) {
    m = free_bits(refcount, p0 + (int64_t)threadIdx.x * kScanPages, n_pages, vec);
    rank = block_exclusive(__popc(m), part, &n);
    found += n;
    ++rounds;
  }
  if (found < want) return false;
  int rank0 = 0;
  for (int64_t p0 = 0; p0 < n_pages && rank0 < want; p0 += kRound) {
    const int64_t p = p0 + (int64_t)threadIdx.x * kScanPages;
    if (rounds > 1) {  // the bits at hand are the last round's
      m = free_bits(refcount, p, n_pages, vec);
      rank = rank0 + block_exclusive(__popc(m), part, &n);
    }
    for (int r = rank; m != 0 && r < want; m &= m - 1, ++r) take(r, (int)(p + __ffs((int)m) - 1));
    rank0 += n;
  }
  return true;
}

// Last index s in [0, n) with pre[s] <= r (pre non-decreasing, pre[0] = 0): the holder of rank r
// among entries with a positive share.
__device__ __forceinline__ int owner_of(const int* pre, int n, int r) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (pre[mid] <= r) lo = mid; else hi = mid;
  }
  return lo;
}
// The same for increasing ranks: starts at the owner of the rank before (-1: none yet).
__device__ __forceinline__ int next_owner(const int* pre, int n, int r, int s) {
  if (s < 0) return owner_of(pre, n, r);
  while (pre[s + 1] <= r) ++s;
  return s;
}

struct ResizeArgs {
  const int32_t* new_len;
  int32_t* seq_len;
  int n_slots, max_pages;
  int32_t* table;
  int32_t* refcount;
  int64_t n_pages;
  int* status;
};

// All requests' pages form one list for each phase (released, then wanted), which the threads share
// evenly whatever the requests' lengths: a position's request is found in the list's exclusive sums.
__global__ void __launch_bounds__(kThreads) pages_resize_kernel(const ResizeArgs a) {
  extern __shared__ int pre[];          // [n_slots + 1]: exclusive sums of the phase's pages
  int* held = pre + a.n_slots + 1;      // [n_slots]: pages held before, -1 for a refused request
  __shared__ int part[32];
  const int tid = threadIdx.x;
  const int most = a.max_pages * kPage;
  // ---- releases -----------------------------------------------------------------------------
  int total = 0, n;
  for (int s0 = 0; s0 < a.n_slots; s0 += kThreads) {
    const int s = s0 + tid;
    int gone = 0;
    if (s < a.n_slots) {
      const int old = a.seq_len[s], now = a.new_len[s];
      const bool ok = old >= 0 && old <= most && now >= 0 && now <= most;
      if (!ok) set_status(a.status, kDevErrBounds);
      held[s] = ok ? pages_of(old) : -1;
      gone = ok ? max(0, pages_of(old) - pages_of(now)) : 0;
    }
    const int at = block_exclusive(gone, part, &n);
    if (s < a.n_slots) pre[s] = total + at;
    total += n;
  }
  if (tid == 0) pre[a.n_slots] = total;
  __syncthreads();
  constexpr int kBatch = 4;  // pages a thread has in flight
  for (int r0 = tid; r0 < total; r0 += kBatch * kThreads) {
    int page[kBatch];
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      const int r = r0 + k * kThreads;
      if (r < total) {
        const int s = owner_of(pre, a.n_slots, r);
        int32_t* e = a.table + (int64_t)s * a.max_pages + held[s] - pre[s + 1] + r;
        page[k] = *e;
        *e = -1;
      }
    }
#pragma unroll
    for (int k = 0; k < kBatch; ++k)
      if (r0 + k * kThreads < total) {
        bool ok = page[k] >= 0 && page[k] < a.n_pages;
        if (ok && atomicSub(&a.refcount[page[k]], 1) <= 0) {
          atomicAdd(&a.refcount[page[k]], 1);
          ok = false;
        }
        if (!ok) set_status(a.status, kDevErrBounds);
      }
  }
  __syncthreads();
  // ---- what each request wants -----------------------------------------------------------------
  total = 0;
  for (int s0 = 0; s0 < a.n_slots; s0 += kThreads) {
    const int s = s0 + tid;
    int need = 0;
    if (s < a.n_slots && held[s] >= 0) {
      const int old = a.seq_len[s], now = a.new_len[s];
      if (now > old) {
        need = pages_of(now) - held[s];
        if (old % kPage != 0) {  // it would write into its last page: that must be its own
          const int p = a.table[(int64_t)s * a.max_pages + old / kPage];
          const bool in = p >= 0 && p < a.n_pages;
          if (!in || a.refcount[p] > 1) {
            set_status(a.status, in ? kDevErrShared : kDevErrBounds);
            held[s] = -1;
            need = 0;
          }
        }
      }
    }
    const int at = block_exclusive(need, part, &n);
    if (s < a.n_slots) pre[s] = total + at;
    total += n;
  }
  if (tid == 0) pre[a.n_slots] = total;
  __syncthreads();
  // ---- allocations -----------------------------------------------------------------------------
  int s_of = -1;
  const bool enough = take_free(a.refcount, a.n_pages, total, part, [&](int r, int page) {
    s_of = next_owner(pre, a.n_slots, r, s_of);
    a.table[(int64_t)s_of * a.max_pages + held[s_of] + (r - pre[s_of])] = page;
    a.refcount[page] = 1;  // each count is read before the block barrier that precedes this write
  });
  __syncthreads();
  if (!enough && tid == 0) set_status(a.status, kDevErrNoPages);
  for (int s = tid; s < a.n_slots; s += kThreads)
    if (held[s] >= 0) {
      const int now = a.new_len[s];
      if (enough || now <= a.seq_len[s]) a.seq_len[s] = now;
    }
}

// A copy of `rows` leading rows of a page to another page, in every layer.
struct CopyJob {
  int32_t src, dst, rows, pad;
};

struct ForkArgs {
  int32_t* seq_len;
  int n_slots, max_pages, n_forks;
  int32_t* table;
  int32_t* refcount;
  int64_t n_pages;
  CopyJob* jobs;  // workspace [n_forks]
  int* status;
  int32_t src[kMaxForks], dst[kMaxForks];
};
static_assert(sizeof(ForkArgs) <= 32764, "kernel parameter block");

__global__ void __launch_bounds__(kThreads) pages_fork_kernel(const __grid_constant__ ForkArgs a) {
  __shared__ int part[32], len[kMaxForks], first[kMaxForks + 1], pre[kMaxForks + 1], fresh[kMaxForks];
  __shared__ int src[kMaxForks], dst[kMaxForks];  // lanes that read parameters at their own place would take turns
  const int f = threadIdx.x;  // a thread a fork where forks are looked at one by one
  const int most = a.max_pages * kPage;
  // ---- sources and destinations: len = rows to fork, or -1 for a refused one; the sources' pages
  //      form one list, shared evenly by the threads --------------------------------------------
  int rows = -1;
  if (f < a.n_forks) {
    src[f] = a.src[f];
    dst[f] = a.dst[f];
    rows = a.seq_len[src[f]];
    if (rows < 0 || rows > most || a.seq_len[dst[f]] != 0) {
      rows = -1;
      set_status(a.status, kDevErrBounds);
    }
    len[f] = rows;
  }
  int pages;
  const int at0 = block_exclusive(rows > 0 ? pages_of(rows) : 0, part, &pages);
  if (f < a.n_forks) first[f] = at0;
  if (f == 0) first[a.n_forks] = pages;
  __syncthreads();
  int g = -1;
  for (int r = threadIdx.x; r < pages; r += kThreads) {
    g = next_owner(first, a.n_forks, r, g);
    const int p = a.table[(int64_t)src[g] * a.max_pages + (r - first[g])];
    if (p < 0 || p >= a.n_pages) {
      set_status(a.status, kDevErrBounds);
      len[g] = -1;
    }
  }
  __syncthreads();
  int total;
  const int need = f < a.n_forks && len[f] > 0 && len[f] % kPage != 0 ? 1 : 0;
  const int at = block_exclusive(need, part, &total);
  if (f < a.n_forks) pre[f] = at;
  if (f == 0) pre[a.n_forks] = total;
  __syncthreads();
  const bool enough = take_free(a.refcount, a.n_pages, total, part, [&](int r, int page) {
    fresh[owner_of(pre, a.n_forks, r)] = page;
  });
  __syncthreads();
  if (!enough && f == 0) set_status(a.status, kDevErrNoPages);
  // ---- the destinations' tables: full pages shared, a fresh one for the partly filled last ------
  g = -1;
  for (int r = threadIdx.x; enough && r < pages; r += kThreads) {
    g = next_owner(first, a.n_forks, r, g);
    if (len[g] < 0) continue;
    const int i = r - first[g], p = a.table[(int64_t)src[g] * a.max_pages + i];
    const bool full = i < len[g] / kPage;
    a.table[(int64_t)dst[g] * a.max_pages + i] = full ? p : fresh[g];
    if (full) {
      atomicAdd(&a.refcount[p], 1);
    } else {
      a.refcount[fresh[g]] = 1;
      a.jobs[g] = CopyJob{p, fresh[g], len[g] % kPage, 0};
    }
  }
  if (f < a.n_forks) {
    if (enough && len[f] >= 0) a.seq_len[dst[f]] = len[f];
    if (!enough || len[f] <= 0 || len[f] % kPage == 0) a.jobs[f] = CopyJob{0, 0, 0, 0};
  }
}

// Copies n 16-byte vectors with the block, six loads of a thread in flight.
__device__ __forceinline__ void copy_vec(const uint4* src, uint4* dst, int n) {
  constexpr int kUnroll = 6;
  for (int i0 = threadIdx.x; i0 < n; i0 += kUnroll * blockDim.x) {
    uint4 v[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u)
      if (i0 + u * (int)blockDim.x < n) v[u] = __ldcs(src + i0 + u * blockDim.x);
#pragma unroll
    for (int u = 0; u < kUnroll; ++u)
      if (i0 + u * (int)blockDim.x < n) __stcs(dst + i0 + u * blockDim.x, v[u]);
  }
}

constexpr int kCopyThreads = 256;

// grid (jobs, layers, parts): a part takes an equal share of the job's vectors
__global__ void __launch_bounds__(kCopyThreads) pages_copy_jobs_kernel(uint4* kv, int64_t layer_vec,
                                                                       const CopyJob* __restrict__ jobs) {
  const CopyJob j = jobs[blockIdx.x];
  const int n = j.rows * kRowVec;
  const int lo = (int)((int64_t)n * blockIdx.z / gridDim.z), hi = (int)((int64_t)n * (blockIdx.z + 1) / gridDim.z);
  uint4* layer = kv + (int64_t)blockIdx.y * layer_vec;
  copy_vec(layer + (int64_t)j.src * kPageVec + lo, layer + (int64_t)j.dst * kPageVec + lo, hi - lo);
}

constexpr int kCopyPairs = 4000;  // pairs of one launch, in its parameters
struct CopyArgs {
  uint4* kv;
  int64_t layer_vec;
  int32_t src[kCopyPairs], dst[kCopyPairs];
};
static_assert(sizeof(CopyArgs) <= 32764, "kernel parameter block");

__global__ void __launch_bounds__(kCopyThreads) pages_copy_kernel(const __grid_constant__ CopyArgs a) {
  const int lo = kPageVec / (int)gridDim.z * (int)blockIdx.z;  // 1, 2, 4, 8 or 16 parts: whole shares
  uint4* layer = a.kv + (int64_t)blockIdx.y * a.layer_vec;
  copy_vec(layer + (int64_t)a.src[blockIdx.x] * kPageVec + lo, layer + (int64_t)a.dst[blockIdx.x] * kPageVec + lo,
           kPageVec / (int)gridDim.z);
}

struct CompactArgs {
  uint4* kv;
  int n_layers, max_pages, max_path;
  int64_t n_pages;
  const int32_t* table;
  const int32_t* base;
  const int32_t* path;
  const int32_t* n_accept;
  int* status;
};
constexpr int kCompactLayers = 4;  // layers of one block

// A thread owns one 16-byte column of a layer's rows, for all rows of the path: since path[k] >= k
// and the path increases, moving k in order never overwrites a row that is still to be read,
// and neither does a batch that is loaded before it is stored.
__global__ void __launch_bounds__(kCompactLayers * kRowVec) pages_compact_kernel(const CompactArgs a) {
  const int s = blockIdx.x;
  const int n = a.n_accept[s], base = a.base[s];
  const int32_t* path = a.path + (int64_t)s * a.max_path;
  const int32_t* row = a.table + (int64_t)s * a.max_pages;
  bool bad = n < 0 || n > a.max_path || base < 0;
  if (!bad)
    for (int k = threadIdx.x; k < n; k += blockDim.x) {
      // path[k] >= k holds on every good path (it starts at 0 or above and increases); asked for by itself,
      // since base + k must lie in the table here even where another thread's step is the bad one
      const int64_t from = (int64_t)base + path[k];
      if (path[k] < k || (k > 0 && path[k] <= path[k - 1]) || from >= (int64_t)a.max_pages * kPage) {
        bad = true;
        break;
      }
      const int p = row[from / kPage], q = row[(base + k) / kPage];
      if (p < 0 || p >= a.n_pages || q < 0 || q >= a.n_pages) bad = true;
    }
  if (__syncthreads_or(bad)) {
    if (threadIdx.x == 0 && blockIdx.y == 0) set_status(a.status, kDevErrBounds);
    return;
  }
  const int layer = (int)blockIdx.y * kCompactLayers + (int)threadIdx.x / kRowVec;
  if (layer >= a.n_layers) return;
  uint4* kv = a.kv + (int64_t)layer * a.n_pages * kPageVec + threadIdx.x % kRowVec;
  auto at = [&](int t) { return kv + ((int64_t)row[t / kPage] * kPage + t % kPage) * kRowVec; };
  constexpr int kBatch = 8;
  for (int k0 = 0; k0 < n; k0 += kBatch) {
    uint4 v[kBatch];
    bool move[kBatch];
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      move[u] = k0 + u < n && path[k0 + u] != k0 + u;
      if (move[u]) v[u] = *at(base + path[k0 + u]);
    }
#pragma unroll
    for (int u = 0; u < kBatch; ++u)
      if (move[u]) *at(base + k0 + u) = v[u];
  }
}

irm_status check_workspace(const void* ws, size_t bytes, size_t need) {
  if (!ws || !aligned(ws, 256) || bytes < need)
    return fail(IRM_ERR_WORKSPACE, "workspace must be 256-byte aligned and hold %zu bytes (got %zu)", need, bytes);
  return IRM_OK;
}

irm_status check_slots(int n_slots, int max_pages, int64_t n_pages) {
  if (n_slots < 1 || n_slots > kMaxSlots) return fail(IRM_ERR_UNSUPPORTED, "n_slots %d outside [1, %d]", n_slots, kMaxSlots);
  if (max_pages < 1 || max_pages > INT32_MAX / kPage) return fail(IRM_ERR_INVALID_ARG, "bad max_pages %d", max_pages);
  if ((int64_t)n_slots * max_pages > kMaxEntries)
    return fail(IRM_ERR_UNSUPPORTED, "a page table of %d x %d has more than 2^30 entries", n_slots, max_pages);
  if (n_pages < 1 || n_pages >= (int64_t(1) << 25)) return fail(IRM_ERR_UNSUPPORTED, "n_pages %lld outside [1, 2^25)", (long long)n_pages);
  return IRM_OK;
}

irm_status check_cache(const void* kv, int n_layers) {
  if (kv == nullptr || !aligned(kv, 16)) return fail(IRM_ERR_INVALID_ARG, "kv must be a 16-byte aligned device pointer");
  if (n_layers < 1 || n_layers > 65535) return fail(IRM_ERR_UNSUPPORTED, "n_layers %d outside [1, 65535]", n_layers);
  return IRM_OK;
}

// Pairs of pages or slots: both in [0, n), destinations distinct and no source of the call.  One
// bit per index, only the touched ones are cleared again.
irm_status check_pairs(const int32_t* src, const int32_t* dst, int m, int64_t n, const char* what) {
  thread_local std::vector<uint64_t> seen;
  try {
    if ((int64_t)seen.size() * 64 < n) seen.resize((size_t)(n + 63) / 64, 0);
  } catch (const std::exception&) {
    return fail(IRM_ERR_INVALID_ARG, "no host memory to check the %s pairs", what);
  }
  irm_status st = IRM_OK;
  int marked = 0;
  for (int i = 0; i < m && st == IRM_OK; ++i) {
    if (src[i] < 0 || src[i] >= n || dst[i] < 0 || dst[i] >= n) {
      st = fail(IRM_ERR_INVALID_ARG, "pair %d: %s %d -> %d outside [0, %lld)", i, what, src[i], dst[i], (long long)n);
      break;
    }
    uint64_t& w = seen[dst[i] >> 6];
    const uint64_t bit = 1ull << (dst[i] & 63);
    if (w & bit) {
      st = fail(IRM_ERR_INVALID_ARG, "pair %d: %s %d is a destination twice", i, what, dst[i]);
      break;
    }
    w |= bit;
    marked = i + 1;
  }
  for (int i = 0; i < m && st == IRM_OK; ++i)
    if (seen[src[i] >> 6] >> (src[i] & 63) & 1)
      st = fail(IRM_ERR_INVALID_ARG, "pair %d: %s %d is a source and a destination", i, what, src[i]);
  for (int i = 0; i < marked; ++i) seen[dst[i] >> 6] = 0;
  return st;
}

// The resize kernel's dynamic shared memory limit belongs to the device: raised once on each, for
// more slots than fit by default.
cudaError_t raise_resize_smem() {
  static std::mutex mu;
  static bool done[128];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  std::lock_guard<std::mutex> lk(mu);
  if (dev >= 0 && dev < 128 && done[dev]) return cudaSuccess;
  e = cudaFuncSetAttribute(pages_resize_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                           (int)((2 * kMaxSlots + 1) * sizeof(int)));
  if (e == cudaSuccess && dev >= 0 && dev < 128) done[dev] = true;
  return e;
}

size_t workspace_need() { return IRM_WORKSPACE_HEADER + kMaxForks * sizeof(CopyJob); }

// Shares of a page that make a few thousand blocks where there are few pages to copy (16 at most,
// 288 vectors each), one where there are many.
int copy_parts(int64_t blocks) {
  int parts = 1;
  while (parts < 16 && blocks * parts < 2432) parts *= 2;  // 152 SMs x 8 resident blocks x 2
  return parts;
}

}  // namespace
}  // namespace irm

extern "C" {

irm_status irm_pages_workspace_size(int n_slots, size_t* bytes) {
  if (bytes == nullptr) return irm::fail(IRM_ERR_INVALID_ARG, "bytes is null");
  if (n_slots < 1 || n_slots > irm::kMaxSlots)
    return irm::fail(IRM_ERR_UNSUPPORTED, "n_slots %d outside [1, %d]", n_slots, irm::kMaxSlots);
  *bytes = irm::workspace_need();
  return IRM_OK;
}

irm_status irm_pages_resize(const int32_t* new_len, int32_t* seq_len, int n_slots, int32_t* page_table, int max_pages,
                            int32_t* refcount, int64_t n_pages, void* workspace, size_t workspace_bytes,
                            cudaStream_t stream) {
  using namespace irm;
  irm_status st = check_slots(n_slots, max_pages, n_pages);
  if (st != IRM_OK) return st;
  if (!new_len || !seq_len || !page_table || !refcount) return fail(IRM_ERR_INVALID_ARG, "null device pointer");
  if (!aligned(new_len, 4) || !aligned(seq_len, 4) || !aligned(page_table, 4) || !aligned(refcount, 4))
    return fail(IRM_ERR_INVALID_ARG, "misaligned device pointer");
  if ((st = check_workspace(workspace, workspace_bytes, workspace_need())) != IRM_OK) return st;
  const ResizeArgs a{new_len, seq_len, n_slots, max_pages, page_table, refcount, n_pages, static_cast<int*>(workspace)};
  const size_t smem = (size_t)(2 * n_slots + 1) * sizeof(int);
  cudaError_t e = smem > 40960 ? raise_resize_smem() : cudaSuccess;
  if (e != cudaSuccess) return cuda_fail(e, "page resize set-up");
  pages_resize_kernel<<<1, kThreads, smem, stream>>>(a);
  e = cudaGetLastError();
  return e == cudaSuccess ? IRM_OK : cuda_fail(e, "page resize launch");
}

irm_status irm_pages_fork(const int32_t* src_host, const int32_t* dst_host, int n_forks, void* kv, int n_layers,
                          int32_t* seq_len, int n_slots, int32_t* page_table, int max_pages, int32_t* refcount,
                          int64_t n_pages, void* workspace, size_t workspace_bytes, cudaStream_t stream) {
  using namespace irm;
  irm_status st = check_slots(n_slots, max_pages, n_pages);
  if (st != IRM_OK) return st;
  if (n_forks < 0 || n_forks > kMaxForks) return fail(IRM_ERR_UNSUPPORTED, "n_forks %d outside [0, %d]", n_forks, kMaxForks);
  if ((n_forks > 0 && (!src_host || !dst_host)) || !seq_len || !page_table || !refcount)
    return fail(IRM_ERR_INVALID_ARG, "null pointer");
  if (!aligned(seq_len, 4) || !aligned(page_table, 4) || !aligned(refcount, 4))
    return fail(IRM_ERR_INVALID_ARG, "misaligned device pointer");
  if ((st = check_cache(kv, n_layers)) != IRM_OK) return st;
  if ((st = check_pairs(src_host, dst_host, n_forks, n_slots, "slot")) != IRM_OK) return st;
  if ((st = check_workspace(workspace, workspace_bytes, workspace_need())) != IRM_OK) return st;
  if (n_forks == 0) return IRM_OK;
  ForkArgs a;
  a.seq_len = seq_len;
  a.n_slots = n_slots;
  a.max_pages = max_pages;
  a.n_forks = n_forks;
  a.table = page_table;
  a.refcount = refcount;
  a.n_pages = n_pages;
  a.jobs = reinterpret_cast<CopyJob*>(static_cast<uint8_t*>(workspace) + IRM_WORKSPACE_HEADER);
  a.status = static_cast<int*>(workspace);
  std::memcpy(a.src, src_host, (size_t)n_forks * sizeof(int32_t));
  std::memcpy(a.dst, dst_host, (size_t)n_forks * sizeof(int32_t));
  std::memset(a.src + n_forks, 0, (size_t)(kMaxForks - n_forks) * sizeof(int32_t));
  std::memset(a.dst + n_forks, 0, (size_t)(kMaxForks - n_forks) * sizeof(int32_t));
  pages_fork_kernel<<<1, kThreads, 0, stream>>>(a);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return cuda_fail(e, "page fork launch");
  const dim3 grid((unsigned)n_forks, (unsigned)n_layers, (unsigned)copy_parts((int64_t)n_forks * n_layers));
  pages_copy_jobs_kernel<<<grid, kCopyThreads, 0, stream>>>(static_cast<uint4*>(kv), n_pages * kPageVec, a.jobs);
  e = cudaGetLastError();
  return e == cudaSuccess ? IRM_OK : cuda_fail(e, "page copy launch");
}

irm_status irm_pages_compact(void* kv, int n_layers, int64_t n_pages, const int32_t* page_table, int max_pages,
                             int n_slots, const int32_t* base, const int32_t* path, int max_path,
                             const int32_t* n_accept, void* workspace, size_t workspace_bytes, cudaStream_t stream) {
  using namespace irm;
  irm_status st = check_slots(n_slots, max_pages, n_pages);
  if (st != IRM_OK) return st;
  if (max_path < 1) return fail(IRM_ERR_INVALID_ARG, "max_path must be positive");
  if (!page_table || !base || !path || !n_accept) return fail(IRM_ERR_INVALID_ARG, "null device pointer");
  if (!aligned(page_table, 4) || !aligned(base, 4) || !aligned(path, 4) || !aligned(n_accept, 4))
    return fail(IRM_ERR_INVALID_ARG, "misaligned device pointer");
  if ((st = check_cache(kv, n_layers)) != IRM_OK) return st;
  if ((st = check_workspace(workspace, workspace_bytes, IRM_WORKSPACE_HEADER)) != IRM_OK) return st;
  const CompactArgs a{static_cast<uint4*>(kv), n_layers, max_pages, max_path, n_pages, page_table, base, path, n_accept,
                      static_cast<int*>(workspace)};
  const dim3 grid((unsigned)n_slots, (unsigned)((n_layers + kCompactLayers - 1) / kCompactLayers));
  pages_compact_kernel<<<grid, kCompactLayers * kRowVec, 0, stream>>>(a);
  const cudaError_t e = cudaGetLastError();
  return e == cudaSuccess ? IRM_OK : cuda_fail(e, "page compaction launch");
}

irm_status irm_pages_copy(void* kv, int n_layers, int64_t n_pages, const int32_t* src_host, const int32_t* dst_host,
                          int n, cudaStream_t stream) {
  using namespace irm;
  irm_status st = check_slots(1, 1, n_pages);
  if (st != IRM_OK) return st;
  if (n < 0) return fail(IRM_ERR_INVALID_ARG, "n must not be negative");
  if (n > 0 && (!src_host || !dst_host)) return fail(IRM_ERR_INVALID_ARG, "null pointer");
  if ((st = check_cache(kv, n_layers)) != IRM_OK) return st;
  if ((st = check_pairs(src_host, dst_host, n, n_pages, "page")) != IRM_OK) return st;
  thread_local CopyArgs a;  // 32 KB: kept off the stack
  a.kv = static_cast<uint4*>(kv);
  a.layer_vec = n_pages * kPageVec;
  for (int i0 = 0; i0 < n; i0 += kCopyPairs) {
    const int m = n - i0 < kCopyPairs ? n - i0 : kCopyPairs;
    std::memcpy(a.src, src_host + i0, (size_t)m * sizeof(int32_t));
    std::memcpy(a.dst, dst_host + i0, (size_t)m * sizeof(int32_t));
    const dim3 grid((unsigned)m, (unsigned)n_layers, (unsigned)copy_parts((int64_t)m * n_layers));
    pages_copy_kernel<<<grid, kCopyThreads, 0, stream>>>(a);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return cuda_fail(e, "page copy launch");
  }
  return IRM_OK;
}

}  // extern "C"
