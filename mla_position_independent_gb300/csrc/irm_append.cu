// New rows into the paged cache (bf16 or 8-bit) with the position rotation on the way, and the
// rotation of queries.
//
//   R(p) turns pair j by p theta_j (irm_rope); the angle is reduced to one turn in exact integer
//   arithmetic for every int32 p, so far positions lose nothing.  cos and sin are multiplied by
//   `factor` (the magnitude that tables scaled for long contexts bring along); the pair is turned in
//   fp32 and rounded to bf16 once.
//   8-bit rows: for each 128 columns e is the smallest exponent with max |c| <= 448 2^e, in [-126, 7];
//   code = e4m3(c 2^-e), to the nearest even, at most 448 in magnitude.  A power of two as scale costs
//   a floating code nothing (its steps are relative), and makes code x scale exact in bf16 (at the least scales
//   too: the values are multiples of bf16's least step, 2^-133, and so is what rounding to a code makes of them): what
//   attention reads is the code's value, rounded nowhere.  The maximum is compared by its
//   bits, so NaN and infinity count as larger than every number; such a group's scale is NaN.
//
// What bounds them: the bytes (1152 in and 656 or 1152 out a token, 256 a query row), and for few tokens
// the launch.  Append: a warp a token, two 16-byte loads of cKV and one pair of k_r a lane, in flight
// together; a lane's 16 columns are one 16-byte store of codes and 8 lanes a group's maximum.  64
// tokens take 2.1 us, 8191 4.6 (8-bit), 16384 6.6 (bf16: 5.8 TB/s, 0.86 of the measured copy), 262144 104 (bf16,
// 5.8 TB/s) and 95 us (8-bit, 5.0 TB/s: in any order of the tokens, rows of 20.5 sectors meet inside
// one that is written twice).  Two tokens a warp: 114 and 108 us.
// Queries: a block takes 256 (token, head) rows, computes each token's 32 (cos, sin) once for
// all its heads, and has 8 16-byte loads a thread in flight: 8192 x 128 rows out of [T, H, 192] in 43.1 us
// (6.2 TB/s, 0.92 of the copy).
#include <cuda_runtime.h>
#include <cmath>
#include <cstdint>
#include <cstring>

#include "irm_common.cuh"
#include "irm_host_util.h"

namespace irm {
namespace {

constexpr uint32_t kFull = 0xffffffffu;
constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kRow8 = IRM_ROW_BYTES8;

struct AppendArgs {
  const uint8_t* c_kv;
  const uint8_t* k_rope;
  int64_t c_stride, k_stride;  // bytes
  int64_t n_tokens;
  uint8_t* kv;
  int64_t n_pages;
  const int32_t* table;
  int n_slots, max_pages;
  const int32_t* row;
  const int32_t* request;
  const int32_t* position;
  int encoded, interleaved;
  float factor;
  int* status;
  RopePhase phase;
};

// Exponent of the scale of a group whose largest magnitude has these fp32 bits (finite).
__device__ __forceinline__ int scale_exponent(uint32_t bits) {
  if (bits == 0) return 0;
  const int e = (int)(bits >> 23) - 127 - 8 + ((bits & 0x7fffffu) > 0x600000u ? 1 : 0);  // 448 = 1.75 x 2^8
  return max(-126, min(7, e));
}

// Two e4m3 codes, `a` in the low byte.
__device__ __forceinline__ uint32_t e4m3_pair(float a, float b) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(b), "f"(a));
  return r;
}

template <bool CODES>
__global__ void __launch_bounds__(kThreads) pages_append_kernel(const __grid_constant__ AppendArgs a) {
  const int lane = threadIdx.x & 31;
  const int64_t t = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5);
  if (t >= a.n_tokens) return;
  const uint8_t* c = a.c_kv + t * a.c_stride;
  const uint8_t* k = a.k_rope + t * a.k_stride;
  // a lane's columns: 16 neighbouring ones (codes), or two vectors 32 apart
  const uint4 v0 = __ldcs(reinterpret_cast<const uint4*>(c) + (CODES ? 2 * lane : lane));
  const uint4 v1 = __ldcs(reinterpret_cast<const uint4*>(c) + (CODES ? 2 * lane + 1 : lane + 32));
  // its pair of k_r
  uint32_t pair;
  if (a.interleaved) {
    pair = reinterpret_cast<const uint32_t*>(k)[lane];
  } else {
    const uint16_t* h = reinterpret_cast<const uint16_t*>(k);
    pair = (uint32_t)h[lane] | (uint32_t)h[lane + 32] << 16;
  }
  const int row = a.row[t];
  if (row < 0) return;  // a token that has no row
  const int64_t s = a.request != nullptr ? (int64_t)a.request[t] : t;
  int page = -1;
  if (s >= 0 && s < a.n_slots && row / kPage < a.max_pages) page = a.table[s * a.max_pages + row / kPage];
  if (page < 0 || page >= a.n_pages) {
    if (lane == 0) set_status(a.status, kDevErrBounds);
    return;
  }
  uint8_t* dst = a.kv + ((int64_t)page * kPage + row % kPage) * (CODES ? kRow8 : 2 * kDRow);
  // ---- k_r ----
  if (!a.encoded) {
    float cs, sn;
    rope_cos_sin(a.position != nullptr ? a.position[t] : row, a.phase.F[lane], cs, sn);
    cs *= a.factor;
    sn *= a.factor;
    const float x = __uint_as_float(pair << 16), y = __uint_as_float(pair & 0xffff0000u);
    const __nv_bfloat162 r = __floats2bfloat162_rn(fmaf(x, cs, -y * sn), fmaf(x, sn, y * cs));
    pair = *reinterpret_cast<const uint32_t*>(&r);
  }
  uint8_t* kd = dst + (CODES ? IRM_ROW8_ROPE : 2 * kDLat);
  if (a.interleaved) {
    reinterpret_cast<uint32_t*>(kd)[lane] = pair;
  } else {
    reinterpret_cast<uint16_t*>(kd)[lane] = (uint16_t)pair;
    reinterpret_cast<uint16_t*>(kd)[lane + 32] = (uint16_t)(pair >> 16);
  }
  // ---- cKV ----
  if (!CODES) {
    reinterpret_cast<uint4*>(dst)[lane] = v0;
    reinterpret_cast<uint4*>(dst)[lane + 32] = v1;
    return;
  }
  const uint32_t w[8] = {v0.x, v0.y, v0.z, v0.w, v1.x, v1.y, v1.z, v1.w};
  uint32_t most = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) most = max(most, max(w[i] << 16 & 0x7fffffffu, w[i] & 0x7fff0000u));
#pragma unroll
  for (int o = 1; o < 8; o <<= 1) most = max(most, __shfl_xor_sync(kFull, most, o));
  const bool finite = most < 0x7f800000u;
  const int e = finite ? scale_exponent(most) : 0;
  const uint32_t scale = finite ? (uint32_t)(e + 127) << 23 : 0x7fc00000u;
  const float inv = __uint_as_float((uint32_t)(127 - e) << 23);
  uint32_t q[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t lo = e4m3_pair(__uint_as_float(w[2 * i] << 16) * inv, __uint_as_float(w[2 * i] & 0xffff0000u) * inv);
    const uint32_t hi = e4m3_pair(__uint_as_float(w[2 * i + 1] << 16) * inv, __uint_as_float(w[2 * i + 1] & 0xffff0000u) * inv);
    q[i] = finite ? lo | hi << 16 : 0u;
  }
  reinterpret_cast<uint4*>(dst)[lane] = make_uint4(q[0], q[1], q[2], q[3]);
  if ((lane & 7) == 0) *reinterpret_cast<uint32_t*>(dst + IRM_ROW8_SCALES + (lane >> 1)) = scale;
}

struct RopeArgs {
  const uint8_t* x;
  uint8_t* out;
  int64_t xt, xh, ot, oh;  // strides in bytes
  int64_t n_tokens;
  int H, hb, tb;           // heads, and heads and tokens of a block
  const int32_t* position;
  int interleaved;
  float factor;
  RopePhase phase;
};

constexpr int kRopeRows = 256;    // (token, head) rows of a block
constexpr int kRopeTokens = 32;   // at most

// Four lanes a row: lane p takes the vectors p and p + 4 (8 pairs in either pairing).
__global__ void __launch_bounds__(kThreads) rope_apply_kernel(const __grid_constant__ RopeArgs a) {
  __shared__ float cs[kRopeTokens][32], sn[kRopeTokens][32];
  const int tid = threadIdx.x;
  const int64_t t0 = (int64_t)blockIdx.x * a.tb;
  const int h0 = (int)blockIdx.y * a.hb;
  const int nt = (int)min((int64_t)a.tb, a.n_tokens - t0), nh = min(a.hb, a.H - h0);
  const int rows = nt * nh;
  constexpr int kPer = kRopeRows * 4 / kThreads;
  uint4 x[kPer], y[kPer];
#pragma unroll
  for (int u = 0; u < kPer; ++u) {
    const int r = (u * kThreads + tid) >> 2, p = tid & 3;
    if (r < rows) {
      const uint4* src = reinterpret_cast<const uint4*>(a.x + (t0 + r / nh) * a.xt + (int64_t)(h0 + r % nh) * a.xh);
      x[u] = src[p];
      y[u] = src[p + 4];
    }
  }
  for (int i = tid; i < nt * 32; i += kThreads) {
    float c, s;
    rope_cos_sin(a.position[t0 + (i >> 5)], a.phase.F[i & 31], c, s);
    cs[i >> 5][i & 31] = c * a.factor;
    sn[i >> 5][i & 31] = s * a.factor;
  }
  __syncthreads();
#pragma unroll
  for (int u = 0; u < kPer; ++u) {
    const int r = (u * kThreads + tid) >> 2, p = tid & 3;
    if (r < rows) {
      const int t = r / nh;
      float c8[8], s8[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const int j = pair_index(a.interleaved, p, p + 4, e);
        c8[e] = cs[t][j];
        s8[e] = sn[t][j];
      }
      rotate_pairs8_any(x[u], y[u], c8, s8, a.interleaved);
      uint4* dst = reinterpret_cast<uint4*>(a.out + (t0 + t) * a.ot + (int64_t)(h0 + r % nh) * a.oh);
      dst[p] = x[u];
      dst[p + 4] = y[u];
    }
  }
}

// Rows of bf16 that vectors of 16 bytes may read.
bool vector_rows(const void* p, int64_t stride) { return aligned(p, 16) && stride % 8 == 0; }

template <bool CODES>
irm_status append(const void* c_kv, int64_t c_stride, const void* k_rope, int64_t k_stride, int64_t n_tokens, void* kv,
                  int64_t n_pages, const int32_t* page_table, int n_slots, int max_pages, const int32_t* row,
                  const int32_t* request, const int32_t* position, const irm_rope* rope, float factor, int encoded,
                  void* workspace, size_t workspace_bytes, cudaStream_t stream) {
  if (n_tokens < 0 || n_tokens > INT32_MAX) return fail(IRM_ERR_INVALID_ARG, "n_tokens %lld outside [0, 2^31)", (long long)n_tokens);
  if (n_slots < 1) return fail(IRM_ERR_INVALID_ARG, "n_slots must be positive");
  if (max_pages < 1 || max_pages > INT32_MAX / kPage) return fail(IRM_ERR_INVALID_ARG, "bad max_pages %d", max_pages);
  if (n_pages < 1 || n_pages >= (int64_t(1) << 25)) return fail(IRM_ERR_UNSUPPORTED, "n_pages %lld outside [1, 2^25)", (long long)n_pages);
  if (request == nullptr && n_tokens > n_slots)
    return fail(IRM_ERR_INVALID_ARG, "%lld tokens without requests, but %d slots", (long long)n_tokens, n_slots);
  if (!c_kv || !k_rope || !kv || !page_table || !row) return fail(IRM_ERR_INVALID_ARG, "null device pointer");
  if (!vector_rows(c_kv, c_stride) || !vector_rows(k_rope, k_stride))
    return fail(IRM_ERR_INVALID_ARG, "rows of c_kv and k_rope must start on 16 bytes");
  if (n_tokens > 1 && (c_stride < kDLat || k_stride < kDRope)) return fail(IRM_ERR_INVALID_ARG, "rows of c_kv or k_rope overlap");
  if (!aligned(kv, 16)) return fail(IRM_ERR_INVALID_ARG, "kv must be 16-byte aligned");
  for (const void* p : {(const void*)page_table, (const void*)row, (const void*)request, (const void*)position})
    if (!aligned(p, 4)) return fail(IRM_ERR_INVALID_ARG, "misaligned device pointer");
  if (encoded != 0 && encoded != 1) return fail(IRM_ERR_INVALID_ARG, "encoded must be 0 or 1");
  if (!encoded && !std::isfinite(factor)) return fail(IRM_ERR_INVALID_ARG, "factor must be finite");
  if (!workspace || !aligned(workspace, 256) || workspace_bytes < IRM_WORKSPACE_HEADER)
    return fail(IRM_ERR_WORKSPACE, "workspace must be 256-byte aligned and hold %d bytes", IRM_WORKSPACE_HEADER);
  AppendArgs a{};
  if (!encoded) {
    const irm_status st = select_rope(rope, a.phase.F, &a.interleaved);
    if (st != IRM_OK) return st;
  }
  if (n_tokens == 0) return IRM_OK;
  a.c_kv = static_cast<const uint8_t*>(c_kv);
  a.k_rope = static_cast<const uint8_t*>(k_rope);
  a.c_stride = 2 * c_stride;
  a.k_stride = 2 * k_stride;
  a.n_tokens = n_tokens;
  a.kv = static_cast<uint8_t*>(kv);
  a.n_pages = n_pages;
  a.table = page_table;
  a.n_slots = n_slots;
  a.max_pages = max_pages;
  a.row = row;
  a.request = request;
  a.position = position;
  a.encoded = encoded;
  a.factor = factor;
  a.status = static_cast<int*>(workspace);
  pages_append_kernel<CODES><<<(unsigned)((n_tokens + kWarps - 1) / kWarps), kThreads, 0, stream>>>(a);
  const cudaError_t e = cudaGetLastError();
  return e == cudaSuccess ? IRM_OK : cuda_fail(e, "page append launch");
}

}  // namespace
}  // namespace irm

extern "C" {

irm_status irm_pages_append(const void* c_kv, int64_t c_stride, const void* k_rope, int64_t k_stride, int64_t n_tokens,
                            void* kv, int64_t n_pages, const int32_t* page_table, int n_slots, int max_pages,
                            const int32_t* row, const int32_t* request, const int32_t* position, const irm_rope* rope,
                            float factor, int encoded, void* workspace, size_t workspace_bytes, cudaStream_t stream) {
  return irm::append<false>(c_kv, c_stride, k_rope, k_stride, n_tokens, kv, n_pages, page_table, n_slots, max_pages, row,
                            request, position, rope, factor, encoded, workspace, workspace_bytes, stream);
}

irm_status irm_pages_append8(const void* c_kv, int64_t c_stride, const void* k_rope, int64_t k_stride, int64_t n_tokens,
                             void* kv, int64_t n_pages, const int32_t* page_table, int n_slots, int max_pages,
                             const int32_t* row, const int32_t* request, const int32_t* position, const irm_rope* rope,
                             float factor, int encoded, void* workspace, size_t workspace_bytes, cudaStream_t stream) {
  return irm::append<true>(c_kv, c_stride, k_rope, k_stride, n_tokens, kv, n_pages, page_table, n_slots, max_pages, row,
                           request, position, rope, factor, encoded, workspace, workspace_bytes, stream);
}

irm_status irm_rope_apply(const void* x, int64_t x_token, int64_t x_head, int64_t n_tokens, int n_heads,
                          const int32_t* position, const irm_rope* rope, float factor, void* out, int64_t out_token,
                          int64_t out_head, cudaStream_t stream) {
  using namespace irm;
  if (n_tokens < 0 || n_tokens > INT32_MAX) return fail(IRM_ERR_INVALID_ARG, "n_tokens %lld outside [0, 2^31)", (long long)n_tokens);
  if (n_heads < 1 || n_heads > 65535) return fail(IRM_ERR_UNSUPPORTED, "n_heads %d outside [1, 65535]", n_heads);
  if (!x || !out || !position) return fail(IRM_ERR_INVALID_ARG, "null device pointer");
  if (!aligned(x, 16) || !aligned(out, 16) || (x_token | x_head | out_token | out_head) % 8 != 0)
    return fail(IRM_ERR_INVALID_ARG, "rows of x and out must start on 16 bytes");
  // one of the strides steps over all of the other's rows
  if ((n_heads > 1 && out_head < kDRope) || (n_tokens > 1 && out_token < kDRope) ||
      (n_heads > 1 && n_tokens > 1 && (__int128)out_head * (n_heads - 1) + kDRope > out_token &&
       (__int128)out_token * (n_tokens - 1) + kDRope > out_head))
    return fail(IRM_ERR_INVALID_ARG, "rows of out overlap");
  if (!aligned(position, 4)) return fail(IRM_ERR_INVALID_ARG, "misaligned device pointer");
  if (!std::isfinite(factor)) return fail(IRM_ERR_INVALID_ARG, "factor must be finite");
  RopeArgs a{};
  const irm_status st = select_rope(rope, a.phase.F, &a.interleaved);
  if (st != IRM_OK) return st;
  if (n_tokens == 0) return IRM_OK;
  a.x = static_cast<const uint8_t*>(x);
  a.out = static_cast<uint8_t*>(out);
  a.xt = 2 * x_token;
  a.xh = 2 * x_head;
  a.ot = 2 * out_token;
  a.oh = 2 * out_head;
  a.n_tokens = n_tokens;
  a.H = n_heads;
  a.hb = n_heads < kRopeRows ? n_heads : kRopeRows;
  a.tb = kRopeRows / a.hb < kRopeTokens ? kRopeRows / a.hb : kRopeTokens;
  a.position = position;
  a.factor = factor;
  const dim3 grid((unsigned)((n_tokens + a.tb - 1) / a.tb), (unsigned)((n_heads + a.hb - 1) / a.hb));
  rope_apply_kernel<<<grid, kThreads, 0, stream>>>(a);
  const cudaError_t e = cudaGetLastError();
  return e == cudaSuccess ? IRM_OK : cuda_fail(e, "rotation launch");
}

}  // extern "C"
