// kv_cache.cu -- operators on the KV cache itself: quantised append (q4_0),
// the choice of the positions that stay when a cache is cut down, and the
// move of their rows.  Only the attention layers "grow a KV cache" ("The Hybrid
// Attention in Qwen3.8-27B"); these bound what it costs.
#include <cuda_fp16.h>
#include <math.h>

#include "common.cuh"
#include "internal.h"

namespace hh {

namespace {

// ---------------------------------------------------------------------------
// kv_append_q4_0.  A thread holds 8 consecutive elements of a row (one 16-byte
// load); four neighbouring threads hold a block of 32.
// ---------------------------------------------------------------------------
constexpr int kAppendThreads = 256;

__global__ void __launch_bounds__(kAppendThreads) kv_append_q4_kernel(const __grid_constant__ KvAppendQ4Args p) {
  const int b = blockIdx.y;
  const bool is_v = blockIdx.z != 0;
  const uint32_t row_units = (uint32_t)p.H_kv * p.d / 8;  // 16-byte units of one token
  const uint32_t u = blockIdx.x * kAppendThreads + threadIdx.x;
  const uint32_t tok = u / row_units, col = u - tok * row_units;
  int n_new = p.n_new ? p.n_new[b] : p.n;
  n_new = n_new < 0 ? 0 : (n_new > p.n ? p.n : n_new);
  const long long len = p.cache_len ? p.cache_len[b] : p.T_cache;
  const long long pos = len - n_new + tok;
  const bool live = tok < (uint32_t)n_new && pos >= 0 && pos < p.T_cache;
  uint32_t w[4] = {0, 0, 0, 0};
  const size_t src = ((size_t)b * p.n + tok) * row_units + col;
  if (live) {
    const uint4 x = __ldg(reinterpret_cast<const uint4 *>(is_v ? p.v : p.k) + src);
    w[0] = x.x, w[1] = x.y, w[2] = x.z, w[3] = x.w;
  }
  // The element of largest magnitude as an integer maximum: bf16 magnitudes order as their bit patterns;
  // below them the block position reversed (the first one wins a tie), then the sign, which only rides along.
  const uint32_t first = 31u - (threadIdx.x & 3) * 8u;
  uint32_t best = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint32_t e = (w[i >> 1] >> ((i & 1) * 16)) & 0xFFFFu;
    best = max(best, ((e & 0x7FFFu) << 6) | ((first - i) << 1) | (e >> 15));
  }
  best = max(best, __shfl_xor_sync(0xffffffffu, best, 1));
  best = max(best, __shfl_xor_sync(0xffffffffu, best, 2));
  const uint32_t mag = best >> 6;
  const float m = __uint_as_float((mag << 16) | (best << 31));
  const bool bad = mag >= 0x7F80u;  // an infinity or a NaN in the block
  // bf16 / 8 is exact in fp32, so the scale is rounded once, to fp16 (11 bits, as the format stores it)
  __half s = __float2half_rn(fminf(fmaxf(m * -0.125f, -65504.f), 65504.f));
  if (bad) s = __ushort_as_half((unsigned short)0x7FFFu);
  const float sf = __half2float(s);
  if (sf == 0.f) s = __ushort_as_half((unsigned short)0);
  // x has 8 significant bits and s has 11: x / s is a tie or at least 2^-16 (relative) away from one, so the
  // fp32 quotient rounds to the code that the exact one gives
  uint32_t codes = 0;
  float held[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint32_t e = w[i >> 1];
    const float x = (i & 1) ? bf16_hi(e) : bf16_lo(e);
    float c = 0.f;
    if (!bad && sf != 0.f) c = fminf(fmaxf(rintf(__fdiv_rn(x, sf)), -8.f), 7.f);
    codes |= (uint32_t)((int)c + 8) << (4 * i);
    held[i] = sf * c;
  }
  if (!live) return;
  const size_t dst = ((size_t)b * p.T_cache + (size_t)pos) * row_units + col;
  reinterpret_cast<uint32_t *>(is_v ? p.v_values : p.k_values)[dst] = codes;
  if ((threadIdx.x & 3) == 0) (is_v ? p.v_scales : p.k_scales)[dst >> 2] = __half_as_ushort(s);
  bf16_t *h = is_v ? p.v_held : p.k_held;
  if (h)
    reinterpret_cast<uint4 *>(h)[src] = make_uint4(pack_bf16(held[0], held[1]), pack_bf16(held[2], held[3]),
                                                   pack_bf16(held[4], held[5]), pack_bf16(held[6], held[7]));
}

// ---------------------------------------------------------------------------
// kv_evict_select.  One CTA per (sequence, kv head).  Weights map to 32-bit
// keys that order as the weights do; the last n_recent positions get the
// largest key.  A radix selection (four passes of 8 bits) finds the key of the
// n_keep-th largest and how many positions of exactly that key stay; a last
// pass writes the positions in order.
// ---------------------------------------------------------------------------
constexpr int kSelThreads = 512;
constexpr int kSelWarps = kSelThreads / 32;

__device__ __forceinline__ uint32_t weight_key(float w) {
  if (w != w) return 0xFFFFFFFEu;                  // a NaN above every number
  const uint32_t u = __float_as_uint(w + 0.f);     // -0 becomes +0
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

__global__ void __launch_bounds__(kSelThreads) kv_select_kernel(const __grid_constant__ KvSelectArgs p) {
  __shared__ uint32_t hist[256];
  __shared__ uint32_t warp_cnt[2][kSelWarps];
  __shared__ uint32_t s_prefix, s_need;
  const int b = blockIdx.y, h = blockIdx.x, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  int len = p.cache_len ? p.cache_len[b] : p.T_cache;
  len = len < 0 ? 0 : (len > p.T_cache ? p.T_cache : len);
  const float *acc = p.acc + ((size_t)b * p.H_kv + h) * p.T_cache;
  int32_t *keep = p.keep + ((size_t)b * p.H_kv + h) * p.n_keep;
  const int n_out = min(len, p.n_keep);
  for (int i = n_out + tid; i < p.n_keep; i += kSelThreads) keep[i] = -1;
  if (len <= p.n_keep) {
    for (int i = tid; i < len; i += kSelThreads) keep[i] = i;
    return;
  }
  const int recent_from = len - p.n_recent;  // > 0: n_recent <= n_keep < len
  auto key_at = [&](int i) { return i >= recent_from ? 0xFFFFFFFFu : weight_key(acc[i]); };
  // key of the n_keep-th largest position
  uint32_t prefix = 0, mask = 0, need = p.n_keep;
  for (int shift = 24; shift >= 0; shift -= 8) {
    if (tid < 256) hist[tid] = 0;
    __syncthreads();
    for (int i = tid; i < len; i += kSelThreads) {
      const uint32_t k = key_at(i);
      if ((k & mask) == prefix) atomicAdd(&hist[(k >> shift) & 255u], 1u);
    }
    __syncthreads();
    if (tid == 0) {
      uint32_t left = need;
      int d = 255;
      while (d > 0 && hist[d] < left) left -= hist[d--];
      s_prefix = prefix | ((uint32_t)d << shift);
      s_need = left;
    }
    __syncthreads();
    prefix = s_prefix;
    need = s_need;
    mask |= 255u << shift;
  }
  // positions above the key, and the first `need` of those that have exactly it, in order
  uint32_t base_gt = 0, base_eq = 0;
  for (int i0 = 0; i0 < len; i0 += kSelThreads) {
    const int i = i0 + tid;
    const uint32_t k = i < len ? key_at(i) : 0u;
    const bool gt = i < len && k > prefix, eq = i < len && k == prefix;
    const uint32_t bg = __ballot_sync(0xffffffffu, gt), be = __ballot_sync(0xffffffffu, eq);
    if (lane == 0) warp_cnt[0][warp] = __popc(bg), warp_cnt[1][warp] = __popc(be);
    __syncthreads();
    uint32_t g = base_gt, e = base_eq;
    for (int w = 0; w < kSelWarps; ++w) {
      if (w < warp) g += warp_cnt[0][w], e += warp_cnt[1][w];
      base_gt += warp_cnt[0][w];
      base_eq += warp_cnt[1][w];
    }
    const uint32_t below = (1u << lane) - 1u;
    g += __popc(bg & below);
    e += __popc(be & below);
    if (gt || (eq && e < need)) keep[g + min(e, need)] = i;
    __syncthreads();
  }
}

// ---------------------------------------------------------------------------
// kv_compact.  One CTA per (sequence, kv head, array) moves the kept rows in
// chunks: a chunk is read whole before any of it is written, and entry i comes
// from a position >= i, so that later chunks still find their rows in place
// when the array is compacted in place.
// ---------------------------------------------------------------------------
constexpr int kMoveThreads = 256;

__global__ void __launch_bounds__(kMoveThreads) kv_compact_kernel(const __grid_constant__ KvCompactArgs p) {
  const int h = blockIdx.x, b = blockIdx.y, a = blockIdx.z, tid = threadIdx.x;
  const int32_t *keep = p.keep + ((size_t)b * p.H_kv + h) * p.n_keep;
  if (a == p.n_arrays) {  // the weights, one 4-byte element a position
    const float *src = p.acc_src + ((size_t)b * p.H_kv + h) * p.T_src;
    float *dst = p.acc_dst + ((size_t)b * p.H_kv + h) * p.T_dst;
    for (int i0 = 0; i0 < p.T_dst; i0 += kMoveThreads) {
      const int i = i0 + tid;
      const int at = i < p.n_keep ? keep[i] : -1;
      const float x = at >= 0 && at < p.T_src ? src[at] : 0.f;
      __syncthreads();
      if (i < p.T_dst) dst[i] = x;
    }
    return;
  }
  const int per_row = p.row_bytes[a] / 8;
  const uint2 *src = reinterpret_cast<const uint2 *>(p.src[a]) + ((size_t)b * p.T_src * p.H_kv + h) * per_row;
  uint2 *dst = reinterpret_cast<uint2 *>(p.dst[a]) + ((size_t)b * p.T_dst * p.H_kv + h) * per_row;
  const size_t stride = (size_t)p.H_kv * per_row;
  const long long total = (long long)p.n_keep * per_row;
  for (long long j0 = 0; j0 < total; j0 += kMoveThreads) {
    const long long j = j0 + tid;
    const int i = (int)(j / per_row), c = (int)(j % per_row);
    const int at = j < total ? keep[i] : -1;
    const bool ok = at >= 0 && at < p.T_src;
    uint2 x = make_uint2(0u, 0u);
    if (ok) x = src[at * stride + c];
    __syncthreads();
    if (ok) dst[i * stride + c] = x;
  }
}

}  // namespace

cudaError_t launch_kv_append_q4(const KvAppendQ4Args &a, cudaStream_t s) {
  const long long units = (long long)a.n * a.H_kv * a.d / 8;
  const dim3 grid((unsigned)((units + kAppendThreads - 1) / kAppendThreads), (unsigned)a.B, 2);
  kv_append_q4_kernel<<<grid, kAppendThreads, 0, s>>>(a);
  return cudaGetLastError();
}

cudaError_t launch_kv_select(const KvSelectArgs &a, cudaStream_t s) {
  kv_select_kernel<<<dim3((unsigned)a.H_kv, (unsigned)a.B), kSelThreads, 0, s>>>(a);
  return cudaGetLastError();
}

cudaError_t launch_kv_compact(const KvCompactArgs &a, cudaStream_t s) {
  const unsigned jobs = (unsigned)a.n_arrays + (a.acc_dst ? 1u : 0u);
  kv_compact_kernel<<<dim3((unsigned)a.H_kv, (unsigned)a.B, jobs), kMoveThreads, 0, s>>>(a);
  return cudaGetLastError();
}

}  // namespace hh
