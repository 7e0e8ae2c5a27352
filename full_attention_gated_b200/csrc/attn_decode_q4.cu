// attn_decode_q4.cu -- one new query per sequence against a q4_0 KV cache
// (grouped-query attention decode), with the step's attention weights
// accumulated per cached position on request.
//
// "The economics of hybrid attention" (table in "What a token of context
// costs") prices the q4_0 cache at 18 KiB per token.  Element i of a block of
// 32 stands for s (c_i - 8): 4-bit code c_i, fp16 scale s (include/hh_kv.h).
//     p = softmax_j(scale q . k_j),  o = sum_j p_j v_j,  o *= sigmoid(gate)
//
// The step is one stream over the cache, so HBM bounds it as long as the codes
// can be opened as fast as they arrive: 32 elements are 18 bytes, and at the
// measured 6.55 TB/s an SM takes in about 40 elements a clock.  What follows is
// chosen for few instructions an element:
//  * Split kernel: CTA = (kv head, split of the cache, sequence).  A producer
//    warp streams tiles of 64 keys: codes by TMA (swizzled for ldmatrix),
//    scales by cp.async (their rows are 8 or 16 bytes; zero past the end, so
//    that whatever a masked row holds never enters a product).  Four consumer
//    warps take 16 keys of a tile each, keys as the M of warp-level MMAs and
//    the group's query heads as N.  (With N = 8 of real columns a tcgen05 tile
//    would need the opened codes written to shared memory first; as register
//    operands they are used where they are opened.)
//  * A nibble in the low bits of an fp16 is the subnormal c 2^-24, one further
//    up in the mantissa c 2^-20: one AND (every other pair a shift too) makes
//    two operands, exactly, and MMAs take subnormals at full rate.  The factor
//    between the two is paid in Q for K and in the output's scale for V.
//  * The offset of 8: for K it is the accumulator's initial value,
//    -8 sum(q) of the block; for V two MMAs with a constant operand add
//    -8 sum(p') to the same accumulators, so that they stay near the result
//    (no cancellation at the end over a long cache).
//  * K's scale multiplies a block's partial logits in fp32; V's multiplies the
//    weights: p' = s p in fp16 (two roundings of 2^-11 at most).  Weights are
//    kept as 2^13 p while every scale of the warp's keys is below 2, as p from
//    the first larger one on: p' neither overflows nor, where it counts,
//    leaves the normal range.
//  * Q is scaled by a power of two per head to [1, 2) before it becomes fp16.
//  * The running maximum is only reduced across the warp, and the accumulators
//    only rescaled, when a logit exceeds it.
// Combine kernel: merges the splits of a query head, applies the gate, rounds
// to bf16 once.  Softmax statistics, logits and sums are fp32.
#include <cuda_fp16.h>
#include <math.h>
#include <string.h>

#include "common.cuh"
#include "internal.h"

namespace hh {

namespace {

constexpr int kTileKeys = 64;
constexpr int kWarps = 4;  // consumers
constexpr int kThreads = (kWarps + 1) * 32;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kSmallExp = 13.f;  // weights are kept as 2^13 p while the scales allow it

struct DecodeQ4Params {
  CUtensorMap tm_k, tm_v;  // codes, 4-D (D/2 bytes, H_kv, T_cache, B), box (D/2, 1, 64, 1)
  const bf16_t *q, *gate;
  const uint16_t *k_scales, *v_scales;
  const int32_t *cache_len;
  bf16_t *o;
  float *part_o;   // [B, H_q, n_splits, D]
  float *part_ml;  // [B, H_q, n_splits, 2]
  float *logits;   // [B, H_q, T_cache], log2 domain (accumulating calls)
  int T_cache, H_q, H_kv, group, n_splits, split_len;
  float scale_log2;
  unsigned *status;
};

template <int D>
struct Q4Smem {
  static constexpr int kRow = D / 2;                    // bytes of codes a key
  static constexpr int kTile = kTileKeys * kRow;        // K (or V) codes of a tile
  static constexpr int kScaleRow = D / 16;              // bytes of scales a key
  static constexpr int kScales = kTileKeys * kScaleRow; // K (or V) scales of a tile
  static constexpr int kStages = D == 256 ? 5 : 8;
  static constexpr int kStage = 2 * kTile + 2 * kScales;
  static_assert(kStage % 1024 == 0, "stages keep the swizzle's alignment");
  static constexpr int kRed = kWarps * 16 * D * 4 + 2 * kWarps * 16 * 4;
  static_assert(kRed <= kStages * kStage, "the reduction reuses the ring");
  static constexpr int kTotal = kStages * kStage + 2 * kStages * 8 + 1024;
  // 16-byte chunk c of row r in a tile, as TMA's 128- or 64-byte swizzle lays it out
  static __device__ __forceinline__ uint32_t at(uint32_t r, uint32_t c) {
    if constexpr (D == 256) return sw128(r, c);
    return r * 64u + ((c ^ ((r >> 1) & 3u)) << 4);
  }
};

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;\n" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ uint32_t mul_f16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;\n" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ float f16_lo(uint32_t w) { return __half2float(__ushort_as_half((unsigned short)(w & 0xFFFFu))); }
__device__ __forceinline__ float f16_hi(uint32_t w) { return __half2float(__ushort_as_half((unsigned short)(w >> 16))); }
// transposes an 8x8 matrix of 16-bit elements held one row pair a lane
__device__ __forceinline__ uint32_t transpose8(uint32_t a) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;\n" : "=r"(r) : "r"(a));
  return r;
}
// D = A B + C, fp16 operands, fp32 accumulation
__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1, float c0, float c1, float c2, float c3) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%11,%12,%13};\n"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(c0), "f"(c1), "f"(c2), "f"(c3));
}
__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
  mma_f16(d, a0, a1, a2, a3, b0, b1, d[0], d[1], d[2], d[3]);
}
// four 4-bit codes of each 16-bit half, opened into two fp16 operands apiece: c 2^-24, c 2^-20, c 2^-24, c 2^-20
struct Opened {
  uint32_t x0, x1, x2, x3;
};
__device__ __forceinline__ Opened open_codes(uint32_t w) {
  const uint32_t u = w >> 8;
  return {w & 0x000F000Fu, w & 0x00F000F0u, u & 0x000F000Fu, u & 0x00F000F0u};
}
// 8 or 16 bytes to shared memory, zero where !valid (src must be readable either way)
template <int N>
__device__ __forceinline__ void cp_async_small(uint32_t dst, const void *src, bool valid) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;\n" ::"r"(dst), "l"(src), "n"(N), "r"(valid ? N : 0));
}
// the barrier counts this thread's arrival once its cp.async operations so far have landed
__device__ __forceinline__ void cp_async_arrive(uint64_t *bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];\n" ::"r"(smem_u32(bar)) : "memory");
}
__device__ __forceinline__ int cached(const int32_t *cache_len, int b, int T_cache) {
  const int len = cache_len ? cache_len[b] : T_cache;
  return len < 0 ? 0 : (len > T_cache ? T_cache : len);
}

template <int D, int NT, bool kAcc>
__global__ void __launch_bounds__(kThreads, (NT == 1 || D == 128) ? 2 : 1)
    q4_split_kernel(const __grid_constant__ DecodeQ4Params p) {
  using L = Q4Smem<D>;
  constexpr int NB = D / 32;  // blocks a row
  extern __shared__ uint8_t smem_raw[];
  uint8_t *ring = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t *full = reinterpret_cast<uint64_t *>(ring + L::kStages * L::kStage);
  uint64_t *empty = full + L::kStages;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int kvh = blockIdx.x, split = blockIdx.y, b = blockIdx.z;
  const int len = cached(p.cache_len, b, p.T_cache);
  const int k_begin = split * p.split_len;
  const int k_end = min(k_begin + p.split_len, len);
  if (k_begin >= len && split > 0) return;  // the combine reads the splits below the length only
  const int n_tiles = k_end > k_begin ? (k_end - k_begin + kTileKeys - 1) / kTileKeys : 0;

  if (threadIdx.x == 0) {
    for (int s = 0; s < L::kStages; ++s) {
      mbar_init(&full[s], 33);  // the codes' expect_tx and the 32 lanes' scales
      mbar_init(&empty[s], kWarps);
    }
    fence_barrier_init();
  }
  __syncthreads();

  if (warp == kWarps) {
    // ---------------- producer warp ----------------
    if (lane == 0 && n_tiles > 0) {
      tma_prefetch_desc(&p.tm_k);
      tma_prefetch_desc(&p.tm_v);
    }
    const size_t srow = (size_t)p.H_kv * L::kScaleRow;
    const uint8_t *ks = reinterpret_cast<const uint8_t *>(p.k_scales) + ((size_t)b * p.T_cache * p.H_kv + kvh) * L::kScaleRow;
    const uint8_t *vs = reinterpret_cast<const uint8_t *>(p.v_scales) + ((size_t)b * p.T_cache * p.H_kv + kvh) * L::kScaleRow;
    int last = -1;
    for (int i = 0; i < n_tiles; ++i) {
      const int s = i % L::kStages;
      bool ok = true;
      if (i >= L::kStages && lane == 0) ok = mbar_wait(&empty[s], ((i / L::kStages) - 1) & 1, p.status);
      if (!__shfl_sync(0xffffffffu, ok, 0)) break;
      last = i;
      const uint32_t dk = smem_u32(ring + s * L::kStage), dv = dk + L::kTile;
      const uint32_t dks = dk + 2 * L::kTile, dvs = dks + L::kScales;
      const int t0 = k_begin + i * kTileKeys;
      if (lane == 0) {
        mbar_arrive_expect_tx(&full[s], 2 * L::kTile);
        tma_load_4d(dk, &p.tm_k, &full[s], 0, kvh, t0, b);
        tma_load_4d(dv, &p.tm_v, &full[s], 0, kvh, t0, b);
      }
#pragma unroll
      for (int r = 0; r < kTileKeys; r += 32) {
        const int t = t0 + r + lane;
        const bool live = t < k_end;
        const size_t off = (size_t)(live ? t : k_begin) * srow;
        cp_async_small<L::kScaleRow>(dks + (r + lane) * L::kScaleRow, ks + off, live);
        cp_async_small<L::kScaleRow>(dvs + (r + lane) * L::kScaleRow, vs + off, live);
      }
      cp_async_arrive(&full[s]);
    }
    // every copy issued above has landed before the CTA can exit (bounded; complete on the normal path)
    for (int i = max(last - L::kStages + 1, 0); i <= last; ++i)
      mbar_wait(&full[i % L::kStages], (i / L::kStages) & 1, p.status);
    return;
  }

  // ---------------- consumer warps ----------------
  const int g = lane >> 2, c4 = lane & 3;
  // Q^T fragments: head nt * 8 + g; a k-step of a block contracts the elements that one AND opens.  b0 goes with
  // the codes at 2^-24 and takes 16 q, b1 with those at 2^-20.
  uint32_t qb[NB][NT][4];
  float init[NB][NT][2];  // -8 sum(q) of the block, for heads nt * 8 + 2 c4 and + 1
  float col[NT][2];       // logit = col * accumulated
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    const int h = nt * 8 + g;
    const bool real = h < p.group;
    const uint4 *q = reinterpret_cast<const uint4 *>(p.q + ((size_t)b * p.H_q + kvh * p.group + (real ? h : 0)) * D + 8 * c4);
    uint32_t top = 0;
#pragma unroll 2
    for (int j = 0; j < NB; ++j) {
      const uint4 w = real ? q[4 * j] : make_uint4(0u, 0u, 0u, 0u);
      const uint32_t e[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) top = max(top, max(e[i] & 0x7FFFu, (e[i] >> 16) & 0x7FFFu));
    }
    top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
    top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
    const uint32_t eb = top >> 7;  // exponent field of the largest |q|
    const uint32_t field = eb == 0 || eb == 255 ? 127u : max(254u - eb, 1u);
    const float f = __uint_as_float(field << 23), inv = __uint_as_float((254u - field) << 23);
#pragma unroll
    for (int j = 0; j < NB; ++j) {
      const uint4 w = real ? q[4 * j] : make_uint4(0u, 0u, 0u, 0u);  // from L1 now
      const float x0 = f * bf16_lo(w.x), x1 = f * bf16_hi(w.x), x2 = f * bf16_lo(w.y), x3 = f * bf16_hi(w.y);
      const float x4 = f * bf16_lo(w.z), x5 = f * bf16_hi(w.z), x6 = f * bf16_lo(w.w), x7 = f * bf16_hi(w.w);
      qb[j][nt][0] = pack_f16(16.f * x0, 16.f * x4);
      qb[j][nt][1] = pack_f16(x1, x5);
      qb[j][nt][2] = pack_f16(16.f * x2, 16.f * x6);
      qb[j][nt][3] = pack_f16(x3, x7);
      float sum = 0.0625f * (f16_lo(qb[j][nt][0]) + f16_hi(qb[j][nt][0]) + f16_lo(qb[j][nt][2]) + f16_hi(qb[j][nt][2])) +
                  f16_lo(qb[j][nt][1]) + f16_hi(qb[j][nt][1]) + f16_lo(qb[j][nt][3]) + f16_hi(qb[j][nt][3]);
      sum += __shfl_xor_sync(0xffffffffu, sum, 1);
      sum += __shfl_xor_sync(0xffffffffu, sum, 2);
      sum *= -8.f / 1048576.f;
      init[j][nt][0] = __shfl_sync(0xffffffffu, sum, 8 * c4);
      init[j][nt][1] = __shfl_sync(0xffffffffu, sum, 8 * c4 + 4);
    }
    col[nt][0] = __shfl_sync(0xffffffffu, inv, 8 * c4) * (1048576.f * p.scale_log2);
    col[nt][1] = __shfl_sync(0xffffffffu, inv, 8 * c4 + 4) * (1048576.f * p.scale_log2);
  }

  float o[2 * NB][NT][4];
#pragma unroll
  for (int mt = 0; mt < 2 * NB; ++mt)
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) o[mt][nt][0] = o[mt][nt][1] = o[mt][nt][2] = o[mt][nt][3] = 0.f;
  float m_run[NT][2], l_run[NT][2];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) m_run[nt][0] = m_run[nt][1] = -INFINITY, l_run[nt][0] = l_run[nt][1] = 0.f;
  float up = kSmallExp;  // weights are 2^up p

  const uint32_t mrow = warp * 16 + (lane & 7) + ((lane >> 3) & 1) * 8;  // ldmatrix: key row of this lane
  for (int i = 0; i < n_tiles; ++i) {
    const int s = i % L::kStages;
    if (!mbar_wait(&full[s], (i / L::kStages) & 1, p.status)) break;
    const uint8_t *st = ring + s * L::kStage;
    const uint32_t kb = smem_u32(st), vb = kb + L::kTile;
    const uint8_t *ksc = st + 2 * L::kTile, *vsc = ksc + L::kScales;
    // ---- logits: S^T = K Q^T, block by block ----
    uint32_t s0[NB / 2], s1[NB / 2];  // the scales of keys g and g + 8
#pragma unroll
    for (int j = 0; j < NB / 2; j += 2) {
      const uint2 u0 = *reinterpret_cast<const uint2 *>(ksc + (warp * 16 + g) * L::kScaleRow + j * 4);
      const uint2 u1 = *reinterpret_cast<const uint2 *>(ksc + (warp * 16 + g + 8) * L::kScaleRow + j * 4);
      s0[j] = u0.x, s0[j + 1] = u0.y, s1[j] = u1.x, s1[j + 1] = u1.y;
    }
    float sc[NT][4];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) sc[nt][0] = sc[nt][1] = sc[nt][2] = sc[nt][3] = 0.f;
#pragma unroll
    for (int j = 0; j < NB; j += 2) {
      uint32_t r[4];  // keys g (r0) and g + 8 (r1) of block j, the same of block j + 1
      ldsm_x4(kb + L::at(mrow, j + (lane >> 4)), r[0], r[1], r[2], r[3]);
#pragma unroll
      for (int jj = 0; jj < 2; ++jj) {
        const Opened a = open_codes(r[2 * jj]), c = open_codes(r[2 * jj + 1]);
        const float f0 = jj ? f16_hi(s0[j / 2]) : f16_lo(s0[j / 2]);
        const float f1 = jj ? f16_hi(s1[j / 2]) : f16_lo(s1[j / 2]);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          float t[4];
          const float *in = init[j + jj][nt];
          mma_f16(t, a.x0, c.x0, a.x1, c.x1, qb[j + jj][nt][0], qb[j + jj][nt][1], in[0], in[1], in[0], in[1]);
          mma_f16(t, a.x2, c.x2, a.x3, c.x3, qb[j + jj][nt][2], qb[j + jj][nt][3]);
          sc[nt][0] = fmaf(f0, t[0], sc[nt][0]);
          sc[nt][1] = fmaf(f0, t[1], sc[nt][1]);
          sc[nt][2] = fmaf(f1, t[2], sc[nt][2]);
          sc[nt][3] = fmaf(f1, t[3], sc[nt][3]);
        }
      }
    }
    const int key0 = k_begin + i * kTileKeys + warp * 16 + g;
    const bool v0 = key0 < k_end, v1 = key0 + 8 < k_end;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      sc[nt][0] = v0 ? sc[nt][0] * col[nt][0] : -INFINITY;
      sc[nt][1] = v0 ? sc[nt][1] * col[nt][1] : -INFINITY;
      sc[nt][2] = v1 ? sc[nt][2] * col[nt][0] : -INFINITY;
      sc[nt][3] = v1 ? sc[nt][3] * col[nt][1] : -INFINITY;
    }
    if constexpr (kAcc) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          const int hd = nt * 8 + 2 * c4 + c;
          if (hd >= p.group) continue;
          float *row = p.logits + ((size_t)b * p.H_q + kvh * p.group + hd) * p.T_cache;
          if (v0) row[key0] = sc[nt][c];
          if (v1) row[key0 + 8] = sc[nt][c + 2];
        }
    }
    // ---- a new maximum, or the first scale of 2 or more: rescale ----
    uint32_t w0[NB / 2], w1[NB / 2], w8[NB / 2], w9[NB / 2];  // V's scales of keys 2 c4, + 1, + 8, + 9
#pragma unroll
    for (int j = 0; j < NB / 2; j += 2) {
      const uint8_t *base = vsc + (warp * 16 + 2 * c4) * L::kScaleRow + j * 4;
      const uint2 u0 = *reinterpret_cast<const uint2 *>(base), u1 = *reinterpret_cast<const uint2 *>(base + L::kScaleRow);
      const uint2 u8 = *reinterpret_cast<const uint2 *>(base + 8 * L::kScaleRow);
      const uint2 u9 = *reinterpret_cast<const uint2 *>(base + 9 * L::kScaleRow);
      w0[j] = u0.x, w0[j + 1] = u0.y, w1[j] = u1.x, w1[j + 1] = u1.y;
      w8[j] = u8.x, w8[j + 1] = u8.y, w9[j] = u9.x, w9[j + 1] = u9.y;
    }
    uint32_t any = 0;
#pragma unroll
    for (int j = 0; j < NB / 2; ++j) any |= w0[j] | w1[j] | w8[j] | w9[j];
    bool change = (any & 0x40004000u) != 0 && up != 0.f;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
      change |= fmaxf(sc[nt][0], sc[nt][2]) > m_run[nt][0] || fmaxf(sc[nt][1], sc[nt][3]) > m_run[nt][1];
    if (__any_sync(0xffffffffu, change)) {
      const float was = up;
      if (__any_sync(0xffffffffu, (any & 0x40004000u) != 0)) up = 0.f;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          float mx = fmaxf(sc[nt][c], sc[nt][c + 2]);
          mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 4));
          mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 8));
          mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 16));
          const float m_new = fmaxf(m_run[nt][c], mx);
          const float alpha = m_new == -INFINITY ? 1.f : ex2(m_run[nt][c] - m_new + (up - was));
          m_run[nt][c] = m_new;
          l_run[nt][c] *= alpha;
#pragma unroll
          for (int mt = 0; mt < 2 * NB; ++mt) {
            o[mt][nt][c] *= alpha;
            o[mt][nt][c + 2] *= alpha;
          }
        }
    }
    // ---- weights, transposed to B fragments: keys 2 c4, + 1 (b0) and + 8, + 9 (b1) of head g ----
    uint32_t pb[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const float z0 = m_run[nt][0] == -INFINITY ? 0.f : m_run[nt][0] - up;
      const float z1 = m_run[nt][1] == -INFINITY ? 0.f : m_run[nt][1] - up;
      const float p0 = ex2(sc[nt][0] - z0), p1 = ex2(sc[nt][1] - z1), p2 = ex2(sc[nt][2] - z0), p3 = ex2(sc[nt][3] - z1);
      l_run[nt][0] += p0 + p2;
      l_run[nt][1] += p1 + p3;
      pb[nt][0] = transpose8(pack_f16(p0, p1));
      pb[nt][1] = transpose8(pack_f16(p2, p3));
    }
    // ---- O^T += V^T P'^T: block J gives elements 4 g, 4 g + 1 (rows g, g + 8 of m-tile 2 J) and 4 g + 2, 4 g + 3 ----
#pragma unroll
    for (int j = 0; j < NB; j += 2) {
      uint32_t r[4];  // keys 0..7 (r0) and 8..15 (r1) of block j, the same of block j + 1
      ldsm_x4_t(vb + L::at(mrow, j + (lane >> 4)), r[0], r[1], r[2], r[3]);
#pragma unroll
      for (int jj = 0; jj < 2; ++jj) {
        const Opened a = open_codes(r[2 * jj]), c = open_codes(r[2 * jj + 1]);
        const uint32_t lo = __byte_perm(w0[j / 2], w1[j / 2], jj ? 0x7632 : 0x5410);
        const uint32_t hi = __byte_perm(w8[j / 2], w9[j / 2], jj ? 0x7632 : 0x5410);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          const uint32_t b0 = mul_f16x2(pb[nt][0], lo), b1 = mul_f16x2(pb[nt][1], hi);
          float(&oa)[4] = o[2 * (j + jj)][nt], (&ob)[4] = o[2 * (j + jj) + 1][nt];
          // -8 at 2^-24 and at 2^-20
          mma_f16(oa, 0x80088008u, 0x80808080u, 0x80088008u, 0x80808080u, b0, b1);
          mma_f16(ob, 0x80088008u, 0x80808080u, 0x80088008u, 0x80808080u, b0, b1);
          mma_f16(oa, a.x0, a.x1, c.x0, c.x1, b0, b1);
          mma_f16(ob, a.x2, a.x3, c.x2, c.x3, b0, b1);
        }
      }
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(&empty[s]);
  }

  // ---------------- merge the warps (the ring is free once all of them are here) ----------------
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      float l = l_run[nt][c];
      l += __shfl_xor_sync(0xffffffffu, l, 4);
      l += __shfl_xor_sync(0xffffffffu, l, 8);
      l += __shfl_xor_sync(0xffffffffu, l, 16);
      l_run[nt][c] = l * ex2(-up);
    }
  const float unit_lo = 16777216.f * ex2(-up), unit_hi = 1048576.f * ex2(-up);  // rows g and g + 8
  asm volatile("bar.sync 1, %0;\n" ::"n"(kWarps * 32) : "memory");
  float *red_o = reinterpret_cast<float *>(ring);
  float *red_m = red_o + kWarps * 16 * D;
  float *red_l = red_m + kWarps * 16;
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    const int hd = nt * 8 + c4 * 2;
#pragma unroll
    for (int mt = 0; mt < 2 * NB; ++mt) {
      const int dd = (mt >> 1) * 32 + 4 * g + (mt & 1) * 2;
      *reinterpret_cast<float2 *>(red_o + (warp * 16 + hd) * D + dd) = make_float2(o[mt][nt][0] * unit_lo, o[mt][nt][2] * unit_hi);
      *reinterpret_cast<float2 *>(red_o + (warp * 16 + hd + 1) * D + dd) = make_float2(o[mt][nt][1] * unit_lo, o[mt][nt][3] * unit_hi);
    }
    if (lane < 4) {
      red_m[warp * 16 + hd] = m_run[nt][0];
      red_m[warp * 16 + hd + 1] = m_run[nt][1];
      red_l[warp * 16 + hd] = l_run[nt][0];
      red_l[warp * 16 + hd + 1] = l_run[nt][1];
    }
  }
  asm volatile("bar.sync 1, %0;\n" ::"n"(kWarps * 32) : "memory");
  for (int idx = threadIdx.x; idx < p.group * D; idx += kWarps * 32) {
    const int hd = idx / D, dd = idx % D;
    float mt = -INFINITY;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) mt = fmaxf(mt, red_m[w * 16 + hd]);
    float lt = 0.f, ot = 0.f;
    if (mt != -INFINITY) {
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const float f = ex2(red_m[w * 16 + hd] - mt);
        lt += red_l[w * 16 + hd] * f;
        ot += red_o[(w * 16 + hd) * D + dd] * f;
      }
    }
    const size_t bh = (size_t)b * p.H_q + kvh * p.group + hd, row = bh * p.n_splits + split;
    if (p.n_splits == 1) {  // the only split: its result is the output
      float res = n_tiles > 0 ? ot / lt : 0.f;
      if (p.gate && n_tiles > 0) res *= 1.f / (1.f + expf(-bf16_to_f(p.gate[bh * D + dd])));
      p.o[bh * D + dd] = f_to_bf16(res);
    } else {
      p.part_o[row * D + dd] = ot;
    }
    if (dd == 0) {
      p.part_ml[row * 2 + 0] = mt;
      p.part_ml[row * 2 + 1] = lt;
    }
  }
}

// Merges the splits that lie below the sequence's length.
template <int D>
__global__ void __launch_bounds__(D) q4_combine_kernel(const __grid_constant__ DecodeQ4Params p) {
  const int h = blockIdx.x, b = blockIdx.y, dd = threadIdx.x;
  const size_t bh = (size_t)b * p.H_q + h;
  const int len = cached(p.cache_len, b, p.T_cache);
  const int n = min(p.n_splits, (len + p.split_len - 1) / p.split_len);
  const float *ml = p.part_ml + bh * p.n_splits * 2;
  const float *po = p.part_o + bh * p.n_splits * D + dd;
  float M = -INFINITY;
  for (int s = 0; s < n; ++s) M = fmaxf(M, ml[2 * s]);
  float res = 0.f;
  if (n > 0) {
    const float base = M == -INFINITY ? 0.f : M;
    float Ls = 0.f, acc = 0.f;
    for (int s = 0; s < n; ++s) {
      const float f = ex2(ml[2 * s] - base);
      Ls += ml[2 * s + 1] * f;
      acc += po[(size_t)s * D] * f;
    }
    res = acc / Ls;
    if (p.gate) res *= 1.f / (1.f + expf(-bf16_to_f(p.gate[bh * D + dd])));
  }
  p.o[bh * D + dd] = f_to_bf16(res);
}

// Splits of the cache.  Two CTAs run on an SM; a CTA takes its tiles and about three tiles' time to start and end.
// The split count with the fewest tile times over all waves of CTAs is taken: one wave that fills the GPU for a few
// long sequences, a few even waves for many.
struct Q4Plan {
  int n_splits, split_len;
};
Q4Plan q4_plan(int B, int H_kv, int T_cache) {
  const int tiles = (T_cache + kTileKeys - 1) / kTileKeys;
  if (tiles <= 1) return {1, kTileKeys};
  const long long pairs = (long long)B * H_kv, slots = 2 * 148;
  long long best = -1;
  int best_per = tiles;
  for (int n = 1; n <= tiles && n <= (int)slots; ++n) {
    const int per = (tiles + n - 1) / n;
    const int real = (tiles + per - 1) / per;
    const long long cost = (pairs * real + slots - 1) / slots * (per + 3);
    if (best < 0 || cost < best) best = cost, best_per = per;
  }
  return {(tiles + best_per - 1) / best_per, best_per * kTileKeys};
}

size_t round256(size_t n) { return (n + 255) & ~size_t(255); }

template <int D, int NT, bool kAcc>
cudaError_t launch_split(const DecodeQ4Params &p, int B, cudaStream_t s) {
  auto kern = q4_split_kernel<D, NT, kAcc>;
  const int smem = Q4Smem<D>::kTotal;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  kern<<<dim3(p.H_kv, p.n_splits, B), kThreads, smem, s>>>(p);
  return cudaGetLastError();
}

template <int D>
cudaError_t launch_d(const DecodeQ4Params &p, int B, bool acc, cudaStream_t s) {
  cudaError_t e;
  if (p.group > 8) e = acc ? launch_split<D, 2, true>(p, B, s) : launch_split<D, 2, false>(p, B, s);
  else e = acc ? launch_split<D, 1, true>(p, B, s) : launch_split<D, 1, false>(p, B, s);
  if (e != cudaSuccess || p.n_splits == 1) return e;
  q4_combine_kernel<D><<<dim3(p.H_q, B), D, 0, s>>>(p);
  return cudaGetLastError();
}

}  // namespace

// statistics, partial outputs (more than one split), logits (accumulating calls)
size_t attn_decode_q4_workspace(int B, int H_q, int H_kv, int d, int T_cache, bool with_acc) {
  const size_t heads = (size_t)B * H_q, n = q4_plan(B, H_kv, T_cache).n_splits;
  return round256(heads * n * 2 * sizeof(float)) + (n > 1 ? round256(heads * n * d * sizeof(float)) : 0) +
         (with_acc ? heads * T_cache * sizeof(float) : 0);
}

cudaError_t launch_attn_decode_q4(const AttnDecodeQ4Args &a, cudaStream_t s) {
  if (a.B == 0) return cudaSuccess;
  const Q4Plan plan = q4_plan(a.B, a.H_kv, a.T_cache);
  const size_t heads = (size_t)a.B * a.H_q, n = plan.n_splits;
  DecodeQ4Params p;
  uint8_t *ws = reinterpret_cast<uint8_t *>(a.workspace);
  p.part_ml = reinterpret_cast<float *>(ws);
  ws += round256(heads * n * 2 * sizeof(float));
  p.part_o = reinterpret_cast<float *>(ws);
  if (n > 1) ws += round256(heads * n * a.d * sizeof(float));
  p.logits = reinterpret_cast<float *>(ws);
  p.q = a.q;
  p.gate = a.gate;
  p.k_scales = a.k_scales;
  p.v_scales = a.v_scales;
  p.cache_len = a.cache_len;
  p.o = a.o;
  p.T_cache = a.T_cache;
  p.H_q = a.H_q;
  p.H_kv = a.H_kv;
  p.group = a.H_q / a.H_kv;
  p.n_splits = plan.n_splits;
  p.split_len = plan.split_len;
  p.scale_log2 = a.scale * kLog2e;
  p.status = device_status_ptr();
  if (a.T_cache > 0) {
    const uint64_t dims[4] = {(uint64_t)a.d / 2, (uint64_t)a.H_kv, (uint64_t)a.T_cache, (uint64_t)a.B};
    const uint64_t strides[3] = {(uint64_t)a.d / 2, (uint64_t)a.H_kv * a.d / 2, (uint64_t)a.T_cache * a.H_kv * a.d / 2};
    const uint32_t box[4] = {(uint32_t)a.d / 2, 1, (uint32_t)kTileKeys, 1};
    const CUtensorMapSwizzle sw = a.d == 256 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B;
    if (encode_tmap(&p.tm_k, CU_TENSOR_MAP_DATA_TYPE_UINT8, 4, a.k_values, dims, strides, box, sw) != CUDA_SUCCESS ||
        encode_tmap(&p.tm_v, CU_TENSOR_MAP_DATA_TYPE_UINT8, 4, a.v_values, dims, strides, box, sw) != CUDA_SUCCESS) {
      set_error("gqa_attn_decode_q4_0: cuTensorMapEncodeTiled failed for the q4_0 cache");
      return cudaErrorInvalidValue;
    }
  } else {
    memset(&p.tm_k, 0, sizeof(p.tm_k));
    memset(&p.tm_v, 0, sizeof(p.tm_v));
  }
  const cudaError_t e = a.d == 256 ? launch_d<256>(p, a.B, a.acc_out, s) : launch_d<128>(p, a.B, a.acc_out, s);
  if (e != cudaSuccess || !a.acc_out) return e;
  return launch_attn_weights({p.logits, p.part_ml, a.cache_len, a.acc_in, a.acc_out, a.B, a.T_cache, a.H_q, a.H_kv,
                              plan.n_splits, plan.split_len},
                             s);
}

}  // namespace hh
