// kv_cache.cu -- operators on the KV cache itself: quantised append (q4_0),
// the choice of the positions that stay when a cache is cut down, and the
// move of their rows.  Only the attention layers "grow a KV cache" ("The Hybrid
// Attention in Qwen3.8-27B"); these bound what it costs.
#include <cooperative_groups.h>
#include <cuda_fp16.h>
#include <math.h>
#include <stddef.h>

#include "common.cuh"
#include "internal_kv.h"

namespace cg = cooperative_groups;

namespace hh {

namespace {

// ---------------------------------------------------------------------------
// kv_append_q4_0.  A thread holds 8 consecutive elements of a K row and the
// same of the V row (one 16-byte load each); four neighbouring threads hold a
// block of 32.
// ---------------------------------------------------------------------------
constexpr int kAppendThreads = 256;

__device__ __forceinline__ uint32_t bf16x2_max(uint32_t a, uint32_t b) {  // a NaN stays
  uint32_t r;
  asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ uint32_t bf16x2_min(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("min.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// two fp32 values in one register pair: a * b, a + b, a * b + c in one instruction each
struct F2 {
  uint64_t v;
  __device__ __forceinline__ F2(float lo, float hi) { asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "f"(lo), "f"(hi)); }
  __device__ __forceinline__ explicit F2(uint64_t x) : v(x) {}
  __device__ __forceinline__ void get(float &lo, float &hi) const {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
  }
};
__device__ __forceinline__ F2 mul2(F2 a, F2 b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a.v), "l"(b.v));
  return F2(r);
}
__device__ __forceinline__ F2 add2(F2 a, F2 b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a.v), "l"(b.v));
  return F2(r);
}
__device__ __forceinline__ F2 fma2(F2 a, F2 b, F2 c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a.v), "l"(b.v), "l"(c.v));
  return F2(r);
}

// 8 elements (w) of a block spread over four neighbouring lanes: their codes, the block's scale, and (kHeld) s c per
// element rounded to bf16.  The instructions bound it (21 an element with all around it, 70% of the issue slots): an
// integer maximum over (magnitude, position, sign) keys, exact divisions and conversions had 30 and took 44 us where
// this takes 31 (18,412 tokens of 4 prompts, 172 MB, 26 us at the copy bandwidth).
template <bool kHeld>
__device__ __forceinline__ uint32_t quantise8(uint32_t (&w)[4], __half &s, uint4 &held) {
  // the block's largest x and largest -x
  const uint32_t hi = bf16x2_max(bf16x2_max(w[0], w[1]), bf16x2_max(w[2], w[3]));
  const uint32_t lo = bf16x2_min(bf16x2_min(w[0], w[1]), bf16x2_min(w[2], w[3])) ^ 0x80008000u;
  uint32_t ends = bf16x2_max(__byte_perm(hi, lo, 0x5410), __byte_perm(hi, lo, 0x7632));
  ends = bf16x2_max(ends, __shfl_xor_sync(0xffffffffu, ends, 1));
  ends = bf16x2_max(ends, __shfl_xor_sync(0xffffffffu, ends, 2));
  const float up = bf16_lo(ends), down = bf16_hi(ends);
  float m = up > down ? up : -down;
  if (__any_sync(0xffffffffu, up == down)) {
    // Both signs reach the largest magnitude: the first element decides.  Magnitudes order as bit patterns; below them
    // the block position reversed, then the sign, which only rides along.
    const uint32_t first = 31u - (threadIdx.x & 3) * 8u;
    uint32_t best = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint32_t e = (w[i >> 1] >> ((i & 1) * 16)) & 0xFFFFu;
      best = max(best, ((e & 0x7FFFu) << 6) | ((first - i) << 1) | (e >> 15));
    }
    best = max(best, __shfl_xor_sync(0xffffffffu, best, 1));
    best = max(best, __shfl_xor_sync(0xffffffffu, best, 2));
    if (up == down) m = __uint_as_float(((best >> 6) << 16) | (best << 31));
  }
  // bf16 / 8 is exact in fp32, so the scale is rounded once, to fp16 (11 bits, as the format stores it)
  const float want = m * -0.125f;
  s = __float2half_rn(fminf(fmaxf(want, -65504.f), 65504.f));
  float sf = __half2float(s);
  if (sf == 0.f) s = __ushort_as_half((unsigned short)0);
  bool bad = false;
  if (!(fabsf(want) >= 0x1p-21f && fabsf(want) <= 65504.f)) {
    bad = !(fmaxf(up, down) < INFINITY);  // a NaN is in both
    // Elements beyond +-8 s become that: under a saturated scale (0x4900: 524288 = 8 x 65536), and under a subnormal one
    // of k 2^-24, k <= 8, which may have been rounded down by up to a third (8 s has four bits: exact in bf16).
    uint32_t end = fabsf(want) > 65504.f ? 0x4900u : __float_as_uint(8.f * fabsf(sf)) >> 16;
    if (bad) {  // an infinity or a NaN in the block: codes of 8
      s = __ushort_as_half((unsigned short)0x7FFFu);
      sf = 0.f;
      w[0] = w[1] = w[2] = w[3] = end = 0u;
    }
    end |= end << 16;
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = bf16x2_max(bf16x2_min(w[i], end), end | 0x80008000u);
  }
  // c = rint(x / s) by an approximate reciprocal and one correction.  x has 8 significant bits and s has 11, so x / s
  // is either an exact tie (k + 1/2, which the correction restores: the residual is exact and its error far below
  // half a unit) or at least 2^-16 (relative) away from one, where a last-bit error does not matter.  |x / s| <= 8.5 (s is
  // m / -8 to 1/16, and m's own quotient is negative), so only +8 is to be clamped: -8.5 is a tie that goes to -8, and
  // adding 1.5 x 2^23 + 8 rounds to the code in the low bits.
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(sf));
  if (sf == 0.f) r = 0.f;
  constexpr float kMagic = 12582912.f + 8.f;
  const F2 r2(r, r), neg_s(-sf, -sf), magic(kMagic, kMagic);
  float t[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const F2 x(bf16_lo(w[i]), bf16_hi(w[i]));
    F2 q = mul2(x, r2);
    q = fma2(r2, fma2(q, neg_s, x), q);
    float q0, q1;
    q.get(q0, q1);
    add2(F2(fminf(q0, 7.f), fminf(q1, 7.f)), magic).get(t[2 * i], t[2 * i + 1]);
  }
  if constexpr (kHeld) {
    const float scale = bad ? __uint_as_float(0x7FC00000u) : sf;
    const F2 scale2(scale, scale), minus(-kMagic, -kMagic);
    uint32_t h[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float h0, h1;
      mul2(add2(F2(t[2 * i], t[2 * i + 1]), minus), scale2).get(h0, h1);
      h[i] = pack_bf16(h0, h1);
    }
    held = make_uint4(h[0], h[1], h[2], h[3]);
  }
  // the low bytes of four even and four odd elements
  auto bytes = [&](int i) {
    return __byte_perm(__byte_perm(__float_as_uint(t[i]), __float_as_uint(t[i + 2]), 0x0040),
                       __byte_perm(__float_as_uint(t[i + 4]), __float_as_uint(t[i + 6]), 0x0040), 0x5410);
  };
  return bytes(0) + (bytes(1) << 4);
}

// kRounds: groups of 8 elements that a thread takes, one after the other
template <bool kHeld, int kRounds>
__global__ void __launch_bounds__(kAppendThreads) kv_append_q4_kernel(const __grid_constant__ KvAppendQ4Args p) {
  const int b = blockIdx.y;
  const uint32_t row_units = (uint32_t)p.H_kv * p.d / 8;  // 16-byte units of one token
  int n_new = p.n_new ? p.n_new[b] : p.n;
  n_new = n_new < 0 ? 0 : (n_new > p.n ? p.n : n_new);
  const long long len = p.cache_len ? p.cache_len[b] : p.T_cache;
#pragma unroll 1
  for (int r = 0; r < kRounds; ++r) {
    const uint32_t u = (blockIdx.x * kRounds + r) * kAppendThreads + threadIdx.x;
    const uint32_t tok = u / row_units, col = u - tok * row_units;
    const long long pos = len - n_new + tok;
    const bool live = tok < (uint32_t)n_new && pos >= 0 && pos < p.T_cache;  // the same in all lanes of a block
    if (!__any_sync(0xffffffffu, live)) continue;
    const size_t src = ((size_t)b * p.n + tok) * row_units + col;
    const size_t dst = ((size_t)b * p.T_cache + (size_t)pos) * row_units + col;
    uint32_t w[2][4] = {};
    if (live) {
      const uint4 x = __ldg(reinterpret_cast<const uint4 *>(p.k) + src);
      const uint4 y = __ldg(reinterpret_cast<const uint4 *>(p.v) + src);
      w[0][0] = x.x, w[0][1] = x.y, w[0][2] = x.z, w[0][3] = x.w;
      w[1][0] = y.x, w[1][1] = y.y, w[1][2] = y.z, w[1][3] = y.w;
    }
#pragma unroll
    for (int side = 0; side < 2; ++side) {
      __half s;
      uint4 held;
      const uint32_t codes = quantise8<kHeld>(w[side], s, held);
      if (!live) continue;
      reinterpret_cast<uint32_t *>(side ? p.v_values : p.k_values)[dst] = codes;
      if ((threadIdx.x & 3) == 0) (side ? p.v_scales : p.k_scales)[dst >> 2] = __half_as_ushort(s);
      if constexpr (kHeld) reinterpret_cast<uint4 *>(side ? p.v_held : p.k_held)[src] = held;
    }
  }
}

// ---------------------------------------------------------------------------
// kv_evict_select.  One cluster of up to eight CTAs per (sequence, kv head),
// each with a contiguous part of the positions.  Weights map to 32-bit keys
// that order as the weights do; the last n_recent positions get the largest
// key.  The n_keep-th largest key is found by radix selection, the histograms
// summed over the cluster through shared memory:
//  1. All positions by a first digit made for weights: exponent and three bits
//     of mantissa (2047 bins; everything negative shares bin 0).
//  2. Positions above the digit found go to a bitmap, those of it to another;
//     the keys of the latter are sent to every CTA of the cluster.
//  3. Each CTA finds the key's other bits in that list, and with them which of
//     its own positions stay; they are written out in order.
// Where list or bitmaps would not fit (more than 4096 weights of one digit,
// parts above 65,536 positions) the later digits are found like the first.
// 16 x 4 rows of up to 131,072 weights (19 MB in the measured lengths, 2.9 us at
// the copy bandwidth): 34 us.  The two passes over all positions (about 15
// instructions each, shared-memory atomics in the first) take 7 of 20 us a CTA,
// the digits, the list and the cluster's barriers the rest.  Half of the time is
// instructions (70 a position with all phases, the list's loops and the bins that
// every CTA scans among them), half latency.  A row of 1500: 7.4 us.
// ---------------------------------------------------------------------------
constexpr int kSelMaxWarps = 32;
constexpr int kSelBins = 2048;
constexpr int kSelList = 4096;       // keys of the first digit found, in the whole row
constexpr int kSelMapPart = 65536;   // positions of a CTA's part that have a bitmap
constexpr int kSelMaxCluster = 8;

struct SelectSmem {
  uint32_t hist[kSelBins];    // this CTA's
  uint32_t merged[kSelBins];  // the cluster's
  uint32_t list[kSelList];
  uint32_t warp_sum[2][kSelMaxWarps];
  uint32_t cta_cnt[2];        // for the CTAs behind: positions above, and of exactly, the digit or key
  uint32_t digit, left, count;
  uint2 map[1];               // bitmaps of the positions above the digit (x) and of it (y)
};

static_assert(offsetof(SelectSmem, merged) % 16 == 0 && offsetof(SelectSmem, map) % 8 == 0, "vector accesses");

__device__ __forceinline__ uint32_t weight_key(float w) {
  if (w != w) return 0xFFFFFFFEu;                  // a NaN above every number
  const uint32_t u = __float_as_uint(w + 0.f);     // -0 becomes +0
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}
// 0 for the keys of negative weights, 1 + exponent and three mantissa bits for the others (the top bin takes the last
// two of them: NaN and the recent positions)
__device__ __forceinline__ int first_digit(uint32_t key) {
  return __vimin_s32_relu((int)(key >> 20) - 2047, kSelBins - 1);  // max(min(a, b), 0)
}

// exclusive sums over the CTA's threads of x and y, and their totals
template <int kThreads>
__device__ __forceinline__ void scan2(SelectSmem &sm, uint32_t &x, uint32_t &y, uint32_t &tx, uint32_t &ty) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  uint32_t ix = x, iy = y;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t u = __shfl_up_sync(0xffffffffu, ix, o), v = __shfl_up_sync(0xffffffffu, iy, o);
    if (lane >= o) ix += u, iy += v;
  }
  __syncthreads();  // the last use of warp_sum is over
  if (lane == 31) sm.warp_sum[0][warp] = ix, sm.warp_sum[1][warp] = iy;
  __syncthreads();
  x = ix - x, y = iy - y;
  tx = ty = 0;
#pragma unroll
  for (int w = 0; w < kThreads / 32; ++w) {
    const uint32_t u = sm.warp_sum[0][w], v = sm.warp_sum[1][w];
    if (w < warp) x += u, y += v;
    tx += u, ty += v;
  }
}

// The bin of the histogram at which the count from the top reaches `left`; leaves it, what `left` still lacks there and
// the bin's count in sm.
template <int kThreads>
__device__ __forceinline__ void pick_bin(SelectSmem &sm, const uint32_t *bins, uint32_t left) {
  constexpr int kPer = kSelBins / kThreads;  // bins a thread, the first thread the highest ones
  static_assert(kPer % 2 == 0, "vectors of bins");
  const int top = kSelBins - 1 - kPer * (int)threadIdx.x;
  uint32_t before = 0, unused = 0, t0, t1;
#pragma unroll
  for (int i = 0; i < kPer; i += 2) {
    const uint2 c = *reinterpret_cast<const uint2 *>(bins + top - 1 - i);
    before += c.x + c.y;
  }
  const uint32_t mine = before;
  scan2<kThreads>(sm, before, unused, t0, t1);
  if (before < left && before + mine >= left) {  // one thread
    uint32_t need = left - before, n;
    int d = top;
    while (need > (n = bins[d])) need -= n, --d;
    sm.digit = (uint32_t)d;
    sm.left = need;
    sm.count = n;
  }
  __syncthreads();
}

// pick_bin on the sum of the cluster's histograms: each CTA sums a slice of the bins and hands it to all.
template <int kThreads>
__device__ __forceinline__ void pick_bin_cluster(SelectSmem &sm, cg::cluster_group &cluster, int n_cta, int rank,
                                                 uint32_t left) {
  if (n_cta == 1) {
    __syncthreads();
    pick_bin<kThreads>(sm, sm.hist, left);
    return;
  }
  cluster.sync();
  const int slice = kSelBins / n_cta;  // n_cta is a power of two
  for (int i = rank * slice + (int)threadIdx.x; i < (rank + 1) * slice; i += kThreads) {
    uint32_t sum = 0;
#pragma unroll
    for (int c = 0; c < kSelMaxCluster; ++c)
      if (c < n_cta) sum += cluster.map_shared_rank(sm.hist, c)[i];
#pragma unroll
    for (int c = 0; c < kSelMaxCluster; ++c)
      if (c < n_cta) cluster.map_shared_rank(sm.merged, c)[i] = sum;
  }
  cluster.sync();
  pick_bin<kThreads>(sm, sm.merged, left);
}

// The bits of the key below its first digit, from the highest on: (mask, prefix) hold what is known.
struct KeyBits {
  uint32_t prefix, mask;
  int shift;
  __device__ __forceinline__ KeyBits(uint32_t d0) {
    if (d0 == 0) {  // all keys below 2^31
      prefix = 0u, mask = 0x80000000u, shift = 21;
    } else {        // the top bin holds two values of the digit
      mask = d0 == kSelBins - 1 ? 0xFFE00000u : 0xFFF00000u;
      prefix = (0x80000000u | ((d0 - 1u) << 20)) & mask;
      shift = 10;
    }
  }
  // digits of 10 or 11 bits: 31..21, 20..10, 9..0, less what is known
  __device__ __forceinline__ uint32_t dmask() const {
    return ((1u << (shift == 10 ? 11 : 10)) - 1u) & ~(mask >> shift);
  }
  __device__ __forceinline__ bool take(uint32_t digit) {  // false: that was the last one
    prefix |= digit << shift;
    mask |= dmask() << shift;
    if (shift == 0) return false;
    shift = shift == 21 ? 10 : 0;
    return true;
  }
};

template <int kThreads>
__global__ void __launch_bounds__(kThreads, 6 * 256 / kThreads)
    kv_select_kernel(const __grid_constant__ KvSelectArgs p) {
  extern __shared__ __align__(16) uint8_t sel_raw[];
  SelectSmem &sm = *reinterpret_cast<SelectSmem *>(sel_raw);
  cg::cluster_group cluster = cg::this_cluster();
  const int n_cta = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
  const int b = blockIdx.z, h = blockIdx.y, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  int len = p.cache_len ? p.cache_len[b] : p.T_cache;
  len = len < 0 ? 0 : (len > p.T_cache ? p.T_cache : len);
  const float *acc = p.acc + ((size_t)b * p.H_kv + h) * p.T_cache;
  int32_t *keep = p.keep + ((size_t)b * p.H_kv + h) * p.n_keep;
  if (len <= p.n_keep) {  // all stay (the same decision in the whole cluster); only then entries are left over
    for (int i = rank * kThreads + tid; i < p.n_keep; i += n_cta * kThreads) keep[i] = i < len ? i : -1;
    return;
  }
  // parts are multiples of 32 positions: words of the bitmaps
  const int part = ((len + n_cta - 1) / n_cta + 31) & ~31, begin = min(rank * part, len), n = min(part, len - begin);
  const int recent = len - p.n_recent - begin;  // of this part: the first recent position (len > n_keep >= n_recent)
  const float *w = acc + begin;
  auto key_at = [&](int i) { return i >= recent ? 0xFFFFFFFFu : weight_key(__ldg(w + i)); };
  // visit(i, key, real) for the part's positions, i of a warp's lanes consecutive from a multiple of 32 (not real past
  // the end); kBatch loads are in flight before the first is used, which the stores of a visit would otherwise forbid
  constexpr int kBatch = 8;
  auto sweep = [&](auto visit) {
    for (int i0 = warp * 32; i0 < part; i0 += kBatch * kThreads) {
      const float *src = w + i0 + lane;
      float x[kBatch];
      if (i0 + (kBatch - 1) * kThreads + 32 <= min(n, recent)) {  // all of the batch: no checks
#pragma unroll
        for (int r = 0; r < kBatch; ++r) x[r] = __ldg(src + r * kThreads);
#pragma unroll
        for (int r = 0; r < kBatch; ++r) visit(i0 + r * kThreads + lane, weight_key(x[r]), true);
      } else {
#pragma unroll
        for (int r = 0; r < kBatch; ++r) x[r] = i0 + r * kThreads + lane < n ? __ldg(src + r * kThreads) : 0.f;
#pragma unroll
        for (int r = 0; r < kBatch; ++r) {
          const int i = i0 + r * kThreads + lane;
          if (i - lane < part) visit(i, i >= recent ? 0xFFFFFFFFu : weight_key(x[r]), i < n);
        }
      }
    }
  };
  auto clear_hist = [&] {
    for (int i = tid; i < kSelBins / 4; i += kThreads)
      reinterpret_cast<uint4 *>(sm.hist)[i] = make_uint4(0u, 0u, 0u, 0u);
  };

  // ---- 1. the first digit ----
  clear_hist();
  __syncthreads();
  sweep([&](int, uint32_t k, bool real) {
    if (real) atomicAdd(&sm.hist[first_digit(k)], 1u);
  });
  pick_bin_cluster<kThreads>(sm, cluster, n_cta, rank, (uint32_t)p.n_keep);
  const uint32_t d0 = sm.digit, count = sm.count;
  uint32_t left = sm.left;
  KeyBits key(d0);

  if (count <= (uint32_t)kSelList && part <= kSelMapPart) {  // the same decision in the whole cluster
    // ---- 2. bitmaps, and the list in the order of positions ----
    uint2 *map = sm.map;
    const uint32_t lo = d0 == 0 ? 0u : 0x80000000u | ((d0 - 1u) << 20);  // its smallest and largest key
    const uint32_t hi = d0 == 0 ? 0x7FFFFFFFu : (d0 == kSelBins - 1 ? 0xFFFFFFFFu : lo + 0xFFFFFu);
    sweep([&](int i, uint32_t k, bool real) {
      const uint32_t up = __ballot_sync(0xffffffffu, real && k > hi), ge = __ballot_sync(0xffffffffu, real && k >= lo);
      if (lane == 0) map[i >> 5] = make_uint2(up, ge & ~up);
    });
    uint32_t off = 0;  // of this CTA's keys in the list
#pragma unroll
    for (int c = 0; c < kSelMaxCluster - 1; ++c)
      if (c < rank) off += cluster.map_shared_rank(sm.hist, c)[d0];
    __syncthreads();
    // a thread's words: consecutive ones, or, where there are fewer words than threads, one spread over the warps
    const int words = part >> 5, per_thread = (words + kThreads - 1) / kThreads;
    const int apart = max(1, kThreads / words), place = tid / apart;
    const int t_begin = tid % apart == 0 ? min(place * per_thread, words) : words;
    const int t_end = min(t_begin + per_thread, words);
    uint32_t n_up = 0, at = 0, all_up, all_in;
    for (int i = t_begin; i < t_end; ++i) n_up += __popc(map[i].x), at += __popc(map[i].y);
    scan2<kThreads>(sm, n_up, at, all_up, all_in);
    at += off;
    uint32_t first = at;
    for (int i = t_begin; i < t_end; ++i)
      for (uint32_t bits = map[i].y; bits; bits &= bits - 1u, ++at) {
        const uint32_t k = key_at(i * 32 + __ffs(bits) - 1);
        for (int c = 0; c < n_cta; ++c) cluster.map_shared_rank(sm.list, c)[at] = k;
      }
    if (tid == 0) sm.cta_cnt[0] = all_up;
    if (n_cta > 1) cluster.sync();
    else __syncthreads();
    // ---- 3. the other bits, from the list; every CTA for itself ----
    if (count <= 256u) {  // a thread a key: how many are larger, how many equal
      const uint32_t own = tid < (int)count ? sm.list[tid] : 0u;
      uint32_t larger = 0, equal = 0;
#pragma unroll 4
      for (int i = 0; i < (int)count; ++i) {
        const uint32_t k = sm.list[i];
        larger += k > own;
        equal += k == own;
      }
      if (tid < (int)count && larger < left && larger + equal >= left) {  // the threads of one key
        sm.digit = own;
        sm.left = left - larger;
      }
      __syncthreads();
      key.prefix = sm.digit;
      left = sm.left;
    } else {
      do {
        const uint32_t dmask = key.dmask();
        clear_hist();
        __syncthreads();
        for (int i = tid; i < (int)count; i += kThreads) {
          const uint32_t k = sm.list[i];
          if ((k & key.mask) == key.prefix) atomicAdd(&sm.hist[(k >> key.shift) & dmask], 1u);
        }
        __syncthreads();
        pick_bin<kThreads>(sm, sm.hist, left);
        left = sm.left;
      } while (key.take(sm.digit));
    }
    // of the digit's positions before this CTA's: those above the key, and of exactly it
    uint32_t gt = 0, eq = 0, out, seen;
    for (int i = tid; i < (int)off; i += kThreads) gt += sm.list[i] > key.prefix, eq += sm.list[i] == key.prefix;
    scan2<kThreads>(sm, gt, eq, out, seen);
#pragma unroll
    for (int c = 0; c < kSelMaxCluster - 1; ++c)
      if (c < rank) out += cluster.map_shared_rank(sm.cta_cnt, c)[0];
    // nobody leaves while its counts are read: arrive before the output's stores, which a later arrival would wait for
    if (n_cta > 1) cluster.barrier_arrive();
    // and of this thread's words
    gt = eq = 0;
    at = first;
    for (int i = t_begin; i < t_end; ++i) {
      const uint32_t in = map[i].y;
      uint32_t up = map[i].x, same = 0;
      for (uint32_t bits = in; bits; bits &= bits - 1u, ++at) {
        const uint32_t k = sm.list[at], bit = bits & (0u - bits);
        up |= k > key.prefix ? bit : 0u;
        same |= k == key.prefix ? bit : 0u;
      }
      map[i] = make_uint2(up, same);
      gt += __popc(up), eq += __popc(same);
    }
    uint32_t t0, t1;
    scan2<kThreads>(sm, gt, eq, t0, t1);
    out += gt;
    seen += eq;
    // Each word's positions: by its thread where the warp's words hold few, else by the warp, a word at a time.
    const uint32_t below = (1u << lane) - 1u;
    for (int r = 0; r < per_thread; ++r) {
      const int i = t_begin + r;
      const uint2 m = i < t_end ? map[i] : make_uint2(0u, 0u);
      uint32_t same = m.y, bits = m.x, to = out + min(seen, left);
      const uint32_t room = left > seen ? left - seen : 0u;
      if ((uint32_t)__popc(same) <= room) {
        bits |= same;
      } else {
        for (uint32_t k = 0; k < room; ++k) bits |= same & (0u - same), same &= same - 1u;
      }
      out += __popc(m.x);
      seen += __popc(m.y);
      if (__reduce_max_sync(0xffffffffu, __popc(bits)) <= 10u) {
        for (; bits; bits &= bits - 1u) keep[to++] = begin + i * 32 + __ffs(bits) - 1;
      } else {
        for (uint32_t owners = __ballot_sync(0xffffffffu, bits != 0u); owners; owners &= owners - 1u) {
          const int l = __ffs(owners) - 1;
          const uint32_t word = __shfl_sync(0xffffffffu, bits, l), first_to = __shfl_sync(0xffffffffu, to, l);
          const int at_word = __shfl_sync(0xffffffffu, i, l);
          if (word >> lane & 1u) keep[first_to + __popc(word & below)] = begin + at_word * 32 + lane;
        }
      }
    }
    if (n_cta > 1) cluster.barrier_wait();
    return;
  }

  // ---- the later digits like the first ----
  do {
    const uint32_t dmask = key.dmask();
    clear_hist();
    __syncthreads();
    sweep([&](int, uint32_t k, bool real) {
      if (real && (k & key.mask) == key.prefix) atomicAdd(&sm.hist[(k >> key.shift) & dmask], 1u);
    });
    pick_bin_cluster<kThreads>(sm, cluster, n_cta, rank, left);
    left = sm.left;
  } while (key.take(sm.digit));
  const int per_warp = ((part + (kThreads / 32) - 1) / (kThreads / 32) + 31) & ~31;
  const int w_begin = min(warp * per_warp, n), w_end = min(w_begin + per_warp, n);
  uint32_t out = 0, seen = 0, all_gt, all_eq;
#pragma unroll 8
  for (int i = w_begin + lane; i < w_end; i += 32) {
    const uint32_t k = key_at(i);
    out += k > key.prefix;
    seen += k == key.prefix;
  }
  scan2<kThreads>(sm, out, seen, all_gt, all_eq);
  out = __shfl_sync(0xffffffffu, out, 0);  // before this warp's positions
  seen = __shfl_sync(0xffffffffu, seen, 0);
  if (n_cta > 1) {
    if (tid == 0) sm.cta_cnt[0] = all_gt, sm.cta_cnt[1] = all_eq;
    cluster.sync();
    for (int c = 0; c < rank; ++c) {
      const uint32_t *cnt = cluster.map_shared_rank(sm.cta_cnt, c);
      out += cnt[0];
      seen += cnt[1];
    }
    cluster.sync();  // nobody leaves while its counts are read
  }
  const uint32_t below = (1u << lane) - 1u;
#pragma unroll 4
  for (int i0 = w_begin; i0 < w_end; i0 += 32) {
    const int i = i0 + lane;
    const uint32_t k = i < w_end ? key_at(i) : 0u;
    const bool above = i < w_end && k > key.prefix, equal = i < w_end && k == key.prefix;
    const uint32_t ba = __ballot_sync(0xffffffffu, above), be = __ballot_sync(0xffffffffu, equal);
    const uint32_t e = seen + __popc(be & below);
    if (above || (equal && e < left)) keep[out + __popc(ba & below) + min(e, left)] = begin + i;
    out += __popc(ba);
    seen += __popc(be);
  }
}

// ---------------------------------------------------------------------------
// kv_compact.  Reads and writes every kept row once.
//
// Into other arrays: CTA = (some (position, kv head) pairs of a sequence in the
// order of the destination, array), about 2048 vectors of 16 bytes, fewer while
// that leaves fewer than four CTAs an SM (one sequence of 84,000 positions cut to
// 16,384: 14.4 -> 12.5 us against two); all writes are contiguous.  The weights have
// CTAs of their own.
//
// In place: a cluster of CTAs = (sequence, kv head, array, part of the row) moves
// its rows in chunks: a chunk is read whole before any of it is written, and
// entry i comes from a position >= i, so that later chunks still find their rows
// in place.  While there are fewer than two CTAs an SM, rows are cut into parts of
// at least 32 bytes (a sector), and clusters grow up to eight CTAs (84,000 -> 16,384
// positions of q4_0: 36 -> 14.6 us).
//
// 16 x 4 heads, a q4_0 cache of d = 256 cut from 32,768 positions to 8192 (308
// MB read and written, 47 us at the copy bandwidth): 65 us.  The
// scales' rows are 16 bytes, and HBM reads 64 for each: with those it is 55 us.  In
// place 87 us.
// One sequence, 5000 bf16 rows of d = 128: 3.3 us.
// ---------------------------------------------------------------------------
constexpr int kMoveThreads = 256;
constexpr int kMoveVectors = 2048;   // of a CTA, at most
constexpr int kShiftThreads = 512;
constexpr int kShiftUnroll = 4;       // with 4 CTAs an SM: 87 us where 8 with two took 100 (the case above)

struct GatherParams {
  KvCompactArgs a;
  unsigned first[kMaxCompactArrays + 1];  // first CTA (blockIdx.x) of each array; the weights' CTAs follow the last
  int pairs[kMaxCompactArrays];           // (position, kv head) pairs of one of its CTAs
};

template <typename V>
__device__ __forceinline__ void gather_rows(const long long *from, const V *src, V *dst, int per_row, int pairs) {
  // from: the source row of each pair, or -1; dst: the first pair's row.  Vectors in the order of the destination.
  const int total = pairs * per_row, shift = 31 - __clz(per_row);
  const bool pow2 = (per_row & (per_row - 1)) == 0;
#pragma unroll 4
  for (int v = threadIdx.x; v < total; v += kMoveThreads) {
    const int pair = pow2 ? v >> shift : v / per_row, c = v - pair * per_row;
    const long long row = from[pair];
    if (row >= 0) dst[v] = src[row * per_row + c];
  }
}

__global__ void __launch_bounds__(kMoveThreads) kv_gather_kernel(const __grid_constant__ GatherParams p) {
  __shared__ long long from[kMoveVectors];
  const KvCompactArgs &a = p.a;
  const int b = blockIdx.y;
  int k = 0;
  while (k < a.n_arrays && blockIdx.x >= p.first[k + 1]) ++k;
  if (k == a.n_arrays) {
    const size_t per = (size_t)a.H_kv * a.T_dst, j0 = (size_t)(blockIdx.x - p.first[k]) * (4 * kMoveThreads);
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const size_t j = j0 + r * kMoveThreads + threadIdx.x;
      if (j >= per) continue;
      const int h = (int)(j / a.T_dst), i = (int)(j - (size_t)h * a.T_dst);
      const size_t row = (size_t)b * a.H_kv + h;
      const int at = i < a.n_keep ? a.keep[row * a.n_keep + i] : -1;
      a.acc_dst[row * a.T_dst + i] = at >= 0 && at < a.T_src ? a.acc_src[row * a.T_src + at] : 0.f;
    }
    return;
  }
  const size_t pair0 = (size_t)(blockIdx.x - p.first[k]) * p.pairs[k], all = (size_t)a.n_keep * a.H_kv;
  const int pairs = (int)(all - pair0 < (size_t)p.pairs[k] ? all - pair0 : (size_t)p.pairs[k]);
  for (int x = threadIdx.x; x < pairs; x += kMoveThreads) {
    const size_t pair = pair0 + x, i = pair / a.H_kv, h = pair - i * a.H_kv;
    const int at = a.keep[((size_t)b * a.H_kv + h) * a.n_keep + i];
    from[x] = at >= 0 && at < a.T_src ? (long long)at * a.H_kv + (long long)h : -1;
  }
  __syncthreads();
  const int R = a.row_bytes[k];
  const uint8_t *src = reinterpret_cast<const uint8_t *>(a.src[k]) + (size_t)b * a.T_src * a.H_kv * R;
  uint8_t *dst = reinterpret_cast<uint8_t *>(a.dst[k]) + ((size_t)b * a.T_dst * a.H_kv + pair0) * R;
  if (R % 16 == 0)
    gather_rows(from, reinterpret_cast<const uint4 *>(src), reinterpret_cast<uint4 *>(dst), R / 16, pairs);
  else
    gather_rows(from, reinterpret_cast<const uint2 *>(src), reinterpret_cast<uint2 *>(dst), R / 8, pairs);
}

struct ShiftParams {
  KvCompactArgs a;                    // the arrays that are compacted in place
  int part_bytes[kMaxCompactArrays];  // bytes of a row that one CTA moves
  int first[kMaxCompactArrays + 1];   // first CTA (blockIdx.x) of each array; the weights' CTA follows the last
};

// the first `per` vectors of rows `stride` vectors apart; thread t of the cluster's n
template <typename V>
__device__ __forceinline__ void shift_rows(const cg::cluster_group &cluster, const int32_t *keep, int n_keep, int T,
                                           V *rows, size_t stride, int per) {
  const long long total = (long long)n_keep * per;
  const int n = (int)cluster.num_blocks() * kShiftThreads, t = (int)cluster.block_rank() * kShiftThreads + threadIdx.x;
  const int shift = (per & (per - 1)) == 0 ? 31 - __clz(per) : -1;  // a 64-bit division is worth a hundred instructions
  for (long long j0 = 0; j0 < total; j0 += (long long)n * kShiftUnroll) {
    V x[kShiftUnroll];
    int to[kShiftUnroll];
#pragma unroll
    for (int r = 0; r < kShiftUnroll; ++r) {
      const long long j = j0 + (long long)r * n + t;
      const int i = (int)(shift >= 0 ? j >> shift : j / per), c = (int)(j - (long long)i * per);
      const int at = j < total ? keep[i] : -1;
      to[r] = at >= 0 && at < T && at != i ? i : -1;  // a row that stays where it is is not touched
      if (to[r] >= 0) x[r] = rows[(size_t)at * stride + c];
    }
    if (cluster.num_blocks() > 1) cluster.sync();
    else __syncthreads();
#pragma unroll
    for (int r = 0; r < kShiftUnroll; ++r) {
      const int c = (int)(j0 + (long long)r * n + t - (long long)to[r] * per);
      if (to[r] >= 0) rows[(size_t)to[r] * stride + c] = x[r];
    }
  }
}

__global__ void __launch_bounds__(kShiftThreads, 4) kv_shift_kernel(const __grid_constant__ ShiftParams p) {
  const KvCompactArgs &a = p.a;
  const cg::cluster_group cluster = cg::this_cluster();
  const int h = blockIdx.y, b = blockIdx.z, job = blockIdx.x / cluster.num_blocks();
  const size_t row = (size_t)b * a.H_kv + h;
  const int32_t *keep = a.keep + row * a.n_keep;
  int k = 0;
  while (k < a.n_arrays && job >= p.first[k + 1]) ++k;
  if (k == a.n_arrays) {  // the weights, and zeros behind them
    float *acc = a.acc_dst + row * a.T_dst;
    shift_rows(cluster, keep, a.n_keep, a.T_src, acc, 1, 1);
    cluster.sync();
    for (int i = (int)cluster.block_rank() * kShiftThreads + threadIdx.x; i < a.T_dst;
         i += (int)cluster.num_blocks() * kShiftThreads) {
      const int at = i < a.n_keep ? keep[i] : -1;
      if (at < 0 || at >= a.T_src) acc[i] = 0.f;
    }
    return;
  }
  const int R = a.row_bytes[k], off = (job - p.first[k]) * p.part_bytes[k], bytes = min(p.part_bytes[k], R - off);
  uint8_t *rows = reinterpret_cast<uint8_t *>(a.dst[k]) + ((size_t)b * a.T_dst * a.H_kv + h) * R + off;
  const size_t stride = (size_t)a.H_kv * R;
  if (R % 16 == 0)
    shift_rows(cluster, keep, a.n_keep, a.T_src, reinterpret_cast<uint4 *>(rows), stride / 16, bytes / 16);
  else
    shift_rows(cluster, keep, a.n_keep, a.T_src, reinterpret_cast<uint2 *>(rows), stride / 8, bytes / 8);
}

}  // namespace

template <int kRounds>
static cudaError_t launch_append(const KvAppendQ4Args &a, cudaStream_t s) {
  const long long units = (long long)a.n * a.H_kv * a.d / 8, cta = kRounds * kAppendThreads;
  const dim3 grid((unsigned)((units + cta - 1) / cta), (unsigned)a.B);
  if (a.k_held) kv_append_q4_kernel<true, kRounds><<<grid, kAppendThreads, 0, s>>>(a);
  else kv_append_q4_kernel<false, kRounds><<<grid, kAppendThreads, 0, s>>>(a);
  return cudaGetLastError();
}

cudaError_t launch_kv_append_q4(const KvAppendQ4Args &a, cudaStream_t s) {
  // two rounds a thread once the CTAs of one fill the GPU several times (4 x up to 8191 tokens 33.0 -> 30.3 us, all of
  // them live 52.8 -> 50.0; below that the second round costs 0.1 us; four rounds: 30.1 and 51.2)
  const long long ctas = ((long long)a.n * a.H_kv * a.d / 8 + kAppendThreads - 1) / kAppendThreads * a.B;
  return ctas > 2 * 148 * 8 ? launch_append<2>(a, s) : launch_append<1>(a, s);
}

template <int kThreads>
static cudaError_t launch_select(const KvSelectArgs &a, int n_cta, size_t smem, cudaStream_t s) {
  static std::atomic<uint64_t> done{0};
  const cudaError_t e = once_per_device(done, [] {
    return cudaFuncSetAttribute(kv_select_kernel<kThreads>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                (int)(sizeof(SelectSmem) + sizeof(uint2) * (kSelMapPart / 32)));
  });
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)n_cta, (unsigned)a.H_kv, (unsigned)a.B);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = (unsigned)n_cta;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kv_select_kernel<kThreads>, a);
}

cudaError_t launch_kv_select(const KvSelectArgs &a, cudaStream_t s) {
  // CTAs a row: parts of 4096 positions and more, up to the eight CTAs of a portable cluster; where that is more than
  // the GPU holds at once, longer parts, up to 32,768 positions (64 x 4 rows of 16,384: 39 -> 29 us, of 40,000: 82 ->
  // 48; with parts of 65,536 rows of 131,072 lose: 110 -> 119)
  int n_cta = 1;
  while (n_cta < kSelMaxCluster && (long long)n_cta * 4096 < a.T_cache) n_cta *= 2;
  while (n_cta > 1 && (long long)n_cta * a.B * a.H_kv > 6 * 148 && a.T_cache <= (n_cta / 2) * 32768LL) n_cta /= 2;
  const int part = ((a.T_cache + n_cta - 1) / n_cta + 31) & ~31;  // the longest
  const int map_words = (part < kSelMapPart ? part : kSelMapPart) / 32;
  const size_t smem = sizeof(SelectSmem) + sizeof(uint2) * (size_t)map_words;
  // Few CTAs with long parts wait for memory: more threads have more loads on their way (1 x 4 rows of 131,072: 22.4 us
  // with 256 threads, 17.9 with 512).  Where the SMs are shared by more of them they cost (16 x 4 rows: 37 -> 39 us).
  if (part >= 8192 && (long long)n_cta * a.H_kv * a.B <= 148) return launch_select<512>(a, n_cta, smem, s);
  return launch_select<256>(a, n_cta, smem, s);
}

cudaError_t launch_kv_compact(const KvCompactArgs &a, cudaStream_t s) {
  // arrays (and weights) that go elsewhere, and those that are compacted in place
  GatherParams g = {a, {}, {}};
  ShiftParams sh = {a, {}, {}};
  g.a.n_arrays = sh.a.n_arrays = 0;
  for (int i = 0; i < a.n_arrays; ++i) {
    KvCompactArgs &t = a.src[i] == a.dst[i] ? sh.a : g.a;
    t.src[t.n_arrays] = a.src[i];
    t.dst[t.n_arrays] = a.dst[i];
    t.row_bytes[t.n_arrays++] = a.row_bytes[i];
  }
  const bool acc_in_place = a.acc_dst && a.acc_src == a.acc_dst;
  const long long pairs = (long long)a.n_keep * a.H_kv;
  unsigned ctas = 0;
  for (int vectors = kMoveVectors;; vectors /= 2) {
    ctas = 0;
    for (int i = 0; i < g.a.n_arrays; ++i) {
      const int R = g.a.row_bytes[i], per_row = R % 16 == 0 ? R / 16 : R / 8;
      g.pairs[i] = vectors > per_row ? vectors / per_row : 1;
      g.first[i] = ctas;
      ctas += (unsigned)((pairs + g.pairs[i] - 1) / g.pairs[i]);
    }
    if ((long long)ctas * a.B >= 4 * 148 || vectors <= kMoveThreads) break;
  }
  g.first[g.a.n_arrays] = ctas;
  if (a.acc_dst && !acc_in_place)
    ctas += (unsigned)(((long long)a.H_kv * a.T_dst + 4 * kMoveThreads - 1) / (4 * kMoveThreads));
  if (ctas > 0) {
    kv_gather_kernel<<<dim3(ctas, (unsigned)a.B), kMoveThreads, 0, s>>>(g);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
  }
  const long long rows = (long long)a.B * a.H_kv;
  int jobs = 0;
  long long parts = 1;  // of every row, where it has that many sectors
  while (rows * sh.a.n_arrays * parts < 2 * 148 && parts < 128) parts *= 2;
  for (int i = 0; i < sh.a.n_arrays; ++i) {
    const int R = sh.a.row_bytes[i];
    long long per = (R + parts - 1) / parts;
    per = per < 32 ? 32 : (per + 31) / 32 * 32;
    sh.first[i] = jobs;
    sh.part_bytes[i] = (int)(per < R ? per : R);
    jobs += (R + sh.part_bytes[i] - 1) / sh.part_bytes[i];
  }
  sh.first[sh.a.n_arrays] = jobs;
  if (acc_in_place) ++jobs;
  if (jobs == 0 || (a.n_keep == 0 && !acc_in_place)) return cudaSuccess;
  unsigned n_cta = 1;  // a cluster
  while (n_cta < 8 && rows * jobs * n_cta < 2 * 148 && a.n_keep > (int)n_cta * kShiftThreads) n_cta *= 2;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)jobs * n_cta, (unsigned)a.H_kv, (unsigned)a.B);
  cfg.blockDim = dim3(kShiftThreads);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = n_cta;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kv_shift_kernel, sh);
}

}  // namespace hh
