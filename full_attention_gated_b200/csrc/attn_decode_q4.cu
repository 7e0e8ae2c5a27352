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
//  * Split kernel: CTA = (kv head, group), one wave of CTAs; a group takes an
//    equal share of all sequences' tiles of 64 or 128 keys in a row, by the
//    lengths on the device, so that uneven lengths leave no SM idle.
//  * Four warps to a tile.  Each warp takes the logits of a quarter of its
//    keys, then a quarter of the row's elements of the weighted sum over all of
//    them, so that a thread holds a quarter of the accumulators and three CTAs
//    fit an SM: the products are chains of short dependent instructions, and
//    warps to switch between are what hides them (with a warp's accumulators
//    over all elements, two or three warps a scheduler: 64 to 83% of the copy
//    bandwidth).
//  * Codes arrive by TMA (swizzled for ldmatrix), and so do scales where their
//    rows have TMA's 16 bytes (D = 256; 8% faster at B = 64 than 16-byte
//    cp.async), else by cp.async.  Keys are the M of warp-level MMAs, the
//    group's query heads N.  (With N = 8 of real columns a tcgen05 tile would
//    need the opened codes written to shared memory first; as register operands
//    they are used where they are opened.)
//  * A nibble in the low bits of an fp16 is the subnormal c 2^-24, one further
//    up in the mantissa c 2^-20, and a whole byte (l + 16 h) 2^-24: one AND (every
//    other pair a shift too) makes two operands, exactly, and MMAs take
//    subnormals at full rate.  K's low and high nibbles meet elements of Q scaled
//    for them.  V's are elements of the output: its rows sum the bytes and the
//    high nibbles, and a subtraction at the end leaves the low ones, which saves
//    the fifth of the instructions that would take them apart (4% of the arithmetic).
//  * The offset of 8 is one MMA for 16 keys on each side, with the scales as an
//    operand: for K, -8 sum_J s_J sum(q)_J (the sums as two fp16 terms) is where
//    the logits start; for V, -8 sum p s_J collects in accumulators of its own
//    and joins the others every 1024 keys, so that little cancels at once.  The
//    sums cancel in fp32: a logit is good to 2^-21 of its scale times sum_J 8 s_J
//    sum |q|_J, which counts where large q meet keys that are small beside others
//    of their block.
//  * K's scale multiplies a block's partial logits in fp32; V's multiplies the
//    weights: p' = s p in fp16 (two roundings of 2^-11 at most).  A block of
//    elements has a power of two of its own, which brings the largest scale S of
//    its keys so far into [1/2, 2), and weights are 2^14 p: p' does not overflow,
//    and is a normal number wherever p s / S >= 2^-27.  Below, a product is off by
//    up to 2^-25, which counts with the code 0..15 (the offset is taken off with
//    the exact product): 2^-34 S a key, 2^-20 of the block's largest value at
//    131,072 keys.  A scale below 2^-13 S is off by up to 2^-24 S: 2^-24 of that
//    value.  (One power for all blocks goes by the largest: under a peaked softmax
//    small blocks beside a large one came out wrong altogether.)
//  * Q is scaled by a power of two per head to [2^10, 2^11) before it becomes
//    fp16.
//  * The running maximum is only reduced across the CTA, and the accumulators
//    only rescaled, when a logit exceeds it.
// attn_finish.cu merges the splits and takes the weights.  Softmax statistics,
// logits and sums are fp32.
//
// Measured whole calls, d = 256, 24 q / 4 kv heads: 64 x 131,072 tokens (9.66 GB)
// 1.51 to 1.53 ms from board to board, 96 to 98% of the copy bandwidth; kept up
// for seconds, where the power limit takes the SMs from 1.96 to 1.53 GHz, 1.8 ms.
// (Without the blocks' powers and the offset's factor, 1.49 ms on the same board;
// its arithmetic alone was 1.15 ms then, its copies alone 1.39 and 1.41 ms.)  One
// sequence of 84,000 tokens (97 MB) 27.2 us, of which 15 are its bytes and the
// rest the time to the first tiles, the last tiles' arithmetic and the merge; 777
// tokens 7.2 us, latency alone.
// Opening the codes bounds the arithmetic (integer pipe 48% busy, tensor 35%,
// issue 50% at 8 x 131,072).
// Not kept: K as e4m3 operands (its high and low nibbles are e4m3 values as they
// are, three instructions for eight; the products come out exact, but the MMAs
// convert them one by one: 1.84 ms); eight warps a CTA and two CTAs (1.69 ms); a
// tile's logits ahead of the last one's product, one full barrier less (1.53 ms).
#include <cuda_fp16.h>
#include <float.h>
#include <math.h>
#include <string.h>

#include "common.cuh"
#include "internal_kv.h"
#include "tc.cuh"

namespace hh {

namespace {

constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;
constexpr float kLog2e = 1.4426950408889634f;
// Keys between two folds of the offset's sums.  Until then a byte's row has grown to 255 p' a key where the result is
// at most 8: 64 fp32 additions of 2^-24 each, 32 times enlarged, are 2^-13 of the largest value.
constexpr int kFoldKeys = 1024;
constexpr float kWeightExp = 14.f;  // weights are kept as 2^14 p, of scales below 2

struct DecodeQ4Params {
  CUtensorMap tm_k, tm_v;    // codes, 4-D (D/2 bytes, H_kv, T_cache, B), box (D/2, 1, tile, 1)
  CUtensorMap tm_ks, tm_vs;  // scales, 4-D (D/32, H_kv, T_cache, B), box (D/32, 1, tile, 1), D = 256 only
  const bf16_t *q, *gate;
  const uint16_t *k_scales, *v_scales;
  const int32_t *cache_len;
  bf16_t *o;
  float *part_o;   // [B + groups, H_q, D]
  float *part_ml;  // [B + groups, H_q, 2]
  int *start;      // [B + 1]: first tile of each sequence, and the share
  float *logits;   // [B, H_q, T_cache], log2 domain (accumulating calls)
  int B, T_cache, H_q, H_kv, group;
  float scale_log2;
  unsigned *status;
};

// CTAs an SM that the registers are bounded for.  U: groups of 16 keys a warp takes of a tile.
constexpr int ctas_per_sm(int D, int NT, int U) {
  return D == 256 ? (NT == 2 && U == 2 ? 2 : 3) : (NT == 1 ? 5 : 4);
}

template <int D, int NT, int U>
struct Q4Smem {
  static constexpr int kTileKeys = kWarps * 16 * U;
  static constexpr int kRow = D / 2;                    // bytes of codes a key
  static constexpr int kTile = kTileKeys * kRow;        // codes of a tile of K (or V)
  static constexpr int kScaleRow = D / 16;              // bytes of scales a key
  static constexpr int kScaleAt = 16;                   // their stride here, whatever D (ldmatrix reads 16-byte rows)
  static constexpr int kScales = kTileKeys * kScaleAt;  // scales of a tile
  static constexpr bool kTmaScales = D == 256;          // TMA copies rows of 16 bytes, not of 8
  static constexpr int kStages = U == 2 ? 2 : 3;        // of K, and of V
  static constexpr int kCodesOff = 0;                   // [stage][K, V]
  static constexpr int kScalesOff = kStages * 2 * kTile;
  static_assert(kTile % 1024 == 0, "tiles keep the swizzle's alignment");
  static constexpr int kPRow = kTileKeys + 8;           // fp16 elements of a head's weights (padded: no bank conflicts)
  static constexpr int kP = kScalesOff + kStages * 2 * kScales;  // weights [8 NT][kPRow]; at times the offset's sums
  static_assert(8 * NT * kPRow * 2 >= kWarps * (D / 32) * NT * 32, "[kWarps][D / 32][8 NT] fp32");
  static constexpr int kStat = kP + 8 * NT * kPRow * 2;          // [kWarps][8 NT] maxima or sums
  static constexpr int kLargest = kStat + kWarps * 8 * NT * 4;   // [kWarps][8] V's largest scales (fp16 bits), by block
  static constexpr int kBars = kLargest + kWarps * 8 * 4;        // [stage][K, V]
  static constexpr int kQ = kBars + kStages * 2 * 8;
  static constexpr int kTotal = kQ + (NT == 1 ? 0 : (D / 32) * NT * 512);
  static_assert(kQ % 16 == 0 && kBars % 8 == 0, "alignment");
  static_assert(ctas_per_sm(D, NT, U) * (kTotal + 1024) <= 233472, "the CTAs' shared memory fits an SM");
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
__device__ __forceinline__ float f16_lo(uint32_t w) {
  return __half2float(__ushort_as_half((unsigned short)(w & 0xFFFFu)));
}
__device__ __forceinline__ float f16_hi(uint32_t w) {
  return __half2float(__ushort_as_half((unsigned short)(w >> 16)));
}
// The power of two that brings a block's scales below 2, as fp16 bits: 2^13 down to 2^-16, from the bits of the largest of
// them; and its reciprocal.
__device__ __forceinline__ uint32_t power_for(uint32_t largest) {
  const uint32_t e = min(max(largest >> 10, 1u), 30u);  // exponent field (infinities and NaN as the largest number)
  return e <= 28u ? (29u - e) << 10 : 0x400u >> (e - 28u);
}
__device__ __forceinline__ float reciprocal(uint32_t power) {
  return __uint_as_float(0x7F000000u - __float_as_uint(f16_lo(power)));
}
// 2^14 exp2((s - m) col), two heads at a time.  The difference comes first: of the products, 2^23 and more, units are lost.
__device__ __forceinline__ void weights2(float &p0, float &p1, float s0, float s1, const float (&m)[2],
                                         const float (&col)[2]) {
  asm("{.reg .b64 s, m, c, e;\n"
      "mov.b64 s, {%2, %3};\nmov.b64 m, {%4, %5};\nmov.b64 c, {%6, %7};\nmov.b64 e, {%8, %8};\n"
      "sub.rn.f32x2 s, s, m;\nfma.rn.f32x2 s, s, c, e;\nmov.b64 {%0, %1}, s;}\n"
      : "=f"(p0), "=f"(p1)
      : "f"(s0), "f"(s1), "f"(m[0]), "f"(m[1]), "f"(col[0]), "f"(col[1]), "f"(kWeightExp));
  p0 = ex2(p0);
  p1 = ex2(p1);
}
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
// two bytes of each 16-bit half: l + 16 h for its codes l and h, at 2^-24, and 16 h; the same of the upper byte
__device__ __forceinline__ Opened open_bytes(uint32_t w) {
  const uint32_t u = __byte_perm(w, 0u, 0x4341);
  return {w & 0x00FF00FFu, w & 0x00F000F0u, u, u & 0x00F000F0u};
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

// four elements of an output row: v / l (0 for an empty sequence: l = 0), gated, rounded to bf16.  The reciprocal and
// the sigmoid are good to 2^-20: the rounding to bf16 hides it, and there is far less code to fetch on a short call.
__device__ __forceinline__ uint2 output4(float4 v, float l, bool gated, uint2 gate) {
  const float inv = l == 0.f ? 0.f : __fdividef(1.f, l);
  float r[4] = {v.x * inv, v.y * inv, v.z * inv, v.w * inv};
  const float gf[4] = {bf16_lo(gate.x), bf16_hi(gate.x), bf16_lo(gate.y), bf16_hi(gate.y)};
  if (gated) {
#pragma unroll
    for (int i = 0; i < 4; ++i) r[i] *= __fdividef(1.f, 1.f + ex2(-kLog2e * gf[i]));
  }
  return make_uint2(pack_bf16(r[0], r[1]), pack_bf16(r[2], r[3]));
}

template <int D, int NT, int U, bool kAcc>
__global__ void __launch_bounds__(kThreads, ctas_per_sm(D, NT, U))
    q4_split_kernel(const __grid_constant__ DecodeQ4Params p) {
  using L = Q4Smem<D, NT, U>;
  constexpr int kTileKeys = L::kTileKeys, S = L::kStages;
  constexpr int NB = D / 32;       // blocks a row
  constexpr int NW = NB / kWarps;  // blocks of a warp's elements
  extern __shared__ __align__(1024) uint8_t smem[];
  uint16_t *p_s = reinterpret_cast<uint16_t *>(smem + L::kP);
  float *stat = reinterpret_cast<float *>(smem + L::kStat);
  uint32_t *largest = reinterpret_cast<uint32_t *>(smem + L::kLargest);
  uint64_t *full = reinterpret_cast<uint64_t *>(smem + L::kBars);  // K's and V's barrier of each stage

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, c4 = lane & 3;
  const int kvh = blockIdx.x, grp = blockIdx.y;
  const uint32_t base = smem_u32(smem);
  if (base & 1023u) {  // the swizzled tiles would be misread: say so and leave (uniform)
    if (threadIdx.x == 0 && p.status) atomicOr(p.status, kStatusTimeout);
    return;
  }
  const int first_len = lane < p.B ? cached(p.cache_len, lane, p.T_cache) : 0;
  if (threadIdx.x == 0) {
    for (int i = 0; i < 2 * S; ++i) mbar_init(&full[i], L::kTmaScales ? 1 : 1 + kThreads);
    fence_barrier_init();
    tma_prefetch_desc(&p.tm_k);
    tma_prefetch_desc(&p.tm_v);
    if (L::kTmaScales) {
      tma_prefetch_desc(&p.tm_ks);
      tma_prefetch_desc(&p.tm_vs);
    }
  }
  __syncthreads();
  // the tiles of all sequences in a row (an empty one counts one, fully masked), an equal share for each of the groups
  auto tiles_of = [&](int len) { return max(1, (len + kTileKeys - 1) / kTileKeys); };
  int total = lane < p.B ? tiles_of(first_len) : 0;
#pragma unroll 4
  for (int i = lane + 32; i < p.B; i += 32) total += tiles_of(cached(p.cache_len, i, p.T_cache));
  total = __reduce_add_sync(0xffffffffu, total);
  const int share = (total + (int)gridDim.y - 1) / (int)gridDim.y, first = grp * share;
  const int mine = min(share, total - first);
  if (mine <= 0) return;
  // attn_finish.cu's kernel may be set up from here on where a CTA has little to do: 777 tokens 7.4 -> 6.8 us
  const bool brief = mine <= 2;
  if (brief) asm volatile("griddepcontrol.launch_dependents;\n");
  int b = 0, before = 0, len = 0;  // the sequence that holds tile `first`, the tiles before it, its length
  for (int from = 0;; from += 32) {
    if (from) len = from + lane < p.B ? cached(p.cache_len, from + lane, p.T_cache) : 0;
    else len = first_len;
    const int own = from + lane < p.B ? tiles_of(len) : 0;
    int incl = own;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += v;
    }
    const unsigned past = __ballot_sync(0xffffffffu, before + incl > first);
    if (past) {  // in the end always: first < total
      const int l = __ffs(past) - 1;
      b = from + l;
      before += __shfl_sync(0xffffffffu, incl - own, l);
      len = __shfl_sync(0xffffffffu, len, l);
      break;
    }
    before += __shfl_sync(0xffffffffu, incl, 31);
  }
  if (kvh == 0 && grp == 0 && threadIdx.x == 0) p.start[p.B] = share;

  // The queries go to L1 ahead of the first tiles, whose loads would hold them up (one 128-byte line a thread; as
  // registers they would cost the main loop spills).
  for (int i = threadIdx.x; i < p.group * D / 64; i += kThreads) {
    uint32_t unused;
    const bf16_t *line = p.q + ((size_t)b * p.H_q + kvh * p.group) * D + i * 64;
    asm volatile("ld.global.ca.u32 %0, [%1];" : "=r"(unused) : "l"(line));
  }

  // Loads run through all of this CTA's sequences, K a tile ahead of V: (load_b, load_tile) is the last tile whose K
  // was loaded.  With TMA for the scales thread 0 alone loads; else everyone copies the scales of one key.
  int load_b = b, load_tile = first - before, load_len = len;
  auto load_side = [&](int stage, int side) {
    if (L::kTmaScales && threadIdx.x != 0) return;
    uint64_t *bar = &full[2 * stage + side];
    const int t0 = load_tile * kTileKeys;
    const uint32_t dst = base + L::kCodesOff + (2 * stage + side) * L::kTile;
    const uint32_t sdst = base + L::kScalesOff + (2 * stage + side) * L::kScales;
    if (threadIdx.x == 0) {
      mbar_arrive_expect_tx(bar, L::kTile + (L::kTmaScales ? L::kScales : 0));
      tma_load_4d(dst, side ? &p.tm_v : &p.tm_k, bar, 0, kvh, t0, load_b);
      if (L::kTmaScales) tma_load_4d(sdst, side ? &p.tm_vs : &p.tm_ks, bar, 0, kvh, t0, load_b);
    }
    if (!L::kTmaScales) {
#pragma unroll
      for (int r = threadIdx.x; r < kTileKeys; r += kThreads) {
        const bool live = t0 + r < load_len;
        const uint8_t *src = reinterpret_cast<const uint8_t *>(side ? p.v_scales : p.k_scales) +
                             (((size_t)load_b * p.T_cache + (live ? t0 + r : 0)) * p.H_kv + kvh) * L::kScaleRow;
        cp_async_small<L::kScaleRow>(sdst + r * L::kScaleAt, src, live);
      }
      cp_async_arrive(bar);
    }
  };
  auto next_tile = [&] {
    if (L::kTmaScales && threadIdx.x != 0) return;
    if (++load_tile * kTileKeys >= load_len) {
      load_tile = 0;
      load_len = cached(p.cache_len, ++load_b, p.T_cache);
    }
  };
#pragma unroll
  for (int i = 0; i < S; ++i)
    if (i < mine) {
      if (i > 0) next_tile();
      load_side(i, 0);
      load_side(i, 1);
    }

  // ldmatrix rows: K, 16 of this warp's keys (lanes 0..15), the next block's codes 16 lanes on; V, 16 keys and the next
  // block's (or, with one block a warp, the next 16 keys').  A step along the row is an XOR of the swizzled address.
  const uint32_t at_k = base + L::kCodesOff + L::at(warp * 16 * U + (lane & 15), lane >> 4);
  const uint32_t at_v = base + L::kCodesOff + L::kTile +
                        (NW == 2 ? L::at(lane & 15, 2 * warp + (lane >> 4)) : L::at(lane, warp));
  const uint32_t at_vs = base + L::kScalesOff + L::kScales + (warp * 16 * U + (lane & (16 * U - 1))) * L::kScaleAt;
  const uint32_t at_p = smem_u32(p_s) + ((lane & 7) * L::kPRow + (lane >> 3) * 8) * 2;
  int s = 0, phase = 0, done = 0;
  bool ok = true;
  for (int tile = first - before; done < mine && ok; ++b, tile = 0) {
    if (done > 0) len = cached(p.cache_len, b, p.T_cache), before = first + done;
    const int n_tiles = tiles_of(len);
    const int seg = min(n_tiles - tile, mine - done), seg_end = tile + seg;  // its tiles here: tile .. seg_end - 1
    const bool whole = seg == n_tiles;
    if (tile == 0 && kvh == 0 && threadIdx.x == 0) p.start[b] = before;
    // Q^T fragments: head nt * 8 + g; a k-step of a block contracts the elements that one AND opens.  b0 goes with
    // the codes at 2^-24 and takes 16 q, b1 with those at 2^-20.  One n-tile's fragments stay in registers, two
    // n-tiles' go to shared memory (every warp makes the same ones; warp 0's are kept).
    uint4 qb[NT == 1 ? NB : 1];
    uint4 *q_s = reinterpret_cast<uint4 *>(smem + L::kQ) + lane;
    // -8 sum(q) of blocks 2 c4, + 1 for head nt * 8 + g, 2^16 times that (up to 2^15), as high and low fp16 terms: what the
    // low one drops is 2^-34 of the largest |q| (2^-18 without the factor: keys whose large channels meet small ones of q
    // got logits off by that)
    uint32_t off[NT][2];
    float col[NT][2];     // logit = col * accumulated, heads nt * 8 + 2 c4, + 1; positive (Q takes the scale's sign)
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const int h = nt * 8 + g;
      const bool real = h < p.group;
      const uint4 *q =
          reinterpret_cast<const uint4 *>(p.q + ((size_t)b * p.H_q + kvh * p.group + (real ? h : 0)) * D + 8 * c4);
      uint32_t top = 0;
#pragma unroll
      for (int j = 0; j < NB; ++j) {
        const uint4 w = real ? q[4 * j] : make_uint4(0u, 0u, 0u, 0u);
        const uint32_t e[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) top = max(top, max(e[i] & 0x7FFFu, (e[i] >> 16) & 0x7FFFu));
      }
      top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
      top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
      const uint32_t eb = top >> 7;  // exponent field of the largest |q|
      const uint32_t field = eb == 0 || eb == 255 ? 127u : min(max(254u - eb, 1u), 239u);  // f16 stays finite
      const float inv = __uint_as_float((254u - field) << 23);
      const float f = (p.scale_log2 < 0.f ? -1024.f : 1024.f) * __uint_as_float(field << 23), f16 = 16.f * f;
      float own[2] = {0.f, 0.f};
#pragma unroll
      for (int j = 0; j < NB; ++j) {
        const uint4 w = real ? q[4 * j] : make_uint4(0u, 0u, 0u, 0u);  // from L1 now
        const float x0 = f16 * bf16_lo(w.x), x4 = f16 * bf16_lo(w.z), x2 = f16 * bf16_lo(w.y), x6 = f16 * bf16_lo(w.w);
        const float x1 = f * bf16_hi(w.x), x5 = f * bf16_hi(w.z), x3 = f * bf16_hi(w.y), x7 = f * bf16_hi(w.w);
        const uint4 f4 = make_uint4(pack_f16(x0, x4), pack_f16(x1, x5), pack_f16(x2, x6), pack_f16(x3, x7));
        if constexpr (NT == 1) qb[j] = f4;
        else if (warp == 0) q_s[(j * NT + nt) * 32] = f4;
        // exact in fp16 down to 2^-27 of the largest (the factor of 16: 2^-31); below, off by up to 2^-35 of it
        float sum = fmaf(0.0625f, (x0 + x4) + (x2 + x6), (x1 + x5) + (x3 + x7));
        sum += __shfl_xor_sync(0xffffffffu, sum, 1);
        sum += __shfl_xor_sync(0xffffffffu, sum, 2);
        if (c4 == j / 2) own[j & 1] = sum * (-8.f / 1048576.f * 65536.f);
      }
      const uint32_t hi = pack_f16(own[0], own[1]);
      off[nt][0] = hi;
      off[nt][1] = pack_f16(own[0] - f16_lo(hi), own[1] - f16_hi(hi));
      // a scale of 0 becomes one whose logits are 0 and whose masked keys still get no weight
      const float unit = fmaxf(1024.f * fabsf(p.scale_log2), 1e-30f);
      col[nt][0] = fmaxf(__shfl_sync(0xffffffffu, inv, 8 * c4) * unit, 1e-37f);
      col[nt][1] = fmaxf(__shfl_sync(0xffffffffu, inv, 8 * c4 + 4) * unit, 1e-37f);
    }
    if constexpr (NT == 2) __syncthreads();

    float o[2 * NW][NT][4];
#pragma unroll
    for (int mt = 0; mt < 2 * NW; ++mt)
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) o[mt][nt][0] = o[mt][nt][1] = o[mt][nt][2] = o[mt][nt][3] = 0.f;
    // sums over the warp's keys, columns the heads 2 c4, + 1: p s of block g (0, 1)
    float sums[NT][4] = {};
    float l_run[NT][2] = {};  // sums of p over the thread's keys, as it is before it is rounded for the products
    // maximum of heads nt * 8 + 2 c4, + 1 over all warps' keys (before col), at first less than any
    float m_run[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) m_run[nt][0] = m_run[nt][1] = -FLT_MAX;
    // block g's power of two, in both halves, that its scales are multiplied with (2^14 until the first rescaling)
    uint32_t power = 0x74007400u;

    for (; tile < seg_end; ++tile, ++done) {
      bool landed = mbar_wait(&full[2 * s], phase, p.status);
      // ---- logits: S^T = K Q^T of the warp's keys (g, g + 8 of each 16), block by block ----
      const uint32_t kb = at_k + 2 * s * L::kTile;
      const uint8_t *ksc = smem + L::kScalesOff + 2 * s * L::kScales + (warp * 16 * U + g) * L::kScaleAt;
      float sc[U][NT][4];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        uint32_t k0 = 0, k1 = 0;  // blocks 2 c4, + 1: scales of keys g and g + 8
        if (NB == 8 || c4 < NB / 2) {
          k0 = *reinterpret_cast<const uint32_t *>(ksc + u * 16 * L::kScaleAt + c4 * 4);
          k1 = *reinterpret_cast<const uint32_t *>(ksc + (u * 16 + 8) * L::kScaleAt + c4 * 4);
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          mma_f16(sc[u][nt], k0, k1, k0, k1, off[nt][0], off[nt][1], 0.f, 0.f, 0.f, 0.f);
#pragma unroll
          for (int c = 0; c < 4; ++c) sc[u][nt][c] *= 1.f / 65536.f;
        }
      }
      uint2 s4[U][2];  // scales of four blocks, keys g and g + 8
#pragma unroll
      for (int j = 0; j < NB; j += 2) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
          uint32_t r[4];  // keys g (r0) and g + 8 (r1) of block j, the same of block j + 1
          ldsm_x4((kb + u * 16 * L::kRow) ^ (j << 4), r[0], r[1], r[2], r[3]);
          if (j % 4 == 0) {
            s4[u][0] = *reinterpret_cast<const uint2 *>(ksc + u * 16 * L::kScaleAt + j * 2);
            s4[u][1] = *reinterpret_cast<const uint2 *>(ksc + (u * 16 + 8) * L::kScaleAt + j * 2);
          }
          const uint32_t s0 = j % 4 == 0 ? s4[u][0].x : s4[u][0].y, s1 = j % 4 == 0 ? s4[u][1].x : s4[u][1].y;
#pragma unroll
          for (int jj = 0; jj < 2; ++jj) {
            const Opened a = open_codes(r[2 * jj]), c = open_codes(r[2 * jj + 1]);
            const float f0 = jj ? f16_hi(s0) : f16_lo(s0), f1 = jj ? f16_hi(s1) : f16_lo(s1);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              uint4 qf;
              if constexpr (NT == 1) qf = qb[j + jj];
              else qf = q_s[((j + jj) * NT + nt) * 32];
              float t[4];
              mma_f16(t, a.x0, c.x0, a.x1, c.x1, qf.x, qf.y, 0.f, 0.f, 0.f, 0.f);
              mma_f16(t, a.x2, c.x2, a.x3, c.x3, qf.z, qf.w);
              sc[u][nt][0] = fmaf(f0, t[0], sc[u][nt][0]);
              sc[u][nt][1] = fmaf(f0, t[1], sc[u][nt][1]);
              sc[u][nt][2] = fmaf(f1, t[2], sc[u][nt][2]);
              sc[u][nt][3] = fmaf(f1, t[3], sc[u][nt][3]);
            }
          }
        }
      }
      landed &= mbar_wait(&full[2 * s + 1], phase, p.status);
      const int key0 = tile * kTileKeys + warp * 16 * U + g;
      if (tile == n_tiles - 1) {
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int c = 0; c < 4; ++c)
              if (key0 + u * 16 + (c >> 1) * 8 >= len) sc[u][nt][c] = -INFINITY;
      }
      if constexpr (kAcc) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            const int hd = nt * 8 + 2 * c4 + c;
            if (hd >= p.group) continue;
            float *row = p.logits + ((size_t)b * p.H_q + kvh * p.group + hd) * p.T_cache + key0;
#pragma unroll
            for (int r = 0; r < 2 * U; ++r)
              if (key0 + r * 8 < len) row[r * 8] = sc[r >> 1][nt][(r & 1) * 2 + c] * col[nt][c];
          }
      }
      // V's scales of the warp's keys, transposed: block g of keys 2 c4, + 1 of every 8
      uint32_t vt[2 * U];
      auto load_vt = [&](uint32_t(&x)[2 * U]) {
        if constexpr (U == 2) ldsm_x4_t(at_vs + 2 * s * L::kScales, x[0], x[1], x[2], x[3]);
        else ldsm_x2_t(at_vs + 2 * s * L::kScales, x[0], x[1]);
      };
      load_vt(vt);
      uint32_t any = 0;
#pragma unroll
      for (int r = 0; r < 2 * U; ++r) {
        if (NB < 8 && g >= NB) vt[r] = 0;
        if (tile == n_tiles - 1) {  // past the end they may hold anything: no weight is given, but 0 x NaN would count
          const int key = tile * kTileKeys + warp * 16 * U + r * 8 + 2 * c4;
          if (key + 1 >= len) vt[r] = key < len ? vt[r] & 0xFFFFu : 0u;
        }
        vt[r] = mul_f16x2(vt[r], power);
        any |= vt[r];
      }
      // ---- a new maximum, or a scale that its block's power leaves at 2 or more: rescale ----
      const bool large = (any & 0x40004000u) && power != 0x01000100u;
      bool change = large || !landed;
      float top[NT][2];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          top[nt][c] = fmaxf(sc[0][nt][c], sc[0][nt][c + 2]);
          if constexpr (U == 2) top[nt][c] = fmaxf(top[nt][c], fmaxf(sc[1][nt][c], sc[1][nt][c + 2]));
          change |= top[nt][c] > m_run[nt][c];
        }
      // the barrier also tells that this tile's K, the last tile's V and the last weights have been read
      const bool rescale = __syncthreads_or(change);
      if (done > 0 && done + S - 1 < mine) load_side(s == 0 ? S - 1 : s - 1, 1);
      if (done + S < mine) {
        next_tile();
        load_side(s, 0);
      }
      if (rescale) {
        if (__syncthreads_or(!landed)) {  // a wait ran out: what is in flight lands (bounded) before the CTA exits
          for (int i = done; i < min(mine, done + S + 1); ++i) {
            mbar_wait(&full[2 * (i % S)], (i / S) & 1, p.status);
            if (i < done + S) mbar_wait(&full[2 * (i % S) + 1], (i / S) & 1, p.status);
          }
          ok = false;
          break;
        }
        if (__syncthreads_or(large)) {
          uint32_t x[2 * U], big = 0;  // as they are (multiplied, they may have overflowed), but zero behind the end
          load_vt(x);
#pragma unroll
          for (int r = 0; r < 2 * U; ++r) {
            x[r] &= ((vt[r] & 0x7FFFu) ? 0xFFFFu : 0u) | ((vt[r] & 0x7FFF0000u) ? 0xFFFF0000u : 0u);
            big = max(big, max(x[r] & 0x7FFFu, (x[r] >> 16) & 0x7FFFu));
          }
          big = max(big, __shfl_xor_sync(0xffffffffu, big, 1));
          big = max(big, __shfl_xor_sync(0xffffffffu, big, 2));
          if (c4 == 0) largest[warp * 8 + g] = big;
          __syncthreads();
#pragma unroll
          for (int w = 0; w < kWarps; ++w) big = max(big, largest[w * 8 + g]);
          const uint32_t now = min(power & 0xFFFFu, power_for(big));
          const float shrink = f16_lo(now) * reciprocal(power);  // of what block g has collected
          power = now * 0x10001u;
#pragma unroll
          for (int r = 0; r < 2 * U; ++r) vt[r] = mul_f16x2(x[r], power);
#pragma unroll
          for (int jj = 0; jj < NW; ++jj) {
            const float own = __shfl_sync(0xffffffffu, shrink, 4 * (warp * NW + jj));  // of the warp's block
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
              for (int c = 0; c < 4; ++c) o[2 * jj][nt][c] *= own, o[2 * jj + 1][nt][c] *= own;
          }
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) sums[nt][0] *= shrink, sums[nt][1] *= shrink;
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            float mx = top[nt][c];
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 4));
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 8));
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 16));
            if (lane < 4) stat[warp * 8 * NT + nt * 8 + 2 * c4 + c] = mx;
          }
        __syncthreads();
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            float m_new = m_run[nt][c];
#pragma unroll
            for (int w = 0; w < kWarps; ++w) m_new = fmaxf(m_new, stat[w * 8 * NT + nt * 8 + 2 * c4 + c]);
            const float alpha = ex2((m_run[nt][c] - m_new) * col[nt][c]);
            m_run[nt][c] = m_new;
            sums[nt][c] *= alpha;
            l_run[nt][c] *= alpha;
#pragma unroll
            for (int mt = 0; mt < 2 * NW; ++mt) {
              o[mt][nt][c] *= alpha;
              o[mt][nt][c + 2] *= alpha;
            }
          }
      }
      // ---- weights to shared memory, as B fragments want them (p_s[head][key]); their sums with V's scales and plain
#pragma unroll
      for (int u = 0; u < U; ++u)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          float p0, p1, p2, p3;
          weights2(p0, p1, sc[u][nt][0], sc[u][nt][1], m_run[nt], col[nt]);
          weights2(p2, p3, sc[u][nt][2], sc[u][nt][3], m_run[nt], col[nt]);
          uint32_t *row = reinterpret_cast<uint32_t *>(p_s + (nt * 8 + g) * L::kPRow + (warp * U + u) * 16 + 2 * c4);
          const uint32_t b0 = transpose8(pack_f16(p0, p1)), b1 = transpose8(pack_f16(p2, p3));
          row[0] = b0;
          row[4] = b1;
          l_run[nt][0] += p0 + p2;
          l_run[nt][1] += p1 + p3;
          mma_f16(sums[nt], vt[2 * u], 0u, vt[2 * u + 1], 0u, b0, b1);
        }
      // V's scales in the order in which the products want them, over the rows that every warp has read by now:
      // [32 keys][block][c4] keys 2 c4, + 1 of each of the four 8-key groups
      uint8_t *vs_t = smem + L::kScalesOff + (2 * s + 1) * L::kScales + c4 * 16;
      if (NB == 8 || g < NB) {
        if constexpr (U == 2)
          *reinterpret_cast<uint4 *>(vs_t + (warp * 8 + g) * 64) = make_uint4(vt[0], vt[1], vt[2], vt[3]);
        else
          *reinterpret_cast<uint2 *>(vs_t + ((warp >> 1) * 8 + g) * 64 + (warp & 1) * 8) = make_uint2(vt[0], vt[1]);
      }
      if (L::kTmaScales) tc::fence_proxy_async_smem();  // ahead of the next copy into this stage
      __syncthreads();
      // ---- O^T += V^T P'^T over the tile's keys, the warp's blocks: block J gives elements 4 g, 4 g + 1 (rows g and
      // g + 8 of m-tile 2 J) and 4 g + 2, 4 g + 3 ----
      const uint32_t vb = at_v + 2 * s * L::kTile;
#pragma unroll
      for (int k = 0; k < kTileKeys; k += 32) {
        uint32_t pb[NT][4];  // weights of head g: keys 2 c4, + 1 of each of the four 8-key groups
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
          ldsm_x4(at_p + (nt * 8 * L::kPRow + k) * 2, pb[nt][0], pb[nt][1], pb[nt][2], pb[nt][3]);
        uint32_t x[2][4];  // [16 keys][keys 0..7, 8..15 of the first block, the same of the second]
        if constexpr (NW == 2) {
          ldsm_x4_t(vb + k * L::kRow, x[0][0], x[0][1], x[0][2], x[0][3]);
          ldsm_x4_t(vb + (k + 16) * L::kRow, x[1][0], x[1][1], x[1][2], x[1][3]);
        } else {
          ldsm_x4_t(vb + k * L::kRow, x[0][0], x[0][1], x[1][0], x[1][1]);
        }
        uint4 sc4[NW];
#pragma unroll
        for (int jj = 0; jj < NW; ++jj)
          sc4[jj] = *reinterpret_cast<const uint4 *>(vs_t + (k / 32 * 8 + warp * NW + jj) * 64);
#pragma unroll
        for (int u = 0; u < 2; ++u) {
#pragma unroll
          for (int jj = 0; jj < NW; ++jj) {
            const Opened a = open_bytes(x[u][2 * jj]), c = open_bytes(x[u][2 * jj + 1]);
            const uint32_t lo = u ? sc4[jj].z : sc4[jj].x, hi = u ? sc4[jj].w : sc4[jj].y;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              const uint32_t b0 = mul_f16x2(pb[nt][2 * u], lo), b1 = mul_f16x2(pb[nt][2 * u + 1], hi);
              float(&oa)[4] = o[2 * jj][nt], (&ob)[4] = o[2 * jj + 1][nt];
              mma_f16(oa, a.x0, a.x1, c.x0, c.x1, b0, b1);
              mma_f16(ob, a.x2, a.x3, c.x2, c.x3, b0, b1);
            }
          }
        }
      }
      if (++s == S) s = 0, phase ^= 1;
      if (tile % (kFoldKeys / kTileKeys) == kFoldKeys / kTileKeys - 1 || tile == seg_end - 1) {
        // the offset's sums over the warps join the accumulators: -8 at 2^-24 and at 2^-20 in rows g, at 2^-20 in g + 8
        float *bias_s = reinterpret_cast<float *>(smem + L::kP);
        __syncthreads();  // the weights have been read
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          if (g < NB)
            *reinterpret_cast<float2 *>(bias_s + ((warp * NB + g) * NT + nt) * 8 + 2 * c4) =
                make_float2(sums[nt][0], sums[nt][1]);
          sums[nt][0] = sums[nt][1] = 0.f;
        }
        __syncthreads();
#pragma unroll
        for (int jj = 0; jj < NW; ++jj)
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int c = 0; c < 2; ++c) {
              float sum = 0.f;
#pragma unroll
              for (int w = 0; w < kWarps; ++w) sum += bias_s[((w * NB + warp * NW + jj) * NT + nt) * 8 + 2 * c4 + c];
#pragma unroll
              for (int mt = 2 * jj; mt < 2 * jj + 2; ++mt) {
                o[mt][nt][c] = fmaf(sum, -136.f / 16777216.f, o[mt][nt][c]);
                o[mt][nt][c + 2] = fmaf(sum, -8.f / 1048576.f, o[mt][nt][c + 2]);
              }
            }
      }
    }

    // else from here on (earlier, it would take issue slots: 2 us at 84,000 tokens)
    if (done == mine && !brief) asm volatile("griddepcontrol.launch_dependents;\n");
    // ---------------- sums over the warps, and the segment's result ----------------
    uint2 gate[NT][2][NW] = {};
    if (whole && p.gate) {  // on their way during the exchange
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int c = 0; c < 2; ++c)
#pragma unroll
          for (int jj = 0; jj < NW; ++jj)
            if (nt * 8 + 2 * c4 + c < p.group)
              gate[nt][c][jj] = *reinterpret_cast<const uint2 *>(
                  p.gate + ((size_t)b * p.H_q + kvh * p.group + nt * 8 + 2 * c4 + c) * D + (warp * NW + jj) * 32 +
                  4 * g);
    }
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        float l = l_run[nt][c];
        l += __shfl_xor_sync(0xffffffffu, l, 4);
        l += __shfl_xor_sync(0xffffffffu, l, 8);
        l += __shfl_xor_sync(0xffffffffu, l, 16);
        if (lane < 4) stat[warp * 8 * NT + nt * 8 + 2 * c4 + c] = l * (1.f / (1 << (int)kWeightExp));
      }
    __syncthreads();
    // what a unit of the products stands for: 2^24 (low nibbles) or 2^20, less the weights' 2^14 and the block's power
    const float unit = reciprocal(power) * (1.f / (1 << (int)kWeightExp));
    float unit_lo[NW], unit_hi[NW];
#pragma unroll
    for (int jj = 0; jj < NW; ++jj) {
      const float of = __shfl_sync(0xffffffffu, unit, 4 * (warp * NW + jj));
      unit_lo[jj] = 16777216.f * of, unit_hi[jj] = 1048576.f * of;
    }
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const int hd = nt * 8 + 2 * c4 + c;
        if (hd >= p.group) continue;
        float l = 0.f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) l += stat[w * 8 * NT + hd];
        const size_t h = kvh * p.group + hd, row = (size_t)(b + grp) * p.H_q + h;  // b + grp: a row a (sequence, group)
        if (warp == 0 && g == 0)
          *reinterpret_cast<float2 *>(p.part_ml + row * 2) =
              make_float2(m_run[nt][c] == -FLT_MAX ? -INFINITY : m_run[nt][c] * col[nt][c], l);
#pragma unroll
        for (int jj = 0; jj < NW; ++jj) {
          const int dd = (warp * NW + jj) * 32 + 4 * g;
          const float lo0 = o[2 * jj][nt][c] - o[2 * jj][nt][c + 2], hi0 = o[2 * jj][nt][c + 2];
          const float lo1 = o[2 * jj + 1][nt][c] - o[2 * jj + 1][nt][c + 2], hi1 = o[2 * jj + 1][nt][c + 2];
          const float4 v = make_float4(lo0 * unit_lo[jj], hi0 * unit_hi[jj], lo1 * unit_lo[jj], hi1 * unit_hi[jj]);
          if (whole)
            *reinterpret_cast<uint2 *>(p.o + ((size_t)b * p.H_q + h) * D + dd) = output4(v, l, p.gate, gate[nt][c][jj]);
          else
            *reinterpret_cast<float4 *>(p.part_o + row * D + dd) = v;
        }
      }
  }
}

// Keys of a tile: 128 (32 a warp: fewer instructions a key, 12% of the time at B = 64 x 131,072), but 64 where the
// caches hold fewer tiles than the GPU has room for, so that more CTAs share the latency.
int q4_groups_of_16(int B, int H_q, int H_kv, int d, int T_cache) {
  const long long tiles = (long long)B * H_kv * ((T_cache + 127) / 128);
  return tiles < 148LL * ctas_per_sm(d, H_q / H_kv > 8 ? 2 : 1, 2) ? 1 : 2;
}

// Groups of CTAs (one CTA a kv head) that share the tiles: as many as fill the GPU once, whatever the lengths are.
int q4_groups(int B, int H_q, int H_kv, int d, int T_cache) {
  const int u = q4_groups_of_16(B, H_q, H_kv, d, T_cache), keys = kWarps * 16 * u;
  const long long tiles = (long long)B * ((T_cache + keys - 1) / keys);
  const long long fill = 148 * ctas_per_sm(d, H_q / H_kv > 8 ? 2 : 1, u) / H_kv, n = fill < tiles ? fill : tiles;
  return n < 1 ? 1 : (int)n;
}

size_t round256(size_t n) { return (n + 255) & ~size_t(255); }

template <int D, int NT, int U>
cudaError_t launch_split(const DecodeQ4Params &p, int groups, bool acc, cudaStream_t s) {
  auto kern = acc ? q4_split_kernel<D, NT, U, true> : q4_split_kernel<D, NT, U, false>;
  const int smem = Q4Smem<D, NT, U>::kTotal;
  static std::atomic<uint64_t> done[2];
  const cudaError_t e = once_per_device(done[acc], [&] {
    const cudaError_t r = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (r != cudaSuccess) return r;  // and all of the SM's memory, for the CTAs that the registers allow
    return cudaFuncSetAttribute(kern, cudaFuncAttributePreferredSharedMemoryCarveout, cudaSharedmemCarveoutMaxShared);
  });
  if (e != cudaSuccess) return e;
  kern<<<dim3(p.H_kv, groups), kThreads, smem, s>>>(p);
  return cudaGetLastError();
}

template <int D>
cudaError_t launch_d(const DecodeQ4Params &p, int groups, int u, bool acc, cudaStream_t s) {
  if (p.group > 8) return u == 2 ? launch_split<D, 2, 2>(p, groups, acc, s) : launch_split<D, 2, 1>(p, groups, acc, s);
  return u == 2 ? launch_split<D, 1, 2>(p, groups, acc, s) : launch_split<D, 1, 1>(p, groups, acc, s);
}

}  // namespace

// first tiles, statistics, partial outputs, logits (accumulating calls)
size_t attn_decode_q4_workspace(int B, int H_q, int H_kv, int d, int T_cache, bool with_acc) {
  const size_t rows = ((size_t)B + q4_groups(B, H_q, H_kv, d, T_cache)) * H_q;
  return round256(((size_t)B + 1) * sizeof(int)) + round256(rows * 2 * sizeof(float)) +
         round256(rows * d * sizeof(float)) + (with_acc ? (size_t)B * H_q * T_cache * sizeof(float) : 0);
}

cudaError_t launch_attn_decode_q4(const AttnDecodeQ4Args &a, cudaStream_t s) {
  if (a.B == 0) return cudaSuccess;
  const int groups = q4_groups(a.B, a.H_q, a.H_kv, a.d, a.T_cache);
  const int u = q4_groups_of_16(a.B, a.H_q, a.H_kv, a.d, a.T_cache), tile = kWarps * 16 * u;
  const size_t rows = ((size_t)a.B + groups) * a.H_q;
  DecodeQ4Params p;
  uint8_t *ws = reinterpret_cast<uint8_t *>(a.workspace);
  p.start = reinterpret_cast<int *>(ws);
  ws += round256(((size_t)a.B + 1) * sizeof(int));
  p.part_ml = reinterpret_cast<float *>(ws);
  ws += round256(rows * 2 * sizeof(float));
  p.part_o = reinterpret_cast<float *>(ws);
  ws += round256(rows * a.d * sizeof(float));
  p.logits = reinterpret_cast<float *>(ws);
  AttnFinishArgs f = {p.part_o, p.part_ml, p.logits, a.cache_len, a.gate,   a.o, a.acc_in, a.acc_out, a.B,
                      a.T_cache, a.H_q,    a.H_kv,   a.d,         groups, tile, p.start};
  if (a.T_cache == 0) {  // nothing to attend: the outputs are zero
    f.start = nullptr;
    return launch_attn_finish(f, s);
  }
  p.q = a.q;
  p.gate = a.gate;
  p.k_scales = a.k_scales;
  p.v_scales = a.v_scales;
  p.cache_len = a.cache_len;
  p.o = a.o;
  p.B = a.B;
  p.T_cache = a.T_cache;
  p.H_q = a.H_q;
  p.H_kv = a.H_kv;
  p.group = a.H_q / a.H_kv;
  p.scale_log2 = a.scale * kLog2e;
  p.status = device_status_ptr();
  const uint64_t dims[4] = {(uint64_t)a.d / 2, (uint64_t)a.H_kv, (uint64_t)a.T_cache, (uint64_t)a.B};
  const uint64_t strides[3] = {(uint64_t)a.d / 2, (uint64_t)a.H_kv * a.d / 2, (uint64_t)a.T_cache * a.H_kv * a.d / 2};
  const uint32_t box[4] = {(uint32_t)a.d / 2, 1, (uint32_t)tile, 1};
  const uint64_t sdims[4] = {(uint64_t)a.d / 32, (uint64_t)a.H_kv, (uint64_t)a.T_cache, (uint64_t)a.B};
  const uint64_t sstrides[3] = {(uint64_t)a.d / 16, (uint64_t)a.H_kv * a.d / 16,
                                (uint64_t)a.T_cache * a.H_kv * a.d / 16};
  const uint32_t sbox[4] = {(uint32_t)a.d / 32, 1, (uint32_t)tile, 1};
  const CUtensorMapSwizzle sw = a.d == 256 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B;
  memset(&p.tm_ks, 0, sizeof(p.tm_ks));
  memset(&p.tm_vs, 0, sizeof(p.tm_vs));
  if (encode_tmap(&p.tm_k, CU_TENSOR_MAP_DATA_TYPE_UINT8, 4, a.k_values, dims, strides, box, sw) != CUDA_SUCCESS ||
      encode_tmap(&p.tm_v, CU_TENSOR_MAP_DATA_TYPE_UINT8, 4, a.v_values, dims, strides, box, sw) != CUDA_SUCCESS ||
      (a.d == 256 && (encode_tmap(&p.tm_ks, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 4, a.k_scales, sdims, sstrides, sbox,
                                  CU_TENSOR_MAP_SWIZZLE_NONE) != CUDA_SUCCESS ||
                      encode_tmap(&p.tm_vs, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 4, a.v_scales, sdims, sstrides, sbox,
                                  CU_TENSOR_MAP_SWIZZLE_NONE) != CUDA_SUCCESS))) {
    set_error("gqa_attn_decode_q4_0: cuTensorMapEncodeTiled failed for the q4_0 cache");
    return cudaErrorInvalidValue;
  }
  const bool acc = a.acc_out != nullptr;
  const cudaError_t e = a.d == 256 ? launch_d<256>(p, groups, u, acc, s) : launch_d<128>(p, groups, u, acc, s);
  return e != cudaSuccess ? e : launch_attn_finish(f, s);
}

}  // namespace hh
