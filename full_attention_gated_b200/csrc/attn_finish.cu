// attn_finish.cu -- the end of a split decode call: the splits of every query
// head merged into the output, and every position's attention weight, summed
// over the query heads of its group, added to what the position has drawn so
// far (the figure that cache eviction goes by; "The economics of hybrid
// attention" prices the cache it bounds).
//
// The split kernels leave per split a maximum m (log2 domain), a sum l and an
// unnormalised output, and, where weights are wanted, the step's logits.  Both
// parts start from the merged statistics M = max m, L = sum l exp2(m - M):
//   output: sum over the splits of exp2(m - M) o / L, gated, rounded to bf16
//   once.  16 threads hold 64 elements of a query head's output; up to 16 such
//   teams share its parts, as many as the parts are on average, and a CTA takes
//   16 teams (64 sequences of a part or two: 8 us; with 16 teams for each unit 27).
//   weights: exp2(logit - M) / L, the group's heads in order, then acc.  CTA = (1024
//   positions, kv head, sequence), one thread for one position of one kv head:
//   no atomics.  Bound by the reads of the logits (4 bytes a query head and
//   position) and of acc.
// One launch for both; it is launched to start while the split kernel drains
// (it waits for that kernel's results itself), which hides its launch.
#include <math.h>

#include "common.cuh"
#include "internal_kv.h"

namespace hh {

namespace {

constexpr int kThreads = 256;
constexpr int kMaxGroup = 16;
constexpr int kSlice = 64;                       // output elements of a team
constexpr int kLanes = kSlice / 4, kTeams = kThreads / kLanes;
constexpr int kPositions = 4 * kThreads;         // a CTA

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}

// the parts of head h of sequence b: n rows from `row` on, `step` apart
struct Parts {
  size_t row, step;
  int n;
};
__device__ __forceinline__ Parts parts_of(const AttnFinishArgs &p, int b, int h, int len) {
  if (!p.start)
    return {((size_t)b * p.H_q + h) * p.n_splits, 1, min(p.n_splits, (len + p.split_len - 1) / p.split_len)};
  const int share = p.start[p.B], first = p.start[b], tiles = max(1, (len + p.split_len - 1) / p.split_len);
  // below n_splits, unless a wait ran out in the split kernel and left `start` unwritten: then only the status counts
  const unsigned last = (unsigned)p.n_splits - 1u, per = (unsigned)max(share, 1);
  const int u0 = (int)min((unsigned)first / per, last), u1 = (int)min(((unsigned)first + tiles - 1u) / per, last);
  return {(size_t)(b + u0) * p.H_q + h, (size_t)p.H_q, max(u1 - u0, 0) + 1};
}

// `teams` (a power of two up to kTeams) share the parts of 64 elements of a head's output
__global__ void __launch_bounds__(kThreads) attn_finish_kernel(const __grid_constant__ AttnFinishArgs p, int teams,
                                                              unsigned merge_ctas) {
  __shared__ float4 acc_s[kTeams][kLanes];
  __shared__ float s_m[kMaxGroup], s_l[kMaxGroup];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (blockIdx.x < merge_ctas) {
    const int team = tid / kLanes, x = tid % kLanes, first = team & ~(teams - 1);  // first: of the teams that share
    const unsigned n_slices = (unsigned)p.d / kSlice, units = (unsigned)p.B * p.H_q * n_slices;
    const unsigned unit = blockIdx.x * (kTeams / teams) + team / teams, slice = unit % n_slices, bh = unit / n_slices;
    const unsigned b = bh / p.H_q;
    const bool real = unit < units;
    int len = 0;
    uint2 gate = make_uint2(0u, 0u);
    const size_t at = (size_t)bh * p.d + slice * kSlice + x * 4;
    if (real) {
      len = p.cache_len ? p.cache_len[b] : p.T_cache;
      len = len < 0 ? 0 : (len > p.T_cache ? p.T_cache : len);
      if (p.gate && team == first) gate = *reinterpret_cast<const uint2 *>(p.gate + at);
    }
    asm volatile("griddepcontrol.wait;\n" ::: "memory");  // the split kernel's results
    Parts parts = {0, 0, 0};
    if (real) parts = parts_of(p, (int)b, (int)(bh - b * p.H_q), len);
    const int n = parts.n;
    const float2 *ml = reinterpret_cast<const float2 *>(p.part_ml) + parts.row;
    const float4 *po = reinterpret_cast<const float4 *>(p.part_o) + parts.row * (p.d / 4) + slice * kLanes + x;
    const bool done = p.start && n == 1;
    // each team's own running merge of its parts, then the teams'
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    float M = -INFINITY, l = 0.f;
    if (!done) {
#pragma unroll 4
      for (int s = team - first; s < n; s += teams) {
        const float4 v = po[s * parts.step * (p.d / 4)];
        const float2 st = ml[s * parts.step];
        const float m_new = fmaxf(M, st.x), base = m_new == -INFINITY ? 0.f : m_new;
        const float f0 = ex2(M - base), f = ex2(st.x - base);
        M = m_new;
        l = l * f0 + st.y * f;
        acc.x = acc.x * f0 + v.x * f;
        acc.y = acc.y * f0 + v.y * f;
        acc.z = acc.z * f0 + v.z * f;
        acc.w = acc.w * f0 + v.w * f;
      }
    }
    if (teams > 1) {
      acc_s[team][x] = acc;
      if (x == 0) s_m[team] = M, s_l[team] = l;
      __syncthreads();
      if (team != first) return;
      for (int i = 1; i < teams; ++i) M = fmaxf(M, s_m[first + i]);
      const float base = M == -INFINITY ? 0.f : M;
      acc = make_float4(0.f, 0.f, 0.f, 0.f);
      l = 0.f;
      for (int i = 0; i < teams; ++i) {
        const float4 v = acc_s[first + i][x];
        const float f = ex2(s_m[first + i] - base);
        l += s_l[first + i] * f;
        acc.x += v.x * f, acc.y += v.y * f, acc.z += v.z * f, acc.w += v.w * f;
      }
    }
    if (done || !real) return;
    float r[4] = {acc.x, acc.y, acc.z, acc.w};
    const float gf[4] = {bf16_lo(gate.x), bf16_hi(gate.x), bf16_lo(gate.y), bf16_hi(gate.y)};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      r[i] = n > 0 ? r[i] / l : 0.f;
      if (p.gate && n > 0) r[i] *= 1.f / (1.f + expf(-gf[i]));
    }
    *reinterpret_cast<uint2 *>(p.o + at) = make_uint2(pack_bf16(r[0], r[1]), pack_bf16(r[2], r[3]));
    return;
  }
  // ---- weights ----
  const unsigned chunks = (p.T_cache + kPositions - 1) / kPositions, cta = blockIdx.x - merge_ctas;
  const unsigned row = cta / chunks, b = row / p.H_kv;  // row: (sequence, kv head)
  const int group = p.H_q / p.H_kv, j0 = (int)(cta % chunks) * kPositions + tid;
  int len = p.cache_len ? p.cache_len[b] : p.T_cache;
  len = len < 0 ? 0 : (len > p.T_cache ? p.T_cache : len);
  if (j0 - tid >= len) return;
  const size_t at = (size_t)row * p.T_cache + j0, head0 = (size_t)row * group;
  float was[4], sum[4] = {};  // the step's weights are summed apart: added one by one, they would be lost in a large total
#pragma unroll
  for (int r = 0; r < 4; ++r) was[r] = p.acc_in && j0 + r * kThreads < len ? p.acc_in[at + r * kThreads] : 0.f;
  asm volatile("griddepcontrol.wait;\n" ::: "memory");
  // the logits of up to eight heads are on their way while the statistics are merged
  const float *lg = p.logits + head0 * p.T_cache + j0;
  float x[8][4];
  auto fetch = [&](int g0) {
#pragma unroll
    for (int g = 0; g < 8; ++g)
#pragma unroll
      for (int r = 0; r < 4; ++r)
        x[g][r] =
            g0 + g < group && j0 + r * kThreads < len ? lg[(size_t)(g0 + g) * p.T_cache + r * kThreads] : -INFINITY;
  };
  fetch(0);
  for (int g = warp; g < group; g += kThreads / 32) {
    const Parts parts = parts_of(p, (int)b, (int)(row - b * p.H_kv) * group + g, len);
    const float2 *ml = reinterpret_cast<const float2 *>(p.part_ml) + parts.row;
    float m = -INFINITY, l = 0.f;
    for (int s = lane; s < parts.n; s += 32) m = fmaxf(m, ml[s * parts.step].x);
    m = warp_max(m);
    for (int s = lane; s < parts.n; s += 32) {
      const float2 st = ml[s * parts.step];
      l += m == -INFINITY ? 0.f : st.y * ex2(st.x - m);
    }
    l = warp_sum(l);
    if (lane == 0) s_m[g] = m, s_l[g] = 1.f / l;
  }
  __syncthreads();
  for (int g0 = 0; g0 < group; g0 += 8) {
    if (g0 > 0) fetch(g0);
#pragma unroll
    for (int g = 0; g < 8; ++g)
      if (g0 + g < group)
#pragma unroll
        for (int r = 0; r < 4; ++r) sum[r] = fmaf(ex2(x[g][r] - s_m[g0 + g]), s_l[g0 + g], sum[r]);
  }
#pragma unroll
  for (int r = 0; r < 4; ++r)
    if (j0 + r * kThreads < len) p.acc_out[at + r * kThreads] = was[r] + sum[r];
}

}  // namespace

cudaError_t launch_attn_finish(const AttnFinishArgs &a, cudaStream_t s) {
  // parts of a sequence: all its splits, or its share of the groups (the rows beyond one a sequence) and the one it
  // begins or ends in
  const int parts = a.start ? (a.n_splits + a.B - 1) / a.B + 1 : a.n_splits;
  int teams = 1;
  while (teams < kTeams && teams < parts) teams *= 2;
  const unsigned units = (unsigned)a.B * a.H_q * (a.d / kSlice), per_cta = kTeams / teams;
  const unsigned merge = (units + per_cta - 1) / per_cta;
  const unsigned weights = a.acc_out ? (unsigned)a.B * a.H_kv * ((a.T_cache + kPositions - 1) / kPositions) : 0;
  if (merge + weights == 0) return cudaSuccess;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(merge + weights);
  cfg.blockDim = dim3(kThreads);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, attn_finish_kernel, a, teams, merge);
}

}  // namespace hh
