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
//   once.  CTA = (64 elements, query head, sequence): 16 groups of threads take
//   every 16th split.
//   weights: exp2(logit - M) / L, the group's heads in order.  CTA = (1024
//   positions, kv head, sequence), one thread for one position of one kv head:
//   no atomics.  Bound by the reads of the logits (4 bytes a query head and
//   position) and of acc.
// One launch for both; it is launched to start while the split kernel drains
// (it waits for that kernel's results itself), which hides its launch.
#include <math.h>

#include "common.cuh"
#include "internal.h"

namespace hh {

namespace {

constexpr int kThreads = 256;
constexpr int kMaxGroup = 16;
constexpr int kSlice = 64;                       // output elements a CTA
constexpr int kLanes = kSlice / 4, kGroups = kThreads / kLanes;
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
  if (!p.start) return {((size_t)b * p.H_q + h) * p.n_splits, 1, min(p.n_splits, (len + p.split_len - 1) / p.split_len)};
  const int share = p.start[p.B], first = p.start[b], tiles = max(1, (len + p.split_len - 1) / p.split_len);
  const int u0 = first / share, u1 = (first + tiles - 1) / share;
  return {(size_t)(b + u0) * p.H_q + h, (size_t)p.H_q, u1 - u0 + 1};
}

__global__ void __launch_bounds__(kThreads) attn_finish_kernel(const __grid_constant__ AttnFinishArgs p, int n_slices,
                                                              unsigned merge_ctas) {
  __shared__ float4 acc_s[kGroups][kLanes];
  __shared__ float s_m[kMaxGroup], s_l[kMaxGroup];
  asm volatile("griddepcontrol.wait;\n" ::: "memory");  // the split kernel's results
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (blockIdx.x < merge_ctas) {
    const unsigned slice = blockIdx.x % n_slices, bh = blockIdx.x / n_slices, b = bh / p.H_q;
    int len = p.cache_len ? p.cache_len[b] : p.T_cache;
    len = len < 0 ? 0 : (len > p.T_cache ? p.T_cache : len);
    const Parts parts = parts_of(p, (int)b, (int)(bh - b * p.H_q), len);
    const int n = parts.n;
    if (p.start && n == 1) return;
    const int grp = tid / kLanes, x = tid % kLanes;
    const float2 *ml = reinterpret_cast<const float2 *>(p.part_ml) + parts.row;
    const float4 *po = reinterpret_cast<const float4 *>(p.part_o) + parts.row * (p.d / 4) + slice * kLanes + x;
    // each group's own running merge of its splits, then the groups'
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    float M = -INFINITY, l = 0.f;
#pragma unroll 4
    for (int s = grp; s < n; s += kGroups) {
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
    acc_s[grp][x] = acc;
    if (x == 0) s_m[grp] = M, s_l[grp] = l;
    __syncthreads();
    if (grp != 0) return;
#pragma unroll
    for (int i = 1; i < kGroups; ++i) M = fmaxf(M, s_m[i]);
    const float base = M == -INFINITY ? 0.f : M;
    float r[4] = {0.f, 0.f, 0.f, 0.f};
    l = 0.f;
#pragma unroll
    for (int i = 0; i < kGroups; ++i) {
      const float4 v = acc_s[i][x];
      const float f = ex2(s_m[i] - base);
      l += s_l[i] * f;
      r[0] += v.x * f, r[1] += v.y * f, r[2] += v.z * f, r[3] += v.w * f;
    }
    const size_t at = (size_t)bh * p.d + slice * kSlice + x * 4;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      r[i] = n > 0 ? r[i] / l : 0.f;
      if (p.gate && n > 0) r[i] *= 1.f / (1.f + expf(-bf16_to_f(p.gate[at + i])));
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
  const size_t head0 = (size_t)row * group;
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
  const float *lg = p.logits + head0 * p.T_cache + j0;
  float w[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 2
  for (int g = 0; g < group; ++g, lg += p.T_cache) {
    float x[4];
#pragma unroll
    for (int r = 0; r < 4; ++r) x[r] = j0 + r * kThreads < len ? lg[r * kThreads] : 0.f;
#pragma unroll
    for (int r = 0; r < 4; ++r) w[r] = fmaf(ex2(x[r] - s_m[g]), s_l[g], w[r]);
  }
  const size_t at = (size_t)row * p.T_cache + j0;
#pragma unroll
  for (int r = 0; r < 4; ++r)
    if (j0 + r * kThreads < len) p.acc_out[at + r * kThreads] = (p.acc_in ? p.acc_in[at + r * kThreads] : 0.f) + w[r];
}

}  // namespace

cudaError_t launch_attn_finish(const AttnFinishArgs &a, cudaStream_t s) {
  const unsigned n_slices = (unsigned)a.d / kSlice;
  const unsigned merge = (unsigned)a.B * a.H_q * n_slices;
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
  return cudaLaunchKernelEx(&cfg, attn_finish_kernel, a, (int)n_slices, merge);
}

}  // namespace hh
