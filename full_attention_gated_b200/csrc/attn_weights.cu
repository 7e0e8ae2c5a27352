// attn_weights.cu -- the last pass of a decode call that accumulates attention
// weights: every position's weight, summed over the query heads of its group,
// added to what the position has drawn so far (the figure that cache eviction
// goes by; "The economics of hybrid attention" prices the cache it bounds).
//
// The split kernels leave the step's logits (log2 domain) and, per split,
// their maximum m and sum l.  With the merged (m, l) of head h the weight of
// position j is exp2(logit - m) / l.  One thread owns one position of one kv
// head: no atomics, the sum runs over the heads in order.  Bound by the reads
// of the logits (4 bytes a query head and position) and of acc.
#include <math.h>

#include "common.cuh"
#include "internal.h"

namespace hh {

namespace {

constexpr int kThreads = 256;
constexpr int kMaxGroup = 16;

__global__ void __launch_bounds__(kThreads) attn_weights_kernel(const __grid_constant__ AttnWeightsArgs p) {
  __shared__ float s_m[kMaxGroup], s_inv[kMaxGroup];
  const int kvh = blockIdx.y, b = blockIdx.z, group = p.H_q / p.H_kv;
  int len = p.cache_len ? p.cache_len[b] : p.T_cache;
  len = len < 0 ? 0 : (len > p.T_cache ? p.T_cache : len);
  if ((int)blockIdx.x * kThreads >= len) return;
  const size_t row0 = (size_t)b * p.H_q + kvh * group;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int n_splits = min(p.n_splits, (len + p.split_len - 1) / p.split_len);
  for (int g = warp; g < group; g += kThreads / 32) {
    const float *ml = p.part_ml + (row0 + g) * p.n_splits * 2;
    float m = -INFINITY, l = 0.f;
    for (int s = lane; s < n_splits; s += 32) m = fmaxf(m, ml[2 * s]);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    for (int s = lane; s < n_splits; s += 32) l += m == -INFINITY ? 0.f : ml[2 * s + 1] * exp2f(ml[2 * s] - m);
    l = warp_sum(l);
    if (lane == 0) s_m[g] = m, s_inv[g] = 1.f / l;
  }
  __syncthreads();
  const int j = blockIdx.x * kThreads + threadIdx.x;
  if (j >= len) return;
  const float *lg = p.logits + row0 * p.T_cache + j;
  float w = 0.f;
  for (int g = 0; g < group; ++g) w = fmaf(exp2f(lg[(size_t)g * p.T_cache] - s_m[g]), s_inv[g], w);
  const size_t at = ((size_t)b * p.H_kv + kvh) * p.T_cache + j;
  p.acc_out[at] = (p.acc_in ? p.acc_in[at] : 0.f) + w;
}

}  // namespace

cudaError_t launch_attn_weights(const AttnWeightsArgs &a, cudaStream_t s) {
  if (a.B == 0 || a.T_cache == 0) return cudaSuccess;
  attn_weights_kernel<<<dim3((a.T_cache + kThreads - 1) / kThreads, a.H_kv, a.B), kThreads, 0, s>>>(a);
  return cudaGetLastError();
}

}  // namespace hh
