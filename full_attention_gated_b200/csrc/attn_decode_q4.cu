// attn_decode_q4.cu -- one new query per sequence against a q4_0 KV cache
// (grouped-query attention decode), with the step's attention weights
// accumulated per cached position on request.
//
// "The economics of hybrid attention" (table in "What a token of context
// costs") prices the q4_0 cache at 18 KiB per token.  Element i of a block of
// 32 stands for s (c_i - 8): 4-bit code c_i, fp16 scale s (include/hh_kv.h).
//     p = softmax_j(scale q . k_j),  o = sum_j p_j v_j,  o *= sigmoid(gate)
// in three passes over the positions: the logits of all query heads (each K
// row read once for its group), one CTA per query head for the softmax and
// the sum over V, and the weights summed over the group.
#include <cuda_fp16.h>
#include <math.h>

#include "common.cuh"
#include "internal.h"

namespace hh {

namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr int kMaxGroup = 16;

struct DecodeQ4Params {
  AttnDecodeQ4Args a;
  float *logits;  // [B, H_q, T_cache], log2 domain
  float *ml;      // [B, H_q, 2]: maximum, sum
  int group;
};

__device__ __forceinline__ int cached(const AttnDecodeQ4Args &a, int b) {
  const int len = a.cache_len ? a.cache_len[b] : a.T_cache;
  return len < 0 ? 0 : (len > a.T_cache ? a.T_cache : len);
}

// thread = position: the logits of the group's heads
__global__ void __launch_bounds__(128) q4_logits_kernel(const __grid_constant__ DecodeQ4Params p) {
  __shared__ float q_s[kMaxGroup][256];
  const AttnDecodeQ4Args &a = p.a;
  const int kvh = blockIdx.y, b = blockIdx.z, j = blockIdx.x * 128 + threadIdx.x;
  const int len = cached(a, b);
  if (blockIdx.x * 128 >= len) return;
  for (int i = threadIdx.x; i < p.group * a.d; i += 128)
    q_s[i / a.d][i % a.d] = bf16_to_f(a.q[((size_t)b * a.H_q + kvh * p.group) * a.d + i]) * a.scale * kLog2e;
  __syncthreads();
  if (j >= len) return;
  const size_t row = ((size_t)b * a.T_cache + j) * a.H_kv + kvh;
  const uint32_t *codes = reinterpret_cast<const uint32_t *>(a.k_values + row * (a.d / 2));
  const uint16_t *scales = a.k_scales + row * (a.d / 32);
  float sum[kMaxGroup];
#pragma unroll
  for (int h = 0; h < kMaxGroup; ++h) sum[h] = 0.f;
  for (int w = 0; w < a.d / 8; ++w) {
    const uint32_t c = codes[w];
    const float s = __half2float(__ushort_as_half(scales[w >> 2]));
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float x = s * (float)((int)((c >> (4 * i)) & 15u) - 8);
#pragma unroll
      for (int h = 0; h < kMaxGroup; ++h)
        if (h < p.group) sum[h] = fmaf(q_s[h][w * 8 + i], x, sum[h]);
    }
  }
#pragma unroll
  for (int h = 0; h < kMaxGroup; ++h)
    if (h < p.group) p.logits[((size_t)b * a.H_q + kvh * p.group + h) * a.T_cache + j] = sum[h];
}

// CTA = query head, thread = element of the row
__global__ void q4_output_kernel(const __grid_constant__ DecodeQ4Params p) {
  __shared__ float red[256];
  const AttnDecodeQ4Args &a = p.a;
  const int h = blockIdx.x, b = blockIdx.y, kvh = h / p.group, i = threadIdx.x;
  const int len = cached(a, b);
  const float *lg = p.logits + ((size_t)b * a.H_q + h) * a.T_cache;
  float m = -INFINITY;
  for (int j = i; j < len; j += a.d) m = fmaxf(m, lg[j]);
  red[i] = m;
  __syncthreads();
  for (int j = 0; j < a.d; ++j) m = fmaxf(m, red[j]);
  float l = 0.f, o = 0.f;
  for (int j = 0; j < len; ++j) {
    const size_t row = ((size_t)b * a.T_cache + j) * a.H_kv + kvh;
    const int c = (a.v_values[row * (a.d / 2) + i / 2] >> ((i & 1) * 4)) & 15;
    const float pj = exp2f(lg[j] - m);
    l += pj;
    o = fmaf(pj, __half2float(__ushort_as_half(a.v_scales[row * (a.d / 32) + i / 32])) * (float)(c - 8), o);
  }
  const size_t at = ((size_t)b * a.H_q + h) * a.d + i;
  float r = len > 0 ? o / l : 0.f;
  if (a.gate && len > 0) r *= 1.f / (1.f + expf(-bf16_to_f(a.gate[at])));
  a.o[at] = f_to_bf16(r);
  if (i == 0) p.ml[((size_t)b * a.H_q + h) * 2] = m, p.ml[((size_t)b * a.H_q + h) * 2 + 1] = l;
}

}  // namespace

size_t attn_decode_q4_workspace(int B, int H_q, int H_kv, int d, int T_cache, bool with_acc) {
  return ((size_t)B * H_q * T_cache + (size_t)B * H_q * 2) * sizeof(float);
}

cudaError_t launch_attn_decode_q4(const AttnDecodeQ4Args &a, cudaStream_t s) {
  DecodeQ4Params p;
  p.a = a;
  p.ml = reinterpret_cast<float *>(a.workspace);
  p.logits = p.ml + (size_t)a.B * a.H_q * 2;
  p.group = a.H_q / a.H_kv;
  if (a.T_cache > 0)
    q4_logits_kernel<<<dim3((a.T_cache + 127) / 128, a.H_kv, a.B), 128, 0, s>>>(p);
  q4_output_kernel<<<dim3(a.H_q, a.B), a.d, 0, s>>>(p);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess || !a.acc_out) return e;
  return launch_attn_weights({p.logits, p.ml, a.cache_len, a.acc_in, a.acc_out, a.B, a.T_cache, a.H_q, a.H_kv, 1}, s);
}

}  // namespace hh
