// internal_kv.h -- what the KV-cache operators (include/hh_kv.h) share beyond internal.h: argument structs and launch
// declarations, and attributes that are set once per device.
#pragma once

#include <atomic>

#include "internal.h"

namespace hh {

// Decode that accumulates the step's attention weights.
struct AttnDecodeAccArgs : AttnDecodeArgs {
  const float *acc_in = nullptr;  // nullable: zeros
  float *acc_out = nullptr;       // nullable: no weights; else the workspace is attn_decode_acc_workspace bytes
};
struct AttnDecodeQ8AccArgs : AttnDecodeQ8Args {
  const float *acc_in = nullptr;
  float *acc_out = nullptr;
};
size_t attn_decode_acc_workspace(int B, int H_q, int d, int T_cache);
cudaError_t launch_attn_decode_acc(const AttnDecodeAccArgs &a, cudaStream_t s);
cudaError_t launch_attn_decode_q8_acc(const AttnDecodeQ8AccArgs &a, cudaStream_t s);

// The end of a split decode call (attn_finish.cu): the splits' partial results merged into the
// output, and acc_out[b, hk, j] = acc_in[b, hk, j] + sum over the group's heads of exp2(logit - m) / l for
// j < cache_len[b] (acc_out nullable).  The parts of head h of sequence b are
//   start == NULL: rows (b H_q + h) n_splits + s, for the splits of split_len positions below cache_len[b];
//   else: rows (b + u) H_q + h, for the groups u that share the sequence's tiles of split_len positions (at least one):
//     start[b] / share .. (start[b] + tiles - 1) / share, share = start[B]; a single group has written the output.
//     n_splits: the groups there are.
struct AttnFinishArgs {
  const float *part_o;   // [rows, d], unnormalised
  const float *part_ml;  // [rows, 2]: maximum (log2 domain), sum
  const float *logits;   // [B, H_q, T_cache], log2 domain, written for j < cache_len[b]
  const int32_t *cache_len;
  const bf16_t *gate;    // nullable
  bf16_t *o;
  const float *acc_in;   // nullable: zeros
  float *acc_out;
  int B, T_cache, H_q, H_kv, d, n_splits, split_len;
  const int *start = nullptr;
};
cudaError_t launch_attn_finish(const AttnFinishArgs &a, cudaStream_t s);

// GQA decode over a q4_0 cache: codes [B, T_cache, H_kv, d/2] and fp16 scales [B, T_cache, H_kv, d/32], for K and V;
// acc_out nullable: the step's attention weights are added to it (acc_in nullable: zeros).
struct AttnDecodeQ4Args {
  const bf16_t *q, *gate;
  const uint8_t *k_values, *v_values;
  const uint16_t *k_scales, *v_scales;
  const int32_t *cache_len;
  bf16_t *o;
  const float *acc_in;
  float *acc_out;
  void *workspace;
  int B, T_cache, H_q, H_kv, d;
  float scale;
};
size_t attn_decode_q4_workspace(int B, int H_q, int H_kv, int d, int T_cache, bool with_acc);
cudaError_t launch_attn_decode_q4(const AttnDecodeQ4Args &a, cudaStream_t s);

// KV-cache operators (kv_cache.cu): quantised append, choice of the positions that stay, compaction.
struct KvAppendQ4Args {
  const bf16_t *k, *v;
  uint8_t *k_values, *v_values;
  uint16_t *k_scales, *v_scales;
  const int32_t *cache_len, *n_new;  // nullable
  bf16_t *k_held, *v_held;           // nullable
  int B, n, T_cache, H_kv, d;
};
cudaError_t launch_kv_append_q4(const KvAppendQ4Args &a, cudaStream_t s);
struct KvSelectArgs {
  const float *acc;
  const int32_t *cache_len;  // nullable
  int32_t *keep;
  int B, T_cache, H_kv, n_keep, n_recent;
};
cudaError_t launch_kv_select(const KvSelectArgs &a, cudaStream_t s);
constexpr int kMaxCompactArrays = 8;
struct KvCompactArgs {
  const int32_t *keep;
  const void *src[kMaxCompactArrays];
  void *dst[kMaxCompactArrays];
  int row_bytes[kMaxCompactArrays];
  int n_arrays;
  const float *acc_src;  // nullable (with acc_dst)
  float *acc_dst;
  int B, T_src, T_dst, H_kv, n_keep;
};
cudaError_t launch_kv_compact(const KvCompactArgs &a, cudaStream_t s);

// Kernel attributes are set once per device and kernel: `done` has a bit a device.
template <typename F>
cudaError_t once_per_device(std::atomic<uint64_t> &done, F set) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = dev < 64 ? 1ull << dev : 0;
  if (done.load(std::memory_order_acquire) & bit) return cudaSuccess;
  e = set();
  if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_release);
  return e;
}

}  // namespace hh
