// abi_kv.cpp -- the extern "C" entry points of include/hh_kv.h: argument
// validation, launch and error mapping.  Every check runs before anything is
// enqueued.
#include "../../include/hh_kv.h"

#include <cuda_runtime.h>
#include <math.h>

#include "internal_kv.h"

using namespace hh;

namespace {

#define HH_FAIL(code, ...)    \
  do {                        \
    hh::set_error(__VA_ARGS__); \
    return (code);            \
  } while (0)

bool al(const void *p, unsigned n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1u)) == 0; }

int launch_result(cudaError_t e, const char *fn) {
  if (e != cudaSuccess) {
    if (!hh::last_error()[0]) hh::set_error("%s: CUDA error: %s", fn, cudaGetErrorString(e));
    return HH_ERR_CUDA;
  }
  return HH_OK;
}

int check_workspace(const char *fn, const void *workspace, size_t ws_bytes, size_t need) {
  if (need && (!workspace || ws_bytes < need))
    HH_FAIL(HH_ERR_INVALID_ARG, "%s: workspace of %zu bytes needed (got %zu)", fn, need, ws_bytes);
  if (!al(workspace, 256)) HH_FAIL(HH_ERR_INVALID_ARG, "%s: workspace must be 256-byte aligned", fn);
  return HH_OK;
}

bool overlap(const void *x, size_t nx, const void *y, size_t ny) {
  const uintptr_t u = reinterpret_cast<uintptr_t>(x), w = reinterpret_cast<uintptr_t>(y);
  return u < w + ny && w < u + nx;
}

int check_acc(const char *fn, const float *acc_in, const float *acc_out, bool need, size_t n) {
  if (need && !acc_out) HH_FAIL(HH_ERR_INVALID_ARG, "%s: acc_out is null", fn);
  if (acc_in && !acc_out) HH_FAIL(HH_ERR_INVALID_ARG, "%s: acc_in without acc_out", fn);
  if (!al(acc_in, 16) || !al(acc_out, 16)) HH_FAIL(HH_ERR_INVALID_ARG, "%s: acc must be 16-byte aligned", fn);
  if (acc_in && acc_in != acc_out && overlap(acc_in, n * sizeof(float), acc_out, n * sizeof(float)))
    HH_FAIL(HH_ERR_INVALID_ARG, "%s: acc_in must be acc_out or not overlap it", fn);
  return HH_OK;
}

}  // namespace

extern "C" {

int kv_append_q4_0(const hh_bf16 *k, const hh_bf16 *v, uint8_t *k_values, uint16_t *k_scales, uint8_t *v_values,
                   uint16_t *v_scales, const int32_t *cache_len, const int32_t *n_new, hh_bf16 *k_held,
                   hh_bf16 *v_held, int B, int n, int T_cache, int H_kv, int d, hh_stream stream) {
  static const char *fn = "kv_append_q4_0";
  hh::clear_error();
  if (B < 0 || n < 0 || T_cache < 0 || H_kv <= 0 || d <= 0)
    HH_FAIL(HH_ERR_INVALID_ARG, "%s: sizes must be positive (B, n, T_cache may be 0)", fn);
  if (d != 128 && d != 256) HH_FAIL(HH_ERR_UNSUPPORTED, "%s: only d = 128 or 256 is built", fn);
  if (B > 65535 || H_kv > 65535 || T_cache > (1 << 30) || (long long)n * H_kv * d / 8 >= (1LL << 31))
    HH_FAIL(HH_ERR_INVALID_ARG, "%s: sizes too large", fn);
  if ((k_held == nullptr) != (v_held == nullptr))
    HH_FAIL(HH_ERR_INVALID_ARG, "%s: k_held and v_held go together", fn);
  if (B == 0 || n == 0 || T_cache == 0) return HH_OK;
  if (!k || !v || !k_values || !k_scales || !v_values || !v_scales)
    HH_FAIL(HH_ERR_INVALID_ARG, "%s: null tensor pointer", fn);
  if (!al(k, 16) || !al(v, 16) || !al(k_values, 16) || !al(v_values, 16) || !al(k_scales, 16) || !al(v_scales, 16) ||
      !al(k_held, 16) || !al(v_held, 16) || !al(cache_len, 4) || !al(n_new, 4))
    HH_FAIL(HH_ERR_INVALID_ARG, "%s: tensors must be 16-byte aligned", fn);
  const size_t in = (size_t)B * n * H_kv * d * sizeof(hh_bf16);
  if (k_held && (overlap(k_held, in, k, in) || overlap(k_held, in, v, in) || overlap(v_held, in, k, in) ||
                 overlap(v_held, in, v, in) || overlap(k_held, in, v_held, in)))
    HH_FAIL(HH_ERR_INVALID_ARG, "%s: k_held and v_held must not overlap k, v or each other", fn);
  if (int r = hh::check_device(fn)) return r;
  KvAppendQ4Args a = {k, v, k_values, v_values, k_scales, v_scales, cache_len, n_new, k_held, v_held, B, n, T_cache,
                      H_kv, d};
  return launch_result(launch_kv_append_q4(a, reinterpret_cast<cudaStream_t>(stream)), fn);
}

size_t gqa_attn_decode_q4_0_workspace_size(int B, int H_q, int H_kv, int d, int T_cache, int with_acc) {
  if (B <= 0 || H_q <= 0 || H_kv <= 0 || d <= 0 || T_cache < 0) return 0;
  return hh::attn_decode_q4_workspace(B, H_q, H_kv, d, T_cache, with_acc != 0);
}

int gqa_attn_decode_q4_0(const hh_bf16 *q, const uint8_t *k_values, const uint16_t *k_scales, const uint8_t *v_values,
                         const uint16_t *v_scales, const int32_t *cache_len, const hh_bf16 *gate, hh_bf16 *o,
                         const float *acc_in, float *acc_out, void *workspace, size_t ws_bytes, int B, int T_cache,
                         int H_q, int H_kv, int d, float scale, hh_stream stream) {
  static const char *fn = "gqa_attn_decode_q4_0";
  hh::clear_error();
  const int v = hh::check_decode_args(fn, q, reinterpret_cast<const hh_bf16 *>(k_values),
                                      reinterpret_cast<const hh_bf16 *>(v_values), cache_len, gate, o, B, T_cache, H_q,
                                      H_kv, d, scale);
  if (v < 0) return v;
  if (int r = check_acc(fn, acc_in, acc_out, false, (size_t)B * H_kv * T_cache)) return r;
  if (v == hh::kNothingToDo) return HH_OK;
  if (T_cache > 0 && (!k_scales || !v_scales)) HH_FAIL(HH_ERR_INVALID_ARG, "%s: null scale pointer", fn);
  if (!al(k_scales, 16) || !al(v_scales, 16))
    HH_FAIL(HH_ERR_INVALID_ARG, "%s: scale arrays must be 16-byte aligned", fn);
  const size_t need = hh::attn_decode_q4_workspace(B, H_q, H_kv, d, T_cache, acc_out != nullptr);
  if (int r = check_workspace(fn, workspace, ws_bytes, need)) return r;
  if (int r = hh::check_device(fn)) return r;
  AttnDecodeQ4Args a = {q,       gate,    k_values,  v_values, k_scales, v_scales, cache_len, o,
                        acc_in,  acc_out, workspace, B,        T_cache,  H_q,      H_kv,      d,
                        scale};
  return launch_result(launch_attn_decode_q4(a, reinterpret_cast<cudaStream_t>(stream)), fn);
}

size_t gqa_attn_decode_acc_workspace_size(int B, int H_q, int d, int T_cache) {
  if (B <= 0 || H_q <= 0 || d <= 0 || T_cache < 0) return 0;
  return hh::attn_decode_acc_workspace(B, H_q, d, T_cache);
}

int gqa_attn_decode_acc(const hh_bf16 *q, const hh_bf16 *k_cache, const hh_bf16 *v_cache, const int32_t *cache_len,
                        const hh_bf16 *gate, hh_bf16 *o, const float *acc_in, float *acc_out, void *workspace,
                        size_t ws_bytes, int B, int T_cache, int H_q, int H_kv, int d, float scale, hh_stream stream) {
  static const char *fn = "gqa_attn_decode_acc";
  hh::clear_error();
  const int v = hh::check_decode_args(fn, q, k_cache, v_cache, cache_len, gate, o, B, T_cache, H_q, H_kv, d, scale);
  if (v < 0) return v;
  if (v == hh::kNothingToDo) return HH_OK;
  if (int r = check_acc(fn, acc_in, acc_out, T_cache > 0, (size_t)B * H_kv * T_cache)) return r;
  if (int r = check_workspace(fn, workspace, ws_bytes, hh::attn_decode_acc_workspace(B, H_q, d, T_cache))) return r;
  if (int r = hh::check_device(fn)) return r;
  AttnDecodeAccArgs a;
  a.q = q;
  a.k_cache = k_cache;
  a.v_cache = v_cache;
  a.gate = gate;
  a.cache_len = cache_len;
  a.o = o;
  a.workspace = workspace;
  a.B = B;
  a.T_cache = T_cache;
  a.H_q = H_q;
  a.H_kv = H_kv;
  a.d = d;
  a.scale = scale;
  a.acc_in = acc_in;
  a.acc_out = acc_out;
  return launch_result(launch_attn_decode_acc(a, reinterpret_cast<cudaStream_t>(stream)), fn);
}

int gqa_attn_decode_q8_0_acc(const hh_bf16 *q, const int8_t *k_values, const uint16_t *k_scales,
                             const int8_t *v_values, const uint16_t *v_scales, const int32_t *cache_len,
                             const hh_bf16 *gate, hh_bf16 *o, const float *acc_in, float *acc_out, void *workspace,
                             size_t ws_bytes, int B, int T_cache, int H_q, int H_kv, int d, float scale,
                             hh_stream stream) {
  static const char *fn = "gqa_attn_decode_q8_0_acc";
  hh::clear_error();
  const int v = hh::check_decode_args(fn, q, reinterpret_cast<const hh_bf16 *>(k_values),
                                      reinterpret_cast<const hh_bf16 *>(v_values), cache_len, gate, o, B, T_cache, H_q,
                                      H_kv, d, scale);
  if (v < 0) return v;
  if (d != 256) HH_FAIL(HH_ERR_UNSUPPORTED, "%s: only d = 256 is built for the q8_0 cache", fn);
  if (v == hh::kNothingToDo) return HH_OK;
  if (T_cache > 0 && (!k_scales || !v_scales)) HH_FAIL(HH_ERR_INVALID_ARG, "%s: null scale pointer", fn);
  if (!al(k_scales, 16) || !al(v_scales, 16))
    HH_FAIL(HH_ERR_INVALID_ARG, "%s: scale arrays must be 16-byte aligned", fn);
  if (int r = check_acc(fn, acc_in, acc_out, T_cache > 0, (size_t)B * H_kv * T_cache)) return r;
  if (int r = check_workspace(fn, workspace, ws_bytes, hh::attn_decode_acc_workspace(B, H_q, d, T_cache))) return r;
  if (int r = hh::check_device(fn)) return r;
  AttnDecodeQ8AccArgs a;
  a.q = q;
  a.gate = gate;
  a.k_values = k_values;
  a.v_values = v_values;
  a.k_scales = k_scales;
  a.v_scales = v_scales;
  a.cache_len = cache_len;
  a.o = o;
  a.workspace = workspace;
  a.B = B;
  a.T_cache = T_cache;
  a.H_q = H_q;
  a.H_kv = H_kv;
  a.d = d;
  a.scale = scale;
  a.acc_in = acc_in;
  a.acc_out = acc_out;
  return launch_result(launch_attn_decode_q8_acc(a, reinterpret_cast<cudaStream_t>(stream)), fn);
}

int kv_evict_select(const float *acc, const int32_t *cache_len, int32_t *keep, int B, int T_cache, int H_kv,
                    int n_keep, int n_recent, hh_stream stream) {
  static const char *fn = "kv_evict_select";
  hh::clear_error();
  if (B < 0 || T_cache < 0 || H_kv < 0 || n_keep < 0)
    HH_FAIL(HH_ERR_INVALID_ARG, "%s: sizes must not be negative", fn);
  if (n_recent < 0 || n_recent > n_keep)
    HH_FAIL(HH_ERR_INVALID_ARG, "%s: n_recent (%d) must be in 0 .. n_keep (%d)", fn, n_recent, n_keep);
  if (B > 65535 || H_kv > 65535 || T_cache > (1 << 30) || n_keep > (1 << 30))
    HH_FAIL(HH_ERR_INVALID_ARG, "%s: sizes too large", fn);
  if (B == 0 || H_kv == 0 || n_keep == 0) return HH_OK;
  if (!keep || (T_cache > 0 && !acc)) HH_FAIL(HH_ERR_INVALID_ARG, "%s: null tensor pointer", fn);
  if (!al(acc, 16) || !al(keep, 16) || !al(cache_len, 4))
    HH_FAIL(HH_ERR_INVALID_ARG, "%s: tensors must be 16-byte aligned", fn);
  if (overlap(keep, (size_t)B * H_kv * n_keep * sizeof(int32_t), acc, (size_t)B * H_kv * T_cache * sizeof(float)))
    HH_FAIL(HH_ERR_INVALID_ARG, "%s: keep and acc overlap", fn);
  if (int r = hh::check_device(fn)) return r;
  KvSelectArgs a = {acc, cache_len, keep, B, T_cache, H_kv, n_keep, n_recent};
  return launch_result(launch_kv_select(a, reinterpret_cast<cudaStream_t>(stream)), fn);
}

int kv_compact(const int32_t *keep, const void *const *src, void *const *dst, const int32_t *row_bytes, int n_arrays,
               const float *acc_src, float *acc_dst, int B, int T_src, int T_dst, int H_kv, int n_keep,
               hh_stream stream) {
  static const char *fn = "kv_compact";
  hh::clear_error();
  if (B < 0 || T_src < 0 || T_dst < 0 || H_kv < 0 || n_keep < 0 || n_arrays < 0)
    HH_FAIL(HH_ERR_INVALID_ARG, "%s: sizes must not be negative", fn);
  if (n_arrays > kMaxCompactArrays)
    HH_FAIL(HH_ERR_UNSUPPORTED, "%s: at most %d arrays", fn, kMaxCompactArrays);
  if (n_keep > T_dst) HH_FAIL(HH_ERR_INVALID_ARG, "%s: n_keep (%d) above T_dst (%d)", fn, n_keep, T_dst);
  if ((acc_src == nullptr) != (acc_dst == nullptr))
    HH_FAIL(HH_ERR_INVALID_ARG, "%s: acc_src and acc_dst go together", fn);
  if (B > 65535 || H_kv > 65535 || T_src > (1 << 30) || T_dst > (1 << 30))
    HH_FAIL(HH_ERR_INVALID_ARG, "%s: sizes too large", fn);
  if (n_arrays > 0 && (!src || !dst || !row_bytes)) HH_FAIL(HH_ERR_INVALID_ARG, "%s: null host array", fn);
  if (B == 0 || H_kv == 0 || T_dst == 0) return HH_OK;
  if (T_src == 0) HH_FAIL(HH_ERR_INVALID_ARG, "%s: T_src must be positive", fn);
  const size_t kept = (size_t)B * H_kv * n_keep * sizeof(int32_t), acc_row = (size_t)B * H_kv * sizeof(float);
  if (acc_dst) {
    if (!al(acc_src, 16) || !al(acc_dst, 16)) HH_FAIL(HH_ERR_INVALID_ARG, "%s: tensors must be 16-byte aligned", fn);
    if (acc_src == acc_dst ? T_src != T_dst : overlap(acc_src, acc_row * T_src, acc_dst, acc_row * T_dst))
      HH_FAIL(HH_ERR_INVALID_ARG, "%s: acc_dst must be acc_src with T_dst = T_src, or not overlap it", fn);
    if (keep && overlap(acc_dst, acc_row * T_dst, keep, kept))
      HH_FAIL(HH_ERR_INVALID_ARG, "%s: acc_dst and keep overlap", fn);
  }
  KvCompactArgs a;
  a.n_arrays = n_arrays;
  for (int i = 0; i < n_arrays; ++i) {
    if (!src[i] || !dst[i]) HH_FAIL(HH_ERR_INVALID_ARG, "%s: null tensor pointer (array %d)", fn, i);
    if (row_bytes[i] <= 0 || row_bytes[i] % 8 != 0 || row_bytes[i] > 4096)
      HH_FAIL(HH_ERR_INVALID_ARG, "%s: row_bytes[%d] = %d is not a multiple of 8 in 8 .. 4096", fn, i, row_bytes[i]);
    if (!al(src[i], 16) || !al(dst[i], 16)) HH_FAIL(HH_ERR_INVALID_ARG, "%s: tensors must be 16-byte aligned", fn);
    const size_t row = (size_t)B * H_kv * row_bytes[i];
    if (src[i] == dst[i] ? T_src != T_dst : overlap(src[i], row * T_src, dst[i], row * T_dst))
      HH_FAIL(HH_ERR_INVALID_ARG, "%s: array %d: dst must be src with T_dst = T_src, or not overlap it", fn, i);
    if (keep && overlap(dst[i], row * T_dst, keep, kept))
      HH_FAIL(HH_ERR_INVALID_ARG, "%s: array %d and keep overlap", fn, i);
    if (acc_dst && (overlap(dst[i], row * T_dst, acc_src, acc_row * T_src) ||
                    overlap(dst[i], row * T_dst, acc_dst, acc_row * T_dst) ||
                    overlap(src[i], row * T_src, acc_dst, acc_row * T_dst)))
      HH_FAIL(HH_ERR_INVALID_ARG, "%s: array %d and the weights overlap", fn, i);
    for (int j = 0; j < n_arrays; ++j) {
      const size_t other = (size_t)B * H_kv * row_bytes[j];
      if (j != i && dst[j] && src[j] &&
          (overlap(dst[i], row * T_dst, dst[j], other * T_dst) || overlap(dst[i], row * T_dst, src[j], other * T_src)))
        HH_FAIL(HH_ERR_INVALID_ARG, "%s: arrays %d and %d overlap", fn, i, j);
    }
    a.src[i] = src[i];
    a.dst[i] = dst[i];
    a.row_bytes[i] = row_bytes[i];
  }
  if (n_keep > 0 && !keep) HH_FAIL(HH_ERR_INVALID_ARG, "%s: keep is null", fn);
  if (!al(keep, 16)) HH_FAIL(HH_ERR_INVALID_ARG, "%s: keep must be 16-byte aligned", fn);
  if (n_arrays == 0 && !acc_dst) return HH_OK;
  if (int r = hh::check_device(fn)) return r;
  a.keep = keep;
  a.acc_src = acc_src;
  a.acc_dst = acc_dst;
  a.B = B;
  a.T_src = T_src;
  a.T_dst = T_dst;
  a.H_kv = H_kv;
  a.n_keep = n_keep;
  return launch_result(launch_kv_compact(a, reinterpret_cast<cudaStream_t>(stream)), fn);
}

}  // extern "C"
