"""The stack over q4_0, q8_0 and bf16 caches with tracked attention weights: prefill (q4_0), decode steps in a CUDA
graph, eviction, and decode steps from the same graph over what is left, against the fp64 reference."""
import numpy as np
import pytest
import torch

from full_attention_gated_b200 import inputs_device as D
from full_attention_gated_b200 import stack as S
from helpers import assert_close, host_f64
from oracle import kv_cache as R

pytestmark = pytest.mark.gpu

SMALL = S.StackShape(n_groups=2, gdn_per_group=1, gdn_qk_heads=1, gdn_v_heads=2, gdn_head_dim=128,
                     attn_q_heads=6, attn_kv_heads=2, attn_head_dim=256)


def _cache_values(st, ai):
    k, v = (x[ai].cpu().float().numpy().astype(np.float64) if st.kv_format == "bf16" else x[ai].cpu().numpy()
            for x in (st.k_cache, st.v_cache))
    if st.kv_format == "bf16":
        return k, v
    ks, vs = st.k_scales[ai].cpu().numpy(), st.v_scales[ai].cpu().numpy()
    if st.kv_format == "q4_0":
        return R.q4_0_values(k, ks), R.q4_0_values(v, vs)
    return tuple(x.astype(np.float64) * np.repeat(s.astype(np.float64), 32, -1) for x, s in ((k, ks), (v, vs)))


def _check_step(st, outs, weights):
    """The attention layers' outputs of the last step; the step's weights are added to `weights`."""
    lens = st.cache_len.cpu().numpy()
    ai = 0
    for li, kind in enumerate(st.shape.kinds()):
        if kind != "attn":
            continue
        k, v = _cache_values(st, ai)
        L = st._dec[li]
        ref, w = R.decode(host_f64(L["q"]), k, v, lens, host_f64(L["G"]), st.shape.attn_head_dim ** -0.5)
        assert_close(host_f64(outs[li]), ref, f"layer {li}")
        weights[ai] += w
        # fp32 sums of a few steps' weights, each good to 2^-10
        np.testing.assert_allclose(host_f64(st.attn_weights[ai]), weights[ai], rtol=2.0 ** -9, atol=1e-9)
        ai += 1


@pytest.mark.parametrize("fmt", ["bf16", "q8_0", "q4_0"])
def test_decode_evict_decode(fmt):
    B, capacity, context, n_keep, n_recent = 2, 300, 250, 64, 16
    st = S.HybridStack(B=B, capacity=capacity, shape=SMALL, kv_format=fmt, track_weights=True)
    st.fill_synthetic_cache(context, seed=5)
    weights = [np.zeros((B, 2, capacity)) for _ in range(2)]
    for step in range(2):
        outs = st.decode_step(seed=3)
        torch.cuda.synchronize()
        _check_step(st, outs, weights)
    before = [[a.cpu().numpy() if a.dtype != torch.bfloat16 else a.view(torch.int16).cpu().numpy()
               for a in st.cache_arrays(ai)] for ai in range(2)]
    acc = [w.cpu().numpy() for w in st.attn_weights]
    lens = st.cache_len.cpu().numpy()
    kept = st.evict(n_keep, n_recent)
    assert st.cache_len.tolist() == [n_keep] * B
    for ai in range(2):
        keep = R.evict_select(acc[ai], lens, n_keep, n_recent)
        np.testing.assert_array_equal(kept[ai].cpu().numpy(), keep)
        for a, b in zip(st.cache_arrays(ai), before[ai]):
            a = a.view(torch.int16) if a.dtype == torch.bfloat16 else a
            np.testing.assert_array_equal(a.cpu().numpy(), R.compact(b, keep, b))
        w = R.compact(acc[ai].transpose(0, 2, 1), keep, np.zeros((B, capacity, 2), np.float32)).transpose(0, 2, 1)
        np.testing.assert_array_equal(st.attn_weights[ai].cpu().numpy(), w)
        weights[ai] = w.astype(np.float64)
    outs = st.decode_step(seed=3)  # the graph captured before the eviction
    torch.cuda.synchronize()
    _check_step(st, outs, weights)


def test_q4_0_prefill_then_decode(oracle_mod):
    B, capacity, T = 2, 140, 100
    st = S.HybridStack(B=B, capacity=capacity, shape=SMALL, kv_format="q4_0", seed=7, track_weights=True)
    outs = st.prefill(T)
    torch.cuda.synchronize()
    assert st.cache_len.tolist() == [T] * B
    ai = 0
    for li, kind in enumerate(SMALL.kinds()):
        if kind != "attn":
            continue
        y = D.attn_inputs(7 * 1000 + li, B, T, 6, 2, 256, gate=True)
        k, v = _cache_values(st, ai)
        for x, got in ((y["k"], k), (y["v"], v)):
            codes, s = R.q4_0_quantise(host_f64(x))
            np.testing.assert_array_equal(got[:, :T], R.q4_0_values(R.q4_0_pack(codes), s))
        # the layer attends the values that the cache stands for (their rounding to bf16 is within the bound)
        ref = oracle_mod.causal_attention(host_f64(y["q"]), k[:, :T], v[:, :T], host_f64(y["G"]), 256 ** -0.5)
        assert_close(host_f64(outs[li]), ref, f"prefill layer {li}")
        ai += 1
    weights = [np.zeros((B, 2, capacity)) for _ in range(2)]
    outs = st.decode_step(seed=2)
    torch.cuda.synchronize()
    _check_step(st, outs, weights)
