"""The stack's q4_0 caches and its eviction on the host: buffer sizes against the page's (golden
tests/golden/page_sizes.json) and refusals.  CPU only: the buffers are allocated on the host and no kernel runs."""
import json
import os

import pytest
import torch

from full_attention_gated_b200 import stack as S

GOLD = json.load(open(os.path.join(os.path.dirname(__file__), "golden", "page_sizes.json")))


def test_held_q4_0_buffers_match_the_page():
    st = S.HybridStack(B=2, capacity=3, kv_format="q4_0", device="cpu")
    want = GOLD["kv_bytes_per_token_q4_0"]["value"]
    assert st.kv_bytes_per_token() == want == S.kv_bytes_per_token(S.STACK_27B, "q4_0") == 18 * 1024
    assert st.k_cache[0].dtype == torch.uint8 and st.k_cache[0].shape == (2, 3, 4, 128)
    assert st.k_scales[0].shape == (2, 3, 4, 8)
    assert [a.dtype for a in st.cache_arrays(0)] == [torch.uint8, torch.uint8, torch.float16, torch.float16]


def test_tracked_weights_are_held_and_counted():
    plain = S.HybridStack(B=2, capacity=5, kv_format="q4_0", device="cpu")
    st = S.HybridStack(B=2, capacity=5, kv_format="q4_0", device="cpu", track_weights=True)
    assert plain.attn_weights is None and len(st.attn_weights) == 16 and st.attn_weights[0].shape == (2, 4, 5)
    assert st.decode_bytes_per_step(5) - plain.decode_bytes_per_step(5) == 16 * 2 * 4 * 5 * 8


def test_refusals():
    with pytest.raises(ValueError, match="unknown KV format"):
        S.HybridStack(B=1, capacity=2, kv_format="q5_0", device="cpu")
    st = S.HybridStack(B=1, capacity=4, device="cpu")
    with pytest.raises(ValueError, match="track_weights"):
        st.evict(2, 1)
    with pytest.raises(ValueError, match="q4_0 caches"):
        st.append(0, None, None)
    st = S.HybridStack(B=1, capacity=4, device="cpu", track_weights=True)
    for n_keep, n_recent in ((5, 1), (2, 3), (2, -1)):
        with pytest.raises(ValueError, match="n_recent <= n_keep <= capacity"):
            st.evict(n_keep, n_recent)
    st = S.HybridStack(B=1, capacity=4, kv_format="q8_0", device="cpu")
    with pytest.raises(ValueError, match="prefill writes bf16 and q4_0"):
        st.prefill(2)
