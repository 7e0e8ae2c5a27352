"""Eviction ahead of the first decode step: no position has drawn a weight, and the lower of equals stay."""
import pytest
import torch

from full_attention_gated_b200 import stack as S

pytestmark = pytest.mark.gpu

SHAPE = S.StackShape(n_groups=2, gdn_per_group=1, gdn_qk_heads=1, gdn_v_heads=2, gdn_head_dim=128, attn_q_heads=6,
                     attn_kv_heads=2, attn_head_dim=256)


def test_keeps_the_first_and_the_last_positions():
    st = S.HybridStack(B=2, capacity=140, shape=SHAPE, kv_format="q4_0", track_weights=True)
    st.prefill(100)
    before = [[a.clone() for a in st.cache_arrays(i)] for i in range(2)]
    want = torch.cat((torch.arange(12), torch.arange(92, 100))).cuda()
    for kept, arrays, was in zip(st.evict(20, 8), map(st.cache_arrays, range(2)), before):
        assert torch.equal(kept, want.int().expand_as(kept))
        for a, b in zip(arrays, was):
            assert torch.equal(a[:, :20], b[:, want])
    assert st.cache_len.tolist() == [20, 20]
    st.decode_step(seed=2)
    torch.cuda.synchronize()
    # three query heads a kv head, each step's weights good to 2^-10
    assert all(torch.all(w[..., :20].sum(-1).sub(3).abs() <= 3 * 2.0 ** -10) and not w[..., 20:].any()
               for w in st.attn_weights)
