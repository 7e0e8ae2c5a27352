"""The decode step's buffers on the host: the attention layers run one after the other on one stream, so one workspace
serves them all (with tracked weights it holds a step's logits: 4 bytes a query head and cached position).  CPU only."""
import pytest
import torch

from full_attention_gated_b200 import stack as S

SHAPE = S.StackShape(n_groups=3, gdn_per_group=1, gdn_qk_heads=1, gdn_v_heads=2, gdn_head_dim=128, attn_q_heads=6,
                     attn_kv_heads=2, attn_head_dim=256)


@pytest.mark.parametrize("fmt", ["bf16", "q8_0", "q4_0"])
@pytest.mark.parametrize("track", [False, True])
def test_attention_layers_share_one_workspace(fmt, track):
    st = S.HybridStack(B=2, capacity=50, shape=SHAPE, kv_format=fmt, device="cpu", track_weights=track)
    st._decode_buffers(1)
    ws = [L["ws"] for L in st._dec if L["kind"] == "attn"]
    assert len(ws) == 3 and len({w.data_ptr() for w in ws}) == 1
    assert ws[0].dtype == torch.uint8 and ws[0].numel() == st._decode_workspace_size() > 0
