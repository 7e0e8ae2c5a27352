"""Cache rows past a sequence's length may hold anything: decode over bf16, q8_0 and q4_0 caches whose rows past
cache_len are NaN gives the same as over clean ones."""
import numpy as np
import pytest
import torch

from full_attention_gated_b200 import binding as hb
from full_attention_gated_b200 import inputs as I
from helpers import dev_bf16

pytestmark = pytest.mark.gpu


def _spoil(t, lens):
    t = t.clone()
    for b, n in enumerate(lens):
        t[b, n:].view(torch.uint8).fill_(0xFF)
    return t


@pytest.mark.parametrize("fmt,d", [("bf16", 128), ("bf16", 256), ("q8_0", 256), ("q4_0", 128), ("q4_0", 256)])
@pytest.mark.parametrize("T,lens", [(200, [200, 0, 1, 63, 64, 65]), (2500, [2500, 2049, 1000, 15, 17, 130])])
def test_rows_past_the_length_do_not_matter(fmt, d, T, lens):
    B, Hq, H = len(lens), 10, 2
    rng = np.random.default_rng(T + d)
    q = dev_bf16(I.f32_to_bf16_bits(rng.standard_normal((B, Hq, d)).astype(np.float32)))
    k, v = (dev_bf16(I.f32_to_bf16_bits(rng.standard_normal((B, T, H, d)).astype(np.float32))) for _ in range(2))
    if fmt == "bf16":
        cache, calls = [k, v], [hb.gqa_attn_decode, lambda *a, **kw: hb.gqa_attn_decode_acc(*a, acc(), **kw)]
    elif fmt == "q8_0":
        cache = [torch.from_numpy(a).cuda() for a in I.q8_0_cache(T, B, T, H, d)]
        calls = [hb.gqa_attn_decode_q8_0, lambda *a, **kw: hb.gqa_attn_decode_q8_0_acc(*a, acc(), **kw)]
    else:
        cache = [torch.empty(s, dtype=t, device="cuda") for s, t in 2 * [((B, T, H, d // 2), torch.uint8),
                                                                        ((B, T, H, d // 32), torch.float16)]]
        hb.kv_append_q4_0(k, v, *cache)
        calls = [hb.gqa_attn_decode_q4_0, lambda *a, **kw: hb.gqa_attn_decode_q4_0(*a, acc_out=acc(), **kw)]

    def acc():
        return torch.zeros((B, H, T), device="cuda")

    ln = torch.tensor(lens, dtype=torch.int32, device="cuda")
    spoiled = [_spoil(t, lens) for t in cache]
    for call in calls:
        clean = call(q, *cache, cache_len=ln, scale=d ** -0.5)
        assert torch.equal(call(q, *spoiled, cache_len=ln, scale=d ** -0.5), clean)
        assert torch.isfinite(clean).all()
    hb.hh_device_status()
