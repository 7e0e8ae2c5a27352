"""kv_compact in place over long caches: many chunks, one CTA or a cluster to a row."""
import pytest
import torch

from full_attention_gated_b200 import binding as hb

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("B,T,H,n_keep,sizes", [
    (1, 60000, 2, 40000, (128, 16)),        # q4_0 rows of d = 256 and their scales, clusters of eight
    (1, 33333, 1, 33000, (512, 24, 8)),     # hardly anything goes; rows that are no power of two
    (3, 20000, 4, 9000, (64, 8)),
    (20, 3000, 8, 2999, (256, 40)),         # a CTA a row
    (1, 9000, 1, 600, (4096,)),
])
def test_in_place_equals_gather(B, T, H, n_keep, sizes):
    gen = torch.Generator(device="cuda").manual_seed(T)
    arrays = [torch.randint(0, 256, (B, T, H, n), generator=gen, device="cuda", dtype=torch.uint8) for n in sizes]
    acc = torch.rand((B, H, T), generator=gen, device="cuda")
    order = torch.rand((B, H, T), generator=gen, device="cuda").argsort(-1)[..., :n_keep].sort(-1).values
    keep = order.int()
    keep[0, 0, n_keep - 7:] = -1            # a sequence that held fewer
    held = (keep >= 0)
    want = []
    for x in arrays:
        y = x.clone()
        idx = order.transpose(1, 2)[..., None].expand(-1, -1, -1, x.shape[-1])
        moved = torch.gather(x, 1, idx)
        y[:, :n_keep] = torch.where(held.transpose(1, 2)[..., None], moved, x[:, :n_keep])
        want.append(y)
    want_acc = torch.zeros_like(acc)
    want_acc[..., :n_keep] = torch.where(held, torch.gather(acc, 2, order), 0.0)
    hb.kv_compact(keep, arrays, acc=acc)
    for x, y in zip(arrays, want):
        assert torch.equal(x, y)
    assert torch.equal(acc, want_acc)
