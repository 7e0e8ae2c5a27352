"""kv_evict_select over more rows than the GPU holds clusters for: fewer CTAs a row, longer parts."""
import numpy as np
import pytest
import torch

from full_attention_gated_b200 import binding as hb

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("B,H,T,n_keep,n_recent", [(60, 4, 20011, 2000, 100), (250, 4, 9001, 511, 0),
                                                   (130, 2, 40000, 5000, 5000), (40, 4, 65000, 1, 0)])
@pytest.mark.parametrize("ties", [False, True])
def test_many_rows(B, H, T, n_keep, n_recent, ties):
    rng = np.random.default_rng(B + T)
    acc = rng.integers(0, 50, (B, H, T)).astype(np.float32) if ties else rng.random((B, H, T), dtype=np.float32) ** 8
    lens = rng.integers(0, T + 1, B).astype(np.int32)
    lens[:3] = (T, n_keep, min(T, n_keep + 1))
    keep = hb.kv_evict_select(torch.from_numpy(acc).cuda(), n_keep, n_recent,
                              cache_len=torch.from_numpy(lens).cuda()).cpu().numpy()
    want = np.full((B, H, n_keep), -1, np.int32)
    for b, n in enumerate(lens):
        if n <= n_keep:
            want[b, :, :n] = np.arange(n)
            continue
        old = n - n_recent
        best = np.argsort(-acc[b, :, :old], axis=-1, kind="stable")[:, :n_keep - n_recent]
        want[b, :, :n_keep - n_recent] = np.sort(best, axis=-1)
        want[b, :, n_keep - n_recent:] = np.arange(old, n)
    np.testing.assert_array_equal(keep, want)
