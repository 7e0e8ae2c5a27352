"""gqa_attn_decode_q4_0 where its work is laid out differently: batches that fill the GPU (the wider tiles, sequences
that share a CTA or are shared by several), many short sequences, many heads, group sizes on both sides of eight, other
scales, and caches past 4 GiB.  Caches are filled by kv_append_q4_0 (checked bit for bit in test_gpu_kv_cache.py); the
bounds are those of test_gpu_kv_cache.py."""
import numpy as np
import pytest
import torch

from full_attention_gated_b200 import binding as hb
from helpers import host_f64
from oracle import kv_cache as R

pytestmark = pytest.mark.gpu


def _normal(gen, shape, scale=1.0):
    return (torch.randn(shape, generator=gen, device="cuda") * scale).bfloat16()


def _filled(gen, B, T, H, d, v_scale=None):
    k, v = _normal(gen, (B, T, H, d)), _normal(gen, (B, T, H, d))
    if v_scale is not None:
        v = (v.float() * v_scale).bfloat16()
    cache = [torch.empty(s, dtype=t, device="cuda") for s, t in 2 * [((B, T, H, d // 2), torch.uint8),
                                                                    ((B, T, H, d // 32), torch.float16)]]
    hb.kv_append_q4_0(k, v, *cache)
    return cache


def _check(q, cache, lens, gate, scale, o, acc_in=None, acc_out=None):
    kx, ks, vx, vs = (t.cpu().numpy() for t in cache)
    kv, vv = R.q4_0_values(kx, ks), R.q4_0_values(vx, vs)
    steps = np.repeat(np.abs(vs.astype(np.float64)), 32, axis=-1)
    qf, gf = host_f64(q), None if gate is None else host_f64(gate)
    ref, w = R.decode(qf, kv, vv, lens, gf, scale)
    A = R.decode(qf, kv, np.abs(vv), lens, gf, scale)[0]
    Sv = R.decode(qf, kv, steps, lens, gf, scale)[0]
    err, tol = np.abs(host_f64(o) - ref), 2.0 ** -8 * np.abs(ref) + 2.0 ** -9 * A + 2.0 ** -8 * Sv + 1e-30
    assert np.all(err <= tol), f"o off by up to {np.max(err / tol):.2f} of the bound"
    if acc_out is not None:
        got, want = host_f64(acc_out), w + host_f64(acc_in)
        for b in range(got.shape[0]):
            n = kv.shape[1] if lens is None else int(lens[b])
            d = np.abs(got[b, :, :n] - want[b, :, :n])
            assert np.all(d <= 2.0 ** -10 * w[b, :, :n] + 2.0 ** -23 * want[b, :, :n] + 1e-30), f"weights of {b}"


def _lens(rng, B, T):
    lens = rng.integers(0, T + 1, B)
    lens[:4] = (0, 1, T, min(T, 129))
    return lens.astype(np.int32)


@pytest.mark.parametrize("B,T,Hq,H,d,gated,acc", [
    (40, 700, 24, 4, 256, True, True),     # 128-key tiles, the 27B heads
    (40, 700, 4, 4, 256, False, False),    # one query head a group
    (64, 800, 16, 2, 128, False, True),
    (64, 800, 16, 1, 256, True, True),     # groups of sixteen
    (70, 1200, 12, 1, 128, True, True),    # groups of twelve
    (3, 700, 11, 1, 256, True, True),      # the same on 64-key tiles
    (3, 700, 16, 1, 128, False, True),
    (1500, 3, 2, 1, 128, True, True),      # many short sequences
    (1, 150, 800, 800, 128, False, True),  # more kv heads than CTAs fit
    (2, 300, 150, 150, 256, True, False),
])
def test_layouts_match_reference(B, T, Hq, H, d, gated, acc):
    gen = torch.Generator(device="cuda").manual_seed(B + T)
    rng = np.random.default_rng(B * T)
    cache, q = _filled(gen, B, T, H, d), _normal(gen, (B, Hq, d))
    gate = _normal(gen, (B, Hq, d)) if gated else None
    lens = _lens(rng, B, T) if B >= 4 else None
    a_in = torch.rand((B, H, T), generator=gen, device="cuda") if acc else None
    a_out = torch.zeros_like(a_in) if acc else None
    ln = None if lens is None else torch.from_numpy(lens).cuda()
    o = hb.gqa_attn_decode_q4_0(q, *cache, cache_len=ln, gate=gate, acc_in=a_in, acc_out=a_out)
    hb.hh_device_status()
    _check(q, cache, lens, gate, d ** -0.5, o, a_in, a_out)


@pytest.mark.parametrize("B,T,H,d", [(2, 300, 2, 256), (48, 900, 4, 256), (2, 300, 2, 128)])
@pytest.mark.parametrize("scale", [-0.06, 0.0, 1e-6])
def test_other_scales(B, T, H, d, scale):
    gen = torch.Generator(device="cuda").manual_seed(T)
    cache, q = _filled(gen, B, T, H, d), _normal(gen, (B, 3 * H, d))
    lens = np.full(B, T - 70, np.int32)
    a_in, a_out = torch.zeros((B, H, T), device="cuda"), torch.zeros((B, H, T), device="cuda")
    o = hb.gqa_attn_decode_q4_0(q, *cache, cache_len=torch.from_numpy(lens).cuda(), acc_in=a_in, acc_out=a_out,
                                scale=scale)
    hb.hh_device_status()
    _check(q, cache, lens, None, scale, o, a_in, a_out)


@pytest.mark.parametrize("B,T,Hq,H,d", [(35, 26, 32, 2, 128), (5, 3, 24, 4, 256), (2, 700, 8, 8, 256),
                                        (48, 200, 6, 1, 128), (1, 4001, 12, 2, 256)])
def test_accumulated_weights_are_fp32(B, T, Hq, H, d):
    """Nothing beneath them is rounded to 16 bits.  A logit (here below 8) is an fp32 sum of d products: its roundings,
    of 2^-24 of at most 8 each and of either sign, add up to about sqrt(256) 2^-24 8 = 8e-6; the exponential (2^-22),
    the sum of the weights and the total are finer.  In the 2-norm that stays below 1e-5 of the weights."""
    gen = torch.Generator(device="cuda").manual_seed(T + d)
    cache, q = _filled(gen, B, T, H, d), _normal(gen, (B, Hq, d))
    kx, ks, vx, vs = (t.cpu().numpy() for t in cache)
    acc = torch.zeros((B, H, T), device="cuda")
    hb.gqa_attn_decode_q4_0(q, *cache, acc_in=acc, acc_out=acc, scale=d ** -0.5)
    hb.hh_device_status()
    w = R.decode(host_f64(q), R.q4_0_values(kx, ks), R.q4_0_values(vx, vs), None, None, d ** -0.5)[1]
    assert np.linalg.norm(host_f64(acc) - w) <= 1e-5 * np.linalg.norm(w)


@pytest.mark.parametrize("size,scale", [(1e-36, 1 / 16), (1e-36, 1e35), (1e-38, 1e-30), (1e18, 1e-19), (1e-20, -1e19)])
def test_queries_of_any_size(size, scale):
    """Queries at the ends of the range: the power of two that scales a head for its products stays finite, and masked
    keys get no weight however small the factor back is."""
    B, T, H, d = 3, 200, 2, 256
    gen = torch.Generator(device="cuda").manual_seed(4)
    cache, q = _filled(gen, B, T, H, d), _normal(gen, (B, 3 * H, d), size)
    lens = np.array([200, 1, 77], np.int32)
    o = hb.gqa_attn_decode_q4_0(q, *cache, cache_len=torch.from_numpy(lens).cuda(), scale=scale)
    hb.hh_device_status()
    _check(q, cache, lens, None, scale, o)


def test_value_scales_that_grow_along_the_cache():
    """Blocks of scale 2 and more turn up late in some sequences (other CTAs, other tiles of one CTA)."""
    B, T, H, d = 48, 900, 4, 256
    gen = torch.Generator(device="cuda").manual_seed(9)
    grow = torch.ones((B, T, 1, d), device="cuda")
    grow[::2, 500:, :, 64:96] = 300.0
    grow[1::2, 10:, :, :32] = 2e-4
    cache, q = _filled(gen, B, T, H, d, grow), _normal(gen, (B, 2 * H, d))
    o = hb.gqa_attn_decode_q4_0(q, *cache)
    hb.hh_device_status()
    _check(q, cache, None, None, d ** -0.5, o)


def test_offsets_past_32_bits():
    """Three sequences of 4,194,304 positions: the last one's rows lie beyond 4 GiB of each array of codes."""
    B, T, H, d, n = 3, 1 << 22, 4, 256, 333
    gen = torch.Generator(device="cuda").manual_seed(1)
    cache = [torch.zeros(s, dtype=t, device="cuda") for s, t in 2 * [((B, T, H, d // 2), torch.uint8),
                                                                    ((B, T, H, d // 32), torch.float16)]]
    k, v, q = _normal(gen, (B, n, H, d)), _normal(gen, (B, n, H, d)), _normal(gen, (B, 2 * H, d))
    ln = torch.tensor([0, n, n], dtype=torch.int32, device="cuda")
    hb.kv_append_q4_0(k, v, *cache, cache_len=ln)
    small = [torch.zeros((B, n) + t.shape[2:], dtype=t.dtype, device="cuda") for t in cache]
    hb.kv_append_q4_0(k, v, *small, cache_len=ln)
    for x, y in zip(cache, small):
        assert torch.equal(x[2, :n], y[2]) and torch.equal(x[1, :n], y[1]) and not x[0, :n].any()
    o = hb.gqa_attn_decode_q4_0(q, *cache, cache_len=ln)
    hb.hh_device_status()
    _check(q, small, ln.cpu().numpy(), None, d ** -0.5, o)
    # the last positions: the same rows appended at the end, the head of the cache moved there by compaction in place
    hb.kv_append_q4_0(k, v, *cache)
    for x, y in zip(cache, small):
        assert torch.equal(x[2, T - n:], y[2])
    keep = torch.full((B, H, 2 * n), -1, dtype=torch.int32, device="cuda")
    keep[:, :, :n] = torch.arange(T - n, T, device="cuda")
    hb.kv_compact(keep, cache)
    for x, y in zip(cache, small):
        assert torch.equal(x[2, :n], y[2]) and torch.equal(x[0, :n], x[0, T - n:])


@pytest.mark.parametrize("fmt", ["bf16", "q8_0", "q4_0"])
@pytest.mark.parametrize("T,lens", [(0, None), (0, [0, 0]), (70, [0, -3])])
def test_nothing_cached(fmt, T, lens):
    """No capacity, or nothing in it: zeros, and weights left as they were."""
    B, Hq, H, d = 2, 8, 2, 256
    q = torch.ones((B, Hq, d), dtype=torch.bfloat16, device="cuda")
    rows = {"bf16": [(d, torch.bfloat16)], "q8_0": [(d, torch.int8), (d // 32, torch.float16)],
            "q4_0": [(d // 2, torch.uint8), (d // 32, torch.float16)]}[fmt]
    cache = [torch.full((B, T, H, n), 7, dtype=t, device="cuda") for n, t in 2 * rows]
    ln = None if lens is None else torch.tensor(lens, dtype=torch.int32, device="cuda")
    acc = torch.full((B, H, T), 3.0, device="cuda")
    o = torch.full_like(q, 5.0)
    call = {"bf16": hb.gqa_attn_decode_acc, "q8_0": hb.gqa_attn_decode_q8_0_acc}.get(fmt)
    if call:
        call(q, *cache, acc, acc, cache_len=ln, o=o)
    else:
        hb.gqa_attn_decode_q4_0(q, *cache, cache_len=ln, o=o, acc_in=acc, acc_out=acc)
    keep = hb.kv_evict_select(acc, 4, 1, cache_len=ln)
    hb.hh_device_status()
    assert torch.count_nonzero(o) == 0 and torch.all(acc == 3.0) and torch.all(keep == -1)
