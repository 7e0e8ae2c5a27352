"""The KV-cache operators on the GPU against the fp64 reference (oracle/kv_cache.py): the q4_0 append, decode over
q4_0 (and the accumulating decode over bf16 and q8_0 caches), the choice of the positions that stay, compaction, and
all of them together in a serving loop.

Bounds.  Decode: with A = sum_j p_j |v_j| (times the gate) an output may be off by its rounding to bf16, 2^-8 |o|,
and by P A, where P counts the roundings of a weight: q4_0 and q8_0 round it to fp16 at most twice (2 x 2^-11), bf16
once to bf16 (2^-8).  The second rounding of q4_0 (weight times scale) meets the code 0..15 before the offset of 8
is taken off with the unrounded product, so it weighs |c s| <= |v| + 8 |s|: 2^-11 sum_j p_j 8 |s_j| more.  2^-10 stays for the logits (fp32 sums of d products; |logit| < 32 in these tests, so
2 x 32 x 2^-20 with 2^-20 for a sum of 256 fp32 terms) and the fp32 denominator.  A weight in acc: 2^-10 of the
step's weight for the same reasons, and fp32 rounding (2^-23) of the total.  Everything else is compared exactly."""
import numpy as np
import pytest
import torch

from full_attention_gated_b200 import binding as hb
from full_attention_gated_b200 import inputs as I
from helpers import dev_bf16, f64, host_f64
from oracle import kv_cache as R

pytestmark = pytest.mark.gpu

WEIGHT_ROUNDINGS = {"q4_0": 2.0 ** -10, "q8_0": 2.0 ** -10, "bf16": 2.0 ** -8}


def _bf(rng, shape, scale=1.0):
    return I.f32_to_bf16_bits((scale * rng.standard_normal(shape)).astype(np.float32))


def _dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def _q4(bits):
    codes, s = R.q4_0_quantise(f64(bits))
    return R.q4_0_pack(codes), s


def _spoil(arr, lens):
    """Rows at and past each sequence's length: bytes that read as NaN (all ones)."""
    for b, n in enumerate(lens):
        arr[b, max(0, n):].view(np.uint8)[...] = 0xFF
    return arr


def _check_decode(fmt, o, q, kv, vv, lens, G, scale, acc_in=None, acc_out=None, acc_was=None, v_scales=None):
    ref, w = R.decode(f64(q), kv, vv, lens, None if G is None else f64(G), scale)
    A, _ = R.decode(f64(q), kv, np.abs(vv), lens, None if G is None else f64(G), scale)
    err = np.abs(host_f64(o) - ref)
    tol = 2.0 ** -8 * np.abs(ref) + (WEIGHT_ROUNDINGS[fmt] + 2.0 ** -10) * A + 1e-30
    if fmt == "q4_0":
        steps = np.repeat(np.abs(np.asarray(v_scales, np.float64)), 32, axis=-1)
        tol += 2.0 ** -8 * R.decode(f64(q), kv, steps, lens, None if G is None else f64(G), scale)[0]
    assert np.all(err <= tol), f"o off by up to {np.max(err / tol):.2f} of the bound"
    if acc_out is not None:
        got, T = host_f64(acc_out), kv.shape[1]
        want = w + (0 if acc_in is None else acc_in.astype(np.float64))
        ok = np.abs(got - want) <= 2.0 ** -10 * w + 2.0 ** -23 * np.abs(want) + 1e-30
        for b in range(got.shape[0]):
            n = T if lens is None else min(max(int(lens[b]), 0), T)
            assert np.all(ok[b, :, :n]), f"weights of sequence {b}"
            np.testing.assert_array_equal(got[b, :, n:], acc_was[b, :, n:])  # not written


# ---------------------------------------------------------------- append
def _append_case(B, n, T, H, d, lens, n_new, x, held=True):
    """Runs the append on a cache of known bytes and compares every byte of it with the reference."""
    fill = np.full((B, T, H, d // 2), 0x5A, np.uint8)
    fill_s = np.full((B, T, H, d // 32), 0.25, np.float16)
    dev = [_dev(fill), _dev(fill_s), _dev(fill), _dev(fill_s)]
    kh, vh = (torch.full((B, n, H, d), 7.0, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    xk, xv = x, x[:, ::-1].copy()
    hb.kv_append_q4_0(dev_bf16(xk), dev_bf16(xv), *dev, cache_len=None if lens is None else _dev(np.int32(lens)),
                      n_new=None if n_new is None else _dev(np.int32(n_new)), k_held=kh if held else None,
                      v_held=vh if held else None)
    ln = [T] * B if lens is None else lens
    nn = [n] * B if n_new is None else n_new
    for side, got_v, got_s, got_h in ((xk, dev[0], dev[1], kh), (xv, dev[2], dev[3], vh)):
        want_v, want_s = R.append(fill, fill_s, f64(side), ln, nn)
        np.testing.assert_array_equal(got_v.cpu().numpy(), want_v)
        np.testing.assert_array_equal(got_s.cpu().numpy(), want_s)
        want_h = np.full((B, n, H, d), 7.0)
        if held:
            for b in range(B):
                m = min(max(nn[b], 0), n)
                for i in range(m):
                    pos = ln[b] - m + i
                    if 0 <= pos < T:
                        val = R.q4_0_values(want_v[b, pos], want_s[b, pos])
                        want_h[b, i] = I.bf16_bits_to_f32(I.f32_to_bf16_bits(val.astype(np.float32)))
        np.testing.assert_array_equal(host_f64(got_h), want_h)


@pytest.mark.parametrize("B,n,T,H,d,lens,n_new", [
    (1, 1, 1, 1, 128, None, None),                       # one token fills the cache
    (3, 1, 40, 4, 256, [1, 17, 40], None),               # a decode step
    (3, 1, 40, 1, 128, [5, 0, 41], [1, 1, 1]),           # positions before the start and past the end are dropped
    (2, 33, 50, 3, 128, [33, 50], [33, 7]),              # ragged prompts
    (4, 21, 30, 2, 256, [30, 25, 3, 30], [0, 99, 10, -4]),  # nothing; clamped; the first tokens fall before 0
    (1, 300, 257, 5, 256, None, None),                   # more tokens than the cache holds
])
def test_append_matches_reference(B, n, T, H, d, lens, n_new):
    x = _bf(np.random.default_rng(n * 31 + T), (B, n, H, d))
    _append_case(B, n, T, H, d, lens, n_new, x)


def test_append_special_values():
    rng = np.random.default_rng(5)
    vals = rng.standard_normal((1, 12, 1, 128)).astype(np.float32)
    vals[0, 0] = 0.0
    vals[0, 1] = -0.0
    vals[0, 2, 0, 7] = np.inf
    vals[0, 3, 0, 40] = -np.inf
    vals[0, 4, 0, 127] = np.nan
    vals[0, 5] *= 1e-7      # fp16 subnormal scales
    vals[0, 6] *= 1e-9      # scales that round to zero
    vals[0, 7] *= 1e37      # scales past fp16
    vals[0, 8] = np.where(np.arange(128) % 2, 4.0, -4.0)  # ties of magnitude
    vals[0, 9] = np.where(np.arange(128) % 2, -4.0, 4.0)
    vals[0, 10] = (np.arange(128) % 33 - 16) * 0.5        # quotients on ties
    vals[0, 11] = 3e5       # scale saturates
    _append_case(1, 12, 12, 1, 128, None, None, I.f32_to_bf16_bits(vals))


# ---------------------------------------------------------------- decode
DECODE = [  # B, T, Hq, Hkv, d, gated, lengths, weights accumulated
    (1, 1, 1, 1, 128, False, None, True),                     # one token, one head
    (3, 1000, 24, 4, 256, False, [1000, 0, 333], True),       # the 27B group of six; an empty sequence
    (2, 77, 12, 1, 128, True, None, False),                   # a group of twelve
    (1, 64, 6, 1, 256, True, None, True),                     # exactly one tile of keys
    (5, 130, 16, 2, 128, True, [128, 65, 1, 64, 129], True),  # ends around tile borders
    (4, 90, 10, 5, 128, False, [90, -3, 500, 89], True),      # lengths outside the cache are clamped
    (2, 9000, 16, 1, 256, False, [9000, 8193], False),        # a long cache, a group of sixteen
    (1, 5003, 3, 3, 256, True, None, True),                   # one query head a group
    (3, 2049, 8, 1, 128, False, [2049, 5, 2048], True),
]


@pytest.mark.parametrize("B,T,Hq,Hkv,d,gated,lens,acc", DECODE)
def test_decode_q4_0_matches_reference(B, T, Hq, Hkv, d, gated, lens, acc):
    rng = np.random.default_rng(B * 100 + T)
    q, G = _bf(rng, (B, Hq, d)), _bf(rng, (B, Hq, d)) if gated else None
    (kx, ks), (vx, vs) = _q4(_bf(rng, (B, T, Hkv, d))), _q4(_bf(rng, (B, T, Hkv, d)))
    kv, vv = R.q4_0_values(kx, ks), R.q4_0_values(vx, vs)
    ln, clean_vs = None if lens is None else np.int32(lens), vs.copy()
    if lens is not None:
        for a in (kx, ks, vx, vs):
            _spoil(a, lens)
    acc_in = rng.random((B, Hkv, T), dtype=np.float32) if acc else None
    out = torch.full((B, Hkv, T), -1.0, device="cuda") if acc else None
    was = None if out is None else host_f64(out)
    args = [_dev(a) for a in (kx, ks, vx, vs)]
    o = hb.gqa_attn_decode_q4_0(dev_bf16(q), *args, cache_len=None if ln is None else _dev(ln),
                                gate=None if G is None else dev_bf16(G), acc_in=None if acc_in is None else _dev(acc_in),
                                acc_out=out, scale=d ** -0.5)
    hb.hh_device_status()
    _check_decode("q4_0", o, q, kv, vv, ln, G, d ** -0.5, acc_in, out, was, v_scales=clean_vs)
    if lens is not None:
        for b, n in enumerate(lens):
            if n <= 0:
                assert np.all(host_f64(o)[b] == 0)


@pytest.mark.parametrize("ks_,vs_,qs_", [(1.0, 1e-6, 1.0), (1.0, 3e4, 1.0), (1e-3, 1.0, 1e3), (300.0, 1.0, 3e-3),
                                         (1.0, 1.0, 1e-4)])
def test_decode_q4_0_value_ranges(ks_, vs_, qs_):
    """Keys, values and queries far from 1, and blocks of very different scales in one cache."""
    B, T, Hq, Hkv, d = 2, 400, 6, 2, 128
    rng = np.random.default_rng(8)
    q = _bf(rng, (B, Hq, d), qs_)
    k, v = rng.standard_normal((B, T, Hkv, d)) * ks_, rng.standard_normal((B, T, Hkv, d)) * vs_
    v[:, 200:, :, 32:64] *= 50.0       # large blocks only later in the cache, beside small ones
    v[:, :, :, 96:] *= 1e-2
    (kx, s1), (vx, s2) = (_q4(I.f32_to_bf16_bits(x.astype(np.float32))) for x in (k, v))
    kv, vv = R.q4_0_values(kx, s1), R.q4_0_values(vx, s2)
    o = hb.gqa_attn_decode_q4_0(dev_bf16(q), _dev(kx), _dev(s1), _dev(vx), _dev(s2), scale=d ** -0.5)
    hb.hh_device_status()
    _check_decode("q4_0", o, q, kv, vv, None, None, d ** -0.5, v_scales=s2)


def test_decode_q4_0_nan_block_reaches_only_its_outputs():
    """A block that held an infinity reads as NaN: where it is attended, and nowhere else."""
    B, T, H, d = 2, 70, 2, 128
    rng = np.random.default_rng(3)
    q, k = _bf(rng, (B, H, d)), _bf(rng, (B, T, H, d))
    (kx, ks), (vx, vs) = _q4(k), _q4(_bf(rng, (B, T, H, d)))
    vs[0, 3, 1, 2] = np.nan
    o = host_f64(hb.gqa_attn_decode_q4_0(dev_bf16(q), _dev(kx), _dev(ks), _dev(vx), _dev(vs), scale=0.1))
    hb.hh_device_status()
    bad = np.zeros((B, H, d), bool)
    bad[0, 1, 64:96] = True
    np.testing.assert_array_equal(np.isnan(o), bad)


@pytest.mark.parametrize("fmt", ["bf16", "q8_0"])
@pytest.mark.parametrize("B,T,Hq,Hkv,gated,lens", [
    (1, 1, 2, 1, False, None), (3, 1000, 24, 4, True, [1000, 0, 333]), (2, 77, 13, 1, False, [64, 65]),
    (1, 2500, 4, 4, True, None)])
def test_accumulating_decode_matches_reference(fmt, B, T, Hq, Hkv, gated, lens):
    d = 256
    rng = np.random.default_rng(T + Hq)
    q, G = _bf(rng, (B, Hq, d)), _bf(rng, (B, Hq, d)) if gated else None
    acc_in = rng.random((B, Hkv, T), dtype=np.float32)
    out = torch.full((B, Hkv, T), -1.0, device="cuda")
    was = host_f64(out)
    ln = None if lens is None else np.int32(lens)
    kw = dict(cache_len=None if ln is None else _dev(ln), gate=None if G is None else dev_bf16(G), scale=d ** -0.5)
    if fmt == "bf16":
        k, v = _bf(rng, (B, T, Hkv, d)), _bf(rng, (B, T, Hkv, d))
        kv, vv, cache, f = f64(k), f64(v), (dev_bf16(k), dev_bf16(v)), hb.gqa_attn_decode_acc
        plain = hb.gqa_attn_decode(dev_bf16(q), *cache, **kw)
    else:
        kx, ks, vx, vs = I.q8_0_cache(T, B, T, Hkv, d)
        deq = lambda x, s: x.astype(np.float64) * np.repeat(s.astype(np.float64), 32, axis=-1)
        kv, vv, cache, f = deq(kx, ks), deq(vx, vs), [_dev(a) for a in (kx, ks, vx, vs)], hb.gqa_attn_decode_q8_0_acc
        plain = hb.gqa_attn_decode_q8_0(dev_bf16(q), *cache, **kw)
    o = f(dev_bf16(q), *cache, out, _dev(acc_in), **kw)
    hb.hh_device_status()
    # the accumulating form splits the cache otherwise: both are within the bound of the reference
    _check_decode(fmt, plain, q, kv, vv, ln, G, d ** -0.5)
    _check_decode(fmt, o, q, kv, vv, ln, G, d ** -0.5, acc_in, out, was)
    # in place, without a start value given
    again = _dev(acc_in)
    f(dev_bf16(q), *cache, again, again, **kw)
    fresh = torch.full((B, Hkv, T), -1.0, device="cuda")
    f(dev_bf16(q), *cache, fresh, None, **kw)
    for b in range(B):
        n = T if lens is None else lens[b]
        assert torch.equal(again[b, :, :n], out[b, :, :n])
        assert torch.equal(again[b, :, n:], _dev(acc_in)[b, :, n:])
    _check_decode(fmt, o, q, kv, vv, ln, G, d ** -0.5, None, fresh, was)


def test_decode_q4_0_repeats_bit_for_bit():
    B, T, Hq, Hkv, d = 3, 3001, 24, 4, 256
    rng = np.random.default_rng(12)
    args = [dev_bf16(_bf(rng, (B, Hq, d)))] + [_dev(a) for pair in (_q4(_bf(rng, (B, T, Hkv, d))),) * 2 for a in pair]
    accs = [torch.zeros((B, Hkv, T), device="cuda") for _ in range(2)]
    outs = [hb.gqa_attn_decode_q4_0(*args, acc_out=a) for a in accs]
    assert torch.equal(*outs) and torch.equal(*accs)
    assert torch.equal(hb.gqa_attn_decode_q4_0(*args), outs[0])  # with and without weights


# ---------------------------------------------------------------- select
@pytest.mark.parametrize("B,H,T,n_keep,n_recent,lens", [
    (1, 1, 1, 1, 0, None), (1, 2, 37, 5, 2, None), (2, 3, 700, 256, 0, [700, 255]), (3, 1, 300, 300, 300, [300, 0, 12]),
    (2, 2, 5000, 1024, 1024, [5000, 1030]), (1, 2, 20011, 4097, 100, None), (2, 1, 70000, 333, 32, [70000, 65537]),
    (4, 1, 50, 60, 7, [50, -1, 99, 49]), (1, 1, 4096, 1, 1, None), (1, 1, 4096, 1, 0, None),
])
@pytest.mark.parametrize("kind", ["spread", "ties", "special"])
def test_select_matches_reference(B, H, T, n_keep, n_recent, lens, kind):
    rng = np.random.default_rng(T + n_keep)
    if kind == "spread":
        acc = np.exp(3 * rng.standard_normal((B, H, T))).astype(np.float32)
    elif kind == "ties":
        acc = rng.integers(0, 4, (B, H, T)).astype(np.float32) / 4
    else:
        acc = rng.standard_normal((B, H, T)).astype(np.float32)
        pick = rng.integers(0, 12, acc.shape)
        for i, x in enumerate((np.nan, np.inf, -np.inf, 0.0, -0.0, np.float32(1e-40), -np.nan)):
            acc[pick == i] = x
    if lens is not None:
        for b, n in enumerate(lens):
            acc[b, :, max(0, n):] = np.inf  # past the end: must not be chosen
    ln = None if lens is None else np.int32(lens)
    keep = hb.kv_evict_select(_dev(acc), n_keep, n_recent, cache_len=None if ln is None else _dev(ln))
    np.testing.assert_array_equal(keep.cpu().numpy(), R.evict_select(acc, ln, n_keep, n_recent))


@pytest.mark.parametrize("kind", ["spread", "ties"])
def test_select_long_rows(kind):
    """Parts longer than the select's bitmap (more than 8 x 65,536 positions)."""
    T, n_keep, n_recent, ln = 600_011, 50_000, 77, 599_999
    rng = np.random.default_rng(6)
    acc = rng.random(T, dtype=np.float32) ** 4 if kind == "spread" else rng.integers(0, 9, T).astype(np.float32)
    keep = hb.kv_evict_select(_dev(acc[None, None]), n_keep, n_recent, cache_len=_dev(np.int32([ln])))
    old = ln - n_recent
    best = np.lexsort((np.arange(old), -acc[:old]))[:n_keep - n_recent]
    want = np.concatenate((np.sort(best), np.arange(old, ln)))
    np.testing.assert_array_equal(keep.cpu().numpy()[0, 0], want)


def test_select_all_weights_equal():
    acc = torch.full((2, 2, 33000), 0.125, device="cuda")
    keep = hb.kv_evict_select(acc, 1000, 10).cpu().numpy()
    want = np.concatenate((np.arange(990), np.arange(32990, 33000)))
    np.testing.assert_array_equal(keep, np.broadcast_to(want, keep.shape))


# ---------------------------------------------------------------- compact
def _rows(rng, B, T, H, row, dtype):
    return rng.integers(0, 256, (B, T, H, row), dtype=np.uint8).view(dtype)


@pytest.mark.parametrize("B,T,H,n_keep,T_out", [(1, 1, 1, 1, 1), (2, 100, 3, 40, 64), (1, 5000, 2, 1300, 1300),
                                                (3, 37, 1, 37, 50), (2, 900, 4, 700, 900), (1, 20, 2, 0, 5)])
@pytest.mark.parametrize("in_place", [False, True])
def test_compact_moves_rows(B, T, H, n_keep, T_out, in_place):
    """bf16 rows (d = 128 and 256), q8_0 and q4_0 rows and scales, 8-byte rows, and the weights, in one call."""
    rng = np.random.default_rng(T * 3 + n_keep)
    arrays = [_rows(rng, B, T, H, r, t) for r, t in ((512, np.uint8), (256, np.int16), (128, np.uint8), (64, np.uint8),
                                                     (16, np.float16), (8, np.float16), (520, np.uint8))]
    arrays = [np.nan_to_num(a) if a.dtype == np.float16 else a for a in arrays]
    acc = rng.random((B, H, T), dtype=np.float32)
    keep = np.full((B, H, n_keep), -1, np.int32)
    for b in range(B):
        for h in range(H):
            m = n_keep if (b + h) % 2 == 0 else n_keep // 2  # some sequences held fewer
            keep[b, h, :m] = np.sort(rng.choice(T, m, replace=False))
    dev = [_dev(a) for a in arrays]
    if in_place:
        T_out = T
        hb.kv_compact(_dev(keep), dev, acc=(d_acc := _dev(acc)))
        got, got_acc, was = dev, d_acc, arrays
    else:
        was = [np.full((B, T_out) + a.shape[2:], 3, a.dtype) for a in arrays]
        got = [_dev(a) for a in was]
        got_acc = torch.full((B, H, T_out), 9.0, device="cuda")
        hb.kv_compact(_dev(keep), dev, got, acc=_dev(acc), acc_out=got_acc)
        for x, y in zip(dev, arrays):
            np.testing.assert_array_equal(x.cpu().numpy(), y)  # the source is left alone
    for x, y, z in zip(got, arrays, was):
        np.testing.assert_array_equal(x.cpu().numpy(), R.compact(y, keep, z))
    want = R.compact(acc.transpose(0, 2, 1), keep, np.zeros((B, T_out, H), np.float32)).transpose(0, 2, 1)
    np.testing.assert_array_equal(got_acc.cpu().numpy(), want)


def test_compact_skips_entries_outside_the_cache():
    src, out = _dev(np.arange(6, dtype=np.int64).reshape(1, 6, 1, 1)), _dev(np.full((1, 6, 1, 1), 50, np.int64))
    keep = _dev(np.array([[[5, -1, 6, 2, -2147483648, 2147483647]]], np.int32))
    acc, acc_out = torch.ones((1, 1, 6), device="cuda"), torch.full((1, 1, 6), 4.0, device="cuda")
    hb.kv_compact(keep, [src], [out], acc=acc, acc_out=acc_out)
    assert out.flatten().tolist() == [5, 50, 50, 2, 50, 50]
    assert acc_out.flatten().tolist() == [1, 0, 0, 1, 0, 0]


# ---------------------------------------------------------------- together
def test_serving_loop_with_eviction():
    """Prompt append, then steps of append -> accumulating decode, cut back to n_keep whenever the cache is full;
    a second stream carries the loop, and the reference keeps the same books in fp64."""
    B, T, Hq, H, d, n0, n_keep, n_recent = 2, 48, 6, 2, 128, 30, 20, 6
    rng = np.random.default_rng(77)
    dev = [torch.full(s, f, dtype=t, device="cuda") for s, f, t in 2 * [((B, T, H, d // 2), 0xFF, torch.uint8),
                                                                       ((B, T, H, d // 32), float("nan"), torch.float16)]]
    acc, acc_ref = torch.zeros((B, H, T), device="cuda"), np.zeros((B, H, T))
    kx, ks, vx, vs = [x.cpu().numpy() for x in dev]
    n_new = np.int32([n0, 17])
    lens = n_new.copy()
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    evictions = 0
    for step in range(60):
        n = n0 if step == 0 else 1
        nn = n_new if step == 0 else np.int32([1, 1])
        if step:
            lens = lens + 1
        k, v, q = _bf(rng, (B, n, H, d)), _bf(rng, (B, n, H, d)), _bf(rng, (B, Hq, d))
        ln, up = _dev(lens), [dev_bf16(k), dev_bf16(v), dev_bf16(q), _dev(nn)]
        stream.wait_stream(torch.cuda.current_stream())
        hb.kv_append_q4_0(up[0], up[1], *dev, cache_len=ln, n_new=up[3], stream=stream)
        o = hb.gqa_attn_decode_q4_0(up[2], *dev, cache_len=ln, acc_in=acc, acc_out=acc, scale=0.125, stream=stream)
        kx, ks = R.append(kx, ks, f64(k), lens, nn)
        vx, vs = R.append(vx, vs, f64(v), lens, nn)
        kv, vv = np.nan_to_num(R.q4_0_values(kx, ks)), np.nan_to_num(R.q4_0_values(vx, vs))
        stream.synchronize()
        _check_decode("q4_0", o, q, kv, vv, lens, None, 0.125, v_scales=np.nan_to_num(vs))
        acc_ref += R.decode(f64(q), kv, vv, lens, None, 0.125)[1]
        if lens.max() == T:
            keep = hb.kv_evict_select(acc, n_keep, n_recent, cache_len=ln, stream=stream)
            # the fp32 books decide; the fp64 ones must agree with them to rounding
            a = host_f64(acc)
            stream.synchronize()
            np.testing.assert_allclose(a, acc_ref, rtol=2.0 ** -9, atol=1e-9)
            keep_h = R.evict_select(acc.cpu().numpy(), lens, n_keep, n_recent)
            np.testing.assert_array_equal(keep.cpu().numpy(), keep_h)
            hb.kv_compact(keep, dev, acc=acc, stream=stream)
            kx, ks, vx, vs = (R.compact(x, keep_h, x) for x in (kx, ks, vx, vs))
            acc_ref = R.compact(acc_ref.transpose(0, 2, 1), keep_h, np.zeros((B, T, H))).transpose(0, 2, 1).copy()
            lens = np.minimum(lens, n_keep).astype(np.int32)
            evictions += 1
            stream.synchronize()
            for x, y in zip(dev, (kx, ks, vx, vs)):
                np.testing.assert_array_equal(x.cpu().numpy(), y)
    assert evictions >= 2


def test_step_captured_and_replayed():
    """append -> accumulating decode in a CUDA graph: replays follow the lengths and inputs in device memory."""
    B, T, Hq, H, d = 2, 200, 6, 2, 256
    rng = np.random.default_rng(4)
    dev = [torch.zeros(s, dtype=t, device="cuda") for s, t in 2 * [((B, T, H, d // 2), torch.uint8),
                                                                  ((B, T, H, d // 32), torch.float16)]]
    acc, o = torch.zeros((B, H, T), device="cuda"), torch.empty((B, Hq, d), dtype=torch.bfloat16, device="cuda")
    k, v = (torch.zeros((B, 1, H, d), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    q, ln = torch.zeros((B, Hq, d), dtype=torch.bfloat16, device="cuda"), torch.zeros(B, dtype=torch.int32, device="cuda")
    ws = torch.empty(hb.gqa_attn_decode_q4_0_workspace_size(B, Hq, H, d, T, True), dtype=torch.uint8, device="cuda")

    def step():
        ln.add_(1)
        hb.kv_append_q4_0(k, v, *dev, cache_len=ln)
        hb.gqa_attn_decode_q4_0(q, *dev, cache_len=ln, o=o, acc_in=acc, acc_out=acc, workspace=ws)

    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for t in [ln, acc] + dev:
        t.zero_()
    kb, vb = _bf(rng, (B, T, H, d)), _bf(rng, (B, T, H, d))
    acc_ref = np.zeros((B, H, T))
    (kx, ks), (vx, vs) = _q4(kb), _q4(vb)
    kv, vv = R.q4_0_values(kx, ks), R.q4_0_values(vx, vs)
    for i in range(70):
        qb = _bf(rng, (B, Hq, d))
        k.copy_(dev_bf16(kb[:, i:i + 1]))
        v.copy_(dev_bf16(vb[:, i:i + 1]))
        q.copy_(dev_bf16(qb))
        g.replay()
        lens = np.int32([i + 1] * B)
        _check_decode("q4_0", o, qb, kv, vv, lens, None, d ** -0.5, v_scales=vs)
        acc_ref += R.decode(f64(qb), kv, vv, lens, None, d ** -0.5)[1]
    np.testing.assert_allclose(host_f64(acc), acc_ref, rtol=2.0 ** -9, atol=1e-9)
    assert ln.tolist() == [70, 70]
