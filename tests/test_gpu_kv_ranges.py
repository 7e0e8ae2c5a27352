"""The KV-cache operators at the ends of the formats' ranges, against the fp64 reference: the append of blocks whose scale
is a small subnormal fp16, bit for bit; decode where values, or channels of keys and queries, differ far in size, where
logits are large, and where weights are small beside their totals."""
import numpy as np
import pytest
import torch

from full_attention_gated_b200 import binding as hb
from full_attention_gated_b200 import inputs as I
from helpers import dev_bf16, f64, host_f64
from oracle import kv_cache as R
from test_gpu_decode_q4_sizes import _check
from test_gpu_kv_cache import _append_case, _check_decode

pytestmark = pytest.mark.gpu


# ---------------------------------------------------------------- append
@pytest.mark.parametrize("size", [3e-7, 5e-7, 1e-6, 2e-6, 4e-6])
def test_append_small_blocks(size):
    """Normal blocks whose scales are k 2^-24 with k of a few bits."""
    x = I.f32_to_bf16_bits((size * np.random.default_rng(1).standard_normal((2, 40, 2, 256))).astype(np.float32))
    s = np.abs(R.q4_0_quantise(f64(x))[1].astype(np.float64))
    assert np.mean((s > 0) & (s < 2.0 ** -14)) > 0.5
    _append_case(2, 40, 40, 2, 256, None, None, x)


def test_append_every_rounding_of_a_subnormal_scale():
    """Blocks whose largest element asks for j/16 x 2^-24, j = 1 .. 255, as a scale: rounded down by up to a third it
    leaves quotients of up to 12.  Both signs, the largest element at an even and an odd place, others behind it."""
    rng = np.random.default_rng(2)
    j = np.repeat(np.arange(1, 256), 4)
    sign, place = np.tile([1, 1, -1, -1], 255), np.tile([4, 13, 22, 31], 255)
    top = sign * j * 2.0 ** -25  # 8 x j/16 x 2^-24, an 8-bit number of a bf16
    x = rng.uniform(-1, 1, (j.size, 32)) * np.abs(top)[:, None]
    x[np.arange(j.size), place] = top
    x = I.f32_to_bf16_bits(x.reshape(1, 255, 1, 128).astype(np.float32))
    s = np.abs(R.q4_0_quantise(f64(x))[1].astype(np.float64)).ravel()
    np.testing.assert_array_equal(s, np.rint(j / 16) * 2.0 ** -24)
    assert np.all(s < 2.0 ** -14) and np.all(s[j > 8] > 0)
    _append_case(1, 255, 255, 1, 128, None, None, x)


# ---------------------------------------------------------------- decode: values
def _one_cta(rng, T, d, q, sink, v_scales):
    """One head's cache, as packed codes and scales: logits of deviation 1 under one of `sink` at position 0 (queries q,
    scale 1), values of the given scales."""
    codes = [rng.integers(0, 16, (T, d), dtype=np.uint8) for _ in range(2)]
    ks = np.full((T, d // 32), np.float16(1 / (4.7 * np.linalg.norm(q))))
    codes[0][0] = 8 + 7 * np.sign(q)
    ks[0] = np.float16(sink / (7 * np.abs(q).sum()))
    return R.q4_0_pack(codes[0]), ks, R.q4_0_pack(codes[1]), np.asarray(v_scales, np.float16)


def _check_heads(H, group, d, T, q, cache):
    """The same cache and queries in every kv head, more of them than CTAs that share a sequence's keys: one CTA walks
    all keys of a head.  All heads have to agree, and the first with the reference, within the bound of
    test_gpu_kv_cache.py."""
    qs = np.stack([q * (1 - g / 32) for g in range(group)]).astype(np.float32)
    qs = I.bf16_bits_to_f32(I.f32_to_bf16_bits(qs))
    dev = [torch.from_numpy(a).cuda()[None, :, None].expand(1, T, H, a.shape[-1]).contiguous() for a in cache]
    o = hb.gqa_attn_decode_q4_0(torch.from_numpy(qs).cuda().bfloat16().repeat(H, 1)[None], *dev, scale=1.0)
    hb.hh_device_status()
    got = host_f64(o).reshape(H, group, d)
    np.testing.assert_array_equal(got, np.broadcast_to(got[:1], got.shape))
    kx, ks, vx, vs = (a[None, :, None] for a in cache)
    kv, vv, steps = R.q4_0_values(kx, ks), R.q4_0_values(vx, vs), np.repeat(np.abs(vs.astype(np.float64)), 32, -1)
    ref, A, S = (R.decode(qs[None].astype(np.float64), kv, x, None, None, 1.0)[0][0] for x in (vv, np.abs(vv), steps))
    err, tol = np.abs(got[0] - ref), 2.0 ** -8 * np.abs(ref) + 2.0 ** -9 * A + 2.0 ** -8 * S
    assert np.all(err <= tol), f"o off by up to {np.max(err / tol):.2f} of the bound"


ONE_CTA = [(256, 224, 2), (128, 372, 1), (256, 149, 12), (128, 297, 9)]  # d, kv heads, group


@pytest.mark.parametrize("d,H,group", ONE_CTA)
@pytest.mark.parametrize("small", [0.05, 0.002])
@pytest.mark.parametrize("at", [5, 6000])
def test_small_value_blocks_beside_a_large_one(d, H, group, small, at):
    """A key that draws nearly all weight while its own values are small, and one block of scale 2 and more: the other
    blocks' outputs are sums of many small products, which the large block must not push out of fp16's range."""
    T = 8201
    rng = np.random.default_rng(d + group)
    q = np.abs(rng.standard_normal(d)) + 0.5
    vs = small * rng.uniform(0.8, 1.2, (T, d // 32))
    vs[0] = 0.01 * small
    vs[at, 1] = 5.0
    _check_heads(H, group, d, T, q, _one_cta(rng, T, d, q, 14.5, vs))


@pytest.mark.parametrize("d,H,group", ONE_CTA)
def test_value_scales_over_the_whole_range(d, H, group):
    """Blocks whose scales grow along the cache from the smallest fp16 to the largest, in steps and at once, fall, are
    zero or negative, under a flat softmax."""
    T = 2077
    rng = np.random.default_rng(d + group)
    q = rng.standard_normal(d)
    vs = rng.uniform(0.5, 1.0, (T, d // 32))
    t = np.arange(T)
    vs[:, 0] = np.minimum(2.0 ** (-24 + t // 50), 65504) * np.where(t % 3, 1, -1)
    vs[:, 1] *= np.where(t < 700, 2.0 ** -24, 65000.0)
    vs[:, 2] *= np.where(t < 700, 65000.0, 1.0)
    vs[:, 3] = np.where(t < 1500, 0.0, 1e-3)
    _check_heads(H, group, d, T, q, _one_cta(rng, T, d, q, 2.0, vs))


# ---------------------------------------------------------------- decode: keys
@pytest.mark.parametrize("B,T,H,group,d", [(2, 400, 2, 3, 128), (2, 400, 2, 3, 256), (2, 300, 1, 12, 256),
                                           (40, 700, 4, 2, 256)])
@pytest.mark.parametrize("ratio", [30, 100, 1000])
def test_keys_and_queries_of_unequal_channels(B, T, H, group, d, ratio):
    """One block of channels large in the queries and small in the keys, another the other way round: their shares of
    the logit are alike.  A logit (below 32) is good to 2^-10, as the bound of test_gpu_kv_cache.py has it."""
    gen = torch.Generator(device="cuda").manual_seed(ratio + d)
    q, k, v = (torch.randn(s, generator=gen, device="cuda") for s in ((B, H * group, d), (B, T, H, d), (B, T, H, d)))
    q[..., :32] *= ratio
    k[..., :32] /= ratio
    q[..., -32:] /= ratio
    k[..., -32:] *= ratio
    q, k, v = (x.bfloat16() for x in (q, k, v))
    cache = [torch.empty(s, dtype=t, device="cuda") for s, t in 2 * [((B, T, H, d // 2), torch.uint8),
                                                                    ((B, T, H, d // 32), torch.float16)]]
    hb.kv_append_q4_0(k, v, *cache)
    acc = torch.zeros((B, H, T), device="cuda")
    o = hb.gqa_attn_decode_q4_0(q, *cache, acc_in=acc, acc_out=acc)
    hb.hh_device_status()
    cache = [x[:2].contiguous() for x in cache]
    _check(q[:2], cache, None, None, d ** -0.5, o[:2], torch.zeros_like(acc[:2]), acc[:2])


@pytest.mark.parametrize("B,T,H,group,d", [(2, 400, 2, 3, 128), (1, 3000, 2, 3, 256), (2, 300, 1, 12, 256),
                                           (40, 700, 4, 2, 256)])
@pytest.mark.parametrize("q_size,k_size", [(1e4, 1e4), (1e7, 1.0), (1e18, 1.0), (1e30, 100.0)])
def test_logits_far_from_zero(B, T, H, group, d, q_size, k_size):
    """Logits of 1e7 and more: the largest one's key draws all the weight (the next is further off than the logits'
    rounding), whatever units an fp32 number of that size has."""
    gen = torch.Generator(device="cuda").manual_seed(T)
    q, k, v = (torch.randn(s, generator=gen, device="cuda") for s in ((B, H * group, d), (B, T, H, d), (B, T, H, d)))
    q, k, v = (q * q_size).bfloat16(), (k * k_size).bfloat16(), v.bfloat16()
    cache = [torch.empty(s, dtype=t, device="cuda") for s, t in 2 * [((B, T, H, d // 2), torch.uint8),
                                                                    ((B, T, H, d // 32), torch.float16)]]
    hb.kv_append_q4_0(k, v, *cache)
    acc = torch.zeros((B, H, T), device="cuda")
    o = hb.gqa_attn_decode_q4_0(q, *cache, acc_in=acc, acc_out=acc)
    hb.hh_device_status()
    cache = [x[:2].contiguous() for x in cache]
    _check(q[:2], cache, None, None, d ** -0.5, o[:2], torch.zeros_like(acc[:2]), acc[:2])


# ---------------------------------------------------------------- weights
@pytest.mark.parametrize("fmt", ["bf16", "q8_0", "q4_0"])
@pytest.mark.parametrize("group", [5, 16])
def test_small_weights_on_a_large_total(fmt, group):
    """Totals of a long session, of which equal weights of 1/4096 a head are less than half a unit: the heads' sum (exact,
    group times a power of two) is rounded once as it is added, so the total is off by at most half a unit, 2^-24 of
    it."""
    B, T, H, d = 2, 4096, 2, 256
    q = torch.zeros((B, H * group, d), dtype=torch.bfloat16, device="cuda")
    rows = {"bf16": [(d, torch.bfloat16)], "q8_0": [(d, torch.int8), (d // 32, torch.float16)],
            "q4_0": [(d // 2, torch.uint8), (d // 32, torch.float16)]}[fmt]
    cache = [torch.ones((B, T, H, n), dtype=t, device="cuda") for n, t in 2 * rows]
    gen = torch.Generator(device="cuda").manual_seed(3)
    acc = 8192 + 8000 * torch.rand((B, H, T), generator=gen, device="cuda")
    want = acc.double() + group / T
    fn = {"bf16": hb.gqa_attn_decode_acc, "q8_0": hb.gqa_attn_decode_q8_0_acc, "q4_0": hb.gqa_attn_decode_q4_0}[fmt]
    fn(q, *cache, acc_in=acc, acc_out=acc)
    hb.hh_device_status()
    # 2^-20 of the step's weight for the exponential and the denominator
    assert torch.all((acc.double() - want).abs() <= 2.0 ** -24 * want + 2.0 ** -20 * group / T)


# ---------------------------------------------------------------- q8_0 with weights
def _q8(x):
    xb = np.asarray(x, np.float64).reshape(x.shape[:-1] + (-1, 32))
    s = (np.abs(xb).max(-1, keepdims=True) / 127).astype(np.float16)
    c = np.divide(xb, s.astype(np.float64), out=np.zeros_like(xb), where=s != 0)
    return np.clip(np.rint(c), -127, 127).astype(np.int8).reshape(x.shape), s[..., 0]


def _check_q8_acc(q, k, v):
    """gqa_attn_decode_q8_0_acc over the cache of k, v (scale 1/16), within the bound of test_gpu_kv_cache.py."""
    q = I.f32_to_bf16_bits(q.astype(np.float32))
    (kx, ks), (vx, vs) = _q8(k), _q8(v)
    deq = lambda x, s: x.astype(np.float64) * np.repeat(s.astype(np.float64), 32, -1)
    acc = torch.zeros(k.shape[0], k.shape[2], k.shape[1], device="cuda")
    o = hb.gqa_attn_decode_q8_0_acc(dev_bf16(q), *(torch.from_numpy(a).cuda() for a in (kx, ks, vx, vs)), acc, acc,
                                    scale=1 / 16)
    hb.hh_device_status()
    zero = np.zeros(acc.shape, np.float32)
    _check_decode("q8_0", o, q, deq(kx, ks), deq(vx, vs), None, None, 1 / 16, zero, acc, zero)


@pytest.mark.parametrize("size", [1e-6, 1e-4, 1.0, 4e4, 1e6])
@pytest.mark.parametrize("group", [3, 12])
def test_q8_0_values_of_any_size(size, group):
    rng = np.random.default_rng(group)
    q, k, v = (rng.standard_normal(s) for s in ((2, 2 * group, 256), (2, 700, 2, 256), (2, 700, 2, 256)))
    v[:, :300, :, :64] *= 1e-2  # scales that grow along the cache
    _check_q8_acc(q, k, v * size)


@pytest.mark.parametrize("group", [3, 12])
def test_q8_0_small_values_under_a_peaked_softmax(group):
    """A key that draws nearly all weight while its own values are small: the others' small products all count."""
    rng = np.random.default_rng(group)
    q, k, v = (rng.standard_normal(s) for s in ((1, group, 256), (1, 3000, 1, 256), (1, 3000, 1, 256)))
    q[:] = q[:, :1]
    k[0, 0, 0] = q[0, 0] * (18 * 16 / (q[0, 0] @ q[0, 0]))  # a logit of 18
    v = 0.05 * np.abs(v)
    v[:, 0] *= 1e-3
    _check_q8_acc(q, k, v)


@pytest.mark.parametrize("size", [1e-4, 1e-2, 1e4, 1e6])
@pytest.mark.parametrize("group", [3, 12])
def test_q8_0_queries_of_any_size(size, group):
    """Queries small or large, the keys the other way round: logits of deviation 1."""
    rng = np.random.default_rng(group)
    q, k, v = (rng.standard_normal(s) for s in ((2, 2 * group, 256), (2, 700, 2, 256), (2, 700, 2, 256)))
    k[..., 32:64] *= 1e-3  # a block of small keys, whose queries are large
    q[..., 32:64] *= 1e3
    _check_q8_acc(q * size, k / size, v)
