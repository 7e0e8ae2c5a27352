"""The KV-cache operators on the host: exports of include/hh_kv.h, refusals before anything reaches a GPU, the
binding's checks, and pins of the fp64 reference that the GPU tests compare against (CPU only)."""
import ctypes
import os
import re

import numpy as np
import pytest
import torch

from full_attention_gated_b200 import binding as hb
from full_attention_gated_b200 import inputs as I
from oracle import kv_cache as R

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
INV, UNS = hb.HH_ERR_INVALID_ARG, hb.HH_ERR_UNSUPPORTED


@pytest.fixture(scope="module")
def lib():
    return hb.load_library()


def _rejects(lib, rc, code, words):
    assert rc == code, (rc, code, lib.hh_last_error())
    assert words.encode() in lib.hh_last_error(), (words, lib.hh_last_error())


def test_exports_every_declared_symbol(lib):
    txt = open(os.path.join(ROOT, "include", "hh_kv.h")).read()
    names = re.findall(r"HH_API\s+[\w\s\*]+?\b(\w+)\s*\(", txt)
    assert sorted(names) == ["gqa_attn_decode_acc", "gqa_attn_decode_acc_workspace_size", "gqa_attn_decode_q4_0",
                             "gqa_attn_decode_q4_0_workspace_size", "gqa_attn_decode_q8_0_acc", "kv_append_q4_0",
                             "kv_compact", "kv_evict_select"]
    for n in names:
        assert hasattr(lib, n), n


def _append(lib, **kw):
    a = dict(k=16, v=16, kv=16, ks=16, vv=16, vs=16, ln=None, nn=None, kh=None, vh=None, B=1, n=4, T=8, H=2, d=256)
    a.update(kw)
    return lib.kv_append_q4_0(*a.values(), None)


def test_append_refuses(lib):
    _rejects(lib, _append(lib, n=-1), INV, "sizes must be positive")
    _rejects(lib, _append(lib, H=0), INV, "sizes must be positive")
    _rejects(lib, _append(lib, d=64), UNS, "only d = 128 or 256")
    _rejects(lib, _append(lib, n=1 << 26, H=8), INV, "sizes too large")
    _rejects(lib, _append(lib, k=None), INV, "null tensor pointer")
    _rejects(lib, _append(lib, vs=None), INV, "null tensor pointer")
    _rejects(lib, _append(lib, kv=24), INV, "16-byte aligned")
    _rejects(lib, _append(lib, kh=16), INV, "k_held and v_held go together")
    for empty in (dict(B=0), dict(n=0), dict(T=0)):
        assert _append(lib, k=None, **empty) == hb.HH_OK


def _decode(lib, **kw):
    a = dict(q=16, kv=16, ks=16, vv=16, vs=16, ln=None, gate=None, o=16, ai=None, ao=None, ws=256, n=1 << 40, B=2,
             T=1000, Hq=8, H=2, d=256, scale=0.1)
    a.update(kw)
    return lib.gqa_attn_decode_q4_0(*a.values(), None)


def test_decode_q4_0_refuses(lib):
    _rejects(lib, _decode(lib, Hq=7), INV, "H_q (7) must be a multiple of H_kv (2)")
    _rejects(lib, _decode(lib, Hq=34), UNS, "at most 16 query heads")
    _rejects(lib, _decode(lib, d=64), UNS, "d = 128 or 256")
    _rejects(lib, _decode(lib, scale=float("nan")), INV, "scale must be finite")
    _rejects(lib, _decode(lib, kv=None), INV, "null tensor pointer")
    _rejects(lib, _decode(lib, ks=None), INV, "null scale pointer")
    _rejects(lib, _decode(lib, vs=8), INV, "scale arrays must be 16-byte aligned")
    _rejects(lib, _decode(lib, ai=16), INV, "acc_in without acc_out")
    _rejects(lib, _decode(lib, ao=24), INV, "acc must be 16-byte aligned")
    _rejects(lib, _decode(lib, ai=32, ao=16), INV, "acc_in must be acc_out or not overlap it")
    need = lib.gqa_attn_decode_q4_0_workspace_size(2, 8, 2, 256, 1000, 0)
    _rejects(lib, _decode(lib, n=need - 1), INV, f"workspace of {need} bytes needed")
    _rejects(lib, _decode(lib, ws=272), INV, "256-byte aligned")
    with_acc = lib.gqa_attn_decode_q4_0_workspace_size(2, 8, 2, 256, 1000, 1)
    assert with_acc >= 2 * 8 * 1000 * 4
    _rejects(lib, _decode(lib, n=with_acc - 1, ao=16), INV, f"workspace of {with_acc} bytes needed")
    assert _decode(lib, B=0) == hb.HH_OK
    assert lib.gqa_attn_decode_q4_0_workspace_size(0, 8, 2, 256, 10, 1) == 0


def test_accumulating_decode_refuses(lib):
    def f(q=16, ln=None, o=16, ai=None, ao=16, ws=256, n=1 << 40, T=100, Hq=8, d=256):
        return lib.gqa_attn_decode_acc(q, 16, 16, ln, None, o, ai, ao, ws, n, 2, T, Hq, 2, d, 0.1, None)

    def g(ks=16, ao=16, d=256):
        return lib.gqa_attn_decode_q8_0_acc(16, 16, ks, 16, 16, None, None, 16, None, ao, 256, 1 << 40, 2, 100, 8, 2, d,
                                            0.1, None)
    _rejects(lib, f(ao=None), INV, "acc_out is null")
    _rejects(lib, f(d=64), UNS, "d = 128 or 256")
    _rejects(lib, f(q=None), INV, "null tensor pointer")
    need = lib.gqa_attn_decode_acc_workspace_size(2, 8, 256, 100)
    assert need >= lib.gqa_attn_decode_workspace_size(2, 8, 256, 100) + 2 * 8 * 100 * 4
    _rejects(lib, f(n=need - 1), INV, f"workspace of {need} bytes needed")
    _rejects(lib, g(ks=None), INV, "null scale pointer")
    _rejects(lib, g(ao=None), INV, "acc_out is null")
    _rejects(lib, g(d=128), UNS, "only d = 256")


def test_select_refuses(lib):
    def f(acc=16, keep=16, B=1, T=100, H=2, n_keep=10, n_recent=2):
        return lib.kv_evict_select(acc, None, keep, B, T, H, n_keep, n_recent, None)
    _rejects(lib, f(n_recent=11), INV, "n_recent (11) must be in 0 .. n_keep (10)")
    _rejects(lib, f(n_recent=-1), INV, "n_recent (-1)")
    _rejects(lib, f(n_keep=-1, n_recent=0), INV, "sizes must not be negative")
    _rejects(lib, f(acc=None), INV, "null tensor pointer")
    _rejects(lib, f(keep=None), INV, "null tensor pointer")
    _rejects(lib, f(acc=8), INV, "16-byte aligned")
    _rejects(lib, f(B=70000), INV, "sizes too large")
    assert f(B=0) == hb.HH_OK and f(n_keep=0, n_recent=0) == hb.HH_OK


def _compact(lib, src, dst, rows, keep=16, acc=(None, None), B=1, Ts=100, Td=100, H=2, n_keep=10, n=None):
    m = len(src)
    s, t = (ctypes.c_void_p * max(m, 1))(*src), (ctypes.c_void_p * max(m, 1))(*dst)
    r = (ctypes.c_int * max(m, 1))(*rows)
    cast = lambda a: ctypes.cast(a, ctypes.c_void_p)
    return lib.kv_compact(keep, cast(s), cast(t), cast(r), m if n is None else n, acc[0], acc[1], B, Ts, Td, H, n_keep,
                          None)


def test_compact_refuses(lib):
    far = 1 << 30
    _rejects(lib, _compact(lib, [16], [far], [100]), INV, "row_bytes[0] = 100 is not a multiple of 8")
    _rejects(lib, _compact(lib, [16], [far], [8192]), INV, "row_bytes[0] = 8192")
    _rejects(lib, _compact(lib, [16], [far], [64], n=9), UNS, "at most 8 arrays")
    _rejects(lib, _compact(lib, [16], [far], [64], n_keep=101), INV, "n_keep (101) above T_dst (100)")
    _rejects(lib, _compact(lib, [16], [16], [64], Td=50), INV, "dst must be src with T_dst = T_src, or not overlap")
    _rejects(lib, _compact(lib, [16], [32], [64]), INV, "dst must be src with T_dst = T_src, or not overlap")
    _rejects(lib, _compact(lib, [1024, far], [1024, 1024], [64, 64]), INV, "arrays 0 and 1 overlap")
    _rejects(lib, _compact(lib, [None], [far], [64]), INV, "null tensor pointer (array 0)")
    _rejects(lib, _compact(lib, [24], [far], [64]), INV, "16-byte aligned")
    _rejects(lib, _compact(lib, [16], [far], [64], keep=None), INV, "keep is null")
    _rejects(lib, _compact(lib, [16], [far], [64], acc=(16, None)), INV, "acc_src and acc_dst go together")
    _rejects(lib, _compact(lib, [16], [far], [64], acc=(16, 32)), INV, "acc_dst must be acc_src")
    _rejects(lib, _compact(lib, [16], [far], [64], Ts=0), INV, "T_src must be positive")
    assert _compact(lib, [16], [far], [64], B=0) == hb.HH_OK


def test_overlapping_arguments_are_refused(lib):
    """Tensors that the kernels read without order while another of the call's is written."""
    far, apart = 1 << 30, dict(k=1 << 20, v=1 << 21, kh=1 << 22, vh=1 << 23)
    for x, y in (("kh", "k"), ("kh", "v"), ("vh", "k"), ("vh", "v"), ("vh", "kh")):
        _rejects(lib, _append(lib, **(apart | {x: apart[y] + 16})), INV, "k_held and v_held must not overlap")
    _rejects(lib, lib.kv_evict_select(1 << 20, None, (1 << 20) + 16, 1, 100, 2, 10, 2, None), INV,
             "keep and acc overlap")
    _rejects(lib, _compact(lib, [16], [far], [64], keep=far + 160), INV, "array 0 and keep overlap")
    _rejects(lib, _compact(lib, [16], [far], [64], acc=(far + 64, 2 * far)), INV, "array 0 and the weights overlap")
    _rejects(lib, _compact(lib, [far], [16], [64], keep=1 << 24, acc=(2 * far, far + 64)), INV, "array 0 and the weights overlap")
    _rejects(lib, _compact(lib, [16], [far], [64], keep=2 * far, acc=(2 * far, 2 * far)), INV,
             "acc_dst and keep overlap")


def test_binding_checks_tensors():
    x = torch.zeros((1, 2, 1, 128), dtype=torch.bfloat16)
    vals, sc = torch.zeros((1, 4, 1, 64), dtype=torch.uint8), torch.zeros((1, 4, 1, 4), dtype=torch.float16)
    with pytest.raises(TypeError, match="k: expected a CUDA tensor"):
        hb.kv_append_q4_0(x, x, vals, sc, vals, sc)
    with pytest.raises(TypeError, match="k: expected torch.bfloat16"):
        hb.kv_append_q4_0(x.float(), x, vals, sc, vals, sc)
    with pytest.raises(ValueError, match="k: expected 4 dimensions"):
        hb.kv_append_q4_0(x[0], x, vals, sc, vals, sc)
    with pytest.raises(TypeError, match="acc: expected a CUDA tensor"):
        hb.kv_evict_select(torch.zeros((1, 1, 4)), 2, 1)
    with pytest.raises(ValueError, match="one tensor per array"):
        hb.kv_compact(torch.zeros((1, 1, 2), dtype=torch.int32), [vals], [])
    with pytest.raises(ValueError, match="nothing to compact"):
        hb.kv_compact(torch.zeros((1, 1, 2), dtype=torch.int32), [])


# ---------------- pins of the reference ----------------
def test_reference_q4_0_closed_forms():
    # a block that is already on a grid of 16 levels comes back exactly
    grid = np.arange(32) % 16 - 8.0
    codes, s = R.q4_0_quantise(grid * 0.5)
    assert s.tolist() == [0.5] and np.array_equal(codes, (np.arange(32) % 16).astype(np.uint8))
    np.testing.assert_array_equal(R.q4_0_values(R.q4_0_pack(codes), s), grid * 0.5)
    # the sign of the first of two elements of equal magnitude decides; the other end clips to 7 / 8 of it
    for first in (3.0, -3.0):
        row = np.zeros(32)
        row[4], row[9] = first, -first
        codes, s = R.q4_0_quantise(row)
        assert float(s[0]) == -first / 8
        assert codes[4] == 0 and codes[9] == 15 and codes[0] == 8
    # zeros, infinities and NaN
    assert R.q4_0_quantise(np.zeros(32))[1][0] == 0
    for bad in (np.inf, -np.inf, np.nan):
        row = np.ones(32)
        row[31] = bad
        codes, s = R.q4_0_quantise(row)
        assert np.isnan(s[0]) and np.all(codes == 8)


def test_reference_q4_0_error_is_at_most_half_a_step():
    rng = np.random.default_rng(1)
    x = I.bf16_bits_to_f32(I.f32_to_bf16_bits(rng.standard_normal((500, 32)).astype(np.float32))).astype(np.float64)
    codes, s = R.q4_0_quantise(x)
    err = np.abs(R.q4_0_values(R.q4_0_pack(codes), s) - x)
    step = np.abs(s.astype(np.float64))
    # at most half a step, except where the far end clips (a whole step at most there, plus the scale's rounding)
    clipped = codes.reshape(-1, 32) == 15
    assert np.all(err[~clipped] <= np.broadcast_to(0.5 * step * (1 + 2 ** -10), err.shape)[~clipped])
    assert np.all(err <= step * (1 + 2 ** -7))


def test_reference_decode_against_the_c_oracle(oracle_mod):
    rng = np.random.default_rng(2)
    q, k, v = rng.standard_normal((2, 4, 8)), rng.standard_normal((2, 30, 2, 8)), rng.standard_normal((2, 30, 2, 8))
    gate = rng.standard_normal((2, 4, 8))
    lens = np.array([30, 11], np.int32)
    o, w = R.decode(q, k, v, lens, gate, 0.3)
    np.testing.assert_allclose(o, oracle_mod.decode_attention(q, k, v, lens, gate, 0.3), atol=1e-12)
    np.testing.assert_allclose(w.sum(-1), 2.0, atol=1e-12)  # the weights of two heads a group
    assert np.all(w[1, :, 11:] == 0)


def test_reference_select_and_compact():
    acc = np.array([[[5, 1, 5, 0, np.nan, 2, -0.0, 9]]], np.float32)
    assert R.evict_select(acc, None, 4, 2)[0, 0].tolist() == [0, 4, 6, 7]
    assert R.evict_select(acc, np.array([4]), 3, 0)[0, 0].tolist() == [0, 1, 2]
    assert R.evict_select(acc, np.array([2]), 3, 1)[0, 0].tolist() == [0, 1, -1]
    rows = np.arange(8).reshape(1, 8, 1, 1)
    out = R.compact(rows, np.array([[[0, 4, -1]]], np.int32), np.full((1, 3, 1, 1), 99))
    assert out.ravel().tolist() == [0, 4, 99]
