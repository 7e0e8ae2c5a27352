"""The KV-cache operators at the ends of the formats' ranges: blocks whose scale is a small subnormal fp16, bit for bit
against the fp64 reference."""
import numpy as np
import pytest

from full_attention_gated_b200 import inputs as I
from helpers import f64
from oracle import kv_cache as R
from test_gpu_kv_cache import _append_case

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
