"""The rotated append's norm where a row's squares, or their sum, pass fp32 while their mean does not: the queries, codes,
scales and zero points are the definition's, bit for bit, and within its rounding of the 64-bit formula (the bound is
tests/test_gpu_rotate.py's: the roundings are the same)."""
import numpy as np
import pytest

from tests import kvq_testutil as U
from tests import serving_reference as R
from tests.test_gpu_rotate import Case

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def kvq():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from attention_group_quantized_gb300 import kvq as K
    K.lib()
    return K


def _rows(kind, T, heads, D, rng):
    """fp32 rows [T][heads][D] whose mean of squares stays below 2^127."""
    if kind == "flat":                                              # magnitudes 2^57 .. 2^63, one of each row and head
        e = 57 + (np.arange(T)[:, None] + np.arange(heads)) % 7
        return np.ldexp(np.where(rng.random((T, heads, D)) < 0.5, -1.0, 1.0), e[..., None]).astype(np.float32)
    if kind == "spread":                                            # (channels within 2^64: their mean is below 2^126)
        e = 55 + (np.arange(T)[:, None] + np.arange(heads)) % 8
        return np.ldexp(np.clip(rng.standard_normal((T, heads, D)), -4, 4), e[..., None]).astype(np.float32)
    x = rng.standard_normal((T, heads, D)).astype(np.float32)       # one large channel among small ones
    at = rng.integers(0, D, (T, heads))
    e = 50 + (np.arange(T)[:, None] + np.arange(heads)) % 17        # 2^66: a mean of 2^125 (D 128) or 2^126 (D 64)
    np.put_along_axis(x, at[..., None], np.ldexp(np.ones((T, heads, 1), np.float32), e[..., None]), 2)
    return x


# (few rows: a head a warp; many: four heads a warp)
@pytest.mark.parametrize("rows", ["few", "many"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("kind", ["flat", "spread", "one_large"])
def test_large_rows_are_normed(kvq, kind, D, rows):
    T = 50 if rows == "few" else {64: 2500, 128: 1300}[D]
    Hq, Hkv = 8, 4
    c = Case(kvq, D + T, [T], [13], Hq, Hkv, D, "mixed", D)
    x = R.bf16_values(c.x).reshape(T, Hq + 2 * Hkv, D).copy()
    x[:, :Hq + Hkv] = _rows(kind, T, Hq + Hkv, D, np.random.default_rng(T))
    c.x = R.bf16_bits(x).reshape(T, -1)
    out = c.run()
    assert int(c.status) == 0
    assert out[:, :, :].float().abs().amax(-1).gt(0.1).all()        # (rows of a root mean square of 1 again)
    c.check(out)


@pytest.mark.parametrize("D", [64, 128])
def test_the_mean_is_infinite_from_two_to_the_128_on(kvq, D):
    """Rows on both sides of the end of fp32: the mean is the exact one, rounded once, and infinite where that is."""
    Hq, Hkv = 4, 1
    below = np.float32(2.0 ** 64 * (1 - 2.0 ** -8))                 # the bf16 value below 2^64
    mags = [2.0 ** 63, below, 2.0 ** 64, 2.0 ** 65, 2.0 ** 100, 2.0 ** 127]
    c = Case(kvq, D, [len(mags)], [0], Hq, Hkv, D, "8", 0, eps=1e-6)
    x = R.bf16_values(c.x).reshape(len(mags), Hq + 2 * Hkv, D).copy()
    sign = np.where(np.random.default_rng(D).random((len(mags), Hq + Hkv, D)) < 0.5, -1, 1)
    x[:, :Hq + Hkv] = sign * np.array(mags, np.float32)[:, None, None]
    c.x = R.bf16_bits(x).reshape(len(mags), -1)
    out = c.run()
    assert int(c.status) == 0
    want = R.turn(c.x.reshape(x.shape)[:, :Hq], c.w[0], None, np.arange(len(mags)), c.eps, False)[0]
    got = out.cpu().view(torch.int16).numpy().view(np.uint16)
    assert np.array_equal(got, want)
    assert (R.bf16_values(want)[:2] != 0).all() and not R.bf16_values(want)[2:].any()
