"""GPU tests of the chunk calls at the edges of what they accept: descriptions that do not hold, values that the
operands cannot hold, windows beyond 32 bits, rows that no sequence has."""
import numpy as np
import pytest

from tests import kvq_testutil as U
from tests.test_gpu_chunk import Batch, _kvq, check

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

# name, Hq, new tokens of the longest sequence, whether its kernel is asked for by max_chunk
KERNELS = [("narrow16", 8, 4, True), ("narrow32", 8, 7, True), ("one_slot", 8, 20, False), ("two_slots", 8, 50, False)]


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    _kvq().lib()


def _ints(*a):
    return torch.tensor(a, dtype=torch.int32, device="cuda")


# ---------------------------------------------------------------- starts that do not ascend

@pytest.mark.parametrize("starts", [(0, 10, 5, 20), (0, 20, 0, 20), (0, 3, 3, -1)], ids=str)
@pytest.mark.parametrize("max_chunk", [15, None], ids=["narrow", "wide"])
def test_starts_that_do_not_ascend_leave_the_attention_out(starts, max_chunk):
    """Rows of two sequences, or more rows in all than the buffer has: reported, and nothing is computed."""
    b = Batch(101, 4, 2, 64, "8", [10, 0, 10], [40, 30, 50], False)
    b.fill()
    b.append_new()
    b.ok()
    b.d_start = _ints(*starts)
    out = torch.full((20, 4, 64), 9.0, device="cuda")
    b.attend(U.to_dev_bf16(b.q), out=out, max_chunk=max_chunk)
    torch.cuda.synchronize()
    assert int(b.status.item()) == 1
    assert (out == 9.0).all()
    # the calls that look rows up stay within the caches and the buffer
    b.status.zero_()
    b.read("k", b.d_start, b.d_lens, 20)
    torch.cuda.synchronize()
    assert int(b.status.item()) == 1


# ---------------------------------------------------------------- values that the fp16 operands cannot hold

def _bf16(x):
    return int(torch.tensor(float(x)).bfloat16().view(torch.int16).item()) & 0xFFFF


def _with_value(kernel, paged, part, head, seq, tok, value, D=128, **kw):
    """The status and whether all outputs are finite, of a call on caches that hold `value` in one channel."""
    _, Hq, n, narrow = kernel
    b = Batch(111, Hq, 2, D, "84", [n, n - 1], [700, 300], paged)
    assert (n * Hq // 2 <= 32) == narrow
    x = b.k if part == "k" else b.v
    x[seq, head, tok if tok >= 0 else b.lens[seq] + tok, 37] = _bf16(value)
    b.fill()
    b.append_new()
    b.ok()                                                   # a legal row of the cache
    out = b.attend(U.to_dev_bf16(b.q), max_chunk=n, **kw)
    torch.cuda.synchronize()
    return int(b.status.item()), bool(torch.isfinite(out).all())


@pytest.mark.parametrize("kernel", KERNELS, ids=[k[0] for k in KERNELS])
@pytest.mark.parametrize("paged", [False, True], ids=["contiguous", "pages"])
@pytest.mark.parametrize("part", ["k", "v"])
def test_values_beyond_fp16_are_reported(kernel, paged, part):
    for seq, tok in ((0, 3), (0, 500), (1, 299), (1, -1)):    # first, whole and last tiles; a new token
        for head in (0, 1):                                   # 8-bit, 4-bit
            assert _with_value(kernel, paged, part, head, seq, tok, 1e5)[0] == 6, (seq, tok, head)
    assert _with_value(kernel, paged, part, 0, 0, 130, -1e5, D=64)[0] == 6
    # scales are rounded up to fp16: 65536 / qmax gives one whose largest value rounds to an infinity, 65280 / qmax does not
    for head in (0, 1):
        assert _with_value(kernel, paged, part, head, 0, 130, 65536.0)[0] == 6
        assert _with_value(kernel, paged, part, head, 0, 130, 65280.0) == (0, True)


@pytest.mark.parametrize("kernel", KERNELS, ids=[k[0] for k in KERNELS])
@pytest.mark.parametrize("part", ["k", "v"])
def test_values_beyond_fp16_that_nothing_sees_are_not(kernel, part):
    n = kernel[2]
    window, sinks = 200, 70                                    # sequence 0: positions 700 .. 699 + n; first key 501
    seen = dict(window=window, sinks=sinks)
    for tok, want in ((69, 6), (70, 0), (300, 0), (500, 0), (501, 6), (640, 6)):
        status, finite = _with_value(kernel, True, part, tok % 2, 0, tok, 1e5, **seen)
        assert status == want and (finite or want), tok
