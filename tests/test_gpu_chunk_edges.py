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
