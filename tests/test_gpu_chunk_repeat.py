"""Chunk attention of few rows called again and again with equal inputs: every call gives the same bits.  The sequences'
last key tiles hold at most 64 tokens, so that the tile's second half is a copy of the first, which arrives early and
goes into the slot that the tile before it was read from."""
import pytest

from tests.test_gpu_chunk_long import Call, _built  # noqa: F401  (the module's fixture)

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


@pytest.mark.parametrize("paged", [False, True], ids=["contiguous", "pages"])
@pytest.mark.parametrize("bits", ["84", "4", "8"])
@pytest.mark.parametrize("D,Hq", [(64, 32), (64, 16), (128, 32)])
def test_equal_calls_agree(D, Hq, bits, paged):
    new = [8] * 16
    ctx = [128 * (60 + 2 * i) + 1 + 3 * i - 8 for i in range(16)]       # last tiles of 1 to 46 tokens
    c = Call(23, Hq, 8, D, bits, new, ctx, paged, 0, 0, False)
    first = c.attend()
    c.check(first, (0, 9))
    wrong = torch.zeros((), dtype=torch.int64, device="cuda")
    for _ in range(300):
        wrong += (c.attend() != first).any()
    torch.cuda.synchronize()
    assert int(c.status.item()) == 0
    assert int(wrong) == 0
