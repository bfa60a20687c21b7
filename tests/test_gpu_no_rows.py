"""Calls over packed rows that are none, from arrays without elements (whose strides are 0): they do nothing."""
import numpy as np
import pytest

from tests import kvq_testutil as U

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def kvq():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from attention_group_quantized_gb300 import kvq as K
    K.lib()
    return K


@pytest.mark.parametrize("paged", [False, True])
def test_no_rows_from_empty_arrays(kvq, paged):
    k, v = ((kvq.empty_page_pool([8, 4], 4, 64) if paged else kvq.empty_cache([8, 4], 2, 128, 64)) for _ in range(2))
    i32 = lambda a: torch.tensor(a, dtype=torch.int32, device="cuda")
    at, sfx = ((i32([[0, 1], [2, 3]]),), "_paged") if paged else ((), "")
    start, lens = i32([0, 0, 0]), i32([5, 0])
    status = i32([0])
    q, kn = (U.to_dev_bf16(np.zeros((2, 0, h, 64), np.uint16)[0]) for h in (4, 2))
    before = [t.clone() for c in (k, v) for t in (c.codes, c.sz)]
    getattr(kvq, "append_chunk" + sfx)(kn, kn, k, v, *at, start, lens, status=status)
    assert getattr(kvq, "rotate_append" + sfx)(q, kn, kn, k, v, *at, start, lens, status=status).shape == (0, 4, 64)
    assert getattr(kvq, "chunk_attention" + sfx)(q, k, v, *at, start, lens, status=status).shape == (0, 4, 64)
    getattr(kvq, "block_bounds" + sfx)(k, kvq.empty_bounds(k), *at, start, lens, 0, status=status)
    assert int(status) == 0
    for a, b in zip(before, [t for c in (k, v) for t in (c.codes, c.sz)]):
        assert torch.equal(a, b)
