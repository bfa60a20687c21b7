"""Forks of sequences whose page table names a page outside the pool: such an entry is copied as it stands and reported,
takes no page, and everything else of the call is as it would be without it."""
import pytest

from tests.test_gpu_pages import Pool, _dev

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def kvq():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from attention_group_quantized_gb300 import kvq as K
    K.lib()
    return K


def _fork(kvq, p, a, b):
    kvq.pages_fork(p.pages, p.k, p.v, _dev(a), _dev(b), bounds=p.bounds, workspace=p.ws, status=p.status)


@pytest.mark.parametrize("bad", [10 ** 6, 20, -1, -2 ** 31])
def test_a_bad_last_page_takes_no_page(kvq, bad):
    p = Pool(kvq, 20, 6, 4)
    p.reserve([100, 70, 0, 0, 0, 0])                                # pages 0, 1 and 2, 3
    p.pages.table[0, 1] = bad
    _fork(kvq, p, [0, 1, 0], [2, 3, 4])
    assert int(p.status) == 1
    assert p.pages.seq_lens.tolist() == [100, 70, 100, 70, 100, 0]
    assert p.pages.table[2, :2].tolist() == p.pages.table[4, :2].tolist() == [0, bad]
    assert p.pages.table[3, :2].tolist() == [2, 4]                  # the only page that is taken
    assert p.pages.refs.tolist() == [3, 1, 2, 1, 1] + [0] * 15
    want = list(range(20))
    want[4] = 3
    for x, first in zip(p.buffers(), p.first):
        assert torch.equal(p.page_bytes(x), first[want])


def test_a_bad_last_page_needs_none_of_a_full_pool(kvq):
    p = Pool(kvq, 3, 3, 2)
    p.reserve([100, 30, 0])
    p.pages.table[0, 1] = 3
    _fork(kvq, p, [0], [2])
    assert int(p.status) == 1                                       # (not "too few free pages")
    assert p.pages.seq_lens.tolist() == [100, 30, 100] and p.pages.table[2].tolist() == [0, 3]
    assert p.pages.refs.tolist() == [2, 1, 1]
    for x, first in zip(p.buffers(), p.first):
        assert torch.equal(p.page_bytes(x), first)


@pytest.mark.parametrize("bad", [10 ** 6, -7])
def test_a_bad_full_page_is_copied_as_it_stands(kvq, bad):
    p = Pool(kvq, 20, 4, 4)
    p.reserve([200, 64, 0, 0])                                      # pages 0 .. 3 and 4
    p.pages.table[0, 1] = bad
    p.pages.table[1, 0] = bad
    _fork(kvq, p, [0, 1], [2, 3])
    assert int(p.status) == 1
    assert p.pages.seq_lens.tolist() == [200, 64, 200, 64]
    assert p.pages.table[2].tolist() == [0, bad, 2, 5] and int(p.pages.table[3, 0]) == bad
    assert p.pages.refs.tolist() == [2, 1, 2, 1, 1, 1] + [0] * 14
    want = list(range(20))
    want[5] = 3
    for x, first in zip(p.buffers(), p.first):
        assert torch.equal(p.page_bytes(x), first[want])
