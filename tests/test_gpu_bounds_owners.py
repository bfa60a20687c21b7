"""Block bounds of batches whose 64-row runs hold the first new rows of many sequences, among them empty ones: every
touched block has its own bounds, whatever its head's width and wherever its page lies."""
import numpy as np
import pytest

from tests import kvq_testutil as U
from tests import serving_reference as R
from tests.test_gpu_blocks import _bits, _dev, _status

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def kvq():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from attention_group_quantized_gb300 import kvq as K
    K.lib()
    return K


@pytest.mark.parametrize("B,D,Hkv,bits,paged,most", [
    (3000, 64, 1, "4", True, 12), (1000, 128, 2, "mixed", True, 14), (1000, 128, 3, "mixed", False, 14),
    (900, 64, 8, "mixed", True, 20), (70, 128, 1, "8", False, 140),                  # 64 rows a warp
    (3000, 128, 2, "mixed", True, 4), (3000, 64, 3, "8", False, 4)])                 # one row a warp: mostly first rows
def test_many_owners(kvq, B, D, Hkv, bits, paged, most):
    rng = np.random.default_rng(most * D + Hkv)
    lens = rng.integers(0, most, B)
    lens[[0, 1, B - 1]] = 0                                         # at both ends as well
    assert lens.sum() > 4096 and (lens.sum() > 4 * B) == (most > 4)
    bits = _bits(bits, Hkv)
    rows, cap = int(lens.sum()), -(-int(lens.max()) // 64) * 64
    n = cap // 64
    x = R.bf16_bits(rng.standard_normal((rows, Hkv, D)).astype(np.float32))
    start = np.concatenate([[0], np.cumsum(lens)])
    if paged:
        pages = rng.permutation(B * n + 5)[:B * n].reshape(B, n)
        k, v = (kvq.empty_page_pool(bits, B * n + 5, D) for _ in range(2))
        at, sfx, place = (_dev(pages),), "_paged", lambda b, i: int(pages[b, i])
    else:
        k, v = (kvq.empty_cache(bits, B, cap, D) for _ in range(2))
        at, sfx, place = (), "", lambda b, i: b * n + i
    rows_dev = U.to_dev_bf16(x)
    st = _status()
    getattr(kvq, "append_chunk" + sfx)(rows_dev, rows_dev, k, v, *at, _dev(start), _dev(lens), status=st)
    b = kvq.empty_bounds(k)
    b.codes.fill_(111)
    getattr(kvq, "block_bounds" + sfx)(k, b, *at, _dev(start), _dev(lens), rows, status=st)
    assert int(st) == 0
    codes, scales = b.codes.cpu().numpy(), b.scales.cpu().numpy()
    touched = np.zeros(codes.shape[1], bool)
    for s in range(B):
        for i in range(-(-int(lens[s]) // 64)):
            touched[place(s, i)] = True
    assert (codes[:, ~touched] == 111).all() and not (codes[:, touched] == 111).all((2, 3, 4)).any()
    for s in list(range(0, B, 11)) + [B // 2]:
        if lens[s] == 0:
            continue
        c, sc = R.bounds(R.stored(x[start[s]:start[s + 1]].transpose(1, 0, 2), bits), int(lens[s]))
        for i in range(c.shape[1]):
            assert np.array_equal(codes[:, place(s, i)], c[:, i]) and np.array_equal(scales[:, place(s, i)], sc[:, i])
