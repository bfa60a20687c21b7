"""Sequences that grow by random chunks, with bounds kept after each of them, and then selection and attention of random rows
over them: shapes drawn over the ranges that the calls take.  Bounds and selections exactly, outputs within the decode's
tolerance of the 64-bit attention over the stored values (tests/kvq_testutil.py)."""
import numpy as np
import pytest

from tests import kvq_testutil as U
from tests import serving_reference as R
from tests.test_gpu_blocks import _dev, _status

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def kvq():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from attention_group_quantized_gb300 import kvq as K
    K.lib()
    return K


@pytest.mark.parametrize("seed", range(24))
def test_growing_sequences(kvq, seed):
    rng = np.random.default_rng(1000 + seed)
    B, D, Hkv = int(rng.integers(1, 7)), int(rng.choice([64, 128])), int(rng.choice([1, 2, 3, 5, 8, 16, 64]))
    rep = int(rng.integers(1, 9))
    bits = [int(x) for x in rng.choice([4, 8], Hkv)]
    most = int(rng.choice([2, 5, 20])) if Hkv < 64 else 4           # pages a sequence
    paged = bool(rng.random() < 0.5)
    n_pages = B * most + 2
    pages = rng.permutation(n_pages)[:B * most].reshape(B, most)
    if paged:
        k, v = (kvq.empty_page_pool(bits, n_pages, D) for _ in range(2))
        at, sfx, place = (_dev(pages),), "_paged", lambda b, i: int(pages[b, i])
    else:
        k, v = (kvq.empty_cache(bits, B, most * 64, D) for _ in range(2))
        at, sfx, place = (), "", lambda b, i: b * most + i
    for c in (k, v):                                                # what no call writes is NaN
        c.codes.fill_(0xFF)
        c.sz.fill_(0x7E007E00)
    bounds = kvq.empty_bounds(k)
    st = _status()
    lens = np.zeros(B, int)
    kept = [[np.zeros((Hkv, 0, D), np.uint16) for _ in range(2)] for _ in range(B)]
    for _ in range(int(rng.integers(2, 6))):
        new = [int(min(rng.choice([0, 1, rng.integers(1, 64 * most + 1)]), 64 * most - lens[b])) for b in range(B)]
        x = R.bf16_bits(rng.standard_normal((2, sum(new), Hkv, D)).astype(np.float32) * rng.uniform(0.1, 3))
        start = np.concatenate([[0], np.cumsum(new)])
        lens = lens + new
        rows = [U.to_dev_bf16(a) for a in x]
        getattr(kvq, "append_chunk" + sfx)(rows[0], rows[1], k, v, *at, _dev(start), _dev(lens), status=st)
        getattr(kvq, "block_bounds" + sfx)(k, bounds, *at, _dev(start), _dev(lens), sum(new), status=st)
        for b in range(B):
            for i in range(2):
                kept[b][i] = np.concatenate([kept[b][i], x[i, start[b]:start[b + 1]].transpose(1, 0, 2)], 1)
    assert int(st) == 0
    stored = [[R.stored(kept[b][i], bits) if lens[b] else np.zeros((Hkv, 0, D)) for i in range(2)] for b in range(B)]
    codes, scales = bounds.codes.cpu().numpy(), bounds.scales.cpu().numpy()
    want = [R.bounds(stored[b][0], int(lens[b])) for b in range(B)]
    for b in range(B):
        for i in range(want[b][0].shape[1]):
            assert np.array_equal(codes[:, place(b, i)], want[b][0][:, i])
            assert np.array_equal(scales[:, place(b, i)], want[b][1][:, i])

    rows = int(rng.choice([1, 3, 9, 40])) if Hkv < 64 else 2
    seq = rng.integers(0, B, rows)
    see = np.array([int(rng.integers(0, lens[s] + 1)) if rng.random() < 0.7 else int(lens[s]) for s in seq])
    first, last = int(rng.choice([0, 1, 2])), int(rng.choice([0, 1, 3]))
    n = int(max(first + last, rng.choice([1, 2, 3, 7, 30]), 1))
    q = R.bf16_bits(rng.standard_normal((rows, Hkv * rep, D)).astype(np.float32) * rng.choice([0.0, 1.0, 1.0, 2.0], (rows, 1, 1)))
    qd = U.to_dev_bf16(q)
    sel = getattr(kvq, "select_blocks" + sfx)(qd, k, bounds, *at, _dev(see), n, first=first, last=last, row_seq=_dev(seq),
                                              status=st)
    out = getattr(kvq, "decode_attention_blocks" + sfx)(qd, k, v, *at, sel, _dev(see), row_seq=_dev(seq), status=st)
    assert int(st) == 0
    sel, out = sel.cpu().numpy(), out.cpu().numpy()
    ref = np.zeros((rows, Hkv * rep, D))
    for r in range(rows):
        c, sc = want[seq[r]]
        m = -(-int(see[r]) // 64)
        score = R.scores(R.bf16_values(q[r]), c[:, :m], sc[:, :m]) if m else np.zeros((Hkv, 0))
        for h in range(Hkv):
            assert np.array_equal(sel[r, h], R.select(score[h], n, first, last)), (r, h)
        kk, vv = stored[seq[r]]
        for h in range(Hkv * rep):
            ref[r, h] = R.attend(R.bf16_values(q[r, h]).astype(np.float64), kk[h // rep], vv[h // rep], sel[r, h // rep],
                                 int(see[r]), D ** -0.5)
    U.assert_close(out, ref)
