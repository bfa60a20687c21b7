"""Bounds, selection and attention over selected blocks against their definitions: bounds and selections exactly, outputs
within the decode's tolerance of the 64-bit attention over the stored values."""
import numpy as np
import pytest

from tests import kvq_testutil as U
from tests import serving_reference as R

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def kvq():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from attention_group_quantized_gb300 import kvq as K
    K.lib()
    return K


def _dev(a, dtype=np.int32):
    return torch.from_numpy(np.ascontiguousarray(np.asarray(a, dtype))).cuda()


def _bits(bits, Hkv):
    return {"8": [8] * Hkv, "4": [4] * Hkv}.get(bits) or [8 if i % 2 else 4 for i in range(Hkv)]


class Store:
    """Sequences in caches or pools, with their stored values; what lies past their ends is NaN."""

    def __init__(self, kvq, seed, lens, Hkv, D, bits, paged, cap=None):
        rng = np.random.default_rng(seed)
        self.kvq, self.Hkv, self.D, self.lens, self.rng = kvq, Hkv, D, list(lens), rng
        self.bits = _bits(bits, Hkv)
        self.cap = cap or max(64, -(-max(lens) // 64) * 64)
        B = len(lens)
        n = self.cap // 64
        make = (lambda: kvq.empty_page_pool(self.bits, B * n + 3, D)) if paged else (lambda: kvq.empty_cache(self.bits, B, self.cap, D))
        self.k, self.v = make(), make()
        for c in (self.k, self.v):
            c.codes.fill_(0xFF)
            c.sz.fill_(0x7E007E00)                                  # scales and zero points NaN
        self.pages = rng.permutation(B * n + 3)[:B * n].reshape(B, n) if paged else None
        self.table = _dev(self.pages) if paged else None
        self.x = []
        self.kv = []
        for L in lens:
            x = rng.standard_normal((2, Hkv, L, D)).astype(np.float32)
            x[0] += np.repeat(rng.standard_normal((Hkv, -(-L // 64), D)).astype(np.float32), 64, 1)[:, :L]
            self.x.append(R.bf16_bits(x))
            self.kv.append([R.stored(self.x[-1][i], self.bits) if L else np.zeros((Hkv, 0, D)) for i in range(2)])
        self.start = np.concatenate([[0], np.cumsum(lens)])
        rows = [torch.cat([U.to_dev_bf16(x[i].transpose(1, 0, 2)) for x in self.x]) for i in range(2)]
        self.write(rows[0], rows[1], self.start, lens)
        self.bounds = kvq.empty_bounds(self.k)
        self.bounds.codes.fill_(111)
        self.bounds.scales.fill_(float("nan"))

    def write(self, k, v, start, lens):
        if self.table is None:
            self.kvq.append_chunk(k, v, self.k, self.v, _dev(start), _dev(lens))
        else:
            self.kvq.append_chunk_paged(k, v, self.k, self.v, self.table, _dev(start), _dev(lens))

    def bound(self, start, lens, rows, status=None):
        if self.table is None:
            self.kvq.block_bounds(self.k, self.bounds, _dev(start), _dev(lens), rows, status=status)
        else:
            self.kvq.block_bounds_paged(self.k, self.bounds, self.table, _dev(start), _dev(lens), rows, status=status)

    def place(self, b, i):
        return b * (self.cap // 64) + i if self.pages is None else int(self.pages[b, i])

    def select(self, q, row_lens, n, **more):
        if self.table is None:
            return self.kvq.select_blocks(q, self.k, self.bounds, row_lens, n, **more)
        return self.kvq.select_blocks_paged(q, self.k, self.bounds, self.table, row_lens, n, **more)

    def attend(self, q, blocks, row_lens, **more):
        if self.table is None:
            return self.kvq.decode_attention_blocks(q, self.k, self.v, blocks, row_lens, **more)
        return self.kvq.decode_attention_blocks_paged(q, self.k, self.v, self.table, blocks, row_lens, **more)


def _status():
    return torch.zeros(1, dtype=torch.int32, device="cuda")


# ---------------------------------------------------------------- bounds

BOUNDS = [
    ("one_token", [1], 1, 64, "8", False),
    ("edges_d64", [64, 63, 65, 0, 128], 3, 64, "mixed", True),
    ("edges_d128", [64, 63, 65, 0, 200], 2, 128, "mixed", False),
    ("int4_pages", [333, 7], 4, 128, "4", True),
    ("prompt", [4500], 2, 64, "8", False),
    ("prompts_pages", [2600, 3100, 90], 2, 128, "mixed", True),
]


@pytest.mark.parametrize("case", BOUNDS, ids=[c[0] for c in BOUNDS])
def test_bounds_of_whole_sequences(kvq, case):
    name, lens, Hkv, D, bits, paged = case
    s = Store(kvq, len(name), lens, Hkv, D, bits, paged)
    st = _status()
    s.bound(s.start, lens, sum(lens), st)
    assert int(st) == 0
    codes, scales = s.bounds.codes.cpu().numpy(), s.bounds.scales.cpu().numpy()
    seen = np.zeros(codes.shape[1], bool)
    for b, L in enumerate(lens):
        c, sc = R.bounds(s.kv[b][0], L)
        for i in range(c.shape[1]):
            at = s.place(b, i)
            seen[at] = True
            assert np.array_equal(codes[:, at], c[:, i]) and np.array_equal(scales[:, at], sc[:, i])
            # no stored value lies outside, to the rounding of the scale and of the product (2^-23 of the value)
            hi = c[:, i, :, 0].astype(np.float64) * sc[:, i][..., None]
            lo = c[:, i, :, 1].astype(np.float64) * sc[:, i][..., None]
            x = s.kv[b][0][:, 64 * i:64 * i + 64].reshape(Hkv, -1, D // 32, 32)
            room = 2.0 ** -22 * np.abs(x).max()
            assert (x <= hi[:, None] + room).all() and (x >= lo[:, None] - room).all()
    assert (codes[:, ~seen] == 111).all() and np.isnan(scales[:, ~seen]).all()
    ids = np.flatnonzero(seen)[::-1].copy()
    values = kvq.bounds_values(s.bounds, _dev(ids)).cpu().numpy()
    want = codes[:, ids].astype(np.float32) * scales[:, ids][..., None, None]
    assert np.array_equal(values, want.transpose(0, 1, 3, 2, 4).reshape(Hkv, len(ids), 2, D))


@pytest.mark.parametrize("paged", [False, True])
def test_bounds_of_new_tokens_only(kvq, paged):
    lens, new = [130, 64, 65, 1, 320], [1, 1, 1, 1, 200]
    s = Store(kvq, 2, lens, 2, 128, "mixed", paged)
    start = np.concatenate([[0], np.cumsum(new)])
    s.bound(start, lens, sum(new))
    codes = s.bounds.codes.cpu().numpy()
    for b, (L, n) in enumerate(zip(lens, new)):
        c, _ = R.bounds(s.kv[b][0], L)
        for i in range(-(-L // 64)):
            if i >= (L - n) // 64:
                assert np.array_equal(codes[:, s.place(b, i)], c[:, i])
            else:
                assert (codes[:, s.place(b, i)] == 111).all()


def test_bounds_many_short_sequences(kvq):
    lens = [1 + i % 3 for i in range(3000)]                         # 6,000 rows: 32 a warp, a block each of few
    s = Store(kvq, 3, lens[:1], 1, 64, "8", False)
    del s
    x = R.bf16_bits(np.random.default_rng(3).standard_normal((sum(lens), 1, 64)).astype(np.float32))
    k, v = kvq.empty_cache([8], 3000, 64, 64), kvq.empty_cache([8], 3000, 64, 64)
    start = np.concatenate([[0], np.cumsum(lens)])
    kvq.append_chunk(U.to_dev_bf16(x), U.to_dev_bf16(x), k, v, _dev(start), _dev(lens))
    b = kvq.empty_bounds(k)
    kvq.block_bounds(k, b, _dev(start), _dev(lens), sum(lens))
    codes, scales = b.codes.cpu().numpy(), b.scales.cpu().numpy()
    for i in range(0, 3000, 7):
        c, sc = R.bounds(R.stored(x[start[i]:start[i + 1]].transpose(1, 0, 2), [8]), lens[i])
        assert np.array_equal(codes[:, i], c[:, 0]) and np.array_equal(scales[:, i], sc[:, 0])


def test_bounds_of_zeros_bad_sequences_and_pages(kvq):
    s = Store(kvq, 4, [70, 80], 2, 64, "8", True)
    zero = torch.zeros((70, 2, 64), dtype=torch.bfloat16, device="cuda")
    s.write(zero, zero, [0, 70, 70], [70, 80])
    st = _status()
    s.bound([0, 70, 70], [70, 80], 70, st)
    assert int(st) == 0
    at = s.place(0, 1)
    assert not s.bounds.codes[:, at].any() and not s.bounds.scales[:, at].any()
    s.bound([0, 70, 150], [70, 9], 150, st)                         # longer than its sequence
    assert int(st) == 1
    st.zero_()
    good = s.table.clone()
    s.table[1, 0] = -5
    s.bound([0, 70, 150], [70, 80], 150, st)
    assert int(st) == 1
    c, _ = R.bounds(s.kv[1][0], 80)
    assert np.array_equal(s.bounds.codes[:, int(good[1, 1])].cpu().numpy(), c[:, 1])
    st.zero_()
    got = kvq.bounds_values(s.bounds, _dev([at, -1, 10 ** 6]), status=st)
    assert int(st) == 1 and not got.any()


def test_bounds_of_non_finite_values_are_reported(kvq):
    s = Store(kvq, 5, [70], 1, 64, "8", False)
    s.k.sz.view(1, 1, 128, 2)[0, 0, 66, 1] = 0x00007C00             # an infinite scale
    st = _status()
    s.bound([0, 70], [70], 70, st)
    assert int(st) == 6


# ---------------------------------------------------------------- selection

def _random_bounds(kvq, rng, B, Hkv, blocks, D):
    """Bounds of a cache of B sequences of `blocks` blocks, as they come."""
    hi = rng.integers(-40, 128, (Hkv, B * blocks, D // 32, 32))
    lo = hi - rng.integers(0, 100, hi.shape)
    codes = np.stack([hi, np.maximum(lo, -127)], 3).astype(np.int8)
    scales = rng.uniform(0.01, 0.05, codes.shape[:3]).astype(np.float32)
    k = kvq.empty_cache([4] * Hkv, B, blocks * 64, D)
    return k, kvq.BlockBounds(_dev(codes, np.int8), _dev(scales, np.float32)), codes, scales


SELECT = [
    # name, B, Hq, Hkv, D, blocks, lens, n_select, first, last
    ("short", 3, 4, 2, 64, 4, [256, 1, 129], 3, 1, 1),
    ("all_of_them", 3, 8, 2, 128, 8, [512, 300, 0], 8, 1, 1),
    ("one_of_many", 2, 2, 2, 64, 300, [19200, 6401], 1, 0, 0),
    ("no_forced", 1, 8, 1, 128, 100, [6400], 17, 0, 0),
    ("forced_only", 2, 6, 2, 128, 50, [3200, 700], 5, 3, 2),
    ("forced_overlap", 2, 6, 2, 128, 50, [3200, 256], 8, 4, 4),
    ("several_chunks", 1, 4, 1, 128, 2000, [127990], 64, 1, 2),
    ("many_rows", 40, 8, 2, 128, 33, [1 + 53 * i for i in range(40)], 9, 1, 1),
    ("long_in_memory", 1, 2, 1, 64, 9000, [575999], 300, 1, 1),
    ("nearly_all", 1, 5, 1, 64, 700, [44800], 699, 1, 1),
]


@pytest.mark.parametrize("case", SELECT, ids=[c[0] for c in SELECT])
def test_selection(kvq, case):
    name, B, Hq, Hkv, D, blocks, lens, n, first, last = case
    rng = np.random.default_rng(len(name))
    k, bounds, codes, scales = _random_bounds(kvq, rng, B, Hkv, blocks, D)
    q = R.bf16_bits(rng.standard_normal((B, Hq, D)).astype(np.float32))
    st = _status()
    ws = kvq.select_workspace(B, Hkv, k.Tcap)
    for call in range(2):                                           # (the workspace's counters are zero again)
        got = kvq.select_blocks(U.to_dev_bf16(q), k, bounds, _dev(lens), n, first=first, last=last, workspace=ws,
                                status=st).cpu().numpy()
        assert int(st) == 0
        for b in range(B):
            m = -(-lens[b] // 64)
            at = slice(b * blocks, b * blocks + m)
            score = R.scores(R.bf16_values(q[b]), codes[:, at], scales[:, at]) if m else np.zeros((Hkv, 0))
            for h in range(Hkv):
                assert np.array_equal(got[b, h], R.select(score[h], n, first, last)), (call, b, h)


def test_equal_scores_go_to_the_lowest_index(kvq):
    rng = np.random.default_rng(1)
    k, bounds, codes, scales = _random_bounds(kvq, rng, 1, 2, 400, 128)
    same = rng.integers(0, 3, 400)                                  # three kinds of blocks
    codes[:], scales[:] = codes[:, same], scales[:, same]
    bounds.codes.copy_(_dev(codes, np.int8))
    bounds.scales.copy_(_dev(scales, np.float32))
    q = R.bf16_bits(rng.standard_normal((1, 4, 128)).astype(np.float32))
    for n, qq in ((150, q), (399, q), (150, np.zeros_like(q))):     # (a zero query: every score 0)
        got = kvq.select_blocks(U.to_dev_bf16(qq), k, bounds, _dev([25600]), n, first=0, last=3).cpu().numpy()
        score = R.scores(R.bf16_values(qq[0]), codes, scales)
        for h in range(2):
            assert np.array_equal(got[0, h], R.select(score[h], n, 0, 3))


def test_rows_of_one_sequence_and_paged(kvq):
    s = Store(kvq, 6, [900, 1300], 2, 128, "mixed", True)
    s.bound(s.start, s.lens, sum(s.lens))
    seq, lens = [1, 1, 1, 0, 1, 0], [1300, 1299, 640, 900, 64, 1]
    q = R.bf16_bits(s.rng.standard_normal((6, 8, 128)).astype(np.float32))
    got = s.select(U.to_dev_bf16(q), _dev(lens), 4, row_seq=_dev(seq)).cpu().numpy()
    for r in range(6):
        # (a row that ends inside a block scores it by the whole block's bounds)
        c, sc = R.bounds(s.kv[seq[r]][0], s.lens[seq[r]])
        m = -(-lens[r] // 64)
        score = R.scores(R.bf16_values(q[r]), c[:, :m], sc[:, :m])
        for h in range(2):
            assert np.array_equal(got[r, h], R.select(score[h], 4, 1, 1))


def test_selection_reports(kvq):
    rng = np.random.default_rng(2)
    k, bounds, _, _ = _random_bounds(kvq, rng, 3, 1, 20, 64)
    q = torch.randn((3, 2, 64), device="cuda").bfloat16()
    for lens, seq in (([-1, 64, 1280], None), ([1281, 64, 1280], None), ([700, 64, 1280], [3, 0, 1]),
                      ([700, 64, 1280], [-1, 0, 1])):
        st = _status()
        got = kvq.select_blocks(q, k, bounds, _dev(lens), 4, row_seq=None if seq is None else _dev(seq), status=st)
        assert int(st) == 1 and (got[0] == -1).all() and (got[1, 0].cpu().numpy() == [0, -1, -1, -1]).all()
    st = _status()
    q[1, 1, 5] = float("nan")
    got = kvq.select_blocks(q, k, bounds, _dev([1280] * 3), 4, status=st).cpu().numpy()
    assert int(st) == 6
    assert all(len(set(r)) == 4 and r.min() >= 0 and r.max() < 20 and (np.diff(r) > 0).all() for r in got[:, 0])


# ---------------------------------------------------------------- attention

ATTEND = [
    # name, lens, Hq, Hkv, D, bits, paged, n_select
    ("one_token", [1], 4, 4, 64, "8", False, 1),
    ("tiny", [500], 4, 4, 64, "8", False, 4),
    ("gqa_pages", [900, 64, 63, 1300], 8, 2, 128, "mixed", True, 5),
    ("gqa_contiguous", [900, 0, 65, 1300], 16, 2, 128, "mixed", False, 5),
    ("int4_odd_group", [2000, 777], 6, 2, 64, "4", True, 9),
    ("more_than_there_are", [130, 1], 5, 1, 128, "4", False, 40),
    ("rep_one", [1500], 3, 3, 128, "8", True, 7),
    ("many_rows", [1 + 41 * i for i in range(40)], 4, 2, 64, "8", False, 6),
]


def _lists(rng, lens, Hkv, n):
    """Random ascending lists for every (row, KV head)."""
    out = np.full((len(lens), Hkv, n), -1, np.int32)
    for r, L in enumerate(lens):
        m = -(-L // 64)
        for h in range(Hkv):
            got = np.sort(rng.permutation(m)[:rng.integers(0, min(n, m) + 1) if n > 1 else min(n, m)])
            out[r, h, :len(got)] = got
    return out


@pytest.mark.parametrize("out_dtype", ["f32", "bf16"])
@pytest.mark.parametrize("case", ATTEND, ids=[c[0] for c in ATTEND])
def test_attention_over_lists(kvq, case, out_dtype):
    name, lens, Hq, Hkv, D, bits, paged, n = case
    s = Store(kvq, len(name), lens, Hkv, D, bits, paged)
    q = R.bf16_bits(s.rng.standard_normal((len(lens), Hq, D)).astype(np.float32))
    lists = _lists(s.rng, lens, Hkv, n)
    st = _status()
    ws = kvq.decode_workspace(len(lens), Hq, Hkv, D)
    for call in range(2):
        got = s.attend(U.to_dev_bf16(q), _dev(lists), _dev(lens), status=st, workspace=ws,
                       out_dtype=kvq.OUT_F32 if out_dtype == "f32" else kvq.OUT_BF16).float().cpu().numpy()
        assert int(st) == 0
        ref = np.zeros((len(lens), Hq, D))
        for r, L in enumerate(lens):
            for h in range(Hq):
                kh = h // (Hq // Hkv)
                ref[r, h] = R.attend(R.bf16_values(q[r, h]).astype(np.float64), s.kv[r][0][kh], s.kv[r][1][kh],
                                     lists[r, kh], L, D ** -0.5)
        U.assert_close(got, ref, name, out_bf16=out_dtype == "bf16")


def test_attention_over_every_block_is_the_decode(kvq):
    s = Store(kvq, 7, [1000, 333], 2, 128, "mixed", False)
    q = torch.randn((2, 8, 128), device="cuda").bfloat16()
    lens = _dev([1000, 333])
    lists = torch.arange(16, dtype=torch.int32, device="cuda").expand(2, 2, 16).contiguous()
    lists[1, :, 6:] = -1
    assert torch.equal(s.attend(q, lists, lens), kvq.decode_attention(q, s.k, s.v, lens))


def test_rows_of_one_sequence(kvq):
    s = Store(kvq, 8, [400, 700], 2, 64, "mixed", True)
    seq, lens = [1, 1, 0, 1], [700, 699, 400, 65]
    q = R.bf16_bits(s.rng.standard_normal((4, 4, 64)).astype(np.float32))
    lists = _lists(s.rng, lens, 2, 5)
    got = s.attend(U.to_dev_bf16(q), _dev(lists), _dev(lens), row_seq=_dev(seq), softmax_scale=0.3).cpu().numpy()
    ref = np.stack([[R.attend(R.bf16_values(q[r, h]).astype(np.float64), s.kv[seq[r]][0][h // 2], s.kv[seq[r]][1][h // 2],
                              lists[r, h // 2], lens[r], float(np.float32(0.3))) for h in range(4)] for r in range(4)])
    U.assert_close(got, ref)


def test_bad_entries_are_left_out_and_reported(kvq):
    s = Store(kvq, 9, [640, 640], 1, 128, "8", False)
    q = R.bf16_bits(s.rng.standard_normal((2, 4, 128)).astype(np.float32))
    for bad, kept in (([3, 3, 5, -1], [3, 5]), ([5, 2, 7, -1], [5, 7]), ([1, 10, -1, -1], [1]), ([-1, 4, -1, -1], []),
                      ([-7, 4, -1, -1], []), ([2, 2 ** 30, -1, -1], [2]), ([-1, -1, -1, 0], []), ([-2, -2, -2, -2], [])):
        st = _status()
        lists = np.array([[bad], [[0, 1, 2, 9]]], np.int32)
        got = s.attend(U.to_dev_bf16(q), _dev(lists), _dev([640, 640]), status=st).cpu().numpy()
        assert int(st) == 1
        for r, use in enumerate((kept, [0, 1, 2, 9])):
            ref = np.stack([R.attend(R.bf16_values(q[r, h]).astype(np.float64), s.kv[r][0][0], s.kv[r][1][0], use, 640,
                                     128 ** -0.5) for h in range(4)])
            U.assert_close(got[r], ref, str(bad))
    # nothing listed at all: zeros, and nothing to report
    st = _status()
    got = s.attend(U.to_dev_bf16(q), _dev(np.full((2, 1, 4), -1)), _dev([640, 640]), status=st)
    assert int(st) == 0 and not got.any()


def test_bad_rows_give_zeros(kvq):
    s = Store(kvq, 10, [640, 640], 1, 64, "8", True)
    q = torch.randn((2, 2, 64), device="cuda").bfloat16()
    lists = _dev(np.array([[[0, 1]], [[0, 1]]]))
    good = s.attend(q, lists, _dev([640, 640]))
    for lens, seq in (([-3, 640], None), ([641, 640], None), ([640, 640], [2, 1]), ([640, 640], [-1, 1]),
                      ([2 ** 31 - 1, 640], None)):
        st = _status()
        got = s.attend(q, lists, _dev(lens), row_seq=None if seq is None else _dev(seq), status=st)
        assert int(st) == 1 and not got[0].any() and torch.equal(got[1], good[1])


def test_a_listed_page_outside_the_pool_is_reported(kvq):
    s = Store(kvq, 11, [640], 1, 64, "8", True)
    q = torch.randn((1, 2, 64), device="cuda").bfloat16()
    s.write(*(torch.randn((640, 1, 64), device="cuda").bfloat16() for _ in range(2)), [0, 640], [640])
    st = _status()
    s.table[0, 5] = 10 ** 6                                         # not listed: not looked at
    s.attend(q, _dev([[[0, 4]]]), _dev([640]), status=st)
    assert int(st) == 0
    s.attend(q, _dev([[[0, 5]]]), _dev([640]), status=st)
    assert int(st) == 1


def test_captured_selection_and_attention_replay(kvq):
    s = Store(kvq, 12, [3000, 1000], 2, 128, "8", True)
    s.bound(s.start, s.lens, sum(s.lens))
    q = torch.randn((2, 8, 128), device="cuda").bfloat16()
    lens = _dev([3000, 1000])
    ws = kvq.select_workspace(2, 2, s.cap), kvq.decode_workspace(2, 8, 2, 128)
    sel = torch.empty((2, 2, 8), dtype=torch.int32, device="cuda")
    out = torch.empty((2, 8, 128), device="cuda")
    def step():
        s.select(q, lens, 8, out=sel, workspace=ws[0])
        s.attend(q, sel, lens, out=out, workspace=ws[1])
    step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for _ in range(3):
        q.copy_(torch.randn_like(q))
        lens[1] -= 100
        g.replay()
        torch.cuda.synchronize()
        a, b = sel.clone(), out.clone()
        step()
        torch.cuda.synchronize()
        assert torch.equal(a, sel) and torch.equal(b, out)
