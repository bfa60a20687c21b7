"""Chunk attention and windowed decode on the GPU against the definition in 64 bits with a bound per row that tells a
lost, doubled or misplaced tile and an edge off by one at every length (tests/chunk_reference.py, itself tested on the
CPU): the kernel for few rows in all its forms, pieces of many tiles, long windows.

The reference works on the values that dequantize reads back (tested bit for bit elsewhere).  Every token that no query
of a call sees is poisoned first: NaN scale words, and page-table entries outside the pool where a whole page is unseen.
"""
import numpy as np
import pytest

from tests.chunk_reference import attention, plant, visible, worst

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


def _kvq():
    from attention_group_quantized_gb300 import kvq
    return kvq


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    _kvq().lib()


def _ints(a):
    return torch.tensor(np.asarray(a), dtype=torch.int32, device="cuda")


class Call:
    """Ragged sequences (new tokens, tokens before them) in quantised caches, and queries of the new tokens."""

    def __init__(self, seed, Hq, Hkv, D, bits, new, ctx, paged, window, sinks, planted):
        kvq = _kvq()
        gen = torch.Generator(device="cuda").manual_seed(seed)
        randn = lambda *s: torch.randn(s, generator=gen, device="cuda")
        self.Hq, self.Hkv, self.D, self.new, self.window, self.sinks = Hq, Hkv, D, new, window, sinks
        self.lens = [n + c for n, c in zip(new, ctx)]
        B, hb = len(new), np.array([int(b) for b in (bits * Hkv)[:Hkv]], np.int8)
        pages = -(-max(self.lens) // 64)
        self.start = np.concatenate([[0], np.cumsum(new)])
        self.d_start, self.d_lens = _ints(self.start), _ints(self.lens)
        self.rows = sum(new)
        # queries strided, as slices of a fused projection
        self.q = randn(self.rows + 1, Hq + 2, D).bfloat16()[:self.rows, 1:Hq + 1]
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")
        self.bt = None
        if paged:
            spare = 3
            perm = torch.randperm(B * pages + spare, generator=gen, device="cuda")
            self.bt = perm[:B * pages].int().view(B, pages).contiguous()
            self.kc, self.vc = (kvq.empty_page_pool(hb, B * pages + spare, D) for _ in "kv")
        else:
            self.kc, self.vc = (kvq.empty_cache(hb, B, pages * 64, D) for _ in "kv")
        for c in (self.kc, self.vc):
            c.codes.fill_(0xA5)
            c.sz.fill_(-1)
        whole = np.concatenate([[0], np.cumsum(self.lens)])
        k, v = [], []
        for b, L in enumerate(self.lens):
            kb = randn(L, Hkv, D)
            qb = self.q[self.start[b]:self.start[b + 1]].float()
            k.append(plant(kb, qb, Hq // Hkv, window, sinks, 8.0) if planted else kb)
            v.append(randn(L, Hkv, D))
        tab = () if self.bt is None else (self.bt,)
        sfx = "" if self.bt is None else "_paged"
        at = (*tab, _ints(whole), self.d_lens)
        getattr(kvq, "append_chunk" + sfx)(torch.cat(k).bfloat16(), torch.cat(v).bfloat16(), self.kc, self.vc, *at,
                                           status=self.status)
        read = getattr(kvq, "dequantize" + sfx)
        self.kd, self.vd = (read(c, *at, int(whole[-1]), out_dtype=kvq.OUT_F32, status=self.status)
                            for c in (self.kc, self.vc))
        self.whole = whole
        self._poison()

    def _poison(self):
        """Tokens before every window of their sequence that are no sinks."""
        if not self.window:
            return
        for c in (self.kc, self.vc):
            words = c.sz.view(self.Hkv, c.B, c.Tcap, self.D // 32)
            for b, (n, L) in enumerate(zip(self.new, self.lens)):
                hidden = torch.arange(min(self.sinks, L), max(L - n - self.window + 1, min(self.sinks, L)), device="cuda")
                if len(hidden) == 0:
                    continue
                if self.bt is None:
                    words[:, b, hidden] = -1
                else:
                    words[:, self.bt[b, hidden // 64].long(), hidden % 64] = -1
        if self.bt is not None:
            for b, (n, L) in enumerate(zip(self.new, self.lens)):
                for page in range(-(-self.sinks // 64), max(L - n - self.window + 1, 0) // 64):
                    self.bt[b, page] = -5 if page % 2 else 1 << 30

    def attend(self, **kw):
        kvq = _kvq()
        kw = dict(window=self.window, sinks=self.sinks, max_chunk=max(self.new), status=self.status, **kw)
        if self.bt is None:
            return kvq.chunk_attention(self.q, self.kc, self.vc, self.d_start, self.d_lens, **kw)
        return kvq.chunk_attention_paged(self.q, self.kc, self.vc, self.bt, self.d_start, self.d_lens, **kw)

    def decode(self):
        kvq = _kvq()
        assert all(n == 1 for n in self.new)
        q = self.q.contiguous()
        if self.bt is None:
            return kvq.decode_attention_window(q, self.kc, self.vc, self.d_lens, self.window, self.sinks, status=self.status)
        return kvq.decode_attention_window_paged(q, self.kc, self.vc, self.bt, self.d_lens, self.window, self.sinks,
                                                 status=self.status)

    def check(self, out, sequences=None):
        torch.cuda.synchronize()
        assert int(self.status.item()) == 0
        rep, most = self.Hq // self.Hkv, 0.0
        for b in range(len(self.new)) if sequences is None else sequences:
            n, L, r0, w0 = self.new[b], self.lens[b], self.start[b], self.whole[b]
            if n == 0:
                continue
            see = visible(n, L, self.window, self.sinks, "cuda")
            for h in range(self.Hq):
                kd, vd = (x[w0:w0 + L, h // rep] for x in (self.kd, self.vd))
                ref, bound = attention(self.q[r0:r0 + n, h], kd, vd, self.D ** -0.5, see)
                most = max(most, worst(out[r0:r0 + n, h], ref, bound))
        assert most <= 1.0, most


# rows of a KV head: new tokens x query heads per KV head
ROWS = {16: (4, 8, 2), 17: (17, 2, 2), 31: (31, 1, 1), 32: (4, 16, 2)}     # longest new, Hq, Hkv
WINDOWS = {"none": (0, 0), "inside_a_tile": (40, 0), "separate_sinks": (700, 5), "wide_sinks": (1000, 300)}


@pytest.mark.parametrize("window", WINDOWS)
@pytest.mark.parametrize("rows", ROWS)
@pytest.mark.parametrize("paged", [False, True], ids=["contiguous", "pages"])
@pytest.mark.parametrize("bits", ["8", "4"])
@pytest.mark.parametrize("D", [64, 128])
def test_few_rows(D, bits, paged, rows, window):
    n, Hq, Hkv = ROWS[rows]
    assert n * Hq // Hkv == rows
    for planted in (True, False):
        c = Call(rows + D, Hq, Hkv, D, bits, [n, n - 1, 1, 0, n], [3001, 1130, 0, 70, 517], paged, *WINDOWS[window], planted)
        c.check(c.attend())


LONG = [
    # name, Hq, Hkv, D, bits, new, ctx, paged, window, sinks
    # whole CTAs' ranges inside one segment: pieces of more than 64 tiles
    ("pieces_of_80_tiles_16", 32, 8, 128, "8", [4] * 16, [11500 + 97 * i for i in range(16)], True, 0, 0),
    ("pieces_of_80_tiles_32", 32, 8, 64, "84", [8] * 16, [12500 - 61 * i for i in range(16)], False, 0, 0),
    ("two_long_segments", 4, 1, 128, "4", [4, 3], [70000, 50000], True, 0, 0),
    ("long_window_32", 8, 2, 128, "48", [8, 5], [40000, 30000], True, 25000, 130),
    ("long_window_16", 8, 4, 64, "8", [7, 8, 8], [30000, 5000, 20000], True, 9000, 1000),
    ("one_slot", 8, 2, 128, "84", [30, 25], [20000, 9000], True, 0, 0),
    ("two_slots", 8, 2, 64, "84", [60, 40], [15000, 9000], True, 0, 0),
    ("blocks_of_rows_window", 8, 2, 128, "4", [150, 90], [12000, 6000], True, 3000, 200),
    ("blocks_of_rows", 4, 4, 128, "8", [300, 20], [6000, 9000], False, 0, 0),
]


@pytest.mark.parametrize("planted", [False, True], ids=["random", "planted"])
@pytest.mark.parametrize("case", LONG, ids=[c[0] for c in LONG])
def test_long_contexts(case, planted):
    c = Call(7, *case[1:], planted)
    out = c.attend()
    c.check(out, None if len(c.new) < 5 else (0, 7, 15))
    assert torch.equal(out, c.attend())


DECODE = [
    ("all", 8, 2, 128, "84", [40000, 1], False, 0, 0),
    ("long_split", 4, 1, 128, "8", [40000], False, 30000, 130),
    ("ragged_pages", 8, 2, 64, "84", [30000, 129, 64, 9000, 25], True, 8000, 70),
    ("many", 8, 4, 128, "4", [1000 + 517 * i for i in range(24)], True, 5000, 4),
]


@pytest.mark.parametrize("planted", [False, True], ids=["random", "planted"])
@pytest.mark.parametrize("case", DECODE, ids=[c[0] for c in DECODE])
def test_long_windowed_decode(case, planted):
    name, Hq, Hkv, D, bits, lens, paged, window, sinks = case
    c = Call(8, Hq, Hkv, D, bits, [1] * len(lens), [L - 1 for L in lens], paged, window, sinks, planted)
    out = c.decode()
    c.check(out, None if len(lens) < 8 else (0, 5, 23))


@pytest.mark.parametrize("n,Hq", [(4, 8), (7, 8)], ids=["16", "32"])
def test_pages_outside_the_pool_with_few_rows(n, Hq):
    """A visible page id outside the pool is reported, and the other sequences are right."""
    c = Call(9, Hq, 2, 128, "84", [n, n - 1, n], [900, 1400, 60], True, 0, 0, False)
    for bad in (-1, c.kc.B, 2 ** 31 - 1):
        table = c.bt.clone()
        c.bt[1, 9] = bad
        out = c.attend()
        torch.cuda.synchronize()
        assert int(c.status.item()) == 1
        c.status.zero_()
        c.bt.copy_(table)
        c.check(out, (0, 2))
    c.check(c.attend())
