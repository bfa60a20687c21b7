"""GPU parity of the chunk calls (ragged append, read-back, chunk attention) and of the windowed decode.

Codes, scales and zero points must equal the oracle's bit for bit, read-back values the oracle's dequantised ones
after one rounding.  Attention is compared with the definition in fp64 on the oracle's dequantised cache; its bound
counts the roundings the kernels may make, element by element (see _bound).
"""
import numpy as np
import pytest

from oracle import kvq_oracle as O
from tests import kvq_testutil as U
import kvq_workloads as W

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

SENT_CODE, SENT_WORD = 0xA5, -1      # 0xFFFFFFFF: a NaN scale and a NaN zero point


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from attention_group_quantized_gb300 import kvq
    kvq.lib()


def _kvq():
    from attention_group_quantized_gb300 import kvq
    return kvq


class Batch:
    """One ragged batch: bf16 K, V rows of whole sequences, the chunk at their ends, caches holding everything but
    the chunk (positions never written hold a NaN sentinel), and the oracle's dequantised values."""

    def __init__(self, seed, Hq, Hkv, D, bits, new, ctx, paged, spare_cap=0):
        kvq = _kvq()
        rng = np.random.default_rng(seed)
        self.Hq, self.Hkv, self.D, self.new = Hq, Hkv, D, list(new)
        self.B = len(new)
        self.lens = [n + c for n, c in zip(new, ctx)]
        self.cap = max(64, -(-(max(self.lens) + spare_cap) // 64) * 64)
        self.bits = np.array([int(b) for b in (bits if len(bits) == Hkv else bits * Hkv)], np.int8)
        T = max(max(self.lens), 1)
        scale = np.ones((Hkv, D), np.float32)
        scale[:, rng.integers(0, D, 2)] *= 5.0
        self.k = W._draw_bf16(rng, (self.B, Hkv, T, D), scale)
        self.v = W._draw_bf16(rng, (self.B, Hkv, T, D))
        self.rows = sum(new)
        self.q = W._draw_bf16(rng, (max(self.rows, 1), Hq, D))[:self.rows]
        self.kp, _, _, self.kd = U.oracle_quantize(self.k, self.bits)
        self.vp, _, _, self.vd = U.oracle_quantize(self.v, self.bits)
        self.start = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
        self.paged = paged
        if paged:
            pages = self.cap // 64
            n = self.B * pages + 5
            self.table = rng.permutation(n)[:self.B * pages].reshape(self.B, pages).astype(np.int32)
            self.kc, self.vc = (kvq.empty_page_pool(self.bits, n, D) for _ in "kv")
            self.bt = torch.from_numpy(self.table).cuda()
        else:
            self.table, self.bt = None, None
            self.kc, self.vc = (kvq.empty_cache(self.bits, self.B, self.cap, D) for _ in "kv")
        for c in (self.kc, self.vc):
            c.codes.fill_(SENT_CODE)
            c.sz.fill_(SENT_WORD)
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")
        self.d_start = torch.from_numpy(self.start).cuda()
        self.d_lens = torch.tensor(self.lens, dtype=torch.int32, device="cuda")

    def packed(self, x):
        """Chunk rows of x[B][H][T][D], packed [rows][H][D]."""
        out = [x[b, :, L - n:L].transpose(1, 0, 2) for b, (n, L) in enumerate(zip(self.new, self.lens))]
        return np.concatenate(out) if self.rows else np.empty((0, x.shape[1], self.D), x.dtype)

    def fill(self, upto=None):
        """Quantise each sequence's first upto[b] tokens (default: all but the chunk) with a call of its own."""
        kvq = _kvq()
        upto = [L - n for n, L in zip(self.new, self.lens)] if upto is None else upto
        start = torch.tensor(np.concatenate([[0], np.cumsum(upto)]), dtype=torch.int32, device="cuda")
        lens = torch.tensor(upto, dtype=torch.int32, device="cuda")
        rows = [np.concatenate([x[b, :, :u].transpose(1, 0, 2) for b, u in enumerate(upto)]) for x in (self.k, self.v)]
        if sum(upto):
            self.append(U.to_dev_bf16(rows[0]), U.to_dev_bf16(rows[1]), start, lens)

    def append(self, k, v, start, lens, **kw):
        kvq = _kvq()
        if self.paged:
            kvq.append_chunk_paged(k, v, self.kc, self.vc, self.bt, start, lens, status=self.status, **kw)
        else:
            kvq.append_chunk(k, v, self.kc, self.vc, start, lens, status=self.status, **kw)

    def append_new(self):
        self.append(U.to_dev_bf16(self.packed(self.k)), U.to_dev_bf16(self.packed(self.v)), self.d_start, self.d_lens)

    def read(self, which, start, lens, rows, **kw):
        kvq = _kvq()
        c = self.kc if which == "k" else self.vc
        if self.paged:
            return kvq.dequantize_paged(c, self.bt, start, lens, rows, status=self.status, **kw)
        return kvq.dequantize(c, start, lens, rows, status=self.status, **kw)

    def attend(self, q, **kw):
        kvq = _kvq()
        kw.setdefault("status", self.status)
        if self.paged:
            return kvq.chunk_attention_paged(q, self.kc, self.vc, self.bt, self.d_start, self.d_lens, **kw)
        return kvq.chunk_attention(q, self.kc, self.vc, self.d_start, self.d_lens, **kw)

    def decode(self, q, window, sinks, **kw):
        kvq = _kvq()
        if self.paged:
            return kvq.decode_attention_window_paged(q, self.kc, self.vc, self.bt, self.d_lens, window, sinks,
                                                     status=self.status, **kw)
        return kvq.decode_attention_window(q, self.kc, self.vc, self.d_lens, window, sinks, status=self.status, **kw)

    def ok(self):
        torch.cuda.synchronize()
        assert int(self.status.item()) == 0

    def reference(self, window=0, sinks=0, scale=None):
        """(fp64 outputs [rows][Hq][D], rounding bounds of the same shape)."""
        scale = self.D ** -0.5 if scale is None else scale
        q = O.bf16_to_f32(self.q).astype(np.float64)
        out, bound = np.zeros(q.shape), np.zeros(q.shape)
        for b, (n, L) in enumerate(zip(self.new, self.lens)):
            if n == 0:
                continue
            r0 = self.start[b]
            pos = np.arange(L - n, L)[:, None]
            j = np.arange(L)[None]
            see = j <= pos
            if window:
                see &= (j > pos - window) | (j < sinks)
            for h in range(self.Hq):
                kvh = h // (self.Hq // self.Hkv)
                o, e = attention_and_bound(q[r0:r0 + n, h], self.kd[b, kvh, :L], self.vd[b, kvh, :L], scale, see)
                out[r0:r0 + n, h], bound[r0:r0 + n, h] = o, e
        return out, bound


def attention_and_bound(q, k, v, scale, see):
    """softmax(scale q k^T) v over the visible keys in fp64, and how far a kernel may be off.

    Roundings counted: K_hat and V_hat to fp16 and P to fp16, each off by at most half a step (2^-11 relative).  A
    score is then off by at most E = scale * 2^-11 * sum_d |q_d k_d| (its largest over the row's visible keys), which
    changes every weight by a factor within e^(2E).  With A = sum_j p_j |v_j| the output is off by at most
    A (2 * 2^-11 + e^(2E) - 1), plus fp32 sums, exp2's approximation and the split's merge, given 2^-13 A."""
    s = np.where(see, scale * (q @ k.T), -np.inf)
    p = O.softmax_rows(s)
    E = scale * 2.0 ** -11 * np.where(see, np.abs(q) @ np.abs(k).T, 0.0).max(1, keepdims=True)
    A = p @ np.abs(v)
    return p @ v, A * (2.0 ** -10 + np.expm1(2 * E) + 2.0 ** -13) + 1e-7


def check(got, ref, bound, bf16, what=""):
    got = got.float().cpu().numpy().astype(np.float64)
    bound = bound + (2.0 ** -8 * (np.abs(ref) + bound) if bf16 else 0.0)     # half a step of the output type
    err = np.abs(got - ref)
    bad = ~(err <= bound)
    if bad.any():
        i = np.unravel_index(np.argmax(np.where(np.isnan(err), np.inf, err - bound)), err.shape)
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.size} off; worst at {i}: got {got[i]!r} ref {ref[i]!r} "
                             f"err {err[i]:.3e} bound {bound[i]:.3e}")


# ---------------------------------------------------------------- append and read-back

LAYOUTS = [
    # name, Hkv, D, bits, new, ctx, paged
    ("one_token_d64", 1, 64, "8", [1], [0], False),
    ("ragged_int8", 2, 128, "8", [5, 0, 64, 129], [3, 70, 0, 127], False),
    ("ragged_int4_pages", 3, 64, "4", [1, 33, 0, 65, 200], [63, 1, 0, 64, 7], True),
    ("mixed_pages", 4, 128, "8448", [17, 1, 90], [111, 255, 0], True),
    ("mixed_many", 2, 128, "48", [(i * 7) % 11 for i in range(70)], [(i * 13) % 40 for i in range(70)], False),
    ("empty_sequences", 2, 64, "8", [0, 0, 3, 0], [0, 5, 0, 0], True),
]


@pytest.mark.parametrize("case", LAYOUTS, ids=[c[0] for c in LAYOUTS])
def test_append_writes_the_oracles_codes_and_nothing_else(case):
    _, Hkv, D, bits, new, ctx, paged = case
    b = Batch(11, Hkv, Hkv, D, bits, new, ctx, paged, spare_cap=64)
    b.append_new()
    b.ok()
    for cache, planes, x in ((b.kc, b.kp, b.k), (b.vc, b.vp, b.v)):
        got, scale, zero = U.read_cache(cache, cache.Tcap)
        _, sc, zr, _ = U.oracle_quantize(x, b.bits)
        written = np.zeros((cache.B, cache.Tcap), bool)
        for s, (n, L) in enumerate(zip(b.new, b.lens)):
            for t in range(L - n, L):
                at = (b.table[s, t // 64], t % 64) if paged else (s, t)
                written[at] = True
                for h in range(Hkv):
                    assert np.array_equal(got[h][at], planes[h][s, t]), (s, t, h)
                    assert np.array_equal(scale[at[0], h, at[1]].view(np.uint16), sc[s, h, t].view(np.uint16))
                    assert np.array_equal(zero[at[0], h, at[1]].view(np.uint16), zr[s, h, t].view(np.uint16))
        for h in range(Hkv):
            assert (got[h][~written] == SENT_CODE).all()
        assert (scale.transpose(0, 2, 1, 3)[~written].view(np.uint16) == 0xFFFF).all()


@pytest.mark.parametrize("case", LAYOUTS, ids=[c[0] for c in LAYOUTS])
@pytest.mark.parametrize("f32", [False, True], ids=["bf16", "f32"])
def test_read_back_gives_the_stored_values(case, f32):
    kvq = _kvq()
    _, Hkv, D, bits, new, ctx, paged = case
    b = Batch(12, Hkv, Hkv, D, bits, new, ctx, paged)
    b.fill()
    b.append_new()
    dt = kvq.OUT_F32 if f32 else kvq.OUT_BF16
    extra = 9                                                # rows of the buffer that belong to no sequence
    for which, deq in (("k", b.kd), ("v", b.vd)):
        # the chunk, and then every sequence whole
        for start, lens, take in ((b.start, b.lens, b.new), (np.concatenate([[0], np.cumsum(b.lens)]), b.lens, b.lens)):
            rows = int(start[-1])
            out = torch.full((rows + extra, Hkv, D), 77.0, dtype=torch.float32 if f32 else torch.bfloat16,
                             device="cuda")
            b.read(which, torch.tensor(start, dtype=torch.int32, device="cuda"), b.d_lens, rows + extra, out=out,
                   out_dtype=dt)
            b.ok()
            ref = np.concatenate([deq[s, :, L - n:L].transpose(1, 0, 2) for s, (n, L) in enumerate(zip(take, lens))])
            ref = torch.from_numpy(ref).to(torch.float32)       # exact: 20 significant bits
            want = ref if f32 else ref.to(torch.bfloat16)
            assert torch.equal(out[:rows].cpu(), want)
            assert (out[rows:] == 77.0).all()


def test_append_takes_rows_of_a_fused_projection_in_place():
    b = Batch(13, 8, 2, 64, "84", [7, 20], [5, 90], False)
    b.fill()
    Hq, Hkv, D = 8, 2, 64
    fused = torch.full((b.rows, Hq + 2 * Hkv, D), float("nan"), dtype=torch.bfloat16, device="cuda")
    fused[:, Hq:Hq + Hkv] = U.to_dev_bf16(b.packed(b.k))
    fused[:, Hq + Hkv:] = U.to_dev_bf16(b.packed(b.v))
    b.append(fused[:, Hq:Hq + Hkv], fused[:, Hq + Hkv:], b.d_start, b.d_lens)
    got = b.read("v", b.d_start, b.d_lens, b.rows, out_dtype=_kvq().OUT_F32)
    b.ok()
    want = torch.from_numpy(np.concatenate([b.vd[s, :, L - n:L].transpose(1, 0, 2)
                                            for s, (n, L) in enumerate(zip(b.new, b.lens))])).float()
    assert torch.equal(got.cpu(), want)


def test_append_reports_non_finite_rows():
    b = Batch(14, 2, 2, 128, "8", [4], [0], False)
    k = U.to_dev_bf16(b.packed(b.k))
    k[2, 1, 77] = float("inf")
    b.append(k, U.to_dev_bf16(b.packed(b.v)), b.d_start, b.d_lens)
    torch.cuda.synchronize()
    assert int(b.status.item()) == 6


# ---------------------------------------------------------------- attention

ATTN = [
    # name, Hq, Hkv, D, bits, new, ctx, paged, window, sinks
    ("one_token", 1, 1, 64, "8", [1], [0], False, 0, 0),
    ("prompt_from_zero", 4, 2, 128, "8", [200, 3], [0, 0], False, 0, 0),
    ("verify_pages", 8, 2, 128, "48", [4, 4, 4], [508, 63, 61], True, 0, 0),
    ("ragged_mixed", 8, 4, 64, "8484", [1, 0, 130, 33], [300, 10, 77, 0], False, 0, 0),
    ("rep3", 6, 2, 128, "4", [87, 2], [170, 127], True, 0, 0),
    ("rep5_d64", 5, 1, 64, "8", [60, 1, 9], [1, 384, 130], False, 0, 0),
    ("rep8", 16, 2, 128, "84", [40, 8], [90, 1000], True, 0, 0),
    ("shared_by_all", 24, 1, 64, "4", [12, 1], [500, 127], False, 0, 0),
    ("window_one", 4, 2, 64, "8", [70, 1], [200, 64], False, 1, 0),
    ("window_one_sink", 4, 2, 128, "48", [5, 130], [300, 0], True, 1, 1),
    ("window_inside_a_tile", 8, 2, 128, "8", [33, 4, 1], [400, 127, 129], True, 20, 4),
    ("window_wider_than_all", 4, 4, 64, "4", [9, 65], [40, 10], False, 5000, 3),
    ("window_edges", 4, 1, 128, "8", [129, 64, 2], [383, 192, 510], False, 128, 64),
    ("sinks_past_the_window", 4, 2, 64, "84", [20, 3], [500, 100], True, 64, 300),
    ("sinks_beyond_the_end", 2, 1, 128, "4", [20, 3], [50, 0], False, 16, 4000),
    ("long", 4, 1, 128, "8", [5], [5000], True, 0, 0),
    ("long_window", 4, 1, 64, "4", [100], [5000], False, 700, 130),
    ("three_row_tiles", 8, 1, 128, "8", [70], [1000], False, 0, 0),
]


@pytest.mark.parametrize("case", ATTN, ids=[c[0] for c in ATTN])
@pytest.mark.parametrize("bf16", [False, True], ids=["f32", "bf16"])
def test_chunk_attention_against_the_definition(case, bf16):
    kvq = _kvq()
    name, Hq, Hkv, D, bits, new, ctx, paged, window, sinks = case
    b = Batch(21, Hq, Hkv, D, bits, new, ctx, paged, spare_cap=100)
    b.fill()
    b.append_new()
    ref, bound = b.reference(window, sinks)
    q = U.to_dev_bf16(b.q)
    ws = kvq.chunk_workspace(b.rows, b.B, Hq, Hkv, D)
    for max_chunk in (None, max(new)):
        out = torch.full((b.rows, Hq, D), float("nan"), dtype=torch.bfloat16 if bf16 else torch.float32, device="cuda")
        b.attend(q, window=window, sinks=sinks, out=out, out_dtype=kvq.OUT_BF16 if bf16 else kvq.OUT_F32, workspace=ws,
                 max_chunk=max_chunk)
        b.ok()
        check(out, ref, bound, bf16, name)
        again = b.attend(q, window=window, sinks=sinks, out_dtype=kvq.OUT_BF16 if bf16 else kvq.OUT_F32, workspace=ws,
                         max_chunk=max_chunk)
        b.ok()
        assert torch.equal(out, again)                        # the same bits on every call


def test_chunk_attention_takes_strided_queries_and_a_scale():
    b = Batch(22, 6, 2, 64, "8", [30, 1], [100, 7], False)
    b.fill()
    b.append_new()
    fused = torch.full((b.rows + 3, 10, 64), float("nan"), dtype=torch.bfloat16, device="cuda")
    fused[:b.rows, :6] = U.to_dev_bf16(b.q)
    got = b.attend(fused[:b.rows, :6], softmax_scale=0.3)
    b.ok()
    ref, bound = b.reference(scale=float(np.float32(0.3)))
    check(got, ref, bound, False)
    # heads outermost: [Hq][rows][D] seen as [rows][Hq][D]
    got2 = b.attend(U.to_dev_bf16(b.q.transpose(1, 0, 2).copy()).transpose(0, 1), softmax_scale=0.3)
    b.ok()
    assert torch.equal(got, got2)


def test_rows_of_no_sequence_are_left_as_they_are():
    b = Batch(23, 4, 2, 128, "8", [5, 140], [60, 20], False)
    b.fill()
    b.append_new()
    q = torch.zeros((b.rows + 70, 4, 128), dtype=torch.bfloat16, device="cuda")
    q[:b.rows] = U.to_dev_bf16(b.q)
    q[b.rows:] = float("nan")
    out = torch.full((b.rows + 70, 4, 128), 5.0, device="cuda")
    b.attend(q, out=out)
    b.ok()
    ref, bound = b.reference()
    check(out[:b.rows], ref, bound, False)
    assert (out[b.rows:] == 5.0).all()


def test_windows_do_not_touch_pages_that_nothing_sees():
    """Pages behind the window hold NaN scales and their table entries are garbage."""
    b = Batch(24, 8, 2, 128, "84", [40, 6], [1200, 900], True)
    b.fill()
    b.append_new()
    window, sinks = 150, 4
    for s, (n, L) in enumerate(zip(b.new, b.lens)):
        for page in range(1, (L - n - window + 1) // 64):
            for c in (b.kc, b.vc):
                c.sz.view(2, c.B, -1)[:, int(b.table[s, page])] = SENT_WORD
            b.bt[s, page] = -7 if page % 2 else 10 ** 6
    ref, bound = b.reference(window, sinks)
    check(b.attend(U.to_dev_bf16(b.q), window=window, sinks=sinks), ref, bound, False)
    b.ok()
    last = U.to_dev_bf16(b.q[b.start[1:] - 1])
    check(b.decode(last, window, sinks), ref[b.start[1:] - 1], bound[b.start[1:] - 1], False)
    b.ok()


DECODE = [
    # name, Hq, Hkv, D, bits, lens, paged, window, sinks
    ("all", 4, 2, 64, "8", [5, 0, 130], False, 0, 0),
    ("one", 8, 2, 128, "84", [300, 1, 64, 65], False, 1, 0),
    ("one_and_a_sink", 8, 1, 128, "8", [300, 1, 2, 129], True, 1, 1),
    ("inside_a_tile", 4, 4, 64, "4", [200, 17, 0, 64], True, 20, 3),
    ("tile_edges", 8, 2, 128, "48", [512, 576, 513, 511], False, 128, 64),
    ("sinks_past_the_window", 6, 2, 64, "8", [500, 100], True, 64, 300),
    ("wider_than_all", 4, 2, 128, "8", [300, 10], False, 10 ** 9, 10 ** 9),
    ("many_sequences", 4, 1, 128, "8", [(i * 37) % 400 for i in range(40)], True, 100, 4),
    ("long_split", 4, 1, 128, "8", [40000], False, 30000, 130),
]


@pytest.mark.parametrize("case", DECODE, ids=[c[0] for c in DECODE])
@pytest.mark.parametrize("bf16", [False, True], ids=["f32", "bf16"])
def test_windowed_decode_against_the_definition(case, bf16):
    kvq = _kvq()
    name, Hq, Hkv, D, bits, lens, paged, window, sinks = case
    new = [min(1, L) for L in lens]
    b = Batch(31, Hq, Hkv, D, bits, new, [L - n for L, n in zip(lens, new)], paged)
    b.fill()
    b.append_new()
    ref, bound = b.reference(window, sinks)
    q = np.zeros((b.B, Hq, D), np.uint16)
    full_ref, full_bound = np.zeros((b.B, Hq, D)), np.zeros((b.B, Hq, D))
    for s, n in enumerate(new):
        if n:
            q[s], full_ref[s], full_bound[s] = b.q[b.start[s]], ref[b.start[s]], bound[b.start[s]]
    ws = kvq.decode_workspace(b.B, Hq, Hkv, D)
    got = b.decode(U.to_dev_bf16(q), window, sinks, out_dtype=kvq.OUT_BF16 if bf16 else kvq.OUT_F32, workspace=ws)
    b.ok()
    check(got, full_ref, full_bound, bf16, name)
    for s, n in enumerate(new):
        if n == 0:
            assert (got[s] == 0).all()                       # an empty sequence: a zero row


def test_a_window_of_everything_gives_the_plain_decodes_bytes():
    kvq = _kvq()
    b = Batch(32, 8, 2, 128, "84", [1, 1, 1], [700, 63, 1300], False)
    b.fill()
    b.append_new()
    q = U.to_dev_bf16(b.q)
    plain = kvq.decode_attention(q, b.kc, b.vc, b.d_lens, status=b.status)
    for window, sinks in ((0, 0), (1301, 0), (5000, 7)):
        assert torch.equal(plain, b.decode(q, window, sinks))
    b.ok()


# ---------------------------------------------------------------- a serving loop

@pytest.mark.parametrize("paged", [False, True], ids=["contiguous", "pages"])
def test_a_prompt_in_chunks_then_drafts_then_single_tokens(paged):
    """Three sequences served together: prompt chunks of different sizes, a few verified drafts, single tokens, with
    one workspace throughout; every step against the definition, the final cache read back against the oracle."""
    kvq = _kvq()
    Hq, Hkv, D, window, sinks = 8, 2, 128, 200, 4
    final = [450, 131, 300]
    full = Batch(41, Hq, Hkv, D, "84", final, [0, 0, 0], paged)
    ws = kvq.chunk_workspace(600, 3, Hq, Hkv, D)
    wd = kvq.decode_workspace(3, Hq, Hkv, D)
    done = [0, 0, 0]
    rng = np.random.default_rng(5)
    for step, new in enumerate([(256, 0, 150), (130, 100, 146), (60, 27, 1), (3, 3, 2), (1, 1, 1)]):
        done = [d + n for d, n in zip(done, new)]
        start = torch.tensor(np.concatenate([[0], np.cumsum(new)]), dtype=torch.int32, device="cuda")
        lens = torch.tensor(done, dtype=torch.int32, device="cuda")
        rows = [np.concatenate([x[b, :, L - n:L].transpose(1, 0, 2) for b, (n, L) in enumerate(zip(new, done))])
                for x in (full.k, full.v)]
        q = W._draw_bf16(rng, (sum(new), Hq, D))
        full.append(U.to_dev_bf16(rows[0]), U.to_dev_bf16(rows[1]), start, lens)
        full.q, full.new, full.lens = q, list(new), list(done)
        full.start, full.d_start, full.d_lens, full.rows = start.cpu().numpy(), start, lens, sum(new)
        out = full.attend(U.to_dev_bf16(q), window=window, sinks=sinks, workspace=ws, max_chunk=max(new))
        full.ok()
        ref, bound = full.reference(window, sinks)
        check(out, ref, bound, False, f"step {step}")
        if new == (1, 1, 1):
            one = full.decode(U.to_dev_bf16(q), window, sinks, workspace=wd)
            full.ok()
            check(one, ref, bound, False, "decode")
    assert done == final
    whole = torch.tensor(np.concatenate([[0], np.cumsum(final)]), dtype=torch.int32, device="cuda")
    for which, deq in (("k", full.kd), ("v", full.vd)):
        got = full.read(which, whole, full.d_lens, sum(final), out_dtype=kvq.OUT_F32)
        full.ok()
        want = np.concatenate([deq[b, :, :L].transpose(1, 0, 2) for b, L in enumerate(final)])
        assert torch.equal(got.cpu(), torch.from_numpy(want).float())


def test_a_captured_step_replays_on_new_lengths():
    """append + attention captured once, replayed while the rows and lengths change in place."""
    kvq = _kvq()
    b = Batch(42, 8, 2, 128, "8", [4, 4], [100, 300], False, spare_cap=64)
    b.fill()
    start = b.d_start
    lens = b.d_lens.clone()
    k, v, q = (U.to_dev_bf16(x) for x in (b.packed(b.k), b.packed(b.v), b.q))
    ws = kvq.chunk_workspace(b.rows, b.B, 8, 2, 128)
    out = torch.zeros((b.rows, 8, 128), device="cuda")
    step = lambda: (kvq.append_chunk(k, v, b.kc, b.vc, start, lens, status=b.status),
                    kvq.chunk_attention(q, b.kc, b.vc, start, lens, out=out, workspace=ws, max_chunk=4,
                                        status=b.status))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
        side.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            step()
    torch.cuda.current_stream().wait_stream(side)
    ref, bound = b.reference()
    out.fill_(float("nan"))
    g.replay()
    b.ok()
    check(out, ref, bound, False)
    # the next step's tokens, four positions further
    rng = np.random.default_rng(3)
    nk, nv = (W._draw_bf16(rng, (b.rows, 2, 128)) for _ in "kv")
    k.copy_(U.to_dev_bf16(nk))
    v.copy_(U.to_dev_bf16(nv))
    lens += 4
    out.fill_(float("nan"))
    g.replay()
    b.ok()
    grow = lambda old, new: np.stack([np.concatenate([old[s, :, :L], new[4 * s:4 * s + 4].transpose(1, 0, 2),
                                                      old[s, :, L:]], 1)[:, :max(b.lens) + 4]
                                      for s, L in enumerate(b.lens)])
    b.k, b.v = grow(b.k, nk), grow(b.v, nv)
    b.kd, b.vd = U.oracle_quantize(b.k, b.bits)[3], U.oracle_quantize(b.v, b.bits)[3]
    b.lens = [L + 4 for L in b.lens]
    ref, bound = b.reference()
    check(out, ref, bound, False)


# ---------------------------------------------------------------- what the device refuses

def test_bad_descriptions_are_reported_and_left_out():
    """Sequence 1 of three is unusable in different ways: reported, its rows and positions untouched, the others
    served."""
    kvq = _kvq()
    for bad in ("longer_than_cap", "fewer_than_new", "negative", "too_many"):
        b = Batch(51, 4, 2, 64, "8", [6, 5, 7], [40, 30, 50], False)
        b.fill()
        b.append_new()
        b.ok()
        lens = list(b.lens)
        lens[1] = {"longer_than_cap": b.cap + 1, "fewer_than_new": 4, "negative": -3, "too_many": lens[1]}[bad]
        start = b.d_start
        max_chunk = None
        if bad == "too_many":
            max_chunk = 4
        b.d_lens = torch.tensor(lens, dtype=torch.int32, device="cuda")
        before = b.kc.codes.clone()
        if bad != "too_many":
            other = torch.randn((b.rows, 2, 64), device="cuda").to(torch.bfloat16)
            keep = b.packed(b.k)
            rows = U.to_dev_bf16(keep).clone()
            rows[6:11] = other[6:11]
            b.append(rows, U.to_dev_bf16(b.packed(b.v)), start, b.d_lens)
            torch.cuda.synchronize()
            assert int(b.status.item()) == 1
            assert torch.equal(b.kc.codes, before), bad
            b.status.zero_()
        out = torch.full((b.rows, 4, 64), 9.0, device="cuda")
        b.attend(U.to_dev_bf16(b.q), out=out, max_chunk=max_chunk)
        torch.cuda.synchronize()
        assert int(b.status.item()) == 1, bad
        ref, bound = b.reference()
        if bad == "too_many":                                # every sequence has more than four rows
            assert (out == 9.0).all()
            continue
        assert (out[6:11] == 9.0).all(), bad
        check(out[:6], ref[:6], bound[:6], False)
        check(out[11:], ref[11:], bound[11:], False)


def test_pages_outside_the_pool_are_reported():
    kvq = _kvq()
    b = Batch(52, 4, 2, 128, "84", [70, 3], [100, 30], True)
    b.fill()
    b.append_new()
    b.ok()
    good = b.bt.clone()
    b.bt[0, 2] = b.kc.B                                      # sequence 0, tokens 128 .. 169
    before = b.kc.codes.clone()
    b.append_new()
    torch.cuda.synchronize()
    assert int(b.status.item()) == 1
    assert torch.equal(b.kc.codes, before)                   # the others were written with the same rows again
    b.status.zero_()
    got = b.read("k", b.d_start, b.d_lens, b.rows, out_dtype=kvq.OUT_F32)
    torch.cuda.synchronize()
    assert int(b.status.item()) == 1
    want = torch.from_numpy(b.packed(b.kd)).float()
    assert torch.equal(got[:28].cpu(), want[:28]) and torch.equal(got[70:].cpu(), want[70:])
    assert (got[28:70] == 0).all()
    b.status.zero_()
    out = b.attend(U.to_dev_bf16(b.q))
    torch.cuda.synchronize()
    assert int(b.status.item()) == 1
    ref, bound = b.reference()
    check(out[70:], ref[70:], bound[70:], False)
    b.bt.copy_(good)
    b.status.zero_()
    check(b.attend(U.to_dev_bf16(b.q)), ref, bound, False)
    b.ok()


def test_non_finite_queries_are_reported():
    b = Batch(53, 4, 2, 128, "8", [5], [100], False)
    b.fill()
    b.append_new()
    q = U.to_dev_bf16(b.q)
    q[3, 1, 5] = float("inf")
    b.attend(q)
    torch.cuda.synchronize()
    assert int(b.status.item()) == 6


# ---------------------------------------------------------------- long walks: many tiles and pieces per CTA

WALKS = [
    # name, Hq, Hkv, D, bits, B, new range, ctx range, paged, window, sinks
    ("many_pieces", 16, 8, 64, "84848484", 24, (1, 230), (900, 2000), False, 0, 0),
    ("many_pieces_pages", 32, 8, 128, "88448844", 16, (1, 300), (500, 3000), True, 0, 0),
    ("windows_pages", 16, 4, 128, "4", 12, (100, 600), (2000, 9000), True, 900, 70),
    ("one_long_prompt", 8, 2, 128, "8", 1, (1500, 1500), (9000, 9000), False, 0, 0),
    ("few_rows_long", 8, 2, 128, "84", 3, (3, 9), (20000, 40000), True, 0, 0),
]


@pytest.mark.parametrize("case", WALKS, ids=[c[0] for c in WALKS])
def test_long_walks_against_the_definition_on_the_device(case):
    """Shapes whose CTAs walk tens of tiles over several segments; the reference is the definition in fp64 on the
    values that dequantize reads back (tested bit for bit above)."""
    kvq = _kvq()
    name, Hq, Hkv, D, bits, B, nr, cr, paged, window, sinks = case
    rng = np.random.default_rng(61)
    new = rng.integers(nr[0], nr[1] + 1, B)
    lens = new + rng.integers(cr[0], cr[1] + 1, B)
    cap = -(-int(lens.max()) // 64) * 64
    hb = np.array([int(b) for b in (bits if len(bits) == Hkv else bits * (Hkv // len(bits)))], np.int8)
    bt = None
    if paged:
        pages = cap // 64
        bt = torch.from_numpy(rng.permutation(B * pages + 3)[:B * pages].reshape(B, pages).astype(np.int32)).cuda()
        kc, vc = (kvq.empty_page_pool(hb, B * pages + 3, D) for _ in "kv")
    else:
        kc, vc = (kvq.empty_cache(hb, B, cap, D) for _ in "kv")
    for c in (kc, vc):
        c.codes.fill_(SENT_CODE)
        c.sz.fill_(SENT_WORD)
    gen = torch.Generator(device="cuda").manual_seed(62)
    dev = lambda a: torch.tensor(np.asarray(a), dtype=torch.int32, device="cuda")
    whole, d_lens = dev(np.concatenate([[0], np.cumsum(lens)])), dev(lens)
    start, rows = np.concatenate([[0], np.cumsum(new)]), int(new.sum())
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    total = int(lens.sum())
    k, v = (torch.randn((total, Hkv, D), generator=gen, device="cuda").bfloat16() for _ in "kv")
    q = torch.randn((rows, Hq, D), generator=gen, device="cuda").bfloat16()
    tab = () if bt is None else (bt,)
    sfx = "" if bt is None else "_paged"
    getattr(kvq, "append_chunk" + sfx)(k, v, kc, vc, *tab, whole, d_lens, status=status)
    read = getattr(kvq, "dequantize" + sfx)
    kd, vd = (read(c, *tab, whole, d_lens, total, out_dtype=kvq.OUT_F32, status=status) for c in (kc, vc))
    ws = kvq.chunk_workspace(rows, B, Hq, Hkv, D)
    attend = getattr(kvq, "chunk_attention" + sfx)
    out = None
    for _ in range(3):
        prev, out = out, attend(q, kc, vc, *tab, dev(start), d_lens, window=window, sinks=sinks, workspace=ws,
                                max_chunk=int(new.max()), status=status)
        torch.cuda.synchronize()
        assert int(status.item()) == 0
        assert prev is None or torch.equal(prev, out)
    off = np.concatenate([[0], np.cumsum(lens)])
    rep = Hq // Hkv
    worst = 0.0
    for b in range(B):
        n, L = int(new[b]), int(lens[b])
        pos = torch.arange(L - n, L, device="cuda")[:, None]
        j = torch.arange(L, device="cuda")[None]
        see = j <= pos
        if window:
            see &= (j > pos - window) | (j < sinks)
        for h in range(Hq):
            kk = kd[off[b]:off[b] + L, h // rep].double()
            vv = vd[off[b]:off[b] + L, h // rep].double()
            qq = q[start[b]:start[b] + n, h].double()
            s = (qq @ kk.T * D ** -0.5).masked_fill_(~see, float("-inf"))
            p = torch.softmax(s, 1)
            A = p @ vv.abs()
            E = D ** -0.5 * 2.0 ** -11 * (qq.abs() @ kk.abs().T).masked_fill_(~see, 0.0).amax(1, keepdim=True)
            bound = A * (2.0 ** -10 + torch.expm1(2 * E) + 2.0 ** -13) + 1e-7      # as attention_and_bound
            err = (out[start[b]:start[b] + n, h].double() - p @ vv).abs()
            worst = max(worst, float((err / bound).max()))
            assert torch.isfinite(err).all()
    assert worst <= 1.0, worst


# ---------------------------------------------------------------- limits, concurrency, the debug library

def test_positions_past_32_bits_of_a_long_cache():
    """One sequence of five million tokens (codes of over 5 GB per cache): its first tokens and its last ones, far
    beyond 2^32 bytes, written, read back and attended through a window with sinks."""
    kvq = _kvq()
    Hq, Hkv, D, L, n, window, sinks, keep = 16, 8, 128, 5_000_000, 5, 150, 4, 300
    cap = -(-L // 64) * 64
    kc, vc = (kvq.empty_cache([8] * Hkv, 1, cap, D) for _ in "kv")
    assert kc.codes.numel() > 2 ** 32
    rng = np.random.default_rng(71)
    k, v = (W._draw_bf16(rng, (1, Hkv, sinks + keep, D)) for _ in "kv")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    dev = lambda *a: torch.tensor(a, dtype=torch.int32, device="cuda")
    rows = [U.to_dev_bf16(np.ascontiguousarray(x[0].transpose(1, 0, 2))) for x in (k, v)]
    kvq.append_chunk(rows[0][:sinks], rows[1][:sinks], kc, vc, dev(0, sinks), dev(sinks), status=status)
    kvq.append_chunk(rows[0][sinks:], rows[1][sinks:], kc, vc, dev(0, keep), dev(L), status=status)
    kd, vd = (U.oracle_quantize(x, [8] * Hkv)[3][0] for x in (k, v))
    got = kvq.dequantize(vc, dev(0, keep), dev(L), keep, out_dtype=kvq.OUT_F32, status=status)
    torch.cuda.synchronize()
    assert torch.equal(got.cpu(), torch.from_numpy(vd[:, sinks:].transpose(1, 0, 2).copy()).float())
    q = W._draw_bf16(rng, (n, Hq, D))
    pos = np.arange(L - n, L)[:, None]
    tok = np.concatenate([np.arange(sinks), np.arange(L - keep, L)])[None]
    see = (tok <= pos) & ((tok > pos - window) | (tok < sinks))
    ref, bound = np.zeros((n, Hq, D)), np.zeros((n, Hq, D))
    for h in range(Hq):
        ref[:, h], bound[:, h] = attention_and_bound(O.bf16_to_f32(q[:, h]).astype(np.float64), kd[h // 2], vd[h // 2],
                                                     D ** -0.5, see)
    for max_chunk in (n, None if n * Hq // Hkv > 32 else 4000):          # both kernels
        out = kvq.chunk_attention(U.to_dev_bf16(q), kc, vc, dev(0, n), dev(L), window=window, sinks=sinks,
                                  max_chunk=max_chunk, status=status)
        torch.cuda.synchronize()
        assert int(status.item()) == 0
        check(out, ref, bound, False, str(max_chunk))
    one = kvq.decode_attention_window(U.to_dev_bf16(q[-1:]), kc, vc, dev(L), window, sinks, status=status)
    torch.cuda.synchronize()
    assert int(status.item()) == 0
    check(one, ref[-1:], bound[-1:], False, "decode")


@pytest.mark.parametrize("new,ctx,window", [(4, 2000, 0), (4, 4000, 0), (30, 2000, 0), (30, 3000, 1700), (70, 2500, 0)])
def test_segments_in_equal_parts(new, ctx, window):
    """Enough CTAs for two or three parts of each segment: ragged lengths, some sequences shorter than their parts,
    single-tile parts, windows; equal calls give equal bits."""
    kvq = _kvq()
    B, Hq, Hkv, D = 6, 16, 8, 64
    ctxs = [ctx, ctx - 300, 0, 100, ctx // 2, ctx - 1]
    b = Batch(74, Hq, Hkv, D, "84848484", [new, new - 1, new, 1, new, new], ctxs, True)
    b.fill()
    b.append_new()
    ref, bound = b.reference(window=window, sinks=3)
    q, ws = U.to_dev_bf16(b.q), kvq.chunk_workspace(b.rows, B, Hq, Hkv, D)
    outs = [b.attend(q, window=window, sinks=3, max_chunk=new, workspace=ws) for _ in range(3)]
    check(outs[0], ref, bound, False)
    assert torch.equal(outs[0], outs[1]) and torch.equal(outs[0], outs[2])
    b.ok()


@pytest.mark.parametrize("B", [2049, 4096])
def test_thousands_of_sequences(B):
    """More sequences than the kernel for few rows has room for, and as many as the calls take; every seventh has no
    new token."""
    kvq = _kvq()
    new = [0 if i % 7 == 3 else 1 + i % 2 for i in range(B)]
    b = Batch(72, 2, 1, 64, "8", new, [(5 * i) % 70 for i in range(B)], True)
    b.fill()
    b.append_new()
    ref, bound = b.reference(window=9, sinks=2)
    check(b.attend(U.to_dev_bf16(b.q), window=9, sinks=2, max_chunk=2), ref, bound, False)
    b.ok()


@pytest.mark.parametrize("new", [(0, 3), (17, 40), (90, 150)], ids=["narrow", "one_slot", "two_slots"])
@pytest.mark.parametrize("B", [1, 2, 9, 19, 38, 77])
def test_batches_of_short_segments(B, new):
    """Segments of one to four key tiles, from fewer than CTAs to several per CTA: ranges of the work list that begin
    or end anywhere in a segment, or hold no tile at all."""
    rng = np.random.default_rng(1000 * B + new[1])
    b = Batch(73, 4, 2, 64, "84", [int(x) for x in rng.integers(new[0], new[1] + 1, B)],
              [int(x) for x in rng.integers(0, 400, B)], B % 2 == 1)
    b.fill()
    b.append_new()
    ref, bound = b.reference(window=0, sinks=0)
    check(b.attend(U.to_dev_bf16(b.q), max_chunk=new[1]), ref, bound, False)
    b.ok()


def test_two_calls_at_once_on_two_streams():
    """Independent calls with workspaces of their own, overlapping: the bits of each call alone."""
    kvq = _kvq()
    bs = [Batch(80 + i, 8, 2, 128, "84", n, c, bool(i)) for i, (n, c) in
          enumerate([([150, 9, 60], [700, 1000, 300]), ([3, 4, 2], [1500, 40, 900])])]
    qs, wss, alone = [], [], []
    for b in bs:
        b.fill()
        b.append_new()
        qs.append(U.to_dev_bf16(b.q))
        wss.append(kvq.chunk_workspace(b.rows, b.B, 8, 2, 128))
        alone.append(b.attend(qs[-1], workspace=wss[-1], max_chunk=max(b.new)))
        b.ok()
    streams = [torch.cuda.Stream() for _ in bs]
    outs = [[torch.empty_like(a) for _ in range(6)] for a in alone]
    torch.cuda.synchronize()
    for r in range(6):
        for b, q, ws, s, o in zip(bs, qs, wss, streams, outs):
            b.attend(q, workspace=ws, max_chunk=max(b.new), stream=s, out=o[r])
    for b, a, o in zip(bs, alone, outs):
        b.ok()
        assert all(torch.equal(a, x) for x in o)


@pytest.mark.parametrize("op", ["narrow", "wide", "decode"])
def test_what_a_call_makes_for_itself_belongs_to_its_stream(op):
    """Without a workspace of the caller's, on another stream than the current one, which is busy: the workspace that
    the call makes is zeroed in the order of the call's stream, over memory that held something else before."""
    n = {"narrow": 4, "wide": 70, "decode": 1}[op]
    b = Batch(90, 8, 2, 128, "84", [n, n], [900, 3000], False)
    b.fill()
    b.append_new()
    q = U.to_dev_bf16(b.q if op != "decode" else b.q.reshape(2, 8, 128))
    call = (lambda **kw: b.decode(q, 0, 0, **kw)) if op == "decode" else (lambda **kw: b.attend(q, max_chunk=n, **kw))
    want = call()
    b.ok()
    side, busy = torch.cuda.Stream(), torch.randn((8192, 8192), device="cuda").bfloat16()
    for s in (torch.cuda.current_stream(), side):       # freed blocks full of ones, of both streams
        with torch.cuda.stream(s):
            junk = [torch.full((m,), 255, dtype=torch.uint8, device="cuda") for m in (1 << 27, 1 << 20, 1 << 16)]
            del junk
    torch.cuda.synchronize()
    for _ in range(20):
        busy @ busy
    got = call(stream=side)
    side.synchronize()
    assert torch.equal(got, want)
    b.ok()


def test_a_step_without_new_rows():
    """No sequence has a new token: empty tensors, nothing written, no error."""
    kvq = _kvq()
    b = Batch(92, 8, 2, 128, "84", [0, 0], [10, 70], False)
    b.fill()
    b.ok()
    before = [(c.codes.clone(), c.sz.clone()) for c in (b.kc, b.vc)]
    row = torch.empty((0, 2, 128), dtype=torch.bfloat16, device="cuda")
    b.append(row, row, b.d_start, b.d_lens)
    assert b.attend(torch.empty((0, 8, 128), dtype=torch.bfloat16, device="cuda")).shape == (0, 8, 128)
    assert b.read("k", b.d_start, b.d_lens, 0).shape == (0, 2, 128)
    b.ok()
    for c, (codes, sz) in zip((b.kc, b.vc), before):
        assert torch.equal(c.codes, codes) and torch.equal(c.sz, sz)


def test_workspaces_and_status_words_elsewhere_are_refused():
    kvq = _kvq()
    b = Batch(91, 8, 2, 128, "84", [4, 1], [10, 20], True)
    b.fill()
    b.append_new()
    q = U.to_dev_bf16(b.q)
    ws = kvq.chunk_workspace(b.rows, b.B, 8, 2, 128)
    cpu = torch.zeros(1, dtype=torch.int32)
    one = U.to_dev_bf16(b.q[:2])
    for bad in (dict(workspace=ws.cpu()), dict(workspace=ws[::2]), dict(status=cpu), dict(status=b.status.float())):
        with pytest.raises(kvq.KvqError):
            b.attend(q, **bad)
    for bad in (dict(workspace=ws.cpu()), dict(workspace=ws[::2])):
        with pytest.raises(kvq.KvqError):
            b.decode(one, 5, 1, **bad)
    with pytest.raises(kvq.KvqError):
        kvq.decode_attention_window_paged(one, b.kc, b.vc, b.bt, b.d_lens, 5, 1, status=cpu)
    with pytest.raises(kvq.KvqError):
        kvq.dequantize_paged(b.kc, b.bt, b.d_start, b.d_lens, b.rows, status=cpu)
    with pytest.raises(kvq.KvqError):
        kvq.append_chunk_paged(one[:, :2], one[:, :2], b.kc, b.vc, b.bt, b.d_start, b.d_lens, status=cpu)
    b.ok()


def test_one_workspace_for_calls_of_different_shapes():
    """Calls of different rows, heads and widths, ordered on a stream, share one workspace (it stays zeroed where it
    has to be)."""
    kvq = _kvq()
    shapes = [(8, 2, 128, [200, 30], [400, 90]), (4, 4, 64, [3, 1], [900, 700]), (16, 2, 128, [4, 2], [1300, 64])]
    bs = [Batch(90 + i, Hq, Hkv, D, "8", n, c, False) for i, (Hq, Hkv, D, n, c) in enumerate(shapes)]
    ws = torch.zeros(max(kvq.chunk_workspace_bytes(b.rows, b.B, b.Hq, b.Hkv, b.D) for b in bs), dtype=torch.uint8,
                     device="cuda")
    for b in bs:
        b.fill()
        b.append_new()
        b.ref = b.reference()
    for _ in range(3):
        for b in bs:
            check(b.attend(U.to_dev_bf16(b.q), workspace=ws, max_chunk=max(b.new)), *b.ref, False)
            b.ok()


@pytest.mark.parametrize("case", [a for a in ATTN if a[0] in ("ragged_mixed", "rep3", "window_edges", "long",
                                                              "sinks_past_the_window", "shared_by_all")],
                         ids=lambda c: c[0])
def test_debug_library_finds_no_index_out_of_range(case):
    """The same calls on the library built with index checks: no failed check, the same bytes."""
    import os
    kvq = _kvq()
    if not os.path.exists(kvq.DEBUG_LIB_PATH):
        from attention_group_quantized_gb300 import build
        build.build(debug=True)
    name, Hq, Hkv, D, bits, new, ctx, paged, window, sinks = case
    results = []
    old = kvq.LIB_PATH, kvq._LIB
    try:
        for path in (kvq.LIB_PATH, kvq.DEBUG_LIB_PATH):
            kvq.LIB_PATH, kvq._LIB = path, None
            b = Batch(95, Hq, Hkv, D, bits, new, ctx, paged)
            b.fill()
            b.append_new()
            q = U.to_dev_bf16(b.q)
            got = [b.attend(q, window=window, sinks=sinks, max_chunk=m) for m in (None, max(new))]
            got += [b.read(x, b.d_start, b.d_lens, b.rows) for x in "kv"]
            b.ok()
            results.append([x.cpu() for x in got])
    finally:
        kvq.LIB_PATH, kvq._LIB = old
    for x, y in zip(*results):
        assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))


def test_guard_bytes_around_outputs_and_workspace():
    """Nothing is written outside the output and the workspace."""
    kvq = _kvq()
    for new, max_chunk in (([3, 2], 3), ([90, 5], None)):
        b = Batch(96, 8, 2, 128, "84", new, [700, 100], True)
        b.fill()
        b.append_new()
        n_out, n_ws = b.rows * 8 * 128 * 4, kvq.chunk_workspace_bytes(b.rows, b.B, 8, 2, 128)
        bufs = [torch.full((512 + n,), 0x5A, dtype=torch.uint8, device="cuda") for n in (n_out, n_ws)]
        out = bufs[0][256:256 + n_out].view(torch.float32).view(b.rows, 8, 128)
        ws = bufs[1][256:256 + n_ws]
        ws.zero_()
        b.attend(U.to_dev_bf16(b.q), out=out, workspace=ws, max_chunk=max_chunk)
        b.ok()
        check(out, *b.reference(), False)
        for buf, n in zip(bufs, (n_out, n_ws)):
            assert (buf[:256] == 0x5A).all() and (buf[256 + n:] == 0x5A).all()
