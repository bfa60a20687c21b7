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


# ---------------------------------------------------------------- rows that no usable sequence has, in a call's own output

BAD = {   # what the second of three sequences [6, 5, 7] on [40, 130, 50] tokens becomes: starts, its length, max_chunk
    "length_beyond_cap": ((0, 6, 11, 18), 10 ** 6, None),
    "fewer_than_new": ((0, 6, 11, 18), 4, None),
    "rows_past_the_buffer": ((0, 6, 11, 90), None, None),
    "max_chunk_too_small": ((0, 6, 11, 18), None, 5),
    "rows_before_the_first": ((2, 6, 11, 18), None, None),
    "fewer_rows_than_the_buffer": ((0, 6, 11, 13), None, None),
    "descending": ((0, 11, 6, 18), None, None),
    "no_rows": ((0, 0, 0, 0), None, None),
}


def _used_again(shape, dtype):
    """Memory that held something else is what the next call makes its output from."""
    torch.cuda.synchronize()
    junk = [torch.full(shape, float("nan"), dtype=dtype, device="cuda") for _ in range(3)]
    del junk


@pytest.mark.parametrize("bad", BAD)
@pytest.mark.parametrize("Hq,bf16", [(2, True), (4, False), (8, True), (128, False)], ids=str)
def test_rows_of_no_sequence_are_zeros_in_an_output_that_the_call_makes(bad, Hq, bf16):
    kvq = _kvq()
    start, length, max_chunk = BAD[bad]
    b = Batch(121, Hq, 2, 64, "84", [6, 5, 7], [40, 130, 50], Hq == 4)
    b.fill()
    b.append_new()
    b.ok()
    b.d_start = _ints(*start)
    if length is not None:
        b.d_lens = _ints(b.lens[0], length, b.lens[2])
    q, dt = U.to_dev_bf16(b.q), torch.bfloat16 if bf16 else torch.float32
    kw = dict(max_chunk=max_chunk, out_dtype=kvq.OUT_BF16 if bf16 else kvq.OUT_F32)
    kept = torch.full((18, Hq, 64), 7.0, dtype=dt, device="cuda")
    b.attend(q, out=kept, **kw)                              # the caller's output: those rows stay as they were
    free = (kept == 7.0).flatten(1).all(1)
    assert bad == "no_rows" or free.any()
    for status in (b.status, None):                          # whether or not anyone asks
        _used_again((18, Hq, 64), dt)
        got = b.attend(q, status=status, **kw)
        assert (got[free] == 0).all() and torch.equal(got[~free], kept[~free])
    rows = torch.full((18, 2, 64), 7.0, dtype=dt, device="cuda")
    b.read("k", b.d_start, b.d_lens, 18, out=rows, out_dtype=kw["out_dtype"])
    free = (rows == 7.0).flatten(1).all(1)
    _used_again((18, 2, 64), dt)
    got = b.read("k", b.d_start, b.d_lens, 18, out_dtype=kw["out_dtype"])
    assert (got[free] == 0).all() and torch.equal(got[~free], rows[~free])


def test_many_padding_rows_are_zeros_in_an_output_that_the_call_makes():
    """More rows than the CTAs take in one turn, few of them a sequence's, with both kernels and by the read-back."""
    kvq = _kvq()
    b = Batch(122, 8, 2, 128, "84", [3, 1], [500, 40], True)
    b.fill()
    b.append_new()
    ref, bound = b.reference()
    q = torch.zeros((9001, 8, 128), dtype=torch.bfloat16, device="cuda")
    q[:4] = U.to_dev_bf16(b.q)
    for max_chunk in (3, None):
        _used_again(q.shape, torch.float32)
        got = b.attend(q, max_chunk=max_chunk)
        b.ok()
        check(got[:4], ref, bound, False)
        assert (got[4:] == 0).all()
    _used_again((9001, 2, 128), torch.bfloat16)
    got = b.read("v", b.d_start, b.d_lens, 9001)
    b.ok()
    assert (got[4:] == 0).all() and (got[:4] != 0).any(2).all()


# ---------------------------------------------------------------- numbers of tokens beyond 32 bits

@pytest.mark.parametrize("kernel", KERNELS, ids=[k[0] for k in KERNELS])
def test_windows_wider_than_32_bits_hide_nothing(kernel):
    kvq = _kvq()
    _, Hq, n, _ = kernel
    b = Batch(131, Hq, 2, 128, "84", [n, n - 1], [700, 300], True)
    b.fill()
    b.append_new()
    q, last = U.to_dev_bf16(b.q), U.to_dev_bf16(b.q[b.start[1:] - 1])
    want, want_last = b.attend(q, max_chunk=n), b.decode(last, 0, 0)
    some = b.attend(q, max_chunk=n, window=9)
    for big in (2 ** 31 - 1, 2 ** 31, 2 ** 32, 2 ** 32 + 5, 2 ** 63 - 1, 2 ** 64 + 9):
        assert torch.equal(want, b.attend(q, max_chunk=n, window=big))
        assert torch.equal(want, b.attend(q, max_chunk=n, window=9, sinks=big))
        assert torch.equal(want, b.attend(q, max_chunk=big)) or n * Hq // 2 <= 32     # (the other kernel's bits)
        assert torch.equal(want_last, b.decode(last, big, 0)) and torch.equal(want_last, b.decode(last, 9, big))
    assert torch.equal(some, b.attend(q, max_chunk=n, window=9, sinks=0))
    for bad in (dict(window=-1), dict(window=-2 ** 32), dict(sinks=-2 ** 32 + 4), dict(max_chunk=-2 ** 32 + 9)):
        with pytest.raises(kvq.KvqError):
            b.attend(q, **{"max_chunk": n, **bad})
    with pytest.raises(kvq.KvqError):
        b.decode(last, -2 ** 32 + 7, 0)
    for rows in (-1, -2 ** 32 + 4, 2 ** 31, 2 ** 32 + 4):
        with pytest.raises(kvq.KvqError):
            b.read("k", b.d_start, b.d_lens, rows)
    b.ok()


def test_scale_words_elsewhere_are_refused():
    """A cache whose codes lie on the GPU and whose words do not never reaches a kernel."""
    kvq = _kvq()
    b = Batch(141, 4, 2, 64, "84", [3, 1], [60, 20], False)
    b.fill()
    b.append_new()
    q, rows = U.to_dev_bf16(b.q), U.to_dev_bf16(b.packed(b.k))
    split = lambda c: kvq.QuantCache(c.codes, c.sz.cpu(), c.head_bits, c.B, c.Hkv, c.Tcap, c.D)
    for k, v in ((split(b.kc), b.vc), (b.kc, split(b.vc))):
        for call in (lambda: kvq.append_chunk(rows, rows, k, v, b.d_start, b.d_lens),
                     lambda: kvq.chunk_attention(q, k, v, b.d_start, b.d_lens),
                     lambda: kvq.decode_attention_window(q[:2], k, v, b.d_lens, 5)):
            with pytest.raises(kvq.KvqError):
                call()
    with pytest.raises(kvq.KvqError):
        kvq.dequantize(split(b.kc), b.d_start, b.d_lens, 4)
    b.ok()


def test_large_scales_that_fit_are_taken():
    """Every group's scale large (values of up to 30000 either way in 8 bits, 60000 in 4): nothing is reported, and the
    outputs are right; words of unseen tokens hold a NaN."""
    for kernel in KERNELS:
        _, Hq, n, _ = kernel
        b = Batch(112, Hq, 2, 128, "84", [n, n - 1], [700, 300], True)
        rng = np.random.default_rng(7)
        top = np.array([3e4, 6e4], np.float32)[None, :, None, None]
        x = (rng.uniform(-1, 1, b.v.shape) * top).astype(np.float32)
        x[..., ::32] = np.where(rng.random(x[..., ::32].shape) < 0.5, -top, top)
        b.v = torch.from_numpy(x).bfloat16().view(torch.int16).numpy().view(np.uint16)
        b.vp, _, _, b.vd = U.oracle_quantize(b.v, b.bits)
        b.fill()
        b.append_new()
        ref, bound = b.reference()
        out = b.attend(U.to_dev_bf16(b.q), max_chunk=n)
        b.ok()
        check(out, ref, bound, False, kernel[0])


# ---------------------------------------------------------------- head layouts, shared pages

@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("rep", [1, 2, 3, 5, 7, 11, 16, 31, 32, 33, 64, 100, 127, 128])
def test_any_number_of_query_heads_per_kv_head(rep, D):
    new = [1, 32 // rep if rep <= 32 else 1, 0, max(1, 300 // rep)]           # rows of a KV head up to about 300
    b = Batch(151, rep, 1, D, "8" if rep % 2 else "4", new, [130, 400, 9, 70], rep % 3 == 0)
    b.fill()
    b.append_new()
    for window, sinks in ((0, 0), (50, 3)):
        ref, bound = b.reference(window, sinks)
        check(b.attend(U.to_dev_bf16(b.q), window=window, sinks=sinks, max_chunk=max(new)), ref, bound, False)
    if rep <= 32:                                                             # the kernel for few rows: single tokens
        one = Batch(152, rep, 1, D, "4" if rep % 2 else "8", [1, 1, 1], [0, 127, 700], rep % 3 == 1)
        one.fill()
        one.append_new()
        ref, bound = one.reference(90, 2)
        check(one.attend(U.to_dev_bf16(one.q), window=90, sinks=2, max_chunk=1), ref, bound, False)
        one.ok()
    b.ok()


@pytest.mark.parametrize("new", [(2, 1), (40, 3)], ids=["narrow", "wide"])
def test_sixty_four_kv_heads(new):
    kvq = _kvq()
    bits = "84" * 20 + "4488" * 6
    b = Batch(153, 128, 64, 64, bits, new, [300, 100], True)
    b.fill()
    b.append_new()
    ref, bound = b.reference()
    check(b.attend(U.to_dev_bf16(b.q), max_chunk=max(new)), ref, bound, False)
    got = b.read("v", b.d_start, b.d_lens, b.rows, out_dtype=kvq.OUT_F32)
    b.ok()
    assert torch.equal(got.cpu(), torch.from_numpy(b.packed(b.vd)).float())


@pytest.mark.parametrize("n", [3, 60], ids=["narrow", "wide"])
def test_sequences_that_share_the_pages_of_a_prefix(n):
    """Two sequences with one prefix of whole pages, stored once; each has tokens of its own behind it."""
    kvq = _kvq()
    b = Batch(154, 8, 2, 128, "84", [n, n], [448, 448], True)
    for x in (b.k, b.v):
        x[1, :, :384] = x[0, :, :384]
    for name in "kv":
        _, _, _, deq = U.oracle_quantize(getattr(b, name), b.bits)
        setattr(b, name + "d", deq)
    b.bt[1, :6] = b.bt[0, :6]
    whole = torch.tensor([0, 384], dtype=torch.int32, device="cuda")
    first = [U.to_dev_bf16(np.ascontiguousarray(x[0, :, :384].transpose(1, 0, 2))) for x in (b.k, b.v)]
    kvq.append_chunk_paged(*first, b.kc, b.vc, b.bt[:1].contiguous(), whole, _ints(384), status=b.status)
    tail = lambda x: U.to_dev_bf16(np.concatenate([x[s, :, 384:448 + n].transpose(1, 0, 2) for s in (0, 1)]))
    b.append(tail(b.k), tail(b.v), _ints(0, 64 + n, 128 + 2 * n), b.d_lens)
    ref, bound = b.reference()
    check(b.attend(U.to_dev_bf16(b.q), max_chunk=n), ref, bound, False)
    b.ok()
