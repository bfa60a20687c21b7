"""The rotated append, the block calls and the page calls at their limits: byte offsets past 2^31, sequences of a quarter of
a million blocks, thousands of rows, one workspace for calls of several shapes, other streams, and the debug build."""
import contextlib

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
    import os
    from attention_group_quantized_gb300 import kvq as K
    if not os.path.exists(K.DEBUG_LIB_PATH):
        from attention_group_quantized_gb300 import build
        build.build(debug=True)
    K.lib()
    return K


def _dev(a, dtype=np.int32):
    return torch.from_numpy(np.ascontiguousarray(np.asarray(a, dtype))).cuda()


def _status():
    return torch.zeros(1, dtype=torch.int32, device="cuda")


def test_a_sequence_whose_second_plane_starts_past_two_gigabytes(kvq):
    T, D, Hq, Hkv, bits = 2 ** 24 + 192, 128, 4, 2, [8, 8]
    rng = np.random.default_rng(1)
    k, v = kvq.empty_cache(bits, 1, T, D), kvq.empty_cache(bits, 1, T, D)
    for c in (k, v):
        c.sz.zero_()                                                # every other token is all zeros, scale 0
    n = 70
    lens, start = _dev([T]), _dev([0, n])
    st = _status()
    x = R.bf16_bits(rng.standard_normal((n, Hq + 2 * Hkv, D)).astype(np.float32))
    rows = U.to_dev_bf16(x)
    table = rng.uniform(-1, 1, (1, 16)).astype(np.float32)
    rotary = torch.from_numpy(table).cuda().expand(T, 16).contiguous()
    q = kvq.rotate_append(rows[:, :Hq], rows[:, Hq:Hq + Hkv], rows[:, Hq + Hkv:], k, v, start, lens, rotary=rotary, status=st)
    pos = np.zeros(n, int)
    want_q = R.turn(x[:, :Hq], None, table, pos, 1e-6, False)[0]
    kb = R.turn(x[:, Hq:Hq + Hkv], None, table, pos, 1e-6, False)[0].transpose(1, 0, 2)
    vb = x[:, Hq + Hkv:].transpose(1, 0, 2)
    assert int(st) == 0 and np.array_equal(q.cpu().view(torch.int16).numpy().view(np.uint16), want_q)
    kk, vv = R.stored(kb, bits), R.stored(vb, bits)
    for c, want in ((k, kk), (v, vv)):
        got = kvq.dequantize(c, start, lens, n, out_dtype=kvq.OUT_F32).cpu().numpy()
        assert np.array_equal(got.transpose(1, 0, 2).astype(np.float64), want)
    # a block in the middle whose keys are those of the last ones
    b = kvq.empty_bounds(k)
    middle = 2 ** 23 + 64 * 1001
    kvq.append_chunk(rows[:64, Hq:Hq + Hkv], rows[:64, Hq + Hkv:], k, v, _dev([0, 64]), _dev([middle + 64]))
    kvq.block_bounds(k, b, _dev([0, 64]), _dev([middle + 64]), 64, status=st)
    kvq.block_bounds(k, b, start, lens, n, status=st)
    blocks = T // 64
    km, vm = R.stored(x[:64, Hq:Hq + Hkv].transpose(1, 0, 2), bits), R.stored(x[:64, Hq + Hkv:].transpose(1, 0, 2), bits)
    # the last 70 tokens lie in the last two blocks, the first of which begins with 58 zero tokens
    tail = np.zeros((Hkv, 128, D))
    tail[:, 58:] = kk
    codes, scales = R.bounds(np.concatenate([km, tail], 1), 192)
    for i, at in enumerate((middle // 64, blocks - 2, blocks - 1)):
        assert np.array_equal(b.codes[:, at].cpu().numpy(), codes[:, i])
        assert np.array_equal(b.scales[:, at].cpu().numpy(), scales[:, i])
    one = q[-1:].contiguous()
    sel = kvq.select_blocks(one, k, b, lens, 6, first=1, last=1, status=st).cpu().numpy()
    score = R.scores(R.bf16_values(want_q[-1]), codes, scales)
    for h in range(Hkv):
        # the three blocks that have anything, then (with scores of 0) the lowest ones
        good = [i for i, s in zip((middle // 64, blocks - 2), score[h]) if s > 0]
        want = sorted([0, blocks - 1] + good + list(range(1, 5 - len(good))))
        assert sel[0, h].tolist() == want
    out = kvq.decode_attention_blocks(one, k, v, _dev([[[0, middle // 64, blocks - 2, blocks - 1]] * Hkv]), lens,
                                      status=st).cpu().numpy()
    assert int(st) == 0
    keys = np.concatenate([np.zeros((Hkv, 64, D)), km, tail], 1)
    vals = np.concatenate([np.zeros((Hkv, 64, D)), vm, np.concatenate([np.zeros((Hkv, 58, D)), vv], 1)], 1)
    ref = np.stack([R.attend(R.bf16_values(want_q[-1, h]).astype(np.float64), keys[h // 2], vals[h // 2], [0, 1, 2, 3], 256,
                             D ** -0.5) for h in range(Hq)])
    U.assert_close(out[0], ref)


def test_pages_past_two_gigabytes_are_copied(kvq):
    n = 2 ** 18 + 9
    k, v = (kvq.empty_page_pool([8], n, 128) for _ in range(2))
    for c in (k, v):
        c.codes.view(n, -1)[n - 2:] = torch.randint(0, 256, (2, 64 * 128), device="cuda", dtype=torch.uint8)
        c.sz.view(n, -1)[n - 2:] = torch.randint(0, 2 ** 30, (2, 64 * 4), device="cuda", dtype=torch.int32)
    kvq.copy_pages(k, v, _dev([n - 1, n - 2]), _dev([3, n - 5]))
    for c in (k, v):
        p, w = c.codes.view(n, -1), c.sz.view(n, -1)
        assert torch.equal(p[3], p[n - 1]) and torch.equal(p[n - 5], p[n - 2])
        assert torch.equal(w[3], w[n - 1]) and torch.equal(w[n - 5], w[n - 2])


def test_thousands_of_rows(kvq):
    """The most rows of a selection, over few sequences, D 64 with eight heads a KV head."""
    B, rows, Hkv, D, blocks = 3, 4096, 1, 64, 40
    rng = np.random.default_rng(3)
    k = kvq.empty_cache([4], B, blocks * 64, D)
    v = kvq.empty_cache([4], B, blocks * 64, D)
    x = R.bf16_bits(rng.standard_normal((2, B * blocks * 64, Hkv, D)).astype(np.float32))
    start, full = _dev(np.arange(B + 1) * blocks * 64), _dev([blocks * 64] * B)
    kvq.append_chunk(U.to_dev_bf16(x[0]), U.to_dev_bf16(x[1]), k, v, start, full)
    b = kvq.empty_bounds(k)
    kvq.block_bounds(k, b, start, full, B * blocks * 64)
    q = R.bf16_bits(rng.standard_normal((rows, 8, D)).astype(np.float32))
    seq, lens = rng.integers(0, B, rows), rng.integers(0, blocks * 64 + 1, rows)
    st = _status()
    sel = kvq.select_blocks(U.to_dev_bf16(q), k, b, _dev(lens), 5, row_seq=_dev(seq), status=st)
    out = kvq.decode_attention_blocks(U.to_dev_bf16(q), k, v, sel, _dev(lens), row_seq=_dev(seq), status=st)
    assert int(st) == 0
    codes, scales = b.codes.cpu().numpy(), b.scales.cpu().numpy()
    sel, out = sel.cpu().numpy(), out.cpu().numpy()
    stored = [[R.stored(x[i, s * blocks * 64:(s + 1) * blocks * 64].transpose(1, 0, 2), [4])[0] for i in range(2)]
              for s in range(B)]
    for r in range(0, rows, 97):
        m = -(-lens[r] // 64)
        at = slice(seq[r] * blocks, seq[r] * blocks + m)
        want = R.select(R.scores(R.bf16_values(q[r]), codes[:, at], scales[:, at])[0], 5, 1, 1) if m else np.full(5, -1)
        assert np.array_equal(sel[r, 0], want)
        ref = np.stack([R.attend(R.bf16_values(q[r, h]).astype(np.float64), *stored[seq[r]], want, lens[r], D ** -0.5)
                        for h in range(8)])
        U.assert_close(out[r], ref)


def test_one_workspace_for_selections_of_every_shape(kvq):
    rng = np.random.default_rng(4)
    ws = kvq.select_workspace(64, 4, 64 * 3000)
    for B, Hkv, blocks, n in ((1, 1, 3000, 40), (64, 4, 300, 8), (2, 2, 2500, 1000), (1, 1, 3000, 40), (16, 1, 700, 3)):
        k = kvq.empty_cache([4] * Hkv, B, blocks * 64, 64)
        b = kvq.empty_bounds(k)
        codes = rng.integers(-127, 128, tuple(b.codes.shape)).astype(np.int8)
        scales = rng.uniform(0, 1, tuple(b.scales.shape)).astype(np.float32)
        b.codes.copy_(_dev(codes, np.int8))
        b.scales.copy_(_dev(scales, np.float32))
        q = R.bf16_bits(rng.standard_normal((B, 2 * Hkv, 64)).astype(np.float32))
        lens = rng.integers(blocks * 32, blocks * 64 + 1, B)
        got = kvq.select_blocks(U.to_dev_bf16(q), k, b, _dev(lens), n, workspace=ws).cpu().numpy()
        for r in range(0, B, 7):
            at = slice(r * blocks, r * blocks - (-lens[r] // 64))
            score = R.scores(R.bf16_values(q[r]), codes[:, at], scales[:, at])
            for h in range(Hkv):
                assert np.array_equal(got[r, h], R.select(score[h], n, 1, 1))


def test_calls_on_another_stream(kvq):
    """Everything that a call makes for itself (outputs, workspaces) belongs to the stream that it runs on."""
    rng = np.random.default_rng(5)
    k, v = kvq.empty_page_pool([8, 4], 64, 64), kvq.empty_page_pool([8, 4], 64, 64)
    b = kvq.empty_bounds(k)
    pages = kvq.empty_page_table(64, 3, 20)
    x = U.to_dev_bf16(R.bf16_bits(rng.standard_normal((900, 8, 64)).astype(np.float32)))
    st = _status()

    def go(stream):
        for t in (pages.refs, pages.seq_lens):
            t.zero_()
        torch.cuda.synchronize()
        kvq.pages_reserve(pages, _dev([900, 0, 0]), status=st, stream=stream)
        start = _dev([0, 900, 900, 900])
        q = kvq.rotate_append_paged(x[:, :4], x[:, 4:6], x[:, 6:], k, v, pages.table, start, pages.seq_lens, status=st,
                                    stream=stream)
        kvq.block_bounds_paged(k, b, pages.table, start, pages.seq_lens, 900, status=st, stream=stream)
        kvq.pages_fork(pages, k, v, _dev([0]), _dev([2]), bounds=b, status=st, stream=stream)
        (stream or torch.cuda.current_stream()).synchronize()
        rows, lens = q[-2:].contiguous(), _dev([899, 900])
        sel = kvq.select_blocks_paged(rows, k, b, pages.table, lens, 4, row_seq=_dev([0, 2]), status=st, stream=stream)
        out = kvq.decode_attention_blocks_paged(rows, k, v, pages.table, sel, lens, row_seq=_dev([0, 2]), status=st,
                                                stream=stream)
        kvq.pages_free(pages, _dev([0]), status=st, stream=stream)
        kvq.pages_compact(pages, k, v, bounds=b, status=st, stream=stream)
        torch.cuda.synchronize()
        assert int(st) == 0
        return [t.clone() for t in (q, sel, out, pages.refs, pages.table[2, :15], pages.seq_lens)]

    for a, c in zip(go(None), go(torch.cuda.Stream())):
        assert torch.equal(a, c)


@contextlib.contextmanager
def _library(K, path):
    old_path, old_lib = K.LIB_PATH, K._LIB
    K.LIB_PATH, K._LIB = path, None
    try:
        K.lib()
        yield
    finally:
        K.LIB_PATH, K._LIB = old_path, old_lib


@pytest.mark.parametrize("D,Hq,Hkv,paged,rows", [(128, 8, 2, True, 700), (64, 3, 3, False, 90), (128, 16, 4, False, 1500)])
def test_the_debug_build_finds_no_index_out_of_range(kvq, D, Hq, Hkv, paged, rows):
    """The same kernels with every index checked: status 0 and the same bytes."""
    results = []
    for path in (kvq.LIB_PATH, kvq.DEBUG_LIB_PATH):
        with _library(kvq, path):
            gen = torch.Generator(device="cuda").manual_seed(1)
            bits = [8 if i % 2 else 4 for i in range(Hkv)]
            st = _status()
            x = torch.randn((rows + 3, Hq + 2 * Hkv, D), generator=gen, device="cuda").bfloat16()
            rotary = torch.rand((rows + 64, D), generator=gen, device="cuda")
            start, lens = _dev([0, rows, rows + 3]), _dev([rows, 3])
            most = -(-rows // 64) + 1
            if paged:
                k, v = (kvq.empty_page_pool(bits, 2 * most + 1, D) for _ in range(2))
                pages = kvq.empty_page_table(2 * most + 1, 3, most)
                kvq.pages_reserve(pages, _dev([rows, 3, 0]), status=st)
                table = pages.table[:2].contiguous()
            else:
                k, v = (kvq.empty_cache(bits, 2, most * 64, D) for _ in range(2))
            for c in (k, v):
                c.codes.zero_()
                c.sz.zero_()
            b = kvq.empty_bounds(k)
            args = (x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:], k, v)
            at = (table,) if paged else ()
            sfx = "_paged" if paged else ""
            q = getattr(kvq, "rotate_append" + sfx)(*args, *at, start, lens, rotary=rotary, status=st)
            getattr(kvq, "block_bounds" + sfx)(k, b, *at, start, lens, rows + 3, status=st)
            two = q[[rows - 1, rows + 2]].contiguous()
            sel = getattr(kvq, "select_blocks" + sfx)(two, k, b, *at, lens, 3, status=st)
            out = getattr(kvq, "decode_attention_blocks" + sfx)(two, k, v, *at, sel, lens, status=st)
            outs = [q, sel, out, b.codes, b.scales, k.codes, k.sz, v.codes, v.sz]
            if paged:
                kvq.pages_fork(pages, k, v, _dev([0]), _dev([2]), bounds=b, status=st)
                kvq.pages_free(pages, _dev([1]), status=st)
                kvq.pages_compact(pages, k, v, bounds=b, status=st)
                outs += [pages.refs, pages.seq_lens, pages.table]
            torch.cuda.synchronize()
            assert int(st) == 0
            results.append([t.clone() for t in outs])
    for a, c in zip(*results):
        assert torch.equal(a.view(torch.uint8), c.view(torch.uint8))


def test_two_graphs_of_different_shapes_share_a_workspace(kvq):
    """Captured selections that share a workspace, replayed in turn: each leaves it as the other needs it."""
    ws = kvq.select_workspace(8, 2, 64 * 3000)
    gen = torch.Generator(device="cuda").manual_seed(6)
    parts = []
    for B, Hkv, blocks, n in ((1, 2, 3000, 50), (8, 1, 900, 7)):
        k = kvq.empty_cache([4] * Hkv, B, blocks * 64, 128)
        b = kvq.empty_bounds(k)
        b.codes.copy_(torch.randint(-127, 128, b.codes.shape, generator=gen, device="cuda", dtype=torch.int8))
        b.scales.copy_(torch.rand(b.scales.shape, generator=gen, device="cuda"))
        q = torch.randn((B, 4 * Hkv, 128), generator=gen, device="cuda").bfloat16()
        lens = _dev([blocks * 64] * B)
        out = torch.empty((B, Hkv, n), dtype=torch.int32, device="cuda")
        want = kvq.select_blocks(q, k, b, lens, n)
        kvq.select_blocks(q, k, b, lens, n, out=out, workspace=ws)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            kvq.select_blocks(q, k, b, lens, n, out=out, workspace=ws)
        parts.append((graph, out, want, (k, b, q, lens)))
    for _ in range(3):
        for graph, out, want, _ in parts:
            out.fill_(-7)
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(out, want)


def test_strides_of_single_rows_and_heads_do_not_matter(kvq):
    """A stride that no index uses may be anything: one KV head, or one row, from tensors laid out differently."""
    gen = torch.Generator(device="cuda").manual_seed(8)
    for rows, Hkv in ((5, 1), (1, 2), (1, 1)):
        k, v = (kvq.empty_cache([8] * Hkv, 1, 64, 64) for _ in range(2))
        start, lens = _dev([0, rows]), _dev([rows])
        x = torch.randn((rows, 4 * Hkv, 64), generator=gen, device="cuda").bfloat16()
        q, kn, vn = x[:, :2 * Hkv], x[:, 2 * Hkv:3 * Hkv], x[:, 3 * Hkv:]
        if rows > 1:                                                # the same row stride, another head stride
            vn = vn.as_strided(vn.shape, (vn.stride(0), 3, 1), vn.storage_offset())
        else:
            vn = vn.as_strided(vn.shape, (7, vn.stride(1) if Hkv > 1 else 5, 1), vn.storage_offset())
        got = kvq.rotate_append(q, kn, vn, k, v, start, lens)
        assert torch.equal(got, q)
        k2, v2 = (kvq.empty_cache([8] * Hkv, 1, 64, 64) for _ in range(2))
        kvq.append_chunk(x[:, 2 * Hkv:3 * Hkv], x[:, 3 * Hkv:], k2, v2, start, lens)
        assert torch.equal(kvq.dequantize(v, start, lens, rows), kvq.dequantize(v2, start, lens, rows))
        assert torch.equal(kvq.dequantize(k, start, lens, rows), kvq.dequantize(k2, start, lens, rows))


@pytest.mark.parametrize("case", range(12))
def test_random_rotated_appends_against_the_append(kvq, case):
    """Without norm and rotation the call is the append; with them, the append of the turned keys: equal caches, byte for
    byte, over random shapes."""
    rng = np.random.default_rng(100 + case)
    B, D, Hkv = int(rng.integers(1, 9)), int(rng.choice([64, 128])), int(rng.choice([1, 2, 3, 5, 8]))
    Hq = Hkv * int(rng.choice([1, 2, 4, 7]))
    bits = [int(x) for x in rng.choice([4, 8], Hkv)]
    new = [int(x) for x in rng.integers(0, int(rng.choice([3, 40, 400])), B)]
    lens = [n + int(rng.integers(0, 200)) for n in new]
    T, cap = sum(new), -(-max(max(lens), 1) // 64) * 64
    x = R.bf16_bits(rng.standard_normal((T, Hq + 2 * Hkv, D)).astype(np.float32))
    rot = int(rng.choice([0, 16, D // 2, D]))
    inter, eps = bool(rng.random() < 0.5), 1e-5
    table = rng.uniform(-1, 1, (cap, rot)).astype(np.float32) if rot else None
    w = R.bf16_bits(rng.uniform(0.5, 2, D).astype(np.float32)) if rng.random() < 0.7 else None
    start = np.concatenate([[0], np.cumsum(new)])
    pos = np.concatenate([np.arange(L - n, L) for n, L in zip(new, lens)] or [[]]).astype(int)
    made = [[kvq.empty_cache(bits, B, cap, D) for _ in range(2)] for _ in range(2)]
    for pair in made:
        for c in pair:
            c.codes.fill_(1)
            c.sz.fill_(2)
    rows = U.to_dev_bf16(x)
    st = _status()
    dev_w = None if w is None else U.to_dev_bf16(w)
    q = kvq.rotate_append(rows[:, :Hq], rows[:, Hq:Hq + Hkv], rows[:, Hq + Hkv:], *made[0], _dev(start), _dev(lens),
                          rotary=None if table is None else _dev(table, np.float32), q_weight=dev_w, k_weight=dev_w,
                          eps=eps, interleaved=inter, status=st)
    if T:
        assert np.array_equal(q.cpu().view(torch.int16).numpy().view(np.uint16),
                              R.turn(x[:, :Hq], w, table, pos, eps, inter)[0])
        turned = U.to_dev_bf16(R.turn(x[:, Hq:Hq + Hkv], w, table, pos, eps, inter)[0])
        kv = torch.stack([turned, rows[:, Hq + Hkv:]])
        kvq.append_chunk(kv[0], kv[1], *made[1], _dev(start), _dev(lens), status=st)
    assert int(st) == 0
    for a, b in zip(*made):
        assert torch.equal(a.codes, b.codes) and torch.equal(a.sz, b.sz)
