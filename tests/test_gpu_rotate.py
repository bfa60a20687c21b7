"""The rotated append against its definition: queries, codes, scales and zero points bit for bit, and the queries against
the 64-bit formula.

The bound of the latter: a rounding to bf16 is off by at most 2^-8 of the value (half a step), and before it an fp32 value
passed at most seven roundings (mean, sum with eps, root, reciprocal, two products, one of rotation's) and the rotation's
sum, each 2^-24 of the terms, so 2^-21 of the terms' size covers them."""
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


def _table(positions, rot, rng):
    angle = np.arange(positions)[:, None] * 10000.0 ** (-np.arange(0, rot, 2) / rot) + rng.uniform(0, 0.1)
    return np.concatenate([np.cos(angle), np.sin(angle)], 1).astype(np.float32)


def _dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


class Case:
    def __init__(self, kvq, seed, new, ctx, Hq, Hkv, D, bits, rot, paged=False, interleaved=False, qw=True, kw=True,
                 pad=0, positions=None, scale=1.5, eps=1e-6):
        rng = np.random.default_rng(seed)
        self.kvq, self.D, self.Hq, self.Hkv, self.eps, self.interleaved = kvq, D, Hq, Hkv, eps, interleaved
        self.bits = {"8": [8] * Hkv, "4": [4] * Hkv}.get(bits) or [8 if i % 2 else 4 for i in range(Hkv)]
        self.new, self.lens = np.array(new), np.array(new) + np.array(ctx)
        self.start = np.concatenate([[0], np.cumsum(new)])
        T, B = int(self.start[-1]), len(new)
        cap = max(64, -(-int(self.lens.max()) // 64) * 64)
        self.cap, self.T, self.B = cap, T, B
        x = rng.standard_normal((T, (Hq + 2 * Hkv) * D + pad)).astype(np.float32) * scale
        self.x = R.bf16_bits(x)
        self.w = [R.bf16_bits(1 + 0.3 * rng.standard_normal(D).astype(np.float32)) if on else None for on in (qw, kw)]
        self.table = _table(positions or cap, rot, rng) if rot else None
        self.pages = None
        if paged:
            self.pages = rng.permutation(B * cap // 64 + 2)[:B * cap // 64].reshape(B, -1).astype(np.int32)
            self.caches = [kvq.empty_page_pool(self.bits, B * cap // 64 + 2, D) for _ in range(2)]
        else:
            self.caches = [kvq.empty_cache(self.bits, B, cap, D) for _ in range(2)]
        for c in self.caches:
            c.codes.fill_(0xA5)
            c.sz.fill_(0x5A5A5A5A)
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")

    def run(self, out=None, x=None, stream=None):
        k = self.kvq
        qkv = U.to_dev_bf16(self.x) if x is None else x
        self.held = qkv
        H = self.Hq + 2 * self.Hkv
        rows = qkv[:, :H * self.D].unflatten(1, (H, self.D))
        w = [None if a is None else U.to_dev_bf16(a) for a in self.w]
        args = [rows[:, :self.Hq], rows[:, self.Hq:self.Hq + self.Hkv], rows[:, self.Hq + self.Hkv:], *self.caches]
        more = dict(rotary=None if self.table is None else _dev(self.table), q_weight=w[0], k_weight=w[1], eps=self.eps,
                    interleaved=self.interleaved, out=out, status=self.status, stream=stream)
        start, lens = _dev(self.start.astype(np.int32)), _dev(self.lens.astype(np.int32))
        if self.pages is None:
            return k.rotate_append(*args, start, lens, **more)
        return k.rotate_append_paged(*args, _dev(self.pages), start, lens, **more)

    def expect(self):
        H, D = self.Hq + 2 * self.Hkv, self.D
        x = self.x[:, :H * D].reshape(self.T, H, D)
        pos = np.concatenate([np.arange(n - m, n) for m, n in zip(self.new, self.lens)]).astype(int)
        q = R.turn(x[:, :self.Hq], self.w[0], self.table, pos, self.eps, self.interleaved)
        k = R.turn(x[:, self.Hq:self.Hq + self.Hkv], self.w[1], self.table, pos, self.eps, self.interleaved)[0]
        return q, k, x[:, self.Hq + self.Hkv:], pos

    def check(self, out, skip=()):
        """Everything but the sequences in skip, which have to be untouched (queries: zeros)."""
        (qb, qz, size), k, v, pos = self.expect()
        got = out.cpu().view(torch.int16).numpy().view(np.uint16)
        live = np.ones(self.T, bool)
        for b in skip:
            live[self.start[b]:self.start[b + 1]] = False
        assert np.array_equal(got[live], qb[live])
        assert not got[~live].any()
        err = np.abs(R.bf16_values(got[live]).astype(np.float64) - qz[live])
        assert (err <= 2.0 ** -8 * np.abs(qz[live]) + 2.0 ** -21 * size[live]).all()
        for cache, rows in zip(self.caches, (k, v)):
            planes, scale, zero = U.read_cache(cache, cache.Tcap)
            want = U.oracle_quantize(np.ascontiguousarray(rows.transpose(1, 0, 2))[None], self.bits)
            done = np.zeros((cache.B, cache.Tcap), bool)
            for b in range(self.B):
                if b in skip:
                    continue
                for r in range(self.start[b], self.start[b + 1]):
                    at = (b, pos[r]) if self.pages is None else (self.pages[b, pos[r] // 64], pos[r] % 64)
                    done[at] = True
                    for h in range(self.Hkv):
                        assert np.array_equal(planes[h][at], want[0][h][0, r]), (b, r, h)
                        assert np.array_equal(scale[at[0], h, at[1]], want[1][0, h, r])
                        assert np.array_equal(zero[at[0], h, at[1]], want[2][0, h, r])
            for h in range(self.Hkv):                               # nothing else is written
                assert (planes[h][~done] == 0xA5).all()


CASES = [
    # new, ctx, Hq, Hkv, D, bits, rot, more
    ("token_small_heads", [1], [0], 4, 4, 64, "8", 64, {}),
    ("one_head", [5], [58], 1, 1, 128, "4", 128, {}),
    ("ragged_gqa_pages", [1, 130, 0, 7], [63, 0, 12, 200], 8, 2, 128, "mixed", 128, {"paged": True}),
    ("interleaved_part", [3, 64], [61, 0], 6, 3, 64, "mixed", 32, {"interleaved": True}),
    ("interleaved_whole", [33], [31], 5, 1, 128, "8", 128, {"interleaved": True, "paged": True}),
    ("turns_sixteen", [9, 2], [0, 64], 3, 1, 64, "4", 16, {}),
    ("half_split_part", [70], [5], 4, 2, 128, "4", 64, {}),
    ("three_quarters", [17], [5], 4, 2, 128, "8", 96, {}),
    ("no_norm", [20, 1], [3, 4], 4, 2, 128, "8", 128, {"qw": False, "kw": False}),
    ("norm_of_keys_only", [20, 1], [3, 4], 7, 1, 64, "mixed", 64, {"qw": False}),
    ("no_rotation", [20, 1], [3, 4], 4, 2, 128, "8", 0, {}),
    ("neither", [20, 1], [3, 4], 4, 2, 64, "4", 0, {"qw": False, "kw": False}),
    ("padded_rows", [19], [0], 4, 2, 128, "mixed", 128, {"pad": 24}),
    ("many_heads", [3], [100], 64, 64, 64, "mixed", 64, {}),
    ("long_enough_for_runs_of_heads", [700, 1, 900], [0, 64, 10], 8, 2, 128, "mixed", 128, {"paged": True}),
    ("long_small_heads", [2600], [3], 6, 3, 64, "mixed", 32, {"interleaved": True}),
    ("far_positions", [4], [100000], 2, 1, 64, "8", 64, {}),
    ("tiny_values", [40], [0], 2, 1, 128, "8", 128, {"scale": 1e-20}),
    ("huge_values", [40], [0], 2, 1, 128, "8", 128, {"scale": 1e25}),
]


@pytest.mark.parametrize("case", CASES, ids=[c[0] for c in CASES])
def test_rotate_append(kvq, case):
    name, new, ctx, Hq, Hkv, D, bits, rot, more = case
    if name == "huge_values":
        # squares pass fp32: the mean is infinite, the norm zero, and values stay out of the caches' fp16 range
        c = Case(kvq, 5, new, ctx, Hq, Hkv, D, bits, rot, **more)
        out = c.run()
        assert not out.float().any()
        assert int(c.status) == 6                                   # (V is not normed)
        return
    c = Case(kvq, len(name), new, ctx, Hq, Hkv, D, bits, rot, **more)
    out = c.run()
    assert int(c.status) == 0
    c.check(out)


@pytest.mark.parametrize("interleaved", [False, True])
def test_a_few_million_queries_bit_for_bit(kvq, interleaved):
    """A product fused into a sum, or a mean that is not the exact one rounded, changes about one bf16 value in 2^15."""
    c = Case(kvq, 12, [6000], [0], 4, 1, 128, "8", 128, interleaved=interleaved)
    out = c.run()
    want = c.expect()[0][0]
    assert np.array_equal(out.cpu().view(torch.int16).numpy().view(np.uint16), want)


def test_equal_calls_give_equal_bits_and_zero_rows_do_nothing(kvq):
    c = Case(kvq, 3, [50, 1], [4, 80], 8, 2, 128, "mixed", 128)
    a, b = c.run(), c.run()
    assert torch.equal(a, b)
    e = Case(kvq, 3, [0, 0], [4, 80], 8, 2, 128, "mixed", 128)
    assert e.run().shape == (0, 8, 128) and int(e.status) == 0


def test_in_place_queries_and_another_stream(kvq):
    c = Case(kvq, 4, [37, 2], [4, 80], 4, 2, 64, "8", 64)
    x = U.to_dev_bf16(c.x)
    q = x.view(c.T, 8, 64)[:, :4].contiguous()
    start, lens = _dev(c.start.astype(np.int32)), _dev(c.lens.astype(np.int32))
    rows = x.view(c.T, 8, 64)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = kvq.rotate_append(q, rows[:, 4:6], rows[:, 6:], *c.caches, start, lens, rotary=_dev(c.table),
                            q_weight=U.to_dev_bf16(c.w[0]), k_weight=U.to_dev_bf16(c.w[1]), out=q, status=c.status,
                            stream=side)
    side.synchronize()
    assert got is q
    c.check(got)


def test_unusable_sequences_are_left_out(kvq):
    c = Case(kvq, 6, [5, 6, 7], [10, 10, 10], 4, 2, 128, "8", 128)
    c.lens[1] = 3                                                   # shorter than its new tokens
    out = c.run()
    assert int(c.status) == 1
    c.lens[1] = 16                                                  # (positions of the others are as they were)
    c.check(out, skip=(1,))


def test_positions_past_the_table_are_left_out(kvq):
    c = Case(kvq, 7, [5, 6], [10, 120], 4, 2, 128, "8", 128, positions=126)
    c.table = np.concatenate([c.table, np.zeros((100, 128), np.float32)])   # (to state what the others give)
    full = c.table
    c.table = full[:120]
    out = c.run()
    assert int(c.status) == 1
    c.table = full
    c.check(out, skip=(1,))


def test_rows_of_no_sequence_and_given_outputs(kvq):
    c = Case(kvq, 8, [5, 6], [10, 20], 4, 2, 64, "8", 64)
    c.start[2] = 9                                                  # the last two rows belong to none
    c.new[1], c.lens[1] = 4, 24
    mark = torch.full((11, 4, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    out = c.run(out=mark)
    assert (out[9:] == 7.0).all() and int(c.status) == 0
    again = c.run()
    assert not again[9:].float().any() and torch.equal(again[:9], out[:9])


def test_a_page_outside_the_pool(kvq):
    c = Case(kvq, 9, [5, 6], [10, 20], 4, 2, 128, "8", 128, paged=True)
    good = c.pages.copy()
    c.pages[0, 0] = 10 ** 6
    out = c.run()
    assert int(c.status) == 1
    c.pages = good
    (qb, _, _), _, _, _ = c.expect()
    assert np.array_equal(out.cpu().view(torch.int16).numpy().view(np.uint16), qb)   # queries are computed all the same
    planes, _, _ = U.read_cache(c.caches[0], 64)
    assert (planes[0][good[0, 0]] == 0xA5).all() and (planes[0][good[1, 0], 20:26] != 0xA5).any()


@pytest.mark.parametrize("where,value", [("k", "nan"), ("k", "inf"), ("v", "nan"), ("v", "-inf")])
def test_non_finite_rows_are_reported(kvq, where, value):
    c = Case(kvq, 10, [5], [10], 4, 2, 64, "8", 64)
    c.x[3, (4 if where == "k" else 6) * 64 + 17] = R.bf16_bits(np.array([float(value.replace("nan", "inf"))], np.float32))[0] if value != "nan" else 0x7FC0
    c.run()
    assert int(c.status) == 6


def test_a_captured_call_replays(kvq):
    c = Case(kvq, 11, [9, 1], [10, 64], 8, 2, 128, "mixed", 128)
    x = U.to_dev_bf16(c.x)
    rows = x.view(c.T, 12, 128)
    start, lens = _dev(c.start.astype(np.int32)), _dev(c.lens.astype(np.int32))
    table, w = _dev(c.table), [U.to_dev_bf16(a) for a in c.w]
    out = torch.empty((c.T, 8, 128), dtype=torch.bfloat16, device="cuda")
    call = lambda: kvq.rotate_append(rows[:, :8], rows[:, 8:10], rows[:, 10:], *c.caches, start, lens, rotary=table,
                                     q_weight=w[0], k_weight=w[1], out=out, status=c.status)
    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    other = np.random.default_rng(1).standard_normal(c.x.shape).astype(np.float32)
    c.x = R.bf16_bits(other)
    x.copy_(U.to_dev_bf16(c.x))
    graph.replay()
    torch.cuda.synchronize()
    c.check(out)
