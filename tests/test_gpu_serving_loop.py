"""The page calls, the rotated append, the bounds, the selection and the attention over it run together, as a serving loop
runs them: prompts, decode steps, forks, sequences that end, a compaction in between, on one pool, eagerly and with the
step captured into a graph.  Every step's selections are compared exactly and its outputs within the decode's tolerance
with what the definitions give for the tokens that each slot has seen."""
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


class Server:
    def __init__(self, kvq, seed, Hq, Hkv, D, bits, slots=6, n_pages=60, most=14, take=4):
        self.kvq, self.Hq, self.Hkv, self.D, self.bits, self.slots, self.take = kvq, Hq, Hkv, D, bits, slots, take
        self.rng = np.random.default_rng(seed)
        self.pages = kvq.empty_page_table(n_pages, slots, most)
        self.k, self.v = (kvq.empty_page_pool(bits, n_pages, D) for _ in range(2))
        self.bounds = kvq.empty_bounds(self.k)
        self.ws = kvq.pages_workspace(n_pages, slots)
        self.select_ws = kvq.select_workspace(slots, Hkv, 64 * most)
        self.decode_ws = kvq.decode_workspace(slots, Hq, Hkv, D)
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")
        angle = np.arange(64 * most)[:, None] * 10000.0 ** (-np.arange(0, D, 2) / D)
        self.table = np.concatenate([np.cos(angle), np.sin(angle)], 1).astype(np.float32)
        self.rotary = torch.from_numpy(self.table).cuda()
        self.w = [R.bf16_bits(1 + 0.3 * self.rng.standard_normal(D).astype(np.float32)) for _ in range(2)]
        self.weights = [U.to_dev_bf16(w) for w in self.w]
        self.seen = [[] for _ in range(slots)]                      # projected rows [Hq + 2 Hkv][D] of every token
        # the step's buffers: one row a slot, empty slots without one
        self.x = torch.zeros((slots, Hq + 2 * Hkv, D), dtype=torch.bfloat16, device="cuda")
        self.start = torch.zeros(slots + 1, dtype=torch.int32, device="cuda")
        self.add = torch.zeros(slots, dtype=torch.int32, device="cuda")
        self.row_seq = torch.zeros(slots, dtype=torch.int32, device="cuda")
        self.row_lens = torch.zeros(slots, dtype=torch.int32, device="cuda")

    def ints(self, a):
        return torch.tensor([int(v) for v in a], dtype=torch.int32, device="cuda")

    def fresh(self, n):
        x = self.rng.standard_normal((n, self.Hq + 2 * self.Hkv, self.D)).astype(np.float32)
        drift = self.rng.standard_normal((-(-n // 40), 1, self.D)).astype(np.float32)
        return R.bf16_bits(x + np.repeat(drift, 40, 0)[:n])

    def append(self, x, start):
        Hq, Hkv = self.Hq, self.Hkv
        q = self.kvq.rotate_append_paged(x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:], self.k, self.v, self.pages.table,
                                         start, self.pages.seq_lens, rotary=self.rotary, q_weight=self.weights[0],
                                         k_weight=self.weights[1], status=self.status)
        self.kvq.block_bounds_paged(self.k, self.bounds, self.pages.table, start, self.pages.seq_lens, x.shape[0],
                                    status=self.status)
        return q

    def prompts(self, lengths):
        x = self.fresh(sum(lengths))
        at = np.concatenate([[0], np.cumsum(lengths)])
        for s in range(self.slots):
            self.seen[s] += list(x[at[s]:at[s + 1]])
        self.kvq.pages_reserve(self.pages, self.ints(lengths), workspace=self.ws, status=self.status)
        self.append(U.to_dev_bf16(x), self.ints(at))

    def feed(self):
        """One token's projected rows for every slot that has a sequence, packed into the step's buffers."""
        live = [s for s in range(self.slots) if self.seen[s]]
        x = self.fresh(self.slots)
        for r, s in enumerate(live):
            self.seen[s].append(x[r])
        start = np.concatenate([[0], np.cumsum([1 if self.seen[s] else 0 for s in range(self.slots)])])
        self.x.copy_(U.to_dev_bf16(x))
        self.start.copy_(self.ints(start))
        self.add.copy_(self.ints([1 if self.seen[s] else 0 for s in range(self.slots)]))
        self.row_seq.copy_(self.ints(live + [0] * (self.slots - len(live))))
        self.row_lens.copy_(self.ints([len(self.seen[s]) for s in live] + [0] * (self.slots - len(live))))
        return live

    def step(self):
        k = self.kvq
        k.pages_reserve(self.pages, self.add, workspace=self.ws, status=self.status)
        q = self.append(self.x, self.start)
        sel = k.select_blocks_paged(q, self.k, self.bounds, self.pages.table, self.row_lens, self.take,
                                    row_seq=self.row_seq, workspace=self.select_ws, status=self.status)
        out = k.decode_attention_blocks_paged(q, self.k, self.v, self.pages.table, sel, self.row_lens,
                                              row_seq=self.row_seq, workspace=self.decode_ws, status=self.status)
        return q, sel, out

    def check(self, live, q, sel, out):
        assert int(self.status) == 0
        assert self.pages.seq_lens.tolist() == [len(t) for t in self.seen]
        got_q = q.cpu().view(torch.int16).numpy().view(np.uint16)
        Hq, Hkv, D = self.Hq, self.Hkv, self.D
        sel, out = sel.cpu().numpy(), out.cpu().numpy()
        for r, s in enumerate(live):
            x = np.stack(self.seen[s])
            n = len(x)
            pos = np.arange(n)
            want_q = R.turn(x[-1:, :Hq], self.w[0], self.table, pos[-1:], 1e-6, False)[0]
            assert np.array_equal(got_q[r], want_q[0])
            kb = R.turn(x[:, Hq:Hq + Hkv], self.w[1], self.table, pos, 1e-6, False)[0]
            kk = R.stored(kb.transpose(1, 0, 2), self.bits)
            vv = R.stored(x[:, Hq + Hkv:].transpose(1, 0, 2), self.bits)
            score = R.scores(R.bf16_values(want_q[0]), *R.bounds(kk, n))
            ref = np.zeros((Hq, D))
            for h in range(Hq):
                kh = h // (Hq // Hkv)
                best = R.select(score[kh], self.take, 1, 1)
                assert np.array_equal(sel[r, kh], best), (r, kh)
                ref[h] = R.attend(R.bf16_values(want_q[0, h]).astype(np.float64), kk[kh], vv[kh], best, n, D ** -0.5)
            U.assert_close(out[r], ref, f"slot {s}")
        assert (sel[len(live):] == -1).all() and not out[len(live):].any()

    def go(self):
        live = self.feed()
        self.check(live, *self.step())

    def fork(self, a, b):
        for f, t in zip(a, b):
            self.seen[t] = list(self.seen[f])
        self.kvq.pages_fork(self.pages, self.k, self.v, self.ints(a), self.ints(b), bounds=self.bounds, workspace=self.ws,
                            status=self.status)

    def free(self, slots):
        for s in slots:
            self.seen[s] = []
        self.kvq.pages_free(self.pages, self.ints(slots), status=self.status)

    def compact(self):
        self.kvq.pages_compact(self.pages, self.k, self.v, bounds=self.bounds, workspace=self.ws, status=self.status)
        live = self.pages.refs.count_nonzero()
        assert (self.pages.refs[:live] > 0).all()


MODELS = [(8, 2, 128, [8, 4]), (4, 4, 64, [8, 8, 4, 4]), (5, 1, 128, [4])]


@pytest.mark.parametrize("model", MODELS, ids=["gqa", "small_heads", "odd_group"])
def test_a_loop(kvq, model):
    s = Server(kvq, 1, *model)
    s.prompts([300, 0, 64, 0, 500, 0])
    s.go()
    s.fork([0, 4, 4], [1, 3, 5])
    s.go()                                                          # forks go on apart
    s.free([4, 2])
    s.go()
    s.compact()
    s.go()
    s.prompts([0, 0, 200, 0, 63, 0])                                # new ones in the pages that were let go
    for _ in range(3):
        s.go()                                                      # (one of them passes a page's end)
    s.prompts([30, 7, 0, 0, 0, 129])                                # and chunks onto sequences that have some
    s.go()


def test_the_step_in_a_graph(kvq):
    s = Server(kvq, 2, 8, 2, 128, [8, 4])
    s.prompts([62, 300, 0, 0, 0, 0])
    s.go()                                                          # (loads every kernel before the capture)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = s.step()
    for i in range(5):
        live = s.feed()
        graph.replay()
        s.check(live, *got)
        if i == 1:
            s.fork([1], [2])
        if i == 2:
            s.free([0])
            s.compact()
