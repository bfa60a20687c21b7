"""The page calls against a model of them on lists: tables, counts, lengths, and every byte of the pools and bounds."""
import random

import numpy as np
import pytest

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


def _dev(a):
    return torch.tensor(a, dtype=torch.int32, device="cuda")


class Pool:
    def __init__(self, kvq, n_pages, slots, max_pages, Hkv=2, D=64, bits=None, bounds=True):
        self.kvq = kvq
        self.model = R.Pages(n_pages, slots, max_pages)
        self.pages = kvq.empty_page_table(n_pages, slots, max_pages)
        bits = bits or [8 if i % 2 else 4 for i in range(Hkv)]
        self.k, self.v = (kvq.empty_page_pool(bits, n_pages, D) for _ in range(2))
        self.bounds = kvq.empty_bounds(self.k) if bounds else None
        n = kvq.pages_workspace(n_pages, slots).numel()
        self.room = torch.full((n + 65536,), 0xEE, dtype=torch.uint8, device="cuda")   # no initial contents
        self.ws = self.room[:n]
        gen = torch.Generator(device="cuda").manual_seed(n_pages)
        for c in (self.k, self.v):
            c.codes.copy_(torch.randint(0, 256, c.codes.shape, generator=gen, device="cuda", dtype=torch.uint8))
            c.sz.copy_(torch.randint(-2 ** 31, 2 ** 31 - 1, c.sz.shape, generator=gen, device="cuda", dtype=torch.int32))
        if bounds:
            self.bounds.codes.copy_(torch.randint(-127, 128, self.bounds.codes.shape, generator=gen, device="cuda", dtype=torch.int8))
            self.bounds.scales.copy_(torch.rand(self.bounds.scales.shape, generator=gen, device="cuda"))
        self.first = [self.page_bytes(x) for x in self.buffers()]
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")

    def buffers(self):
        n = self.k.B
        out = []
        for c in (self.k, self.v):
            for h in range(c.Hkv):
                size = 64 * c.D * int(c.head_bits[h]) // 8
                off = c.head_offset(h)
                out.append(c.codes[off:off + n * size].view(n, size))
            out.append(c.sz.view(c.Hkv, n, -1).transpose(0, 1))
        if self.bounds is not None:
            out += [self.bounds.codes.transpose(0, 1), self.bounds.scales.transpose(0, 1)]
        return out

    @staticmethod
    def page_bytes(x):
        return x.reshape(x.shape[0], -1).cpu().clone()

    def check(self, want=()):
        m = self.model
        assert self.pages.refs.tolist() == m.refs
        assert self.pages.seq_lens.tolist() == m.lens
        assert self.pages.table.tolist() == m.table
        for x, first in zip(self.buffers(), self.first):
            assert torch.equal(self.page_bytes(x), first[m.data])
        assert (self.room[self.ws.numel():] == 0xEE).all()          # the calls keep to their workspace
        got = int(self.status)
        assert got in want if want else got == 0, (got, want)
        self.status.zero_()

    def reserve(self, add):
        self.kvq.pages_reserve(self.pages, _dev(add), workspace=self.ws, status=self.status)
        self.check(self.model.reserve(add))

    def fork(self, a, b):
        self.kvq.pages_fork(self.pages, self.k, self.v, _dev(a), _dev(b), bounds=self.bounds, workspace=self.ws,
                            status=self.status)
        self.check(self.model.fork(a, b))

    def free(self, slots):
        self.kvq.pages_free(self.pages, _dev(slots), status=self.status)
        self.check(self.model.free(slots))

    def compact(self):
        n = torch.zeros(1, dtype=torch.int32, device="cuda")
        self.kvq.pages_compact(self.pages, self.k, self.v, bounds=self.bounds, n_live=n, workspace=self.ws,
                               status=self.status)
        want = self.model.compact()
        assert int(n) == want
        self.check()


@pytest.mark.parametrize("D,bits", [(64, [8]), (64, [4]), (128, [8, 4, 4]), (128, [4]), (128, [8] * 8)])
def test_a_life(kvq, D, bits):
    p = Pool(kvq, 40, 8, 10, len(bits), D, bits)
    p.reserve([1, 64, 65, 0, 300, 0, 0, 0])
    p.reserve([0, 0, 0, 0, 0, 0, 0, 0])
    p.reserve([63, 1, 62, 0, 20, 0, 0, 0])
    p.fork([4, 1, 4], [3, 5, 6])                                    # a partly filled last page, a full one
    p.reserve([5, 5, 5, 5, 5, 5, 5, 0])
    p.free([4, 0])
    p.compact()
    p.compact()                                                     # nothing left to move
    p.reserve([640, 0, 0, 0, 100, 0, 0, 0])
    p.free([0, 1, 2, 3, 4, 5, 6, 7])
    p.compact()


def test_a_pool_that_runs_out(kvq):
    p = Pool(kvq, 7, 5, 7)
    p.reserve([130, 64, 0, 0, 0])                                   # 3 + 1 of 7
    p.reserve([0, 63, 300, 1, 1])                                   # slot 1 gets one, 2 none, and so 3 and 4
    p.reserve([3, 1, 64, 0, 0])                                     # no new page, no new page, one
    p.fork([0, 1, 0, 1], [3, 4, 3, 4])                              # a copy; a full one shares; the others' tos are taken
    p.free([2])
    p.fork([0], [2])
    p.free([3])
    p.fork([0, 4], [2, 3])


def test_refused_pairs_and_slots(kvq):
    p = Pool(kvq, 20, 6, 4)
    p.reserve([100, 70, 0, 0, 0, 0])
    p.fork([0, 0, -1, 6, 1, 1], [0, 1, 2, 2, -1, 6])                # onto used slots, from and to nowhere
    p.fork([0, 1, 0, 2], [3, 3, 3, 4])                              # the first of one to; an empty one stays empty
    p.free([3, 3, -1, 6, 5])                                        # twice, nowhere, an empty one
    p.reserve([-1, 300, 20, 0, 0, 2 ** 31 - 1])                     # negative, past the table's pages
    n = p.pages.seq_lens
    n[5] = 64 * 4 + 1                                               # a length that cannot be
    kvq.pages_reserve(p.pages, _dev([0, 0, 0, 0, 0, 0]), workspace=p.ws, status=p.status)
    kvq.pages_compact(p.pages, p.k, p.v, bounds=p.bounds, workspace=p.ws)
    assert int(p.status) == 1
    p.status.zero_()
    kvq.pages_free(p.pages, _dev([5]), status=p.status)
    assert int(p.status) == 1 and int(n[5]) == 0


def test_free_of_a_page_that_is_free_or_outside(kvq):
    p = Pool(kvq, 10, 3, 4)
    p.reserve([100, 70, 10])
    p.pages.table[1, 1] = 10 ** 6
    p.pages.refs[0] = 0                                             # slot 0's first page
    before = p.pages.refs.clone()
    kvq.pages_free(p.pages, _dev([0, 1]), status=p.status)
    assert int(p.status) == 1
    assert p.pages.refs.tolist() == [0, 0, 0, int(before[3])] + before[4:].tolist()


def test_copy_pages(kvq):
    p = Pool(kvq, 12, 1, 1, 3, 128)
    kvq.copy_pages(p.k, p.v, _dev([3, 3, -1, 5, 7]), _dev([0, 1, 2, -1, 7]), bounds=p.bounds, status=p.status)
    p.model.data[0] = p.model.data[1] = 3
    p.check()
    kvq.copy_pages(p.k, p.v, _dev([12, 4]), _dev([2, 2 ** 31 - 1]), bounds=p.bounds, status=p.status)
    assert int(p.status) == 1
    p.status.zero_()
    p.check()
    q = Pool(kvq, 12, 1, 1, 3, 64, bounds=False)
    kvq.copy_pages(q.k, q.v, _dev([11]), _dev([0]))
    q.model.data[0] = 11
    q.check()
    kvq.copy_pages(q.k, q.v, _dev([]), _dev([]))
    q.check()


@pytest.mark.parametrize("seed", range(6))
def test_random_lives(kvq, seed):
    rng = random.Random(seed)
    slots, most = rng.choice([3, 9, 40]), rng.choice([2, 6, 30])
    n = rng.choice([5, 30, 200, 1500])
    p = Pool(kvq, n, slots, most, rng.choice([1, 3]), rng.choice([64, 128]), bounds=rng.random() < 0.5)
    for _ in range(25):
        op = rng.random()
        if op < 0.45:
            p.reserve([rng.choice([0, 0, 1, rng.randint(0, 64 * most)]) for _ in range(slots)])
        elif op < 0.65:
            k = rng.randint(1, slots)
            p.fork([rng.randrange(slots) for _ in range(k)], [rng.randrange(slots) for _ in range(k)])
        elif op < 0.9:
            p.free([rng.randrange(slots) for _ in range(rng.randint(1, slots))])
        else:
            p.compact()


def test_a_large_pool(kvq):
    """More pages and slots than the planning CTA has threads, several for each."""
    p = Pool(kvq, 5000, 2500, 3, 1, 64, [4])
    rng = random.Random(1)
    p.reserve([rng.randint(0, 150) for _ in range(2500)])
    p.free(rng.sample(range(2500), 1500))
    empty = [s for s in range(2500) if p.model.lens[s] == 0]
    full = [s for s in range(2500) if p.model.lens[s]]
    p.fork([rng.choice(full) for _ in empty], empty)
    p.free(rng.sample(range(2500), 1200))
    p.compact()


def test_captured_fork_and_compaction_replay(kvq):
    p = Pool(kvq, 30, 6, 8)
    p.reserve([200, 0, 100, 0, 0, 0])
    p.free([0])
    p.reserve([0, 300, 0, 0, 0, 0])
    a, b, gone = _dev([1, 2]), _dev([3, 4]), _dev([3, 4])
    def step():
        kvq.pages_free(p.pages, gone, status=p.status)
        kvq.pages_fork(p.pages, p.k, p.v, a, b, bounds=p.bounds, workspace=p.ws, status=p.status)
        kvq.pages_compact(p.pages, p.k, p.v, bounds=p.bounds, workspace=p.ws, status=p.status)
    def model():
        p.model.free([3, 4])
        p.model.fork([1, 2], [3, 4])
        p.model.compact()
    step()
    model()
    torch.cuda.synchronize()
    p.check()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for _ in range(3):
        g.replay()
        torch.cuda.synchronize()
        model()
        p.check()
