"""Bounded waits of the chunk attention kernels on the GPU.

The policy's test-only issue limit makes every CTA withhold the queries of all pieces of its work but the first few,
so that the waits of every role run out; the kernels then end with nothing in flight and report it, and the next call on the same context,
with the workspace zero-filled again, gives the bits that it gave before.  No fault is provoked.
"""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

TIMEOUT = 5
# name, Hq, Hkv, D, bits, new tokens, tokens before them, pages, window
CASES = [
    ("narrow16", 8, 2, 128, "84", (4, 3, 4, 1), (20000, 9000, 30000, 15000), False, 0),
    ("narrow16_pages_d64", 4, 2, 64, "84", (5, 8, 2), (40000, 30000, 20000), True, 0),
    ("narrow32_pages", 8, 2, 128, "48", (7, 8, 5), (30000, 20000, 25000), True, 0),
    ("narrow32_d64", 8, 2, 64, "8", (8, 6), (50000, 60000), False, 20000),
    ("one_slot", 8, 2, 128, "8", (30, 20), (40000, 30000), False, 0),
    ("two_slots_pages", 8, 2, 128, "84", (300, 64, 200), (9000, 20000, 12000), True, 0),
    ("two_slots_d64", 4, 1, 64, "4", (900, 100), (20000, 30000), False, 6000),
    # more segments than CTAs, some of one tile: the waits run out after pieces that went through
    ("short_pieces", 8, 4, 64, "8", (3,) * 200, tuple(1 + 7 * i for i in range(200)), True, 0),
    ("short_pieces_narrow32", 16, 4, 128, "84", (7,) * 100, tuple(1 + 17 * i for i in range(100)), False, 0),
    ("short_pieces_one_slot", 8, 4, 128, "4", (40,) * 60, tuple(1 + 31 * i for i in range(60)), False, 0),
    ("short_pieces_two_slots", 8, 4, 64, "84", (120,) * 90, tuple(1 + 19 * i for i in range(90)), True, 300),
]


def _setup(case):
    from attention_group_quantized_gb300 import kvq
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    _, Hq, Hkv, D, bits, new, ctx, paged, window = case
    gen = torch.Generator(device="cuda").manual_seed(5)
    B, rows = len(new), sum(new)
    lens = [n + c for n, c in zip(new, ctx)]
    hb = np.array([int(b) for b in (bits * Hkv)[:Hkv]], np.int8)
    pages = -(-max(lens) // 64)
    mk = (lambda: kvq.empty_page_pool(hb, B * pages, D)) if paged else (lambda: kvq.empty_cache(hb, B, pages * 64, D))
    caches = [mk() for _ in "kv"]
    word = int(np.float16(0.02).view(np.uint16)) | int(np.float16(7).view(np.uint16)) << 16
    for c in caches:
        c.codes.random_(0, 256, generator=gen)
        c.sz.fill_(word)
    dev = lambda a: torch.tensor(a, dtype=torch.int32, device="cuda")
    start = dev([0] + np.cumsum(new).tolist())
    table = torch.randperm(B * pages, generator=gen, device="cuda").int().view(B, pages) if paged else None
    q = torch.randn((rows, Hq, D), generator=gen, device="cuda").bfloat16()
    ws = kvq.chunk_workspace(rows, B, Hq, Hkv, D)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")

    def call(policy=None):
        tab = () if table is None else (table,)
        f = kvq.chunk_attention if table is None else kvq.chunk_attention_paged
        out = f(q, *caches, *tab, start, dev(lens), window=window, sinks=3, workspace=ws, max_chunk=max(new),
                status=status, policy=policy)
        torch.cuda.synchronize()
        return out

    return kvq, call, ws, status


@pytest.mark.parametrize("case", CASES, ids=[c[0] for c in CASES])
def test_a_wait_that_runs_out_is_reported_and_the_context_stays_usable(case):
    kvq, call, ws, status = _setup(case)
    want = call()
    assert int(status.item()) == 0 and torch.isfinite(want).all()
    assert torch.equal(want, call(kvq.policy(wait_limit_us=500_000)))
    assert int(status.item()) == 0
    # the queries of so many pieces of a CTA's work are made ready; with more segments than that many per CTA, some CTA
    # has a piece whose queries are not
    segments = len(case[5]) * case[2]
    limits = [i for i in (0, 1, 2, 4) if i * torch.cuda.get_device_properties(0).multi_processor_count < segments]
    for limit in limits:
        call(kvq.policy(wait_limit_us=2000, test_issue_limit=limit))
        assert int(status.item()) == TIMEOUT, limit
        ws.zero_()
        status.zero_()
        assert torch.equal(want, call()), limit
        assert int(status.item()) == 0
