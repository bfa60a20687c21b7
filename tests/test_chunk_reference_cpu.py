"""The per-row bound of the long chunk tests tells a lost, doubled or misplaced tile and an edge off by one from
rounding, at every length (the mistakes are made in the reference, on the CPU)."""
import pytest

torch = pytest.importorskip("torch")

from tests.chunk_reference import attention, plant, visible, worst


def _data(n, L, D, window, sinks, planted, seed=3):
    gen = torch.Generator().manual_seed(seed)
    mk = lambda *s: torch.randn(s, generator=gen, dtype=torch.float64)
    q, k, v = mk(n, 1, D), mk(L, 1, D), mk(L, D)
    return q[:, 0], (plant(k, q, 1, window, sinks, 8.0) if planted else k)[:, 0], v


def _rounded(q, k, v, scale, see):
    """What a kernel computes: K, V and the weights in fp16, the weights against a maximum that lags behind by up to 2^8,
    sums of the weights before their rounding."""
    h = lambda x: x.half().double()
    s = (q @ h(k).T * scale).masked_fill(~see, float("-inf"))
    e = torch.exp(s - s.amax(1, keepdim=True))
    return (h(e) @ h(v)) / e.sum(1, keepdim=True)


CASES = [(5, 300, 64, 0, 0), (4, 30000, 128, 0, 0), (30, 40000, 64, 0, 0), (4, 30000, 64, 20000, 130), (8, 5000, 128, 700, 70)]


@pytest.mark.parametrize("n,L,D,window,sinks", CASES)
@pytest.mark.parametrize("planted", [False, True])
def test_the_bound_passes_rounding(n, L, D, window, sinks, planted):
    q, k, v = _data(n, L, D, window, sinks, planted)
    see = visible(n, L, window, sinks, "cpu")
    ref, bound = attention(q, k, v, D ** -0.5, see)
    assert worst(_rounded(q, k, v, D ** -0.5, see), ref, bound) < 1.0
    assert worst(torch.full_like(ref, float("nan")), ref, bound) == float("inf")


@pytest.mark.parametrize("n,L,D,window,sinks", CASES)
def test_the_bound_rejects_lost_doubled_and_misplaced_tiles(n, L, D, window, sinks):
    q, k, v = _data(n, L, D, window, sinks, False)
    scale = D ** -0.5
    see = visible(n, L, window, sinks, "cpu")
    ref, bound = attention(q, k, v, scale, see)
    rng = torch.arange(L)
    for t in ([0, (L - window // 2) // 128] if window else [0, (L // 128) // 2, (L - n) // 128 - 1]):
        inside = (rng >= 128 * t) & (rng < 128 * t + 128)
        lost, _ = attention(q, k, v, scale, see & ~inside)
        assert worst(lost, ref, bound) > 2.0, f"tile {t} lost"
        order = torch.cat([rng, rng[inside]])                                  # met twice
        doubled, _ = attention(q, k[order], v[order], scale, see[:, order])
        assert worst(doubled, ref, bound) > 2.0, f"tile {t} twice"
        page = (rng >= 128 * t) & (rng < 128 * t + 64)
        other = torch.where(page, (rng + 64) % L, rng)                         # another page's rows in a page's place
        wrong, _ = attention(q, k[other], v[other], scale, see)
        assert worst(wrong, ref, bound) > 2.0, f"page of tile {t} misplaced"


@pytest.mark.parametrize("n,L,D,window,sinks", CASES)
def test_planted_keys_make_it_reject_edges_off_by_one(n, L, D, window, sinks):
    q, k, v = _data(n, L, D, window, sinks, True)
    scale = D ** -0.5
    ref, bound = attention(q, k, v, scale, visible(n, L, window, sinks, "cpu"))
    pos, j = torch.arange(L - n, L)[:, None], torch.arange(L)[None]
    for off in (-1, 1):
        causal = (j <= pos + off) & (((j > pos - window) | (j < sinks)) if window else True)
        o, _ = attention(q, k, v, scale, causal)
        assert worst(o, ref, bound) > 2.0, f"causal edge off by {off}"
        if window:
            o, _ = attention(q, k, v, scale, (j <= pos) & ((j > pos - window + off) | (j < sinks)))
            assert worst(o, ref, bound) > 2.0, f"window off by {off}"
            o, _ = attention(q, k, v, scale, (j <= pos) & ((j > pos - window) | (j < sinks + off)))
            assert worst(o, ref, bound) > 2.0, f"sinks off by {off}"
