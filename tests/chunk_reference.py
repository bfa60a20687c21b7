"""The definition of windowed causal attention in 64 bits, and a bound per row whose sensitivity does not fall with the
context's length.

A worst-case bound (every rounding off by its most, all in one direction) stays as large as the values while the outputs
of L keys fall like 1 / sqrt(L): on long contexts it passes with tiles missing.  Here roundings count as what they are,
independent errors.  A rounding to fp16 is uniform within half a step, 2^-11 relative at most, so its standard deviation
is at most R = 2^-11 / sqrt(3).  With p the weights of a row, o its output:
  K_hat to fp16      moves score j by s_j = scale R sqrt(sum_d q_d^2 k_jd^2), the output by p_j s_j (v_j - o)
  P to fp16          the output by p_j R v_j; weights below fp16's normal range by 2^-25 of the largest one instead
  V_hat to fp16      channel d by p_j R v_jd
The variances add up over the keys and channels, and an error's norm passes SIGMAS of the resulting deviations for no row
of these tests (a chance of 1e-8 a row if it were normal; the largest single term, uniform, ends at sqrt(3)).  2^-16 of
the output's norm is for fp32 sums, exp2 and the merge.
"""
import torch

SIGMAS = 6.0
R = 2.0 ** -11 / 3 ** 0.5


def visible(n, L, window, sinks, device):
    """[n][L]: the tokens that the queries of the last n positions see."""
    pos = torch.arange(L - n, L, device=device)[:, None]
    j = torch.arange(L, device=device)[None]
    see = j <= pos
    return see & ((j > pos - window) | (j < sinks)) if window else see


def attention(q, k, v, scale, see):
    """Outputs [n][D] of q [n][D] over k, v [L][D] (64 bits), and the bound of each row's error norm."""
    q, k, v = q.double(), k.double(), v.double()
    s = (q @ k.T * scale).masked_fill_(~see, float("-inf"))
    p = torch.softmax(s, 1)
    o = p @ v
    moved = scale * R * ((q * q) @ (k * k).T).sqrt_()                          # K_hat
    weight = (p * R).square_() + (2.0 ** -25 * p.amax(1, keepdim=True)).square_() * see
    v2 = (v * v).sum(1)
    var = (p * moved).square() @ v2 + (p * moved).square().sum(1) * (o * o).sum(1)   # |v - o|^2 <= 2 (|v|^2 + |o|^2), halved
    var = 2 * var + weight @ v2 + (p * R).square() @ v2
    return o, SIGMAS * var.sqrt() + 2.0 ** -16 * o.norm(dim=1)


def worst(got, ref, bound):
    """The largest error norm over its bound; not finite counts as infinite."""
    e = (got.double() - ref).norm(dim=-1) / bound
    return float(torch.where(torch.isfinite(e), e, torch.full_like(e, float("inf"))).max())


def plant(k, q, rep, window, sinks, strength):
    """Keys that tell on a wrong edge, added to k [L][Hkv][D] for the queries q [n][Hq][D] of the last n positions (the
    first query head of each KV head): every query has aligned keys at its own position, the first that it may not see
    after it, the first and last ones on either side of its window and of the sinks."""
    n, L = q.shape[0], k.shape[0]
    D = q.shape[2]
    q0 = q[:, ::rep].to(k.dtype)
    a = q0 * (strength * D ** 0.5 / (q0 * q0).sum(2, keepdim=True))            # q . a / sqrt(D) = strength
    for i in range(n):
        pos = L - n + i
        at = {pos, pos + 1}
        if window:
            at |= {pos - window, pos - window + 1}
        for t in at:
            if 0 <= t < L:
                k[t] += a[i]
    if window and sinks:
        for t in (sinks - 1, sinks):
            if t < L:
                k[t] += a.sum(0)
    return k
