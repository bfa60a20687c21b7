"""More operators of a serving step over the group-quantised KV cache, as a user's program calls them, with plain forms.

A case names one operator and the sizes of one call:

  rotate    the fused projection's rows of a ragged batch: queries and keys normed per head (root mean square, weights)
            and rotated by their positions, queries returned, keys and values quantised into the caches, and the written
            rows read back as values
  bounds    per 64-token block of the keys that new tokens touch: the channels' least and greatest stored values, held in
            8 bits, returned as the values that they stand for
  blocks    for every query row: the blocks of its sequence that a score from those bounds selects, and attention over them
  fork      sequences of a page pool let go, forked again (full pages shared, the last one copied) and given room for new
            tokens
  compact   a pool's live pages moved together into its first ones, tables and counts with them

New rows are packed: sequence b's are rows start[b] .. start[b + 1] - 1 and sit at cache positions
lens[b] - (start[b + 1] - start[b]) .. lens[b] - 1.  Caches hold 8- or 4-bit codes per KV head with an fp16 scale and
zero point per 32 channels, contiguous per sequence or in 64-token pages behind a block table.

Rotated keys are rounded to bf16 before they are quantised, as a projection's output would be.  What is rounded to whole
numbers is computed in 32 bits, one rounding per operation; the mean of squares is the exact one, rounded once.
"""
import functools
import math
import random

import torch

own = False

GROUP, PAGE = 32, 64
EPS = 1e-6


# ---------------------------------------------------------------- cases

def _rotate(B, Hq, Hkv, D, bits, ctx, new, paged, rot, norm=True, interleaved=False):
    return {"op": "rotate", "B": B, "Hq": Hq, "Hkv": Hkv, "D": D, "bits": bits, "ctx_lo": ctx[0], "ctx_hi": ctx[1],
            "new_lo": new[0], "new_hi": new[1], "paged": paged, "rot": rot, "norm": norm, "interleaved": interleaved}


def _bounds(B, Hkv, D, bits, ctx, new, paged):
    return {"op": "bounds", "B": B, "Hq": Hkv, "Hkv": Hkv, "D": D, "bits": bits, "ctx_lo": ctx[0], "ctx_hi": ctx[1],
            "new_lo": new[0], "new_hi": new[1], "paged": paged}


def _blocks(B, Hq, Hkv, D, bits, ctx, new, paged, take, first=1, last=1):
    return {"op": "blocks", "B": B, "Hq": Hq, "Hkv": Hkv, "D": D, "bits": bits, "ctx_lo": ctx[0], "ctx_hi": ctx[1],
            "new_lo": new, "new_hi": new, "paged": paged, "take": take, "first": first, "last": last}


def _fork(B, Hkv, D, bits, ctx, children, room, bounds):
    return {"op": "fork", "B": B, "Hkv": Hkv, "D": D, "bits": bits, "ctx_lo": ctx[0], "ctx_hi": ctx[1],
            "children": children, "room": room, "bounds": bounds}


def _compact(pages, Hkv, D, bits, live, length, bounds):
    return {"op": "compact", "pages": pages, "Hkv": Hkv, "D": D, "bits": bits, "live": live, "length": length,
            "bounds": bounds}


def listed():
    return [
        # the next token of one short conversation, small heads: latency
        dict(_rotate(1, 4, 4, 64, "8", (500, 500), (1, 1), False, 64), name="rotate_token"),
        # a scheduler's step: sequences with one new token next to prompt chunks, pages, INT8 and INT4 heads
        dict(_rotate(16, 32, 8, 128, "mixed", (1000, 8000), (1, 512), True, 128), name="rotate_mixed_pages"),
        # a whole 32K prompt into an INT4 cache, half of each head's channels rotated, pairs side by side
        dict(_rotate(1, 32, 8, 128, "4", (0, 0), (32768, 32768), False, 64, True, True), name="rotate_prompt_int4"),
        # one new token for each of sixteen sequences in pages: the last block of each
        dict(_bounds(16, 8, 128, "mixed", (1000, 8000), (1, 1), True), name="bounds_tokens_pages"),
        # four prompts of about 32K
        dict(_bounds(4, 8, 128, "8", (0, 0), (30001, 32768), False), name="bounds_prompts"),
        # half a thousand tokens, four blocks of eight, one sequence: latency
        dict(_blocks(1, 4, 4, 64, "8", (499, 499), 1, False, 4), name="blocks_tiny"),
        # eight sequences of 32K, 2048 tokens of each seen
        dict(_blocks(8, 32, 8, 128, "8", (32000, 32767), 1, False, 32), name="blocks_32k"),
        # four long INT4 sequences in pages, 4096 tokens of each seen
        dict(_blocks(4, 32, 8, 128, "4", (43000, 115000), 1, True, 64, 1, 2), name="blocks_long_int4"),
        # four drafted tokens verified for each of eight sequences of about 8K
        dict(_blocks(8, 32, 8, 128, "mixed", (7900, 8188), 4, True, 16, 1, 1), name="blocks_drafts"),
        # one short conversation continued twice: latency
        dict(_fork(1, 4, 64, "8", (500, 500), 2, 1, False), name="fork_two"),
        # four samples of each of thirty-two prompts
        dict(_fork(32, 8, 128, "mixed", (500, 8000), 4, 70, True), name="fork_samples"),
        # a pool half of whose 8192 pages were let go here and there
        dict(_compact(8192, 8, 128, "8", 0.5, 4000, True), name="compact_half"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rotate", "rotate", "bounds", "blocks", "blocks", "blocks", "fork", "compact"])
    D = rng.choice([64, 128, 128])
    Hkv = rng.choice([1, 2, 4, 8])
    rep = rng.choice([1, 2, 3, 4, 4, 5, 8])
    bits = rng.choice(["8", "4", "mixed"])
    paged = rng.random() < 0.5
    B = _log(rng, 1, 32)
    if op in ("rotate", "bounds"):
        hi = _log(rng, 1, 24000 // B)
        ctx, new = (0, _log(rng, 1, 4000)), (rng.randint(1, hi), hi)
        if op == "bounds":
            return _bounds(B, Hkv, D, bits, ctx, new, paged)
        if rep * Hkv > 32:
            rep = 4
        return _rotate(B, Hkv * rep, Hkv, D, bits, ctx, new, paged, rng.choice([0, D // 4, D // 2, D, D, D]),
                       rng.random() < 0.8, rng.random() < 0.4)
    if op == "blocks":
        hi = _log(rng, 16, 100000 if B <= 4 else 32000 if B <= 8 else 8000)
        first, last = rng.choice([0, 1, 1, 2]), rng.choice([1, 1, 2, 5])
        return _blocks(B, Hkv * rep, Hkv, D, bits, (rng.randint(0, hi), hi), rng.choice([1, 1, 1, 2, 5]), paged,
                       max(_log(rng, 1, 64), first + last), first, last)
    if op == "fork":
        return _fork(B, Hkv, D, bits, (0, _log(rng, 1, 8000)), rng.randint(1, 4), _log(rng, 1, 200), rng.random() < 0.5)
    return _compact(_log(rng, 64, 8000), Hkv, D, bits, rng.choice([0.1, 0.3, 0.5, 0.7, 0.9, 0.98]), _log(rng, 1, 8000),
                    rng.random() < 0.5)


def _key(c):
    return "|".join("%s=%s" % (k, c[k]) for k in sorted(c) if k != "name")


def _lengths(c):
    """(new tokens, cached length including them) of each sequence: fixed by the case."""
    rng = random.Random(_key(c))
    new = [_log(rng, c["new_lo"], c["new_hi"]) for _ in range(c["B"])]
    return new, [n + rng.randint(c["ctx_lo"], c["ctx_hi"]) for n in new]


def _head_bits(c):
    if c["bits"] != "mixed":
        return [int(c["bits"])] * c["Hkv"]
    rng = random.Random("bits %d %d" % (c["Hkv"], c["D"]))
    return [8 if rng.random() < 0.5 else 4 for _ in range(c["Hkv"])]


def _fork_sizes(c):
    rng = random.Random(_key(c))
    lens = [rng.randint(c["ctx_lo"], c["ctx_hi"]) for _ in range(c["B"])]
    slots = c["B"] * (1 + c["children"])
    most = -(-(max(lens) + c["room"]) // PAGE)
    need = sum(-(-x // PAGE) for x in lens) + sum(c["children"] * (-(-(x + c["room"]) // PAGE) - x // PAGE) for x in lens)
    return lens, slots, max(most, 1), need + 5


def _compact_lens(c):
    """Lengths of the sequences that hold the live pages, the last one cut."""
    rng = random.Random(_key(c))
    left, lens = int(c["pages"] * c["live"]), []
    while left:
        x = max(1, min(rng.randint(c["length"] // 2, c["length"]), left * PAGE))
        lens.append(x)
        left -= -(-x // PAGE)
    return lens or [1]


def _compact_places(c):
    """Pages of the pool that are live, as places in the order in which sequences have them."""
    rng = random.Random(_key(c) + "|places")
    used = sum(-(-x // PAGE) for x in _compact_lens(c))
    return rng.sample(range(c["pages"]), used)


def work(c):
    D, bits = c["D"], _head_bits(c)
    row = sum(D * b // 8 + 4 * (D // GROUP) for b in bits)          # one token's codes and scale words, all KV heads
    block = c["Hkv"] * (2 * D + 4 * (D // GROUP))                   # one block's bounds, all KV heads
    page = 2 * PAGE * row + (block if c.get("bounds") else 0)
    if c["op"] == "fork":
        lens, slots, most, _ = _fork_sizes(c)
        copies = c["children"] * sum(1 for x in lens if x % PAGE)
        # pages copied; entries of the parents read and of the children written, three times for counts
        used = sum(-(-x // PAGE) for x in lens)
        return {"bytes": 2 * copies * page + 4 * c["children"] * used * 6, "flops": 0}
    if c["op"] == "compact":
        places = _compact_places(c)
        moved = sum(1 for p in places if p >= len(places))
        return {"bytes": 2 * moved * page + 2 * 4 * c["pages"] + 2 * 4 * len(places), "flops": 0}
    new, lens = _lengths(c)
    T = sum(new)
    pages = (4 * sum(-(-x // PAGE) for x in lens) if c["paged"] else 0)
    index = 4 * (2 * c["B"] + 1) + pages
    if c["op"] == "rotate":      # rows in; queries and codes out; keys and values read back
        rows = T * (c["Hq"] + 2 * c["Hkv"]) * D * 2
        table = 4 * sum(new) * c["rot"]
        return {"bytes": rows + T * c["Hq"] * D * 2 + 2 * T * row + 2 * T * (row + c["Hkv"] * D * 2) + table + index,
                "flops": T * ((c["Hq"] + c["Hkv"]) * D * 10 + 2 * c["Hkv"] * D * 6)}
    if c["op"] == "bounds":      # the blocks that new tokens lie in, read whole; bounds out, and as 32-bit values
        touched = tokens = 0
        for n, x in zip(new, lens):
            a = (x - n) // PAGE
            touched += -(-x // PAGE) - a
            tokens += x - a * PAGE
        return {"bytes": tokens * row + touched * (2 * block + c["Hkv"] * 2 * D * 4) + index, "flops": tokens * c["Hkv"] * D * 4}
    # every row: the bounds of its blocks, once a sequence; the taken blocks' keys and values of each row
    tokens = scored = dots = 0
    for n, x in zip(new, lens):
        scored += -(-x // PAGE)
        for i in range(n):
            seen = x - n + 1 + i
            k = min(c["take"], -(-seen // PAGE))
            tokens += min(k * PAGE, seen)
            dots += -(-seen // PAGE)
    return {"bytes": scored * block + 2 * tokens * row + 2 * T * c["Hq"] * D * 2 + 4 * T * c["Hkv"] * c["take"] + index,
            "flops": 4 * tokens * c["Hq"] * D + 4 * dots * c["Hkv"] * D}


# ---------------------------------------------------------------- inputs

def _values(gen, shape, outlier):
    x = torch.randn(shape, generator=gen, device="cuda")
    return (x * outlier).to(torch.bfloat16)


def _quantise(x, bits):
    """Codes (uint8, one per channel), fp16 scales and zero points of rows x[..., D], groups of 32 channels."""
    g = x.float().unflatten(-1, (-1, GROUP))
    qmax = float(2 ** bits - 1)
    lo = g.amin(-1).clamp(max=0.0)
    hi = g.amax(-1).clamp(min=0.0)
    want = (hi - lo) / torch.full_like(hi, qmax)                    # (by a number, torch multiplies by its reciprocal)
    half = want.to(torch.float16)
    up = (half.view(torch.int16) + 1).view(torch.float16)           # the next larger value: scales are positive
    s = torch.where(half.float() < want, up, half)
    s = torch.where(hi == lo, torch.ones_like(s), s)
    sf = s.float()
    z = torch.round(-lo / sf).clamp(0.0, qmax)
    code = (torch.round(g / sf.unsqueeze(-1)) + z.unsqueeze(-1)).clamp(0.0, qmax)
    return code.flatten(-2).to(torch.uint8), s, z.to(torch.float16)


def _words(s, z):
    return (s.view(torch.int16).int() & 0xFFFF) | (z.view(torch.int16).int() << 16)


def _planes(state, codes):
    """Views of the code buffer: 8-bit heads [n8][rows][slots][D], 4-bit heads [n4][rows][slots][D / 2]."""
    n8, n4, S, C, D = len(state["h8"]), len(state["h4"]), state["stores"], state["slots"], state["D"]
    cut = n8 * S * C * D
    return codes[:cut].view(n8, S, C, D), codes[cut:cut + n4 * S * C * D // 2].view(n4, S, C, D // 2)


def _put(state, codes, words, at, x):
    """Quantise rows x [Hkv][N][D] into the buffers at (store, slot) index tensors `at`."""
    p8, p4 = _planes(state, codes)
    w = words.view(state["Hkv"], state["stores"], state["slots"], state["D"] // GROUP)
    if state["h8"]:
        c, s, z = _quantise(x[state["i8"]], 8)
        p8[:, at[0], at[1]] = c
        w[state["i8"][:, None], at[0], at[1]] = _words(s, z)
    if state["h4"]:
        c, s, z = _quantise(x[state["i4"]], 4)
        p4[:, at[0], at[1]] = c[..., 0::2] | (c[..., 1::2] << 4)
        w[state["i4"][:, None], at[0], at[1]] = _words(s, z)


def _int32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _storage(state, bits):
    state["bits"] = bits
    state["h8"] = [h for h in range(len(bits)) if bits[h] == 8]
    state["h4"] = [h for h in range(len(bits)) if bits[h] == 4]
    state["i8"] = torch.tensor(state["h8"], dtype=torch.long, device="cuda")
    state["i4"] = torch.tensor(state["h4"], dtype=torch.long, device="cuda")
    state["order"] = torch.argsort(torch.cat([state["i8"], state["i4"]]))    # KV head -> place among the planes


def _prepare_pool(c, seed):
    """A page pool of stored rows (bytes as they come: nothing here computes with them), its tables and counts."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    D, Hkv, bits = c["D"], c["Hkv"], _head_bits(c)
    state = {"op": c["op"], "Hkv": Hkv, "D": D, "slots": PAGE, "keep": {}, "with_bounds": c["bounds"]}
    _storage(state, bits)
    if c["op"] == "fork":
        lens, n, most, pages = _fork_sizes(c)
        B, kids = c["B"], c["children"]
        places = torch.randperm(pages, generator=gen, device="cuda").tolist()
        state["parents"] = _int32([b for b in range(B) for _ in range(kids)])
        state["children"] = _int32([B + b * kids + i for b in range(B) for i in range(kids)])
        state["add"] = _int32([0] * B + [c["room"]] * (B * kids))
        lens = lens + [0] * (B * kids)
    else:
        lens, pages = _compact_lens(c), c["pages"]
        n, most = len(lens), max(-(-x // PAGE) for x in lens)
        places = _compact_places(c)
        rng = random.Random(seed)
        rng.shuffle(places)
    rows, refs, at = [], [0] * pages, 0
    for x in lens:
        used = -(-x // PAGE)
        mine = places[at:at + used]
        at += used
        for p in mine:
            refs[p] += 1
        rows.append(mine + [0] * (most - used))
    state["stores"], state["seqs"], state["most"] = pages, n, most
    state["table0"], state["refs0"], state["lens0"] = _int32(rows), _int32(refs), _int32(lens)
    for name in ("table", "refs", "lens"):
        state[name] = state[name + "0"].clone()
    size = sum(D * b // 8 for b in bits) * pages * PAGE
    for name in ("k", "v"):
        state[name + "_codes"] = torch.randint(0, 256, (size,), generator=gen, device="cuda", dtype=torch.uint8)
        state[name + "_words"] = torch.randint(0, 1 << 30, (Hkv * pages * PAGE * (D // GROUP),), generator=gen,
                                               device="cuda", dtype=torch.int32)
    if c["bounds"]:
        state["b_codes"] = torch.randint(-127, 128, (Hkv, pages, D // GROUP, 2, GROUP), generator=gen, device="cuda",
                                         dtype=torch.int8)
        state["b_scales"] = torch.rand((Hkv, pages, D // GROUP), generator=gen, device="cuda")
    return state


def _rotary_table(positions, rot):
    """Cosines and sines of the usual angles, position * 10000 ** (-2 i / rot), as a model keeps them."""
    freq = 10000.0 ** (-torch.arange(0, rot, 2, device="cuda", dtype=torch.float64) / max(rot, 1))
    angle = torch.arange(positions, device="cuda", dtype=torch.float64)[:, None] * freq
    return torch.cat([angle.cos(), angle.sin()], 1).float()


def prepare(c, seed):
    if c["op"] in ("fork", "compact"):
        return _prepare_pool(c, seed)
    gen = torch.Generator(device="cuda").manual_seed(seed)
    new, lens = _lengths(c)
    B, Hq, Hkv, D, T = c["B"], c["Hq"], c["Hkv"], c["D"], sum(new)
    cap = -(-max(lens) // PAGE) * PAGE
    start = [0]
    for n in new:
        start.append(start[-1] + n)
    state = {"op": c["op"], "B": B, "Hq": Hq, "Hkv": Hkv, "D": D, "T": T, "cap": cap, "new_max": max(new),
             "len_max": max(lens), "start": _int32(start), "lens": _int32(lens), "table": None, "keep": {}}
    _storage(state, _head_bits(c))
    if c["paged"]:
        pages = cap // PAGE
        state["stores"], state["slots"] = B * pages + 3, PAGE
        state["table"] = torch.randperm(B * pages + 3, generator=gen, device="cuda")[:B * pages].int().view(B, pages)
    else:
        state["stores"], state["slots"] = B, cap
    # both caches, filled with quantised rows: some channels of each head are several times the others, and keys drift
    # along the sequence, so that blocks differ
    outlier = torch.where(torch.rand((Hkv, 1, 1, D), generator=gen, device="cuda") < 2.0 / D, 5.0, 1.0)
    store = torch.arange(state["stores"], device="cuda").repeat_interleave(state["slots"])
    slot = torch.arange(state["slots"], device="cuda").repeat(state["stores"])
    n8, n4 = len(state["h8"]), len(state["h4"])
    for name in ("k", "v"):
        codes = torch.empty((2 * n8 + n4) * state["stores"] * state["slots"] * D // 2, dtype=torch.uint8, device="cuda")
        words = torch.empty(Hkv * state["stores"] * state["slots"] * (D // GROUP), dtype=torch.int32, device="cuda")
        x = torch.randn((Hkv, state["stores"], state["slots"], D), generator=gen, device="cuda")
        if name == "k":
            x = x.view(Hkv, -1, PAGE, D)
            x += torch.randn((Hkv, x.shape[1], 1, D), generator=gen, device="cuda")
            x = x.view(Hkv, state["stores"], state["slots"], D).mul_(outlier)
        _put(state, codes, words, (store, slot), x.to(torch.bfloat16).flatten(1, 2))
        state[name + "_codes"], state[name + "_words"] = codes, words
        del x
    if c["op"] == "rotate":
        state.update(rot=c["rot"], interleaved=c["interleaved"], norm=c["norm"])
        state["qkv"] = _values(gen, (T, (Hq + 2 * Hkv) * D), 1.5)
        if c["norm"]:
            state["q_weight"] = (1.0 + 0.2 * torch.randn(D, generator=gen, device="cuda")).to(torch.bfloat16)
            state["k_weight"] = (1.0 + 0.2 * torch.randn(D, generator=gen, device="cuda")).to(torch.bfloat16)
        if c["rot"]:
            state["rotary"] = _rotary_table(cap, c["rot"])
        return state
    state["blocks"] = state["stores"] * state["slots"] // PAGE
    G = D // GROUP
    state["b_codes"] = torch.zeros((Hkv, state["blocks"], G, 2, GROUP), dtype=torch.int8, device="cuda")
    state["b_scales"] = torch.zeros((Hkv, state["blocks"], G), dtype=torch.float32, device="cuda")
    if c["op"] == "bounds":                                         # the blocks that the new tokens lie in
        ids = [(b, i) for b in range(B) for i in range((lens[b] - new[b]) // PAGE, -(-lens[b] // PAGE))]
        at = torch.tensor(ids, device="cuda").unbind(1)
        state["touched"] = _block_of(state, *at).int()
    else:
        state.update(take=c["take"], first=c["first"], last=c["last"])
        state["q"] = _values(gen, (T, Hq, D), 1.0)
        state["row_seq"] = _int32([b for b in range(B) for _ in range(new[b])])
        state["row_lens"] = _int32([x - n + 1 + i for n, x in zip(new, lens) for i in range(n)])
        _fill_bounds(state, torch.zeros(B, dtype=torch.long, device="cuda"))
    return state


# ---------------------------------------------------------------- plain forms

def _where(state, seq, pos):
    """(store, slot) of cache position pos of sequence seq."""
    if state["table"] is None:
        return seq, pos
    return state["table"].long()[seq, pos // PAGE], pos % PAGE


def _rows(state):
    """Sequence, index in its chunk and cache position of every packed row."""
    start = state["start"].long()
    r = torch.arange(state["T"], device="cuda")
    seq = torch.searchsorted(start[1:], r, right=True)
    i = r - start[seq]
    return seq, i, state["lens"].long()[seq] - (start[seq + 1] - start[seq]) + i


def _read(state, name, at):
    """Stored values at (store, slot) in 32 bits, [Hkv] + at's shape + [D]."""
    p8, p4 = _planes(state, state[name + "_codes"])
    c4 = p4[:, at[0], at[1]]
    c = torch.cat([p8[:, at[0], at[1]], torch.stack([c4 & 15, c4 >> 4], -1).flatten(-2)])[state["order"]]
    w = state[name + "_words"].view(state["Hkv"], state["stores"], state["slots"], -1)[:, at[0], at[1]]
    s = (w & 0xFFFF).to(torch.int16).view(torch.float16).float()
    z = (w >> 16).to(torch.int16).view(torch.float16).float()
    return ((c.float().unflatten(-1, (-1, GROUP)) - z.unsqueeze(-1)) * s.unsqueeze(-1)).flatten(-2)


def _turn(x, weight, state, pos):
    """Rows x [T][heads][D], normed and rotated by their positions, in bf16."""
    y = x.float()
    if weight is not None:
        mean = (x.double() * x.double()).mean(-1, keepdim=True).float()
        root = torch.sqrt(mean + EPS)
        y = y * (torch.ones_like(root) / root) * weight.float()
    rot = state["rot"]
    if rot:
        cos, sin = state["rotary"][pos].unsqueeze(1).split(rot // 2, -1)
        part, rest = y[..., :rot], y[..., rot:]
        if state["interleaved"]:
            a, b = part[..., 0::2], part[..., 1::2]
            y = torch.cat([torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2), rest], -1)
        else:
            a, b = part.chunk(2, -1)
            y = torch.cat([a * cos - b * sin, b * cos + a * sin, rest], -1)
    return y.to(torch.bfloat16)


def _plain_rotate(state):
    seq, _, pos = _rows(state)
    at = _where(state, seq, pos)
    Hq, Hkv, D = state["Hq"], state["Hkv"], state["D"]
    q, k, v = state["qkv"].view(-1, Hq + 2 * Hkv, D).split([Hq, Hkv, Hkv], 1)
    q = _turn(q, state.get("q_weight"), state, pos)
    _put(state, state["k_codes"], state["k_words"], at, _turn(k, state.get("k_weight"), state, pos).transpose(0, 1))
    _put(state, state["v_codes"], state["v_words"], at, v.transpose(0, 1))
    return {"q": q, "k": _read(state, "k", at).transpose(0, 1).to(torch.bfloat16),
            "v": _read(state, "v", at).transpose(0, 1).to(torch.bfloat16)}


def _block_of(state, seq, block):
    """Which of the storage's 64-token blocks holds block `block` of sequence seq."""
    if state["table"] is None:
        return seq * (state["cap"] // PAGE) + block
    return state["table"].long()[seq, block]


def _fill_bounds(state, since):
    """Bounds of every sequence's blocks from the one that holds position since[b] on."""
    lens = state["lens"].long()
    block = torch.arange(state["cap"] // PAGE, device="cuda").expand(state["B"], -1)
    seq = torch.arange(state["B"], device="cuda")[:, None].expand_as(block)
    touched = (block >= since[:, None] // PAGE) & (block * PAGE < lens[:, None])
    seq, block = seq[touched], block[touched]
    pos = block[:, None] * PAGE + torch.arange(PAGE, device="cuda")
    x = _read(state, "k", _where(state, seq[:, None].expand_as(pos), pos))             # [Hkv][blocks][64][D]
    out = (pos >= lens[seq][:, None])[None, ..., None]
    lo = x.masked_fill(out, float("inf")).amin(2).unflatten(-1, (-1, GROUP))           # [Hkv][blocks][G][32]
    hi = x.masked_fill(out, float("-inf")).amax(2).unflatten(-1, (-1, GROUP))
    most = torch.maximum(-lo, hi).amax(-1)
    scale = most / torch.full_like(most, 127.0)
    unit = torch.where(scale > 0, scale, torch.ones_like(scale)).unsqueeze(-1)
    codes = torch.stack([torch.ceil(hi / unit), torch.floor(lo / unit)], -2).clamp(-127, 127)
    to = _block_of(state, seq, block)
    state["b_codes"][:, to] = codes.to(torch.int8)
    state["b_scales"][:, to] = scale


def _plain_bounds(state):
    start = state["start"].long()
    _fill_bounds(state, state["lens"].long() - (start[1:] - start[:-1]))
    i = state["touched"].long()
    v = state["b_codes"][:, i].float() * state["b_scales"][:, i, :, None, None]        # [Hkv][blocks][G][2][32]
    return {"values": v.transpose(2, 3).reshape(state["Hkv"], i.numel(), 2, state["D"])}


def _scores(state, lens, seq):
    """Scores of the blocks of every row's sequence, [rows][Hkv][blocks]; whole products of 8-bit values are exact."""
    T, Hkv, D, rep = state["T"], state["Hkv"], state["D"], state["Hq"] // state["Hkv"]
    q = state["q"].float().view(T, Hkv, rep, D)
    up = functools.reduce(torch.add, q.clamp(min=0.0).unbind(2))
    down = functools.reduce(torch.add, q.clamp(max=0.0).unbind(2))
    qs = torch.stack([up, down], 2).unflatten(-1, (-1, GROUP)).transpose(2, 3)         # [T][Hkv][G][2][32]
    most = qs.abs().amax((-2, -1))
    scale = most / torch.full_like(most, 127.0)
    unit = torch.where(scale > 0, scale, torch.ones_like(scale))
    code = torch.round(qs / unit[..., None, None])
    n = -(-state["len_max"] // PAGE)
    at = _block_of(state, seq[:, None], torch.arange(n, device="cuda"))                # [T][n]
    b = state["b_codes"][:, at].float()                                                # [Hkv][T][n][G][2][32]
    dots = (b * code.transpose(0, 1).unsqueeze(2)).sum((-2, -1)).transpose(0, 1)       # [T][Hkv][n][G]
    term = (scale.unsqueeze(2) * state["b_scales"][:, at].transpose(0, 1)) * dots
    return functools.reduce(torch.add, term.unbind(-1))


def _plain_blocks(state):
    T, Hq, Hkv, D = state["T"], state["Hq"], state["Hkv"], state["D"]
    lens, seq, K = state["row_lens"].long(), state["row_seq"].long(), state["take"]
    score = _scores(state, lens, seq)
    n = score.shape[-1]
    block = torch.arange(n, device="cuda")
    held = (lens + PAGE - 1) // PAGE
    kept = (block < state["first"]) | (block >= held[:, None] - state["last"])
    score = score.masked_fill(kept[:, None], float("inf")).masked_fill((block >= held[:, None])[:, None], float("-inf"))
    best = torch.sort(score, dim=-1, descending=True, stable=True).indices[..., :K]
    best = torch.where(best < held[:, None, None], best, torch.full_like(best, n))     # (more asked for than there are)
    best = torch.nn.functional.pad(best, (0, K - best.shape[-1]), value=n)
    best = torch.sort(best, -1).values
    sel = torch.where(best < n, best, torch.full_like(best, -1)).int()
    # attention over the tokens of the selected blocks
    pos = (best.unsqueeze(-1) * PAGE + torch.arange(PAGE, device="cuda")).flatten(-2)  # [T][Hkv][K * 64]
    see = pos < lens[:, None, None]
    at = _where(state, seq[:, None, None].expand_as(pos), pos.clamp(max=state["cap"] - 1))
    k, v = (_read_heads(state, name, at) for name in ("k", "v"))                       # [T][Hkv][K * 64][D]
    q = state["q"].float().view(T, Hkv, Hq // Hkv, D)
    x = (q @ k.transpose(2, 3)).mul_(1.0 / math.sqrt(D))
    x.masked_fill_(~see.unsqueeze(2), float("-inf"))
    x = x.sub_(x.amax(-1, keepdim=True).clamp(min=-3e38)).exp_()
    out = (x @ v) / x.sum(-1, keepdim=True).clamp(min=1e-30)
    return {"sel": sel, "out": out.reshape(T, Hq, D).to(torch.bfloat16)}


def _read_heads(state, name, at):
    """Stored values at (store, slot) [T][Hkv][N], each KV head's own, in 32 bits: [T][Hkv][N][D]."""
    D, (p8, p4) = state["D"], _planes(state, state[name + "_codes"])
    T, Hkv, N = at[0].shape
    c = torch.empty((T, Hkv, N, D), device="cuda")
    h = torch.arange(Hkv, device="cuda")[None, :, None]
    if state["h8"]:
        i = state["i8"]
        c[:, i] = p8[torch.arange(len(i), device="cuda")[None, :, None], at[0][:, i], at[1][:, i]].float()
    if state["h4"]:
        i = state["i4"]
        c4 = p4[torch.arange(len(i), device="cuda")[None, :, None], at[0][:, i], at[1][:, i]]
        c[:, i] = torch.stack([c4 & 15, c4 >> 4], -1).flatten(-2).float()
    w = state[name + "_words"].view(Hkv, state["stores"], state["slots"], -1)[h, at[0], at[1]]
    s = (w & 0xFFFF).to(torch.int16).view(torch.float16).float()
    z = (w >> 16).to(torch.int16).view(torch.float16).float()
    return ((c.unflatten(-1, (-1, GROUP)) - z.unsqueeze(-1)) * s.unsqueeze(-1)).flatten(-2)


def _move(state, src, dst):
    """Pages src to pages dst: codes and words of both caches, and their bounds."""
    for name in ("k", "v"):
        for p in _planes(state, state[name + "_codes"]):
            p[:, dst] = p[:, src]
        w = state[name + "_words"].view(state["Hkv"], state["stores"], -1)
        w[:, dst] = w[:, src]
    if state["with_bounds"]:
        state["b_codes"][:, dst] = state["b_codes"][:, src]
        state["b_scales"][:, dst] = state["b_scales"][:, src]


def _pool(state):
    """All that a page operator may change."""
    return [state[n] for n in ("table", "refs", "lens", "k_codes", "k_words", "v_codes", "v_words", "b_codes", "b_scales")
            if n in state]


def _plain_fork(state):
    table, refs, lens = state["table"], state["refs"], state["lens"]
    col = torch.arange(state["most"], device="cuda")
    kids, parents = state["children"].long(), state["parents"].long()
    gone = col < (lens[kids, None] + PAGE - 1) // PAGE                       # let go
    refs.index_add_(0, table[kids][gone].long(), -torch.ones_like(table[kids][gone]))
    size = lens[parents]                                                     # forked
    full = col < size[:, None] // PAGE
    table[kids] = torch.where(full, table[parents], table[kids])
    refs.index_add_(0, table[kids][full].long(), torch.ones_like(table[kids][full]))
    cut = torch.nonzero(size % PAGE)[:, 0]
    fresh = torch.nonzero(refs == 0)[:cut.numel(), 0]
    last = size[cut].long() // PAGE
    _move(state, table[parents[cut], last].long(), fresh)
    table[kids[cut], last] = fresh.int()
    refs[fresh] = 1
    lens[kids] = size
    have = (lens + PAGE - 1) // PAGE                                         # room for new tokens
    more = (lens + state["add"] + PAGE - 1) // PAGE
    want = (col >= have[:, None]) & (col < more[:, None])
    fresh = torch.nonzero(refs == 0)[:, 0]
    place = torch.cumsum(want.flatten().long(), 0).view_as(want) - 1
    table.copy_(torch.where(want, fresh.int()[place.clamp(min=0, max=fresh.numel() - 1)], table))
    refs[table[want].long()] = 1
    lens += state["add"]
    return _pool(state)


def _plain_compact(state):
    table, refs, lens = (state[n].copy_(state[n + "0"]) for n in ("table", "refs", "lens"))   # what the last pass began with
    live = refs > 0
    page = torch.arange(refs.numel(), device="cuda")
    n = live.sum()
    src, dst = torch.nonzero(live & (page >= n))[:, 0], torch.nonzero(~live & (page < n))[:, 0]
    _move(state, src, dst)
    to = page.index_copy(0, src, dst)
    used = torch.arange(state["most"], device="cuda") < (lens[:, None] + PAGE - 1) // PAGE
    table.copy_(torch.where(used, to[table.long()].int(), table))
    refs[dst] = refs[src]
    refs[src] = 0
    return _pool(state)


_PLAIN = {"rotate": _plain_rotate, "bounds": _plain_bounds, "blocks": _plain_blocks, "fork": _plain_fork,
          "compact": _plain_compact}


# ---------------------------------------------------------------- the framework's calls

def _kept(state, kvq):
    """The cache objects and the workspaces that a serving program makes once."""
    keep = state["keep"]
    if not keep:
        for name in ("k", "v"):
            keep[name] = kvq.QuantCache(state[name + "_codes"], state[name + "_words"], state["bits"],
                                        state["stores"], state["Hkv"], state["slots"], state["D"])
        if "b_codes" in state:
            keep["bounds"] = kvq.BlockBounds(state["b_codes"], state["b_scales"])
        if state["op"] == "blocks":
            keep["select"] = kvq.select_workspace(state["T"], state["Hkv"], state["cap"])
            keep["attend"] = kvq.decode_workspace(state["T"], state["Hq"], state["Hkv"], state["D"])
        if state["op"] in ("fork", "compact"):
            keep["pages"] = kvq.PageTable(state["refs"], state["table"], state["lens"])
            keep["ws"] = kvq.pages_workspace(state["stores"], state["seqs"])
    return keep


def _own_rotate(state, kvq):
    keep = _kept(state, kvq)
    k, v, start, lens, table = keep["k"], keep["v"], state["start"], state["lens"], state["table"]
    Hq, Hkv = state["Hq"], state["Hkv"]
    rows = state["qkv"].view(state["T"], Hq + 2 * Hkv, state["D"])
    args = (rows[:, :Hq], rows[:, Hq:Hq + Hkv], rows[:, Hq + Hkv:], k, v)
    more = {"rotary": state.get("rotary"), "q_weight": state.get("q_weight"), "k_weight": state.get("k_weight"),
            "eps": EPS, "interleaved": state["interleaved"]}
    if table is None:
        return {"q": kvq.rotate_append(*args, start, lens, **more),
                "k": kvq.dequantize(k, start, lens, state["T"], out_dtype=kvq.OUT_BF16),
                "v": kvq.dequantize(v, start, lens, state["T"], out_dtype=kvq.OUT_BF16)}
    return {"q": kvq.rotate_append_paged(*args, table, start, lens, **more),
            "k": kvq.dequantize_paged(k, table, start, lens, state["T"], out_dtype=kvq.OUT_BF16),
            "v": kvq.dequantize_paged(v, table, start, lens, state["T"], out_dtype=kvq.OUT_BF16)}


def _own_bounds(state, kvq):
    keep = _kept(state, kvq)
    if state["table"] is None:
        kvq.block_bounds(keep["k"], keep["bounds"], state["start"], state["lens"], state["T"])
    else:
        kvq.block_bounds_paged(keep["k"], keep["bounds"], state["table"], state["start"], state["lens"], state["T"])
    return {"values": kvq.bounds_values(keep["bounds"], state["touched"])}


def _own_blocks(state, kvq):
    keep = _kept(state, kvq)
    k, v, q, seq, lens, table = keep["k"], keep["v"], state["q"], state["row_seq"], state["row_lens"], state["table"]
    pick = {"first": state["first"], "last": state["last"], "row_seq": seq, "workspace": keep["select"]}
    more = {"row_seq": seq, "out_dtype": kvq.OUT_BF16, "workspace": keep["attend"]}
    if table is None:
        sel = kvq.select_blocks(q, k, keep["bounds"], lens, state["take"], **pick)
        return {"sel": sel, "out": kvq.decode_attention_blocks(q, k, v, sel, lens, **more)}
    sel = kvq.select_blocks_paged(q, k, keep["bounds"], table, lens, state["take"], **pick)
    return {"sel": sel, "out": kvq.decode_attention_blocks_paged(q, k, v, table, sel, lens, **more)}


def _own_fork(state, kvq):
    keep = _kept(state, kvq)
    pages, ws = keep["pages"], keep["ws"]
    kvq.pages_free(pages, state["children"])
    kvq.pages_fork(pages, keep["k"], keep["v"], state["parents"], state["children"], bounds=keep.get("bounds"),
                   workspace=ws)
    kvq.pages_reserve(pages, state["add"], workspace=ws)
    return _pool(state)


def _own_compact(state, kvq):
    keep = _kept(state, kvq)
    state["table"].copy_(state["table0"])                                    # what the last pass began with
    state["refs"].copy_(state["refs0"])
    state["lens"].copy_(state["lens0"])
    kvq.pages_compact(keep["pages"], keep["k"], keep["v"], bounds=keep.get("bounds"), workspace=keep["ws"])
    return _pool(state)


_OWN = {"rotate": _own_rotate, "bounds": _own_bounds, "blocks": _own_blocks, "fork": _own_fork, "compact": _own_compact}


def run(state):
    if own:
        from attention_group_quantized_gb300 import kvq
        return _OWN[state["op"]](state, kvq)
    return _PLAIN[state["op"]](state)


# ---------------------------------------------------------------- in 64 bits

def _stored64(state, name, b, h, count):
    """The first `count` stored rows of sequence b, KV head h, as the values they stand for."""
    S, C, D, bits = state["stores"], state["slots"], state["D"], state["bits"]
    size = [S * C * D * x // 8 for x in bits]
    off = sum(size[g] for g in range(len(bits)) if (bits[g] != 8, g) < (bits[h] != 8, h))
    raw = state[name + "_codes"][off:off + size[h]].view(S, C, -1)
    word = state[name + "_words"].view(len(bits), S, C, -1)[h]
    if state["table"] is None:
        raw, word = raw[b, :count], word[b, :count]
    else:
        ids = state["table"][b, :-(-count // PAGE)].long()
        raw, word = raw[ids].flatten(0, 1)[:count], word[ids].flatten(0, 1)[:count]
    if bits[h] == 4:
        c = torch.empty(count, D, dtype=torch.float64, device=raw.device)
        c[:, 0::2], c[:, 1::2] = (raw % 16).double(), (raw // 16).double()
    else:
        c = raw.double()
    pair = word.contiguous().view(torch.float16).view(count, -1, 2).double()
    return (c - pair[..., 1].repeat_interleave(GROUP, 1)) * pair[..., 0].repeat_interleave(GROUP, 1)


def _round_trip64(x, bits):
    """What quantising rows x[N][D] keeps of them: the range over the number of steps is rounded to 32 bits and then up
    to 16, as the format says; the rest is whole numbers."""
    y = x.double().view(x.shape[0], -1, GROUP)
    steps = 2 ** bits - 1
    low, high = y.min(2).values.clamp(max=0), y.max(2).values.clamp(min=0)
    step = ((high - low).float().double() / steps).float().double()
    near = step.to(torch.float16)
    near = torch.where(near.double() < step, torch.nextafter(near.cpu(), torch.tensor(float("inf"), dtype=torch.float16)).cuda(), near)
    unit = torch.where(high > low, near.double(), 1.0)[..., None]
    zero = (-low[..., None] / unit).round().clamp(0, steps)
    return ((((y / unit).round() + zero).clamp(0, steps) - zero) * unit).view(x.shape)


def _exact_rotate(c, state, new, lens):
    Hq, Hkv, D, rot = c["Hq"], c["Hkv"], c["D"], c["rot"]
    x = state["qkv"].view(-1, Hq + 2 * Hkv, D)
    pos = torch.cat([torch.arange(n - m, n, device="cuda") for m, n in zip(new, lens)])
    outs = []
    for part, weight in ((x[:, :Hq], "q_weight"), (x[:, Hq:Hq + Hkv], "k_weight")):
        y = part.double()
        if c["norm"]:
            y = y * (y.pow(2).mean(2, keepdim=True) + EPS).rsqrt() * state[weight].double()
        if rot:
            turn = torch.complex(state["rotary"][pos, :rot // 2].double(), state["rotary"][pos, rot // 2:].double())[:, None]
            i = torch.arange(rot // 2, device="cuda")
            one, two = (2 * i, 2 * i + 1) if c["interleaved"] else (i, i + rot // 2)
            z = torch.complex(y[..., one], y[..., two]) * turn
            y = y.clone()
            y[..., one], y[..., two] = z.real, z.imag
        outs.append(y)
    q, k = outs
    got = {"q": q}
    k = k.to(torch.bfloat16)                                        # (quantised from its rounded value)
    for name, rows in (("k", k), ("v", x[:, Hq + Hkv:])):
        got[name] = torch.stack([_round_trip64(rows[:, h], state["bits"][h]) for h in range(Hkv)], 1)
    return got


def _exact_bounds(state, since, lens):
    """Bounds of the touched blocks as values, zero elsewhere: [Hkv][blocks][2][D], and the scales [Hkv][blocks][G]."""
    Hkv, D, G = state["Hkv"], state["D"], state["D"] // GROUP
    codes = torch.zeros(Hkv, state["blocks"], 2, D, dtype=torch.float64, device="cuda")
    scales = torch.zeros(Hkv, state["blocks"], G, dtype=torch.float64, device="cuda")
    for b, n in enumerate(lens):
        blocks = torch.arange(since[b] // PAGE, -(-n // PAGE), device="cuda")
        to = blocks + b * (state["cap"] // PAGE) if state["table"] is None else state["table"][b, blocks].long()
        for h in range(Hkv):
            x = _stored64(state, "k", b, h, n)
            pad = blocks.shape[0] * PAGE - (n - since[b] // PAGE * PAGE)
            x = x[since[b] // PAGE * PAGE:]
            x = torch.cat([x, x[-1:].expand(pad, D)]).view(-1, PAGE, D)
            low, high = x.min(1).values, x.max(1).values
            most = torch.maximum(low.abs(), high.abs()).view(-1, G, GROUP).max(2).values
            s = (most / 127).float().double()                       # (kept in 32 bits, as the format says)
            unit = torch.where(s > 0, s, 1.0).repeat_interleave(GROUP, 1)
            codes[h, to, 0] = (high / unit).float().ceil().clamp(-127, 127).double()
            codes[h, to, 1] = (low / unit).float().floor().clamp(-127, 127).double()
            scales[h, to] = s
    return codes, scales


def _exact_blocks(c, state, new, lens):
    D, Hkv, G = state["D"], state["Hkv"], state["D"] // GROUP
    rep, T = state["Hq"] // Hkv, state["T"]
    codes, scales = _exact_bounds(state, [0] * len(lens), lens)
    sel = torch.full((T, Hkv, c["take"]), -1, dtype=torch.int32, device="cuda")
    out = torch.zeros(T, state["Hq"], D, dtype=torch.float64, device="cuda")
    f32 = lambda v: v.float().double()                              # the score is kept in 32 bits, one rounding a step
    row = 0
    for b, (n, length) in enumerate(zip(new, lens)):
        for h in range(Hkv):
            k, v = _stored64(state, "k", b, h, length), _stored64(state, "v", b, h, length)
            for i in range(n):
                seen = length - n + 1 + i
                m = -(-seen // PAGE)
                ids = torch.arange(m, device="cuda")
                at = ids + b * (state["cap"] // PAGE) if state["table"] is None else state["table"][b, ids].long()
                q = state["q"][row + i, h * rep:(h + 1) * rep].double()
                up, down = torch.zeros(D, device="cuda").double(), torch.zeros(D, device="cuda").double()
                for r in range(rep):
                    up, down = f32(up + q[r].clamp(min=0)), f32(down + q[r].clamp(max=0))
                most = torch.maximum(up, -down).view(G, GROUP).max(1).values
                unit = f32(most / 127)
                div = torch.where(unit > 0, unit, 1.0).repeat_interleave(GROUP)
                dots = (f32(up / div).round() * codes[h, at, 0] + f32(down / div).round() * codes[h, at, 1]).view(m, G, GROUP).sum(2)
                term = f32(f32(unit * scales[h, at]) * dots)
                score = term[:, 0]
                for g in range(1, G):
                    score = f32(score + term[:, g])
                score[:c["first"]] = math.inf
                score[max(0, m - c["last"]):] = math.inf
                best = torch.sort(-score, dim=-1, stable=True).indices[:c["take"]].sort().values
                sel[row + i, h, :best.shape[0]] = best.int()
                take = (best[:, None] * PAGE + torch.arange(PAGE, device="cuda")).flatten()
                take = take[take < seen]
                out[row + i, h * rep:(h + 1) * rep] = torch.softmax(q @ k[take].T / D ** 0.5, 1) @ v[take]
        row += n
    return {"sel": sel, "out": out}


def exact(c, seed):
    if c["op"] in ("fork", "compact"):
        return None                                                 # pages are moved, nothing is computed
    state = prepare(c, seed)
    new, lens = _lengths(c)
    if c["op"] == "rotate":
        return _exact_rotate(c, state, new, lens)
    if c["op"] == "blocks":
        return _exact_blocks(c, state, new, lens)
    codes, scales = _exact_bounds(state, [x - n for n, x in zip(new, lens)], lens)
    return {"values": (codes * scales.repeat_interleave(GROUP, 2).unsqueeze(2))[:, state["touched"].long()]}
