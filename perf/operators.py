"""The serving operators around a group-quantised KV cache, as a user's program calls them, with plain forms.

A case names one operator and the sizes of one call:

  append         write a ragged batch of new K and V rows into the caches (quantised as they are written), then read
                 the written rows back as values
  readback       read ragged ranges of one cache back as bf16 rows
  chunk          attention of a chunk of new tokens per sequence over the cache that already holds them: prompt
                 chunks, verification of drafted tokens, or a batch that mixes both; with `window`, a query sees the
                 last `window` tokens and the first `sinks` ones
  decode_window  one query token per sequence with the same window and sinks

New rows are packed: sequence b's are rows start[b] .. start[b + 1] - 1 and sit at cache positions
lens[b] - (start[b + 1] - start[b]) .. lens[b] - 1.  Caches hold 8- or 4-bit codes per KV head with an fp16 scale and
zero point per 32 channels, contiguous per sequence or in 64-token pages behind a block table.  Group quantisation
rounds as its definition says, in 32 bits; attention is softmax over the visible keys of the stored values.
"""
import math
import random

import torch

own = False

GROUP, PAGE = 32, 64


# ---------------------------------------------------------------- cases

def _case(op, B, Hq, Hkv, D, bits, ctx, new, paged, window=0, sinks=0):
    return {"op": op, "B": B, "Hq": Hq, "Hkv": Hkv, "D": D, "bits": bits, "ctx_lo": ctx[0], "ctx_hi": ctx[1],
            "new_lo": new[0], "new_hi": new[1], "paged": paged, "window": window, "sinks": sinks}


def listed():
    return [
        # a few tokens of a short conversation, small heads: latency
        dict(_case("append", 1, 4, 4, 64, "8", (496, 496), (16, 16), False), name="append_tiny"),
        # a scheduler's step: sequences with one new token next to prompt chunks, pages, INT8 and INT4 heads
        dict(_case("append", 16, 32, 8, 128, "mixed", (1000, 8000), (1, 512), True), name="append_mixed_pages"),
        # a whole 32K prompt into an INT4 cache
        dict(_case("append", 1, 32, 8, 128, "4", (0, 0), (32768, 32768), False), name="append_prompt_int4"),
        # a short prefix out of pages, as for handing it to another worker
        dict(_case("readback", 2, 8, 2, 64, "8", (0, 0), (333, 1000), True), name="readback_prefix_pages"),
        # four long sequences back to bf16, as for re-quantising or checking a cache
        dict(_case("readback", 4, 32, 8, 128, "mixed", (100, 900), (5000, 8192), False), name="readback_long_mixed"),
        # five tokens on half a thousand, one sequence, no shared heads
        dict(_case("chunk", 1, 4, 4, 64, "8", (507, 507), (5, 5), False), name="chunk_tiny"),
        # four drafted tokens verified for each of eight sequences of about 8K
        dict(_case("chunk", 8, 32, 8, 128, "8", (7900, 8188), (4, 4), True), name="chunk_verify_8k"),
        # a mixed batch: one token here, a prompt chunk there
        dict(_case("chunk", 16, 32, 8, 128, "mixed", (1000, 8000), (1, 512), True), name="chunk_mixed_batch"),
        # a 2K chunk of a prompt whose first 32K are cached
        dict(_case("chunk", 1, 32, 8, 128, "8", (32768, 32768), (2048, 2048), False), name="chunk_prompt_32k"),
        # about a thousand tokens on long INT4 sequences, window of 4096 and four sinks
        dict(_case("chunk", 4, 32, 8, 128, "4", (43000, 100000), (700, 1100), False, 4096, 4), name="chunk_window_int4"),
        # single tokens of eight 32K sequences, window of 4096 and four sinks
        dict(_case("decode_window", 8, 32, 8, 128, "8", (32700, 32767), (1, 1), False, 4096, 4), name="decode_window_int8"),
        # sixteen sequences from pages, small heads, odd window
        dict(_case("decode_window", 16, 16, 4, 64, "mixed", (300, 9000), (1, 1), True, 1000, 130),
             name="decode_window_pages"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "readback", "chunk", "chunk", "decode_window"])
    D = rng.choice([64, 128, 128])
    Hkv = rng.choice([1, 2, 4, 8])
    rep = rng.choice([1, 2, 3, 4, 4, 5, 8])
    bits = rng.choice(["8", "4", "mixed"])
    paged = rng.random() < 0.5
    B = _log(rng, 1, 32)
    window, sinks = 0, 0
    if op == "append":
        hi = _log(rng, 1, 32768 // B)
        return _case(op, B, Hkv * rep, Hkv, D, bits, (0, _log(rng, 1, 4000)), (rng.randint(1, hi), hi), paged)
    if op == "readback":
        hi = _log(rng, 1, 32768 // B)
        return _case(op, B, Hkv * rep, Hkv, D, bits, (0, _log(rng, 1, 4000)), (rng.randint(1, hi), hi), paged)
    if rng.random() < 0.5 or op == "decode_window":
        window, sinks = _log(rng, 1, 8000), rng.choice([0, 1, 4, 64, 130])
    if op == "decode_window":
        hi = _log(rng, 16, 65536 if B <= 8 else 16384)
        return _case(op, B, Hkv * rep, Hkv, D, bits, (rng.randint(0, hi), hi), (1, 1), paged, window, sinks)
    hi = _log(rng, 1, 1024 // B) if rng.random() < 0.7 else rng.randint(1, 8)
    ctx = _log(rng, 16, 16384 if B <= 8 else 4096)
    return _case(op, B, Hkv * rep, Hkv, D, bits, (rng.randint(0, ctx), ctx), (rng.randint(1, hi), hi), paged, window,
                 sinks)


def _lengths(c):
    """(new tokens, cached length including them) of each sequence: fixed by the case."""
    key = "|".join("%s=%s" % (k, c[k]) for k in sorted(c) if k != "name")
    rng = random.Random(key)
    new = [_log(rng, c["new_lo"], c["new_hi"]) for _ in range(c["B"])]
    return new, [n + rng.randint(c["ctx_lo"], c["ctx_hi"]) for n in new]


def _head_bits(c):
    if c["bits"] != "mixed":
        return [int(c["bits"])] * c["Hkv"]
    rng = random.Random("bits %d %d" % (c["Hkv"], c["D"]))
    return [8 if rng.random() < 0.5 else 4 for _ in range(c["Hkv"])]


def _seen(c, n, length):
    """Cache tokens that n queries at the end of a sequence see among them, and (query, key) pairs."""
    w, s = c["window"], c["sinks"]
    if not w:
        return length, n * length - n * (n - 1) // 2
    first = max(0, length - n - w + 1)
    pairs = 0
    for p in range(length - n, length):
        lo = max(0, p - w + 1)
        pairs += p - lo + 1 + min(s, lo)
    return length - first + min(s, first), pairs


def work(c):
    new, lens = _lengths(c)
    D, bits = c["D"], _head_bits(c)
    row = sum(D * b // 8 + 4 * (D // GROUP) for b in bits)          # one token's codes and scale words, all KV heads
    T = sum(new)
    index = 4 * (2 * c["B"] + 1) + (4 * sum(-(-x // PAGE) for x in lens) if c["paged"] else 0)
    if c["op"] == "append":      # rows in, codes out, and back as values
        return {"bytes": 2 * T * (c["Hkv"] * D * 2 + row) + 2 * T * (row + c["Hkv"] * D * 2) + index,
                "flops": 2 * T * c["Hkv"] * D * 8}
    if c["op"] == "readback":
        return {"bytes": T * (row + c["Hkv"] * D * 2) + index, "flops": 2 * T * c["Hkv"] * D}
    keys = pairs = 0
    for n, x in zip(new, lens):
        k, p = _seen(c, n, x)
        keys, pairs = keys + k, pairs + p
    return {"bytes": 2 * keys * row + 2 * T * c["Hq"] * D * 2 + index, "flops": 4 * pairs * c["Hq"] * D}


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


def prepare(c, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    new, lens = _lengths(c)
    B, Hq, Hkv, D, T = c["B"], c["Hq"], c["Hkv"], c["D"], sum(new)
    bits = _head_bits(c)
    cap = -(-max(lens) // PAGE) * PAGE
    dev = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")
    start = [0]
    for n in new:
        start.append(start[-1] + n)
    state = {"op": c["op"], "B": B, "Hq": Hq, "Hkv": Hkv, "D": D, "T": T, "cap": cap, "bits": bits,
             "window": c["window"], "sinks": c["sinks"], "new_max": max(new), "len_max": max(lens),
             "h8": [h for h in range(Hkv) if bits[h] == 8], "h4": [h for h in range(Hkv) if bits[h] == 4],
             "start": dev(start), "lens": dev(lens), "table": None, "keep": {}}
    state["i8"] = torch.tensor(state["h8"], dtype=torch.long, device="cuda")
    state["i4"] = torch.tensor(state["h4"], dtype=torch.long, device="cuda")
    order = torch.cat([state["i8"], state["i4"]])
    state["order"] = torch.argsort(order)                           # KV head -> place among the planes
    if c["paged"]:
        pages = cap // PAGE
        state["stores"], state["slots"] = B * pages + 3, PAGE
        state["table"] = torch.randperm(B * pages + 3, generator=gen, device="cuda")[:B * pages].int().view(B, pages)
    else:
        state["stores"], state["slots"] = B, cap
    # both caches, filled with quantised rows: some channels of each head are several times the others
    outlier = torch.where(torch.rand((Hkv, 1, 1, D), generator=gen, device="cuda") < 2.0 / D, 5.0, 1.0)
    store = torch.arange(state["stores"], device="cuda").repeat_interleave(state["slots"])
    slot = torch.arange(state["slots"], device="cuda").repeat(state["stores"])
    n8, n4 = len(state["h8"]), len(state["h4"])
    for name in ("k", "v"):
        codes = torch.empty((2 * n8 + n4) * state["stores"] * state["slots"] * D // 2, dtype=torch.uint8, device="cuda")
        words = torch.empty(Hkv * state["stores"] * state["slots"] * (D // GROUP), dtype=torch.int32, device="cuda")
        x = _values(gen, (Hkv, state["stores"], state["slots"], D), outlier if name == "k" else 1.0)
        _put(state, codes, words, (store, slot), x.flatten(1, 2))
        state[name + "_codes"], state[name + "_words"] = codes, words
        del x
    if c["op"] == "append":
        for name in ("k_new", "v_new"):
            state[name] = _values(gen, (T, Hkv, D), outlier[:, 0, 0] if name == "k_new" else 1.0)
    elif c["op"] != "readback":
        state["q"] = _values(gen, (T, Hq, D), 1.0)
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


def _attend(state):
    """Attention of every packed query over its sequence's visible keys, sequences padded to one length."""
    B, Hkv, D, N = state["B"], state["Hkv"], state["D"], state["new_max"]
    rep = state["Hq"] // Hkv
    lens, start = state["lens"].long(), state["start"].long()
    n = start[1:] - start[:-1]
    w, s = state["window"], state["sinks"]
    L = state["len_max"]
    if w and s + w + N - 1 < L:                                   # only the sinks and the last queries' windows
        first = (lens - n - w + 1).clamp(min=s)
        a = torch.arange(w + N - 1, device="cuda")
        key = torch.cat([torch.arange(s, device="cuda").expand(B, s), first[:, None] + a], 1)
    else:
        key = torch.arange(L, device="cuda").expand(B, L)
    held = key < lens[:, None]
    seq = torch.arange(B, device="cuda")[:, None]
    at = _where(state, seq, key.clamp(max=state["cap"] - 1))
    k = _read(state, "k", at).transpose(0, 1)                       # [B][Hkv][L][D]
    v = _read(state, "v", at).transpose(0, 1)
    i = torch.arange(N, device="cuda")
    q = state["q"].float()[(start[:-1, None] + i).clamp(max=state["T"] - 1)]          # [B][N][Hq][D]
    q = q.view(B, N, Hkv, rep, D).permute(0, 2, 3, 1, 4).reshape(B, Hkv, rep * N, D)
    pos = (lens - n)[:, None] + i                                   # [B][N]
    see = held[:, None] & (key[:, None] <= pos[..., None])
    if w:
        see = see & ((key[:, None] > pos[..., None] - w) | (key[:, None] < s))
    x = (q @ k.transpose(2, 3)).mul_(1.0 / math.sqrt(D)).view(B, Hkv, rep, N, -1)
    x.masked_fill_(~see[:, None, None], float("-inf"))
    x = x.sub_(x.amax(-1, keepdim=True).clamp(min=-3e38)).exp_()
    total = x.sum(-1, keepdim=True)
    o = (x.flatten(2, 3) @ v).view(B, Hkv, rep, N, D) / total.clamp(min=1e-30)
    seq, i, _ = _rows(state)
    return o.permute(0, 3, 1, 2, 4).reshape(B, N, state["Hq"], D)[seq, i].to(torch.bfloat16)


def _plain(state):
    if state["op"] in ("append", "readback"):
        seq, _, pos = _rows(state)
        at = _where(state, seq, pos)
        if state["op"] == "readback":
            return {"rows": _read(state, "k", at).transpose(0, 1).to(torch.bfloat16)}
        _put(state, state["k_codes"], state["k_words"], at, state["k_new"].transpose(0, 1))
        _put(state, state["v_codes"], state["v_words"], at, state["v_new"].transpose(0, 1))
        return {"k": _read(state, "k", at).transpose(0, 1).to(torch.bfloat16),
                "v": _read(state, "v", at).transpose(0, 1).to(torch.bfloat16)}
    return {"out": _attend(state)}


# ---------------------------------------------------------------- the framework's calls

def _kept(state, kvq):
    """The cache objects and the workspace that a serving program makes once."""
    keep = state["keep"]
    if not keep:
        for name in ("k", "v"):
            keep[name] = kvq.QuantCache(state[name + "_codes"], state[name + "_words"], state["bits"],
                                        state["stores"], state["Hkv"], state["slots"], state["D"])
        if state["op"] == "chunk":
            keep["ws"] = kvq.chunk_workspace(state["T"], state["B"], state["Hq"], state["Hkv"], state["D"])
        elif state["op"] == "decode_window":
            keep["ws"] = kvq.decode_workspace(state["B"], state["Hq"], state["Hkv"], state["D"])
    return keep


def _own(state):
    from attention_group_quantized_gb300 import kvq
    keep = _kept(state, kvq)
    k, v, start, lens, table = keep["k"], keep["v"], state["start"], state["lens"], state["table"]
    if state["op"] == "readback":
        if table is None:
            return {"rows": kvq.dequantize(k, start, lens, state["T"], out_dtype=kvq.OUT_BF16)}
        return {"rows": kvq.dequantize_paged(k, table, start, lens, state["T"], out_dtype=kvq.OUT_BF16)}
    if state["op"] == "append":
        if table is None:
            kvq.append_chunk(state["k_new"], state["v_new"], k, v, start, lens)
            return {"k": kvq.dequantize(k, start, lens, state["T"], out_dtype=kvq.OUT_BF16),
                    "v": kvq.dequantize(v, start, lens, state["T"], out_dtype=kvq.OUT_BF16)}
        kvq.append_chunk_paged(state["k_new"], state["v_new"], k, v, table, start, lens)
        return {"k": kvq.dequantize_paged(k, table, start, lens, state["T"], out_dtype=kvq.OUT_BF16),
                "v": kvq.dequantize_paged(v, table, start, lens, state["T"], out_dtype=kvq.OUT_BF16)}
    more = {"window": state["window"], "sinks": state["sinks"], "out_dtype": kvq.OUT_BF16, "workspace": keep["ws"]}
    if state["op"] == "chunk":
        more["max_chunk"] = state["new_max"]
        if table is None:
            return {"out": kvq.chunk_attention(state["q"], k, v, start, lens, **more)}
        return {"out": kvq.chunk_attention_paged(state["q"], k, v, table, start, lens, **more)}
    if table is None:
        return {"out": kvq.decode_attention_window(state["q"], k, v, lens, **more)}
    return {"out": kvq.decode_attention_window_paged(state["q"], k, v, table, lens, **more)}


def run(state):
    return _own(state) if own else _plain(state)


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


def exact(c, seed):
    state = prepare(c, seed)
    new, lens = _lengths(c)
    D, Hkv, T = state["D"], state["Hkv"], state["T"]
    rep = state["Hq"] // Hkv
    if c["op"] == "append":
        got = {}
        for name in ("k", "v"):
            got[name] = torch.stack([_round_trip64(state[name + "_new"][:, h], state["bits"][h]) for h in range(Hkv)], 1)
        return got
    if c["op"] == "readback":
        out = torch.empty(T, Hkv, D, dtype=torch.float64, device="cuda")
    else:
        out = torch.zeros(T, state["Hq"], D, dtype=torch.float64, device="cuda")
    row = 0
    for b, (n, length) in enumerate(zip(new, lens)):
        for h in range(Hkv):
            k = _stored64(state, "k", b, h, length)
            if c["op"] == "readback":
                out[row:row + n, h] = k[length - n:]
                continue
            v = _stored64(state, "v", b, h, length)
            at = 0
            if c["window"]:                                        # tokens before every window, but for the sinks
                at = max(min(c["sinks"], length), length - n - c["window"] + 1)
            take = torch.cat([torch.arange(min(c["sinks"], at)), torch.arange(at, length)]).cuda()
            k, v = k[take], v[take]
            for j in range(rep):
                for i in range(0, n, 512):
                    m = min(512, n - i)
                    q = state["q"][row + i:row + i + m, h * rep + j].double()
                    p = torch.arange(length - n + i, length - n + i + m, device="cuda")[:, None]
                    x = q @ k.T / D ** 0.5
                    hide = take[None] > p
                    if c["window"]:
                        hide |= (take[None] <= p - c["window"]) & (take[None] >= c["sinks"])
                    x[hide] = -math.inf
                    out[row + i:row + i + m, h * rep + j] = torch.softmax(x, 1) @ v
        row += n
    return {("rows" if c["op"] == "readback" else "out"): out}
