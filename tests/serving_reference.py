"""What the rotated append, the block bounds, the selection and the page calls are defined to give, in numpy on the CPU.

Values that the definitions round are rounded as they say (np.float32 arithmetic rounds every operation once); the rest is
64 bits.  The page table is a plain Python model."""
import numpy as np

from oracle import kvq_oracle as O

F = np.float32


def bf16_bits(x):
    """float32 -> bf16 bit patterns, round to nearest even (finite values)."""
    u = np.ascontiguousarray(x, F).view(np.uint32).astype(np.uint64)
    return ((u + 0x7FFF + ((u >> 16) & 1)) >> 16).astype(np.uint16)


def bf16_values(bits):
    return (np.ascontiguousarray(bits, np.uint16).astype(np.uint32) << 16).view(F)


def turn(x, weight, table, pos, eps, interleaved):
    """Rows x [T][heads][D] (bf16 bits), normed and rotated at positions pos [T]: (bf16 bits as defined, the formula's
    64-bit values, the size of the terms that each value is the sum of)."""
    y = bf16_values(x)
    z = y.astype(np.float64)
    if weight is not None:
        w = bf16_values(weight)
        mean64 = (z * z).mean(-1, keepdims=True)
        with np.errstate(over="ignore"):
            mean = mean64.astype(F)
        r = F(1) / np.sqrt(mean + F(eps))
        y = (y * r) * w
        z = z / np.sqrt(mean64 + np.float64(F(eps))) * w.astype(np.float64)
    size = np.abs(z)
    if table is not None:
        rot = table.shape[1]
        h = rot // 2
        c, s = table[pos, :h][:, None], table[pos, h:][:, None]
        i = np.arange(h)
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + h)
        y, z, size = y.copy(), z.copy(), size.copy()
        ya, yb, za, zb = y[..., a], y[..., b], z[..., a], z[..., b]
        y[..., a], y[..., b] = ya * c - yb * s, yb * c + ya * s
        size[..., a] = np.abs(za * c) + np.abs(zb * s)
        size[..., b] = np.abs(zb * c) + np.abs(za * s)
        z[..., a], z[..., b] = za * c - zb * s, zb * c + za * s
    return bf16_bits(y), z, size


def bounds(k, tokens):
    """Codes [Hkv][blocks][G][2][32] and scales [Hkv][blocks][G] of stored values k [Hkv][len][D] (64 bits, exact in 32),
    blocks of 64 tokens, the last one cut at len = tokens."""
    Hkv, _, D = k.shape
    n = -(-tokens // 64)
    codes = np.zeros((Hkv, n, D // 32, 2, 32), np.int8)
    scales = np.zeros((Hkv, n, D // 32), F)
    for i in range(n):
        x = k[:, 64 * i:min(64 * i + 64, tokens)].astype(F)
        hi = x.max(1).reshape(Hkv, -1, 32)
        lo = x.min(1).reshape(Hkv, -1, 32)
        a = np.maximum(np.abs(hi), np.abs(lo)).max(-1)
        s = a / F(127)
        u = np.where(s > 0, s, F(1))[..., None]
        codes[:, i, :, 0] = np.clip(np.ceil(hi / u), -127, 127)
        codes[:, i, :, 1] = np.clip(np.floor(lo / u), -127, 127)
        scales[:, i] = s
    return codes, scales


def scores(q, codes, scales):
    """Scores [Hkv][blocks] of one row's queries q [Hq][D] (float32) over bounds [Hkv][blocks][G][2][32]."""
    Hkv, n, G, _, _ = codes.shape
    rep = q.shape[0] // Hkv
    up = np.zeros((Hkv, G * 32), F)
    down = np.zeros((Hkv, G * 32), F)
    for r in range(rep):
        up = up + np.maximum(q[r::rep], F(0))
        down = down + np.minimum(q[r::rep], F(0))
    up, down = up.reshape(Hkv, G, 32), down.reshape(Hkv, G, 32)
    u = np.maximum(up, -down).max(-1) / F(127)
    div = np.where(u > 0, u, F(1))[..., None]
    cp, cn = np.rint(up / div).astype(np.int64), np.rint(down / div).astype(np.int64)
    c = codes.astype(np.int64)
    dots = (c[:, :, :, 0] * cp[:, None] + c[:, :, :, 1] * cn[:, None]).sum(-1)      # [Hkv][n][G]
    t = (u[:, None] * scales) * dots.astype(F)
    score = t[..., 0]
    for g in range(1, G):
        score = score + t[..., g]
    return score


def select(score, n_select, first, last):
    """The selected blocks of scores [blocks], ascending, padded with -1."""
    n = len(score)
    forced = (np.arange(n) < first) | (np.arange(n) >= n - last)
    order = sorted(range(n), key=lambda i: (not forced[i], -float(score[i]), i))
    got = sorted(order[:n_select])
    return np.array(got + [-1] * (n_select - len(got)), np.int32)


def attend(q, k, v, blocks, tokens, scale):
    """softmax over the tokens below `tokens` of the listed blocks: q [D], k and v [len][D], 64 bits."""
    at = [t for i in blocks if i >= 0 for t in range(64 * i, min(64 * i + 64, tokens))]
    if not at:
        return np.zeros(v.shape[1])
    s = k[at] @ q * scale
    p = np.exp(s - s.max())
    return (p / p.sum()) @ v[at]


def stored(x, head_bits):
    """bf16 bits x [Hkv][T][D] -> the values that their codes stand for (64 bits)."""
    return np.stack([O.dequantize(*O.quantize_groups(x[h], int(head_bits[h]))) for h in range(len(head_bits))])


class Pages:
    """The page calls on lists.  `data` maps a page to what it holds."""

    def __init__(self, n_pages, slots, max_pages):
        self.refs = [0] * n_pages
        self.table = [[0] * max_pages for _ in range(slots)]
        self.lens = [0] * slots
        self.max_pages = max_pages
        self.data = list(range(n_pages))
        self.status = 0

    def _report(self, code):
        self.status = self.status or code

    def _free_list(self):
        return [p for p, r in enumerate(self.refs) if r == 0]

    def reserve(self, add):
        free, out = self._free_list(), False
        codes = []
        for s, a in enumerate(add):
            n = self.lens[s]
            if a < 0 or n < 0 or n + a > 64 * self.max_pages:
                codes.append(1)
                continue
            have, need = -(-n // 64), -(-(n + a) // 64) - -(-n // 64)
            if need and (out or need > len(free)):
                out = True
                codes.append(8)
                continue
            for j in range(need):
                p = free.pop(0)
                self.table[s][have + j] = p
                self.refs[p] = 1
            self.lens[s] = n + a
        for c in codes:
            self._report(c)
        return set(codes)

    def fork(self, src, dst):
        free, lens, taken, out = self._free_list(), list(self.lens), set(), False
        codes = []
        for f, t in zip(src, dst):
            S = len(lens)
            if not (0 <= f < S and 0 <= t < S) or lens[t] != 0 or not 0 <= lens[f] <= 64 * self.max_pages or t in taken:
                codes.append(1)
                continue
            taken.add(t)
            n = lens[f]
            full = n // 64
            if n % 64:
                if out or not free:
                    out = True
                    codes.append(8)
                    continue
                p = free.pop(0)
                self.data[p] = self.data[self.table[f][full]]
                self.table[t][full] = p
                self.refs[p] = 1
            for j in range(full):
                self.table[t][j] = self.table[f][j]
                self.refs[self.table[f][j]] += 1
            self.lens[t] = n
        return set(codes)

    def free(self, slots):
        codes = []
        for s in slots:
            if not 0 <= s < len(self.lens):
                codes.append(1)
                continue
            for j in range(-(-self.lens[s] // 64)):
                self.refs[self.table[s][j]] -= 1
            self.lens[s] = 0
        return set(codes)

    def compact(self):
        live = [p for p, r in enumerate(self.refs) if r > 0]
        n = len(live)
        move = dict(zip([p for p in live if p >= n], [p for p, r in enumerate(self.refs) if r == 0 and p < n]))
        for a, b in move.items():
            self.data[b] = self.data[a]
            self.refs[b], self.refs[a] = self.refs[a], 0
        for s, row in enumerate(self.table):
            for j in range(-(-self.lens[s] // 64)):
                row[j] = move.get(row[j], row[j])
        return n
