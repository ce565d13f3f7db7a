"""The 4-bit KV cache in plain numpy: places of tokens, rows in 64 bits from
their bytes, attention by its formula, and the page moves by loops over
Python lists.  Used by the cache's tests only; shares no code with the HIP
library (rows are quantized by the oracle)."""
import math

import numpy as np

import oracle
import workloads

BLOCK = {"nvfp4": 16, "mxfp4": 32, "mxfp4_oas": 32}
LEVELS = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def hadamard(seed):
    """Row vector times this = its 16-point RHT."""
    signs = oracle.rht_signs(seed)
    h = np.array([[(-1.0) ** bin(i & j).count("1") for j in range(16)] for i in range(16)])
    d = np.array([-1.0 if signs >> i & 1 else 1.0 for i in range(16)])
    return d[:, None] * h / 4.0


def quantize_rows(x, fmt, factor, rht, seed):
    """(codes, scales) of rows [..., D] (uint16 BF16 bits or float32)."""
    flat = np.ascontiguousarray(x.reshape(-1, x.shape[-1]))
    c, s, _ = oracle.quantize(flat, fmt, "row", "rtne", rht, seed, 0,
                              tensor_scale=factor if fmt == "nvfp4" else None)
    return c.reshape(*x.shape[:-1], -1), s.reshape(*x.shape[:-1], -1)


def values(codes, scales, fmt, factor, rht, seed):
    """Rows [..., D] that bytes stand for, float64, rotation undone."""
    c = np.stack((codes & 15, codes >> 4), -1).reshape(*codes.shape[:-1], -1).astype(int)
    v = LEVELS[c & 7] * np.where(c & 8, -1.0, 1.0)
    s = scales.astype(int)
    if fmt == "nvfp4":
        e, m = s >> 3, (s & 7).astype(float)
        d = np.where(e == 0, m * 2.0 ** -9, (1 + m / 8) * 2.0 ** (e - 7.0)) * float(np.float32(factor))
    else:
        d = 2.0 ** (s - 127.0)
    v = (v.reshape(*scales.shape, -1) * d[..., None]).reshape(v.shape)
    if rht:
        v = (v.reshape(*v.shape[:-1], -1, 16) @ hadamard(seed).T).reshape(v.shape)
    return v


def visible(p, kv_len, window, sinks):
    """Positions that a token at position p sees (a boolean of kv_len)."""
    j = np.arange(kv_len)
    see = j <= p
    if window:
        see &= (j > p - window) | (j < sinks)
    return see


def attention(q, k, v, q_len, window, sinks, scale, held=None):
    """q [q_len, Hq, D], k, v [kv_len, H, D] float64 -> (out, lse, bounds).

    bounds[t, h, d] is what the kernels' roundings may move an output by, per
    unit of: (score) |delta s| <= 1 for each score, (prob) a relative error
    of 1 of each probability."""
    n, hq, dim = q.shape
    kv_len, heads = k.shape[:2]
    out = np.zeros((n, hq, dim))
    lse = np.full((n, hq), -np.inf)
    mean = np.zeros((n, hq, dim))   # sum_j w_j |v_j|
    dot = np.zeros((n, hq))         # max_j scale * <|q|, |k_j|>
    floor = np.zeros((n, hq, dim))  # sum_j |v_j| over visible keys
    for t in range(n):
        see = visible(kv_len - q_len + t, kv_len, window, sinks)
        if held is not None:
            see = see & held
        if not see.any():
            continue
        for h in range(hq):
            kk, vv = k[see, h * heads // hq], v[see, h * heads // hq]
            s = kk @ q[t, h] * scale
            m = s.max()
            w = np.exp(s - m)
            lse[t, h] = m + math.log(w.sum())
            w /= w.sum()
            out[t, h] = w @ vv
            mean[t, h] = w @ np.abs(vv)
            dot[t, h] = (np.abs(kk) @ np.abs(q[t, h])).max() * abs(scale)
            floor[t, h] = np.abs(vv).sum(0)
    return out, lse, (mean, dot, floor)


class Case:
    """A random cache with sequences in it: bytes as the oracle quantizes them,
    every place that no token holds poisoned (0xFF: NaN scales)."""

    def __init__(self, fmt, dim, page, heads, lens, seed, rht=False, spare=3, factor=24 / 2688.0,
                 rht_seed=5, layers=1, layer=0, spread=1.0, columns=None, bf16=True):
        rng = np.random.default_rng(seed)
        self.fmt, self.dim, self.page, self.heads, self.lens = fmt, dim, page, heads, list(lens)
        self.rht, self.rht_seed, self.factor = rht, rht_seed, factor
        self.layers, self.layer = layers, layer
        used = [-(-max(n, 0) // page) for n in lens]
        self.pages = sum(used) + spare
        cols = max(used + [1]) + 1 if columns is None else columns
        ids = rng.permutation(self.pages)[: sum(used)]
        self.table = np.full((len(lens), cols), -1, np.int32)
        at = 0
        for b, n in enumerate(used):
            self.table[b, :n] = ids[at: at + n]
            at += n
        half, nsc = dim // 2, dim // BLOCK[fmt]
        shape = (layers, self.pages, heads, page)
        self.codes = {x: np.full(shape + (half,), 0xFF, np.uint8) for x in "kv"}
        self.scales = {x: np.full(shape + (nsc,), 0xFF, np.uint8) for x in "kv"}
        self.rows = {}  # (x, sequence): BF16 bits or float32 [len, heads, dim]
        for x in "kv":
            for b, n in enumerate(lens):
                a = rng.standard_normal((n, heads, dim)) * spread
                a[..., rng.integers(0, dim)] *= 6.0
                r = workloads.to_bf16_bits(a) if bf16 else a.astype(np.float32)
                self.rows[x, b] = r

    def place(self, b, t):
        return int(self.table[b, t // self.page]), t % self.page

    def fill(self, upto=None):
        """Write the tokens (of sequence b the first upto[b]) into the bytes."""
        for x in "kv":
            for b, n in enumerate(self.lens):
                m = n if upto is None else upto[b]
                if not m:
                    continue
                c, s = quantize_rows(self.rows[x, b][:m], self.fmt, self.factor, self.rht, self.rht_seed)
                for t in range(m):
                    pg, off = self.place(b, t)
                    if pg < 0:
                        continue
                    self.codes[x][self.layer, pg, :, off] = c[t]
                    self.scales[x][self.layer, pg, :, off] = s[t]
        return self

    def read(self, x, b):
        """Rows of a sequence from the bytes, float64 [len, heads, dim]."""
        n = self.lens[b]
        out = np.zeros((n, self.heads, self.dim))
        for t in range(n):
            pg, off = self.place(b, t)
            if pg >= 0:
                out[t] = values(self.codes[x][self.layer, pg, :, off], self.scales[x][self.layer, pg, :, off],
                                self.fmt, self.factor, self.rht, self.rht_seed)
        return out


# ------------------------------------------------------------------ page moves
def fork(table, lens, refs, parents, children, page):
    """Lists of moves (src, dst, tokens) and the forks that failed; the tables
    (numpy arrays) are changed in place."""
    free = [i for i in range(len(refs)) if refs[i] == 0]
    moves, failed = [], 0
    plan = []
    for p, c in zip(parents, children):
        full, rem = divmod(int(lens[p]), page)
        last = int(table[p, full]) if rem else -1
        if rem and last >= 0:
            if not free:
                failed += 1
                plan.append((p, c, None))
                continue
            new = free.pop(0)
            moves.append((last, new, rem))
            plan.append((p, c, new))
        else:
            plan.append((p, c, -1))
    rows, ns = table.copy(), lens.copy()
    for p, c, new in plan:
        table[c] = -1
        lens[c] = 0
        if new is None:
            continue
        full = int(ns[p]) // page
        lens[c] = ns[p]
        for j in range(full):
            if rows[p, j] >= 0:
                table[c, j] = rows[p, j]
                refs[rows[p, j]] += 1
        if new >= 0:
            table[c, full] = new
            refs[new] = 1
    return moves, failed


def free(table, lens, refs, seqs, page, window, sinks):
    for s in seqs:
        for c in range(table.shape[1]):
            if table[s, c] < 0:
                continue
            if window and (c * page < sinks or (c + 1) * page > lens[s] - window):
                continue
            refs[table[s, c]] -= 1
            table[s, c] = -1
        if not window:
            lens[s] = 0


def compact(table, refs):
    n = int((refs > 0).sum())
    holes = [i for i in range(n) if refs[i] <= 0]
    movers = [i for i in range(n, len(refs)) if refs[i] > 0]
    place = np.where(refs > 0, np.arange(len(refs)), -1).astype(np.int32)
    for s, d in zip(movers, holes):
        place[s] = d
        refs[d], refs[s] = refs[s], 0
    for r in table:
        for c in range(len(r)):
            r[c] = place[r[c]] if r[c] >= 0 else -1
    return list(zip(movers, holes)), place, n
