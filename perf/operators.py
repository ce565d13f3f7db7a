"""What is measured of the 4-bit KV cache: writing and reading it, attention over it, and moving its pages.

Each case is one call (or the short sequence of calls) that a serving program
makes.  ``own`` false computes it with elementary torch operations in 32 bits;
``own`` true calls ``block_scaled_bit_fp4_amd``.

The cache: ``k_codes`` / ``v_codes`` [layers, pages, heads, page, dim / 2]
(element 2j in the low nibble of byte j), ``k_scales`` / ``v_scales`` [layers,
pages, heads, page, dim / block] (E4M3 per 16 elements and one float32 factor
per layer for nvfp4; E8M0 per 32 elements for mxfp4), both optionally of rows
rotated by the 16-point random Hadamard transform.  A batch: ``page_table``
[sequences, pages of a sequence], ``kv_lens`` (tokens of each sequence, the new
ones included), ``cu_q`` (first new token of each sequence): new token i of a
sequence stands at position kv_len - q_len + i.
"""
import math

import torch

own = False

RHT_SEED = 7
RHT_SIGNS = 0xED90  # the sign mask of that seed: bit j set, element j of a 16-group is negated
LEVELS = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
BLOCK = {"nvfp4": 16, "mxfp4": 32}


# ------------------------------------------------------------------ the cases
def listed():
    return [
        # writing the cache and reading the rows back
        # one new token of each of 32 running sequences, after the fused q, k, v projection
        dict(name="append_tokens", op="append", batch=32, q_len=1, kv_len=2048, ragged=True, heads=32, kv_heads=8,
             dim=128, page=64, fmt="nvfp4", rht=True, dtype="bf16", out="bf16"),
        # the prompts of four sequences, lengths apart and no multiple of a page
        dict(name="append_prompts", op="append", batch=4, q_len=16381, kv_len=16381, ragged=True, heads=32,
             kv_heads=8, dim=128, page=64, fmt="mxfp4", rht=False, dtype="f32", out="f32"),
        # attention, one new token per sequence
        # a single short conversation: the smallest call, latency counts
        dict(name="decode_single_517", op="attention", batch=1, q_len=1, kv_len=517, ragged=False, heads=32,
             kv_heads=8, dim=128, page=64, fmt="nvfp4", rht=True, window=0, sinks=0),
        # an ordinary serving batch, lengths apart
        dict(name="decode_batch_64x8192", op="attention", batch=64, q_len=1, kv_len=8192, ragged=True, heads=32,
             kv_heads=8, dim=128, page=64, fmt="nvfp4", rht=True, window=0, sinks=0),
        # two very long documents
        dict(name="decode_long_2x262144", op="attention", batch=2, q_len=1, kv_len=262144, ragged=False, heads=64,
             kv_heads=8, dim=128, page=128, fmt="mxfp4", rht=False, window=0, sinks=0),
        # streaming: a window and the first tokens, narrow heads
        dict(name="decode_window_48x30011", op="attention", batch=48, q_len=1, kv_len=30011, ragged=True, heads=64,
             kv_heads=8, dim=64, page=16, fmt="mxfp4", rht=True, window=4096, sinks=4),
        # several drafted tokens checked at once, wide heads
        dict(name="draft_5_of_16x4099", op="attention", batch=16, q_len=5, kv_len=4099, ragged=True, heads=16,
             kv_heads=4, dim=256, page=32, fmt="nvfp4", rht=True, window=0, sinks=0),
        # attention, prompts: two whole prompts
        dict(name="prompt_2x4096", op="attention", batch=2, q_len=4096, kv_len=4096, ragged=False, heads=32,
             kv_heads=8, dim=128, page=64, fmt="nvfp4", rht=True, window=0, sinks=0),
        # one chunk of a long prompt under a window with first tokens
        dict(name="chunk_4001_of_16384_window", op="attention", batch=2, q_len=4001, kv_len=16384, ragged=True,
             heads=32, kv_heads=8, dim=128, page=64, fmt="mxfp4", rht=True, window=2048, sinks=16),
        # pages: a few samples of one answer (fork, and giving the forks back)
        dict(name="fork_4", op="fork", layers=4, pages=96, heads=8, dim=128, page=64, fmt="nvfp4", seqs=4, row=16,
             children=4, used=0.5),
        # pages: 256 beams of 64 sequences over all layers
        dict(name="fork_256", op="fork", layers=16, pages=2048, heads=8, dim=128, page=64, fmt="mxfp4", seqs=64,
             row=64, children=256, used=0.5),
        # pages: what fell out of the window is given back, and the pool packed
        dict(name="trim_and_compact", op="compact", layers=16, pages=2048, heads=8, dim=128, page=64, fmt="nvfp4",
             seqs=64, row=64, window=1024, sinks=4, used=0.9),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["append", "attention", "attention", "attention", "fork", "compact"])
    fmt = rng.choice(["nvfp4", "mxfp4"])
    page = rng.choice([16, 32, 64, 128])
    if op == "append":
        batch, kv_heads, dim = _log(rng, 1, 64), rng.choice([1, 2, 4, 8]), rng.choice([64, 128, 256])
        q_len = _log(rng, 1, max(1, (1 << 25) // (batch * kv_heads * dim)))
        q_len = min(q_len, 16384)
        return dict(op="append", batch=batch, q_len=q_len, kv_len=q_len + _log(rng, 1, 4096) - 1, ragged=True,
                    heads=kv_heads * rng.choice([1, 4, 5]), kv_heads=kv_heads, dim=dim, page=page, fmt=fmt,
                    rht=rng.random() < 0.5, dtype=rng.choice(["bf16", "f32"]), out=rng.choice(["bf16", "f32"]))
    if op == "attention":
        dim = rng.choice([64, 128, 128, 256])
        kv_heads = rng.choice([1, 2, 4, 8])
        heads = kv_heads * rng.choice([1, 2, 4, 5, 8])
        window, sinks = rng.choice([(0, 0), (_log(rng, 1, 8192), rng.choice([0, 1, 4, 100]))])
        kind = rng.choice(["single", "few", "prompt"])
        if kind == "single":
            batch = _log(rng, 1, 64)
            kv_len, q_len = _log(rng, 1, min(262144, 400_000_000 // (batch * kv_heads * dim))), 1
        elif kind == "few":
            batch, q_len = _log(rng, 1, 32), rng.randint(2, 17)
            kv_len = q_len + _log(rng, 1, min(32768, (1 << 28) // (batch * kv_heads * dim)))
        else:
            batch, q_len = _log(rng, 1, 4), _log(rng, 18, 4096)
            kv_len = q_len + rng.choice([0, _log(rng, 1, 8192)])
            # at most the pairs of the largest prompt case
            heads = max(kv_heads, min(heads, (1 << 31) // (batch * q_len * kv_len) // kv_heads * kv_heads))
        return dict(op="attention", batch=batch, q_len=q_len, kv_len=kv_len, ragged=rng.random() < 0.7, heads=heads,
                    kv_heads=kv_heads, dim=dim, page=page, fmt=fmt, rht=rng.random() < 0.5, window=window,
                    sinks=sinks)
    layers, heads, dim = _log(rng, 1, 16), rng.choice([1, 4, 8]), rng.choice([64, 128])
    seqs, row = _log(rng, 1, 64), _log(rng, 2, 64)
    pages = min(seqs * row + _log(rng, 8, 512), (1 << 31) // (layers * heads * page * dim))
    if op == "fork":
        return dict(op=op, layers=layers, pages=pages, heads=heads, dim=dim, page=page, fmt=fmt, seqs=seqs, row=row,
                    children=_log(rng, 1, 256), used=rng.uniform(0.2, 0.8))
    return dict(op=op, layers=layers, pages=pages, heads=heads, dim=dim, page=page, fmt=fmt, seqs=seqs, row=row,
                window=_log(rng, 1, row * page), sinks=rng.choice([0, 4, 20]), used=rng.uniform(0.3, 1.0))


def _lengths(case):
    """(new tokens, all tokens) of each sequence: of the case alone, so that its work is known."""
    b = range(case["batch"])
    if not case["ragged"]:
        return [case["q_len"] for _ in b], [case["kv_len"] for _ in b]
    spread = [(i * 40503 % 65536) / 65536 for i in b]  # 0 for the first sequence
    q = [max(1, case["q_len"] - int(f * 0.5 * case["q_len"])) for f in spread]
    kv = [max(n, case["kv_len"] - int((f * 7 % 1) * 0.75 * case["kv_len"])) for f, n in zip(spread, q)]
    return q, kv


def _visible(q, kv, window, sinks):
    """(keys that any of the q last positions sees, pairs of a position and a key it sees)"""
    first = kv - q
    if not window:
        return kv, q * first + q * (q + 1) // 2
    lowest = max(0, first - window + 1)
    pairs = sum(min(p + 1, window + min(sinks, max(0, p + 1 - window))) for p in range(first, kv))
    keys = min(sinks, lowest) + kv - lowest
    return keys, pairs


def work(case):
    row = case["dim"] // 2 + case["dim"] // BLOCK[case["fmt"]]  # bytes of one K or V row in the cache
    if case["op"] == "append":
        n = sum(_lengths(case)[0]) * case["kv_heads"] * 2
        size = {"bf16": 2, "f32": 4}
        return {"bytes": n * (case["dim"] * (size[case["dtype"]] + size[case["out"]]) + 2 * row), "flops": 0}
    if case["op"] == "attention":
        q, kv = _lengths(case)
        seen = [_visible(a, b, case["window"], case["sinks"]) for a, b in zip(q, kv)]
        return {"bytes": sum(k for k, _ in seen) * case["kv_heads"] * 2 * row + sum(q) * case["heads"] * case["dim"] * 4,
                "flops": 4 * case["dim"] * case["heads"] * sum(p for _, p in seen)}
    token = 2 * row * case["heads"] * case["layers"]
    lens = _page_lengths(case)
    if case["op"] == "fork":
        tokens = sum(lens[i % case["seqs"]] % case["page"] for i in range(case["children"]))
        return {"bytes": 2 * tokens * token + 8 * case["children"] * case["row"] + 8 * case["pages"], "flops": 0}
    kept = [_kept(n, case) for n in lens]
    n = sum(len(k) for k in kept)
    # pages lie at random: those past the first n are moved
    return {"bytes": max(1.0, 2 * n * (1 - n / case["pages"])) * case["page"] * token + 8 * case["seqs"] * case["row"]
            + 8 * case["pages"], "flops": 0}


# ----------------------------------------------------- pages of the page cases
def _page_lengths(case):
    """Tokens of each sequence: as many pages in all as the case's share of the pool, the rows at most full."""
    per = max(1, min(case["row"] - 1, int(case["used"] * case["pages"] / case["seqs"])))
    return [max(1, per * case["page"] - (i * 37 % (case["page"] * max(1, per // 2)))) for i in range(case["seqs"])]


def _kept(n, case):
    """Columns of a row of n tokens that hold one of its first `sinks` or last `window` tokens."""
    cols = -(-n // case["page"])
    return [c for c in range(cols) if c * case["page"] < case["sinks"] or (c + 1) * case["page"] > n - case["window"]]


# ------------------------------------------------------------------- plain form
def _stage(t, h):
    g = t.reshape(*t.shape[:-1], 16 // (2 * h), 2, h)
    u, v = g[..., 0, :], g[..., 1, :]
    return torch.stack((u + v, u - v), -2).reshape(t.shape)


def _butterfly(t):
    return _stage(_stage(_stage(_stage(t, 1), 2), 4), 8) * 0.25


def _signs(device):
    bits = (torch.tensor(RHT_SIGNS, device=device) >> torch.arange(16, device=device)) & 1
    return 1.0 - 2.0 * bits.float()


def _rotate(x):
    """The 16-point random Hadamard transform of each aligned 16-group of the last axis, float32."""
    g = x.reshape(*x.shape[:-1], -1, 16)
    return _butterfly(g * _signs(x.device)).reshape(x.shape)


def _rotate_back(y):
    g = y.reshape(*y.shape[:-1], -1, 16)
    return (_butterfly(g) * _signs(y.device)).reshape(y.shape)


def _encode(x, fmt, factor, rht):
    """(codes, scale bytes) of float rows, as the library's quantizer defines them."""
    y = _rotate(x.float()) if rht else x.float()
    b = y.reshape(*y.shape[:-1], -1, BLOCK[fmt])
    amax = b.abs().amax(-1)
    if fmt == "nvfp4":
        s = (amax / (factor * 6.0)).clamp(max=448.0).to(torch.float8_e4m3fn)
        d = factor * s.float()
        inv = torch.where(d > 0, 1.0 / d, torch.zeros_like(d))
        byte = s.view(torch.uint8)
    else:
        e = torch.where(amax > 0, torch.frexp(amax).exponent - 3, torch.full_like(amax, -127).int()).clamp(-127, 127)
        inv = torch.ldexp(torch.ones_like(amax), -e)
        byte = (e + 127).to(torch.uint8)
    v = b * inv[..., None]
    m = v.abs()
    k = torch.where(m < 2, (m * 2).round(), torch.where(m < 4, m.round() + 2, (m * 0.5).round() + 4)).clamp(max=7)
    c = (k.to(torch.uint8) | (torch.signbit(v).to(torch.uint8) << 3)).reshape(*y.shape[:-1], -1, 2)
    return c[..., 0] | (c[..., 1] << 4), byte


def _decode(codes, byte, fmt, factor):
    """The values that codes and scale bytes stand for, float32 (of rotated rows: still rotated)."""
    level = torch.tensor(LEVELS + tuple(-v for v in LEVELS), device=codes.device)
    c = torch.stack((codes & 15, codes >> 4), -1).flatten(-2).int()
    if fmt == "nvfp4":
        d = factor * byte.view(torch.float8_e4m3fn).float()
    else:
        d = torch.ldexp(torch.ones((), device=codes.device), byte.int() - 127)
    v = level[c].reshape(*byte.shape, BLOCK[fmt]) * d[..., None]
    return v.reshape(*codes.shape[:-1], -1)


def _places(s):
    """Pages and offsets of positions 0.. of each sequence up to the longest, and whether each is held."""
    at = torch.arange(s["longest"], device=s["kv_lens"].device)
    page = s["page_table"][:, at // s["page"]].long()
    held = (at < s["kv_lens"][:, None]) & (page >= 0)
    return page.clamp(min=0), (at % s["page"]).expand_as(page), held


def _new_tokens(s):
    """Sequence and position of each new token."""
    t = torch.arange(s["tokens"], device=s["cu_q"].device)
    b = torch.searchsorted(s["cu_q"][1:], t, right=True)
    return b, s["kv_lens"][b] - s["cu_q"][b + 1] + t


def _plain_append(s):
    b, at = _new_tokens(s)
    page, off = s["page_table"][b, at // s["page"]].long(), at % s["page"]
    out = []
    fmt, rht = s["fmt"], s["rht"]

    def one(x, codes, scales, factor):
        c, y = _encode(x, fmt, factor, rht)
        codes[0][page, :, off] = c
        scales[0][page, :, off] = y
        v = _decode(codes[0][page, :, off], scales[0][page, :, off], fmt, factor)
        return (_rotate_back(v) if rht else v).to(s["out"])

    out.append(one(s["k"], s["k_codes"], s["k_scales"], s["k_scale"]))
    out.append(one(s["v"], s["v_codes"], s["v_scales"], s["v_scale"]))
    return out


def _plain_attention(s):
    page, off, held = _places(s)
    fmt = s["fmt"]
    k = _decode(s["k_codes"][0][page, :, off], s["k_scales"][0][page, :, off], fmt, s["k_scale"])  # B, S, H, D
    v = _decode(s["v_codes"][0][page, :, off], s["v_scales"][0][page, :, off], fmt, s["v_scale"])
    k, v = k.transpose(1, 2).contiguous(), v.transpose(1, 2).contiguous()
    batch, heads, _, dim = k.shape
    group = s["q"].shape[1] // heads
    q = s["q"].float()
    q = _rotate(q) if s["rht"] else q
    b, at = _new_tokens(s)
    i = torch.arange(s["tokens"], device=b.device) - s["cu_q"][b]
    pad = torch.zeros(batch, s["q_len"], heads * group, dim, device=q.device)
    pad[b, i] = q
    pos = torch.full((batch, s["q_len"]), -1, device=q.device, dtype=torch.long)
    pos[b, i] = at.long()
    rows = pad.reshape(batch, s["q_len"], heads, group, dim).permute(0, 2, 3, 1, 4).reshape(batch, heads, -1, dim)
    t = torch.matmul(rows, k.transpose(2, 3).contiguous()) * s["scale"]
    t = t.reshape(batch, heads, group, s["q_len"], -1)
    j = torch.arange(s["longest"], device=q.device)
    seen = held[:, None] & (j <= pos[..., None])
    if s["window"]:
        seen = seen & ((j > pos[..., None] - s["window"]) | (j < s["sinks"]))
    t = t.masked_fill(~seen[:, None, None], -math.inf)
    top = t.amax(-1, keepdim=True).clamp(min=-3e38)
    p = (t - top).exp_()
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p.reshape(batch, heads, -1, s["longest"]), v).reshape(batch, heads, group, s["q_len"], dim)
    o = torch.where(total > 0, o / total, torch.zeros_like(o))
    o = o.permute(0, 3, 1, 2, 4).reshape(batch, s["q_len"], heads * group, dim)[b, i]
    return (_rotate_back(o) if s["rht"] else o).to(torch.bfloat16)


def _move(buffer, src, dst, tokens):
    """Page dst[i] takes the first tokens[i] tokens of page src[i], in every layer."""
    some = torch.arange(buffer.shape[3], device=buffer.device) < tokens[:, None]
    buffer[:, dst] = torch.where(some[None, :, None, :, None], buffer[:, src], buffer[:, dst])


def _plain_fork(s):
    table, lens, refs, page = s["table"].clone(), s["lens"].clone(), s["refs"].clone(), s["page"]
    parents, children = s["parents"].long(), s["children"].long()
    n = lens[parents].long()
    full, rem = n // page, n % page
    rows = table[parents]
    col = torch.arange(table.shape[1], device=table.device)
    last = rows.gather(1, full.clamp(max=table.shape[1] - 1)[:, None])[:, 0].long()
    need = (rem > 0) & (last >= 0)
    rank = torch.cumsum(need.long(), 0) - 1
    free = torch.argsort((refs > 0).int(), stable=True)
    ok = ~need | (rank < (refs == 0).sum())
    new = free[rank.clamp(min=0, max=refs.numel() - 1)]
    copied = need & ok
    shared = ok[:, None] & (col < full[:, None]) & (rows >= 0)
    refs.index_add_(0, rows.clamp(min=0).long().reshape(-1), shared.reshape(-1).to(refs.dtype))
    out = torch.where(shared, rows, torch.full_like(rows, -1))
    out = torch.where((col == full[:, None]) & copied[:, None], new[:, None].to(rows.dtype), out)
    table[children] = out
    lens[children] = torch.where(ok, n, torch.zeros_like(n)).to(lens.dtype)
    refs[new[copied]] = 1
    _move(s["k_codes"], last[copied], new[copied], rem[copied])
    _move(s["k_scales"], last[copied], new[copied], rem[copied])
    _move(s["v_codes"], last[copied], new[copied], rem[copied])
    _move(s["v_scales"], last[copied], new[copied], rem[copied])
    forked = table.clone(), lens.clone(), refs.clone()
    _plain_free(table, lens, refs, children, page, 0, 0)
    return [*forked, refs, s["k_codes"], s["k_scales"], s["v_codes"], s["v_scales"]]


def _plain_free(table, lens, refs, seqs, page, window, sinks):
    rows, n = table[seqs], lens[seqs].long()[:, None]
    col = torch.arange(table.shape[1], device=table.device)
    gone = rows >= 0
    if window:
        gone = gone & (col * page >= sinks) & ((col + 1) * page <= n - window)
    refs.index_add_(0, rows.clamp(min=0).long().reshape(-1), -gone.reshape(-1).to(refs.dtype))
    table[seqs] = torch.where(gone, torch.full_like(rows, -1), rows)
    if not window:
        lens[seqs] = 0


def _plain_compact(s):
    table, lens, refs, page = s["table"].clone(), s["lens"].clone(), s["refs"].clone(), s["page"]
    _plain_free(table, lens, refs, s["seqs"].long(), page, s["window"], s["sinks"])
    used = refs > 0
    ids = torch.arange(refs.numel(), device=refs.device)
    n = used.sum()
    moved = used & (ids >= n)
    order = torch.argsort(used.int(), stable=True)  # the free pages first, ascending
    to = order[(torch.cumsum(moved.long(), 0) - 1).clamp(min=0)]
    place = torch.where(moved, to, torch.where(used, ids, torch.full_like(ids, -1)))
    src, dst = ids[moved], place[moved]
    s["k_codes"][:, dst] = s["k_codes"][:, src]
    s["k_scales"][:, dst] = s["k_scales"][:, src]
    s["v_codes"][:, dst] = s["v_codes"][:, src]
    s["v_scales"][:, dst] = s["v_scales"][:, src]
    table = torch.where(table >= 0, place[table.clamp(min=0).long()], torch.full_like(ids[:1], -1)).int()
    packed = torch.zeros_like(refs)
    packed[place[used]] = refs[used]
    return [table, packed, place.int(), n.int().reshape(1), s["k_codes"], s["k_scales"], s["v_codes"], s["v_scales"]]


# -------------------------------------------------------------------- one pass
def run(s):
    if not own:
        return {"append": _plain_append, "attention": _plain_attention, "fork": _plain_fork,
                "compact": _plain_compact}[s["op"]](s)
    import block_scaled_bit_fp4_amd as fp4

    cache = fp4.KVCache(s["k_codes"], s["k_scales"], s["v_codes"], s["v_scales"], s.get("k_scale"), s.get("v_scale"),
                        s["fmt"], s.get("rht", False), RHT_SEED)
    if s["op"] == "append":
        batch = fp4.KVBatch(s["page_table"], s["kv_lens"], s["cu_q"], s["q_len"])
        fp4.kv_append(cache, s["k"], s["v"], batch)
        return list(fp4.kv_gather(cache, batch, s["tokens"], out_dtype=s["out"]))
    if s["op"] == "attention":
        batch = fp4.KVBatch(s["page_table"], s["kv_lens"], s["cu_q"], s["q_len"], s["longest"])
        return fp4.kv_attention(s["q"], cache, batch, scale=s["scale"], window=s["window"], sinks=s["sinks"])
    table, lens, refs = s["table"].clone(), s["lens"].clone(), s["refs"].clone()
    if s["op"] == "fork":
        fp4.kv_fork(cache, table, lens, refs, s["parents"], s["children"])
        forked = table.clone(), lens.clone(), refs.clone()
        fp4.kv_free(table, lens, refs, s["children"], s["page"])
        return [*forked, refs, s["k_codes"], s["k_scales"], s["v_codes"], s["v_scales"]]
    fp4.kv_free(table, lens, refs, s["seqs"], s["page"], window=s["window"], sinks=s["sinks"])
    place, n = fp4.kv_compact(cache, table, refs)
    return [table, refs, place, n, s["k_codes"], s["k_scales"], s["v_codes"], s["v_scales"]]


# ---------------------------------------------------------------------- inputs
def _rows(g, batch, n, heads, dim):
    """Keys or values of running text: normal, a few channels of each head five times larger."""
    x = torch.randn(batch, n, heads, dim, generator=g, device="cuda")
    gain = 1.0 + 4.0 * (torch.rand(heads, dim, generator=g, device="cuda") < 0.03)
    return x * gain


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    page, dim, fmt = case["page"], case["dim"], case["fmt"]
    s = {"op": case["op"], "page": page, "fmt": fmt}
    if case["op"] in ("fork", "compact"):
        return _prepare_pages(case, s, g)
    q_lens, kv_lens = _lengths(case)
    batch, heads, kv_heads = case["batch"], case["heads"], case["kv_heads"]
    longest, row = max(kv_lens), -(-max(kv_lens) // page)
    used = [-(-n // page) for n in kv_lens]
    pages = sum(used) + 3
    ids = torch.randperm(pages, generator=g, device="cuda")[: sum(used)]
    first = torch.tensor([sum(used[:i]) for i in range(batch)], device="cuda")
    col = torch.arange(row, device="cuda")
    count = torch.tensor(used, device="cuda")
    table = torch.where(col < count[:, None], ids[(first[:, None] + col).clamp(max=len(ids) - 1)], -1)
    cu = [0]
    for n in q_lens:
        cu.append(cu[-1] + n)
    s |= dict(page_table=table.int().contiguous(), kv_lens=torch.tensor(kv_lens, device="cuda", dtype=torch.int32),
              cu_q=torch.tensor(cu, device="cuda", dtype=torch.int32), tokens=cu[-1], q_len=max(q_lens),
              longest=longest, rht=case["rht"])
    # the layer's factors come from a calibration: the largest rotated value maps to the top of the format
    s["k_scale"] = torch.full((1,), 24.0 / (6 * 448), device="cuda")
    s["v_scale"] = torch.full((1,), 24.0 / (6 * 448), device="cuda")
    shape = (1, pages, kv_heads, page)
    for name in ("k", "v"):
        s[name + "_codes"] = torch.zeros(*shape, dim // 2, dtype=torch.uint8, device="cuda")
        s[name + "_scales"] = torch.zeros(*shape, dim // BLOCK[fmt], dtype=torch.uint8, device="cuda")
    if case["op"] == "append":
        dtype = {"bf16": torch.bfloat16, "f32": torch.float32}
        # one row of the fused projection: the queries' part, then keys, then values
        x = _rows(g, 1, cu[-1], heads + 2 * kv_heads, dim)[0].to(dtype[case["dtype"]])
        s |= dict(k=x[:, heads:heads + kv_heads], v=x[:, heads + kv_heads:], out=dtype[case["out"]])
        return s
    for name in ("k", "v"):
        for b in range(batch):  # a sequence at a time: a long one has 32-bit copies of several GB
            n = used[b] * page
            c, y = _encode(_rows(g, 1, n, kv_heads, dim)[0], fmt, s[name + "_scale"], case["rht"])
            at = table[b, : used[b]].long()
            s[name + "_codes"][0, at] = c.reshape(used[b], page, kv_heads, -1).transpose(1, 2)
            s[name + "_scales"][0, at] = y.reshape(used[b], page, kv_heads, -1).transpose(1, 2)
    q = torch.randn(cu[-1], heads + 2 * kv_heads, dim, generator=g, device="cuda") * 1.5
    s |= dict(q=q.to(torch.bfloat16)[:, :heads], scale=1.0 / math.sqrt(dim), window=case["window"],
              sinks=case["sinks"])
    return s


def _prepare_pages(case, s, g):
    page, pages, seqs, row = case["page"], case["pages"], case["seqs"], case["row"]
    lens = _page_lengths(case)
    children = case.get("children", 0)
    used = [-(-n // page) for n in lens]
    ids = torch.randperm(pages, generator=g, device="cuda")
    count = torch.tensor(used + [0] * children, device="cuda")[:, None]
    col = torch.arange(row, device="cuda")
    at = sum(used)
    place = (torch.cumsum(count, 0) - count + col).clamp(max=pages - 1)
    table = torch.where(col < count, ids[place], -1).int().contiguous()
    refs = torch.zeros(pages, dtype=torch.int32, device="cuda")
    refs[ids[:at]] = 1
    s |= dict(table=table, refs=refs, lens=torch.tensor(lens + [0] * children, dtype=torch.int32, device="cuda"))
    shape = (case["layers"], pages, case["heads"], page)
    for name in ("k", "v"):
        for part, n in (("_codes", case["dim"] // 2), ("_scales", case["dim"] // BLOCK[case["fmt"]])):
            s[name + part] = torch.randint(0, 256, (*shape, n), generator=g, device="cuda", dtype=torch.uint8)
    if case["op"] == "fork":
        s["parents"] = (torch.arange(children, device="cuda") % seqs).int()
        s["children"] = (seqs + torch.randperm(children, generator=g, device="cuda")).int()
    else:
        s |= dict(seqs=torch.arange(seqs, device="cuda").int(), window=case["window"], sinks=case["sinks"])
    return s


# -------------------------------------------------------- the definition in 64 bits
def _hadamard(device):
    """diag(signs), then the Sylvester matrix over 4: a row times this is its transform."""
    i = torch.arange(16)
    parity = sum(((i[:, None] & i[None]) >> k) & 1 for k in range(4)) % 2
    sign = 1 - 2 * ((RHT_SIGNS >> i) & 1)
    return (sign[:, None] * (1 - 2 * parity) / 4.0).double().to(device)


def _values64(codes, byte, case, factor):
    """The rows that pages hold, in the basis they came in, float64."""
    grid = torch.tensor(LEVELS, dtype=torch.float64, device=codes.device)
    low, high = codes.int() & 15, codes.int() >> 4
    v = torch.zeros(*codes.shape[:-1], 2 * codes.shape[-1], dtype=torch.float64, device=codes.device)
    v[..., 0::2] = grid[low & 7] * (1 - (low >> 3) * 2)
    v[..., 1::2] = grid[high & 7] * (1 - (high >> 3) * 2)
    e = byte.int()
    if case["fmt"] == "nvfp4":
        m, x = (e & 7).double(), e >> 3
        d = torch.where(x > 0, (1 + m / 8) * 2.0 ** (x - 7).double(), m * 2.0 ** -9) * float(factor)
    else:
        d = 2.0 ** (e - 127).double()
    v = v * d.repeat_interleave(BLOCK[case["fmt"]], -1)
    return (v.unflatten(-1, (-1, 16)) @ _hadamard(v.device).T).flatten(-2) if case["rht"] else v


def _rounded64(x, case, factor):
    """The values that rows stand for after the write, float64."""
    h = _hadamard(x.device)
    y = x.double()
    y = (y.unflatten(-1, (-1, 16)) @ h).flatten(-2) if case["rht"] else y
    b = y.unflatten(-1, (-1, BLOCK[case["fmt"]]))
    amax = b.abs().amax(-1, keepdim=True)
    if case["fmt"] == "nvfp4":
        r = amax / (6 * float(factor))
        step = 2.0 ** (torch.floor(torch.log2(r.clamp(min=2.0 ** -6))) - 3)
        d = torch.clamp(torch.round(r / step) * step, max=448.0) * float(factor)
    else:
        d = 2.0 ** (torch.floor(torch.log2(amax.clamp(min=2.0 ** -125))) - 2)
    m = torch.where(d > 0, b.abs() / d, torch.zeros_like(b))
    k = ((m > 0.25).int() + (m >= 0.75).int() + (m > 1.25).int() + (m >= 1.75).int() + (m > 2.5).int()
         + (m >= 3.5).int() + (m > 5).int())
    v = (torch.tensor(LEVELS, dtype=torch.float64, device=x.device)[k] * torch.sign(b) * d).flatten(-2)
    return (v.unflatten(-1, (-1, 16)) @ h.T).flatten(-2) if case["rht"] else v


def exact(case, seed):
    if case["op"] in ("fork", "compact"):
        return None  # bytes and whole numbers
    s = prepare(case, seed)
    if case["op"] == "append":
        return [_rounded64(s["k"], case, s["k_scale"]), _rounded64(s["v"], case, s["v_scale"])]
    q_lens, kv_lens = _lengths(case)
    group = case["heads"] // case["kv_heads"]
    out = torch.empty(s["tokens"], case["heads"], case["dim"], dtype=torch.float64, device="cuda")
    first = 0
    for b, (nq, nk) in enumerate(zip(q_lens, kv_lens)):
        at = s["page_table"][b, : -(-nk // case["page"])].long()
        p = torch.arange(nk - nq, nk, device="cuda")[:, None]
        j = torch.arange(nk, device="cuda")[None]
        dark = j > p
        if case["window"]:
            dark = dark | ((j <= p - case["window"]) & (j >= case["sinks"]))
        for h in range(case["kv_heads"]):
            k = _values64(s["k_codes"][0, at, h], s["k_scales"][0, at, h], case, s["k_scale"]).flatten(0, 1)[:nk]
            v = _values64(s["v_codes"][0, at, h], s["v_scales"][0, at, h], case, s["v_scale"]).flatten(0, 1)[:nk]
            for i in range(h * group, (h + 1) * group):
                x = (s["q"][first: first + nq, i].double() @ k.T) * s["scale"]
                out[first: first + nq, i] = torch.softmax(x.masked_fill(dark, -math.inf), -1) @ v
        first += nq
    return out
