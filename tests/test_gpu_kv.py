"""The 4-bit KV cache on the GPU against plain numpy in 64 bits.

Writing is compared byte for byte with the oracle's quantizer; reading within
the inverse transform's binary32 rounding.  Attention is held to a bound
that follows from the roundings the kernels make (tests/kv_ref.py gives the
sums it multiplies):

- a score is a binary32 sum of D exact products of K with a q that has been
  rounded: not at all without the transform (FP16 takes BF16's 8 bits after a
  power-of-two scaling of the row; what falls under FP16's smallest step is
  below 2^-24 of the row's largest), by 2^-11 relative in FP16 and 2^-16 in
  two BF16 parts with it (rotation in binary32 included):
  |ds| <= (e_q + D * 2^-23) * max_j scale * <|q|, |K_j|>;
- a probability rounds by e_p = 2^-11 (FP16) or 2^-8 (BF16), exp2 and its
  argument by 2^-20 * (1 + |s| * 2^-4), and one that is below 2^-14 of the
  largest loses up to 2^-24 of it in FP16;
- the sums over N keys round by N * 2^-23.
A relative error e of every weight moves a weighted mean of V by at most
2 e sum_j w_j |v_j|.  The result's own rounding adds 2^-8 of it in BF16."""
import numpy as np
import pytest
import torch

import block_scaled_bit_fp4_amd as fp4
from tests import kv_ref
from tests.gpu_util import DEV, assert_bytes_equal, note, to_device, to_host

pytestmark = pytest.mark.gpu


def ints(a):
    return torch.tensor(np.asarray(a, dtype=np.int32), device=DEV)


def device_cache(c):
    f = c.factor if c.fmt == "nvfp4" else None
    k = torch.full((c.layers,), float("nan"), device=DEV)
    if f is not None:
        k[c.layer] = f
    return fp4.KVCache(to_device(c.codes["k"].copy()), to_device(c.scales["k"].copy()),
                       to_device(c.codes["v"].copy()), to_device(c.scales["v"].copy()),
                       k if f is not None else None, k.clone() if f is not None else None, c.fmt,
                       c.rht, c.rht_seed)


def device_batch(c, q_lens, max_q=None, max_kv=0):
    cu = np.concatenate(([0], np.cumsum(q_lens)))
    return fp4.KVBatch(ints(c.table), ints(c.lens), ints(cu),
                       max([1, *q_lens]) if max_q is None else max_q, max_kv)


def new_rows(c, x, q_lens):
    return np.concatenate([c.rows[x, b][len(c.rows[x, b]) - n:] for b, n in enumerate(q_lens)])


# --------------------------------------------------------------- write and read
@pytest.mark.parametrize("fmt,rht", [("nvfp4", True), ("nvfp4", False), ("mxfp4", True),
                                     ("mxfp4_oas", False), ("mxfp4_oas", True)])
@pytest.mark.parametrize("dim,page,heads,lens,q_lens", [
    (64, 16, 3, [1, 17, 40], [1, 5, 40]),
    (128, 64, 2, [64, 63, 0, 130], [64, 1, 0, 129]),
    (256, 32, 1, [33], [2]),
])
@pytest.mark.parametrize("bf16", [True, False])
def test_append_and_gather(fmt, rht, dim, page, heads, lens, q_lens, bf16):
    note("kv append %s rht=%s dim %d page %d bf16=%s" % (fmt, rht, dim, page, bf16))
    c = kv_ref.Case(fmt, dim, page, heads, lens, 11, rht=rht, layers=2, layer=1, bf16=bf16)
    before = [n - m for n, m in zip(lens, q_lens)]
    c.fill(before)
    cache, batch = device_cache(c), device_batch(c, q_lens)
    # keys and values as views of one wider tensor: strides that are not dense
    k, v = to_device(new_rows(c, "k", q_lens)), to_device(new_rows(c, "v", q_lens))
    both = torch.cat((torch.zeros_like(k), k, v), 1)
    fp4.kv_append(cache, both[:, heads:2 * heads], both[:, 2 * heads:], batch, layer=1)
    got = fp4.kv_gather(cache, batch, sum(q_lens), layer=1, out_dtype=torch.float32)
    half = fp4.kv_gather(cache, batch, sum(q_lens), layer=1)
    torch.cuda.synchronize()
    c.fill()
    for x, codes, scales in (("k", cache.k_codes, cache.k_scales), ("v", cache.v_codes, cache.v_scales)):
        assert_bytes_equal(to_host(scales), c.scales[x], "scales of " + x)
        assert_bytes_equal(to_host(codes), c.codes[x], "codes of " + x)
    for x, g, h in (("k", got[0], half[0]), ("v", got[1], half[1])):
        want = np.concatenate([c.read(x, b)[n - m:] for b, (n, m) in enumerate(zip(lens, q_lens))])
        # one product, four binary32 sums of 16 values: 2^-21 of their magnitudes
        mag = np.abs(want.reshape(*want.shape[:-1], -1, 16)).max(-1).repeat(16, -1) * 16
        assert np.all(np.abs(to_host(g) - want) <= 2.0 ** -21 * mag)
        assert torch.equal(h, g.to(torch.bfloat16))


def test_append_skips_what_has_no_place():
    """Positions before the first token, past the table, pages of -1 or out of
    range, new tokens past max_q: left out, nothing else touched."""
    note("kv append without a place")
    c = kv_ref.Case("nvfp4", 64, 16, 2, [20, 40, 10], 3)
    cache = device_cache(c)
    table = ints([[0, -1], [1, c.pages + 5], [-7, 2]])
    lens = ints([20, 40, 10])  # 40 tokens, but columns for 32
    rows = 20 + 40 + 30  # the last has more new tokens than tokens
    x = torch.randn(rows, 2, 64, device=DEV).to(torch.bfloat16)
    batch = fp4.KVBatch(table, lens, ints([0, 20, 60, 90]), 40)
    fp4.kv_append(cache, x, x, batch)
    k, v = fp4.kv_gather(cache, batch, rows, out_dtype=torch.float32)
    torch.cuda.synchronize()
    wrote = [(0, t) for t in range(16)] + [(1, t) for t in range(16)]
    codes = to_host(cache.k_codes)[0]
    for pg in range(c.pages):
        for t in range(16):
            assert (codes[pg, :, t] != 0xFF).any() == ((pg, t) in wrote), (pg, t)
    host = to_host(k)
    for r in range(rows):
        held = r < 16 or 20 <= r < 36
        assert (host[r] != 0).any() == held, r
    # max_q cuts: only the first two new tokens of each
    cache2 = device_cache(c)
    fp4.kv_append(cache2, x, x, batch._replace(max_q=2))
    torch.cuda.synchronize()
    codes = to_host(cache2.k_codes)[0]
    assert sum(int((codes[p, :, t] != 0xFF).any()) for p in range(c.pages) for t in range(16)) == 4


# -------------------------------------------------------------------- attention
def check_attention(c, q_lens, group, window=0, sinks=0, out_dtype=torch.bfloat16, seed=0,
                    scale=None, max_kv=0, held=None, q_gain=1.0, cache=None, batch=None):
    dim, hq = c.dim, c.heads * group
    rng = np.random.default_rng(1000 + seed)
    tokens = sum(q_lens)
    wide = to_device(kv_ref.workloads.to_bf16_bits(rng.standard_normal((tokens, hq + 2, dim)) * q_gain))
    q = wide[:, 1:hq + 1]  # strided
    cache = device_cache(c) if cache is None else cache
    batch = device_batch(c, q_lens, max_kv=max_kv) if batch is None else batch
    out = torch.full((tokens, hq, dim), float("nan"), dtype=out_dtype, device=DEV)
    lse = torch.full((tokens, hq), float("nan"), device=DEV)
    ws = fp4.kv_attention_workspace_bytes(cache, batch, hq, tokens, window, sinks)
    work = torch.full((ws,), 0xFF, dtype=torch.uint8, device=DEV)  # contents: any
    fp4.kv_attention(q, cache, batch, layer=c.layer, scale=scale, window=window, sinks=sinks, out=out,
                     lse=lse, workspace=work)
    torch.cuda.synchronize()
    got, got_lse = out.double().cpu().numpy(), lse.double().cpu().numpy()
    scale = 1.0 / np.sqrt(dim) if scale is None else scale
    mx = c.fmt != "nvfp4"
    e_q = (2.0 ** -16 if mx else 2.0 ** -11) if c.rht else 2.0 ** -23
    e_p = 2.0 ** -8 if mx else 2.0 ** -11
    at = 0
    for b, n in enumerate(q_lens):
        if n == 0:
            continue
        qb = q[at:at + n].double().cpu().numpy()
        want, wlse, (mean, dot, floor) = kv_ref.attention(
            qb, c.read("k", b), c.read("v", b), n, window, sinks, scale,
            None if held is None else held[b])
        keys = max(c.lens[b], 1)
        # the rotated rows' products bound the sums that the kernel takes
        amp = 4.0 if c.rht else 1.0
        ds = (e_q + dim * 2.0 ** -23) * dot * amp + 2.0 ** -20 * (1 + 2.0 ** -4 * np.abs(np.where(np.isfinite(wlse), wlse, 0)))
        rel = 2 * (ds + e_p + keys * 2.0 ** -23)
        vmag = mean.reshape(*mean.shape[:-1], -1, 16).max(-1).repeat(16, -1) * amp if c.rht else mean
        fmag = floor.reshape(*floor.shape[:-1], -1, 16).max(-1).repeat(16, -1) * amp if c.rht else floor
        bound = rel[..., None] * vmag + 2.0 ** -24 * fmag
        if out_dtype == torch.bfloat16:
            bound = bound * (1 + 2.0 ** -8) + 2.0 ** -8 * np.abs(want)
        err = np.abs(got[at:at + n] - want)
        bad = np.argwhere(~(err <= bound))
        assert bad.size == 0, "%s: %d out of bound, first %s: got %r want %r bound %r" % (
            (c.fmt, dim, b), len(bad), tuple(bad[0]), got[at:at + n][tuple(bad[0])],
            want[tuple(bad[0])], bound[tuple(bad[0])])
        g = got_lse[at:at + n]
        assert np.array_equal(np.isneginf(g), np.isneginf(wlse))
        fin = np.isfinite(wlse)
        # the sum of the rounded probabilities: their errors and the scores'
        assert np.all(np.abs(g - wlse)[fin] <= (rel + 2.0 ** -22 * np.abs(wlse) * 4)[fin])
        at += n
    return out


FORMATS = [("nvfp4", False), ("nvfp4", True), ("mxfp4", False), ("mxfp4_oas", True)]


@pytest.mark.parametrize("fmt,rht", FORMATS)
@pytest.mark.parametrize("dim,page,heads,group", [(64, 16, 2, 8), (128, 64, 2, 4), (256, 32, 1, 3),
                                                  (128, 256, 1, 1), (64, 128, 1, 16)])
def test_single_tokens(fmt, rht, dim, page, heads, group):
    note("kv attention single %s rht=%s dim %d page %d group %d" % (fmt, rht, dim, page, group))
    lens = [1, 15, 16, 17, 64, 65, 200, 333]
    c = kv_ref.Case(fmt, dim, page, heads, lens, 7, rht=rht, layers=2, layer=1).fill()
    check_attention(c, [1] * len(lens), group)
    check_attention(c, [1] * len(lens), group, out_dtype=torch.float32)


@pytest.mark.parametrize("fmt,rht", FORMATS)
@pytest.mark.parametrize("dim,group,q_lens", [(64, 4, [5, 1, 8, 3]), (128, 7, [2, 3, 1, 9]),
                                              (256, 4, [5, 6, 1, 7]), (128, 32, [1, 2, 2, 1])])
def test_few_tokens(fmt, rht, dim, group, q_lens):
    """Rows of 17 to 64: two row tiles of a workgroup, several workgroups."""
    note("kv attention few %s rht=%s dim %d group %d" % (fmt, rht, dim, group))
    c = kv_ref.Case(fmt, dim, 32, 1, [5, 90, 8, 300], 8, rht=rht).fill()
    check_attention(c, q_lens, group)


@pytest.mark.parametrize("fmt,rht", FORMATS)
@pytest.mark.parametrize("dim,heads,group,lens,q_lens", [
    (64, 2, 4, [150, 99, 1], [150, 77, 1]),
    (128, 1, 5, [130, 400], [130, 65]),
    (128, 1, 1, [70, 257], [70, 257]),
    (256, 1, 4, [100, 65], [100, 33]),
])
def test_prompts(fmt, rht, dim, heads, group, lens, q_lens):
    note("kv attention prompt %s rht=%s dim %d group %d" % (fmt, rht, dim, group))
    c = kv_ref.Case(fmt, dim, 32, heads, lens, 9, rht=rht).fill()
    check_attention(c, q_lens, group)
    check_attention(c, q_lens, group, out_dtype=torch.float32)


@pytest.mark.parametrize("fmt,rht", [("nvfp4", True), ("mxfp4", False)])
@pytest.mark.parametrize("q_lens", [[1, 1, 1], [6, 2, 9], [120, 40, 75]])
@pytest.mark.parametrize("window,sinks", [(1, 0), (17, 3), (64, 64), (100, 33), (1000, 5), (40, 500)])
def test_window_and_sinks(fmt, rht, q_lens, window, sinks):
    note("kv attention window %d sinks %d %s" % (window, sinks, q_lens))
    c = kv_ref.Case(fmt, 64, 16, 1, [120, 333, 75], 10, rht=rht).fill()
    check_attention(c, q_lens, 4, window, sinks)


@pytest.mark.parametrize("q_lens", [[4, 3, 1, 0], [90, 70, 100, 2]])
def test_rows_that_see_nothing(q_lens):
    """More new tokens than tokens (the first stand before position 0), and
    empty sequences: zeros and lse -inf; every other row as always."""
    note("kv attention empty rows %s" % q_lens)
    c = kv_ref.Case("nvfp4", 128, 16, 2, [2, 0, 1, 40], 12).fill()
    check_attention(c, q_lens, 4)


@pytest.mark.parametrize("q_len", [1, 80])
def test_pages_given_back(q_len):
    """Under a window the pages that fell out of it are gone (-1, their bytes
    poisoned by another use): results as before, also where one page inside
    the window is missing."""
    note("kv attention with missing pages, %d new" % q_len)
    c = kv_ref.Case("nvfp4", 64, 16, 1, [300, 200], 13).fill()
    window, sinks = 70, 20
    full = check_attention(c, [q_len, 1], 2, window, sinks)
    first = [300 - q_len - window + 1, 200 - window]
    for b in (0, 1):
        for col in range(c.table.shape[1]):
            if (col + 1) * 16 <= first[b] and col * 16 >= sinks and c.table[b, col] >= 0:
                for x in "kv":
                    c.codes[x][0, c.table[b, col]] = 0xFF
                    c.scales[x][0, c.table[b, col]] = 0xFF
                c.table[b, col] = -1
    assert torch.equal(full, check_attention(c, [q_len, 1], 2, window, sinks))
    # a page inside what is seen: its tokens are not attended to
    c.table[1, 9] = -1
    held = [np.ones(300, bool), np.ones(200, bool)]
    held[1][9 * 16:10 * 16] = False
    check_attention(c, [q_len, 1], 2, window, sinks, held=held)


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
@pytest.mark.parametrize("q_lens,lens", [([1, 1], [5000, 777]), ([3, 9], [4100, 50]), ([100, 130], [4000, 3000])])
def test_split_keys(fmt, q_lens, lens):
    """Long rows and few of them: the keys are split and joined; a max_kv that
    is too small only costs balance; the result does not depend on what the
    workspace held, and repeats bit for bit."""
    note("kv attention split %s %s" % (fmt, lens))
    c = kv_ref.Case(fmt, 64, 64, 1, lens, 14, rht=True).fill()
    cache, batch = device_cache(c), device_batch(c, q_lens)
    assert fp4.kv_attention_workspace_bytes(cache, batch, 4, sum(q_lens)) > 0
    a = check_attention(c, q_lens, 4)
    assert torch.equal(a, check_attention(c, q_lens, 4))
    check_attention(c, q_lens, 4, max_kv=max(lens))
    check_attention(c, q_lens, 4, max_kv=1000)
    check_attention(c, q_lens, 4, window=2500, sinks=70)


def test_large_scores_and_scales():
    """Scores of some hundreds (one key takes all the weight), a negative and a
    zero scale, large and tiny q, keys and values."""
    note("kv attention magnitudes")
    for i, (fmt, spread, gain, scale) in enumerate([
            ("nvfp4", 1.0, 40.0, None), ("mxfp4", 30.0, 10.0, None), ("nvfp4", 1.0, 1.0, -0.3),
            ("nvfp4", 1.0, 1.0, 0.0), ("mxfp4", 1e-6, 1e-6, 1e10), ("mxfp4", 1e8, 1e-9, None),
            ("nvfp4", 1.0, 1e-20, 1e18), ("nvfp4", 1.0, 1e20, 1e-21)]):
        for q_lens in ([1, 2], [70, 90]):
            c = kv_ref.Case(fmt, 64, 32, 1, [100, 95], 20 + i, spread=spread, rht=i % 2 == 1).fill()
            check_attention(c, q_lens, 2, scale=scale, q_gain=gain, out_dtype=torch.float32)


def test_rows_of_no_sequence_and_other_stream():
    """Rows past the last sequence stay as they are; a call on another stream
    is ordered there and allocates there."""
    note("kv attention stream and padding rows")
    c = kv_ref.Case("nvfp4", 64, 16, 2, [2100, 30], 15).fill()
    cache, batch = device_cache(c), device_batch(c, [1, 1])
    q = torch.randn(5, 8, 64, device=DEV).to(torch.bfloat16)
    out = torch.full((5, 8, 64), 7.0, dtype=torch.bfloat16, device=DEV)
    fp4.kv_attention(q, cache, batch, out=out)
    torch.cuda.synchronize()
    assert torch.all(out[2:] == 7.0) and not torch.any(out[:2] == 7.0)
    s = torch.cuda.Stream()
    big = torch.randn(4096, 4096, device=DEV)
    with torch.cuda.stream(s):
        for _ in range(4):
            big = big @ big * 1e-3
        q2 = q.clone()
    other = fp4.kv_attention(q2, cache, batch, stream=s)
    s.synchronize()
    assert torch.equal(other[:2], out[:2])


def test_attention_in_a_graph():
    """Append and attention captured together; lengths, tables and rows change
    in place between the replays."""
    note("kv graph")
    c = kv_ref.Case("nvfp4", 128, 16, 2, [900, 1500], 16, rht=True)
    cache = device_cache(c)
    batch = device_batch(c, [1, 1])
    k, v = (torch.zeros(2, 2, 128, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    q = torch.zeros(2, 8, 128, dtype=torch.bfloat16, device=DEV)
    out = torch.zeros_like(q)
    n = fp4.kv_attention_workspace_bytes(cache, batch, 8, 2)
    ws = torch.empty(max(n, 16), dtype=torch.uint8, device=DEV)
    s = torch.cuda.Stream()
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g, stream=s):
        fp4.kv_append(cache, k, v, batch, stream=s)
        fp4.kv_attention(q, cache, batch, out=out, workspace=ws, stream=s)
    fresh = device_cache(c)
    for step in range(4):
        lens = [1 + 37 * step, 700 + 200 * step]
        for b in (0, 1):  # everything before the new token
            batch.kv_lens[b] = lens[b]
        torch.cuda.synchronize()
        for x, t in (("k", k), ("v", v)):
            t.copy_(to_device(np.stack([c.rows[x, b][lens[b] - 1] for b in (0, 1)])))
        q.copy_(torch.randn(q.shape, device=DEV))
        pre = fp4.KVBatch(batch.page_table, ints(lens), ints(np.cumsum([0] + lens)), max(lens))
        for t in (cache, fresh):
            fp4.kv_append(t, to_device(np.concatenate([c.rows["k", b][:lens[b]] for b in (0, 1)])),
                          to_device(np.concatenate([c.rows["v", b][:lens[b]] for b in (0, 1)])), pre)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        want = fp4.kv_attention(q, fresh, batch, workspace=ws)
        torch.cuda.synchronize()
        assert torch.equal(out, want), step


def test_far_pages():
    """A layer of more than 2^32 bytes: the pages at its end."""
    note("kv far pages")
    pages, page, heads, dim = 36000, 256, 8, 128  # 4.7e9 code bytes a layer
    cache = fp4.new_kv_cache(pages, page, heads, dim, "mxfp4")
    table = ints([[pages - 1, pages - 2, 1], [0, 2, pages - 3]])
    lens = [600, 515]
    rng = np.random.default_rng(2)
    rows = kv_ref.workloads.to_bf16_bits(rng.standard_normal((sum(lens), heads, dim)))
    k = to_device(rows)
    batch = fp4.KVBatch(table, ints(lens), ints([0, 600, 1115]), 600)
    fp4.kv_append(cache, k, k, batch)
    back, _ = fp4.kv_gather(cache, batch, 1115, out_dtype=torch.float32)
    q = torch.randn(2, 8, dim, device=DEV).to(torch.bfloat16)
    one = fp4.KVBatch(table, ints(lens), ints([0, 1, 2]), 1)
    out = fp4.kv_attention(q, cache, one, out_dtype=torch.float32)
    torch.cuda.synchronize()
    c, s = kv_ref.quantize_rows(rows, "mxfp4", None, False, 0)
    want = kv_ref.values(c, s, "mxfp4", None, False, 0)
    assert np.array_equal(to_host(back), want.astype(np.float32))
    for b, at in ((0, 0), (1, 600)):
        r = want[at:at + lens[b]]
        o, _, (mean, _, _) = kv_ref.attention(q[b:b + 1].double().cpu().numpy(), r, r, 1, 0, 0, dim ** -0.5)
        assert np.all(np.abs(to_host(out)[b] - o[0]) <= 2 * (2.0 ** -8 + 2.0 ** -10) * mean[0])


# ------------------------------------------------------------------------ pages
def pool(rng, layers, pages, heads, page, fmt, dim):
    half, nsc = dim // 2, dim // kv_ref.BLOCK[fmt]
    return [rng.integers(0, 256, (layers, pages, heads, page, n), dtype=np.uint8)
            for n in (half, nsc, half, nsc)]


def pool_cache(arrays, fmt):
    return fp4.KVCache(*[to_device(a.copy()) for a in arrays], fmt=fmt)


def sequences(rng, seqs, cols, page, pages, spare_rows):
    """Rows of pages, some pages shared by two rows."""
    table = np.full((seqs + spare_rows, cols), -1, np.int32)
    lens = np.zeros(seqs + spare_rows, np.int32)
    refs = np.zeros(pages, np.int32)
    ids = list(rng.permutation(pages))
    for s in range(seqs):
        lens[s] = rng.integers(0, cols * page + 1)
        for c in range(-(-int(lens[s]) // page)):
            share = s and c * page + page <= lens[s] and c * page + page <= lens[s - 1] and rng.random() < 0.3
            if not share and not ids:
                lens[s] = c * page
                break
            p = table[s - 1, c] if share else ids.pop()
            table[s, c] = p
            refs[p] += 1
    return table, lens, refs


def move_bytes(arrays, moves):
    for a in arrays:
        old = a.copy()
        for s, d, *n in moves:
            n = n[0] if n else a.shape[3]
            a[:, d, :, :n] = old[:, s, :, :n]


@pytest.mark.parametrize("fmt,dim", [("nvfp4", 64), ("nvfp4", 256), ("mxfp4", 64), ("mxfp4_oas", 128)])
@pytest.mark.parametrize("page", [16, 64])
def test_copy_pages(fmt, dim, page):
    note("kv copy pages %s %d %d" % (fmt, dim, page))
    rng = np.random.default_rng(4)
    arrays = pool(rng, 3, 20, 5, page, fmt, dim)
    cache = pool_cache(arrays, fmt)
    src, dst, n = [0, 3, 3, 7, 9, -1, 25, 8], [10, 11, 12, 13, 14, 15, 16, 40], [page, 1, page - 1, 0, 7, 5, 5, 5]
    fp4.kv_copy_pages(cache, ints(src[:3]), ints([17, 18, 19]))
    fp4.kv_copy_pages(cache, ints(src), ints(dst), ints(n))
    torch.cuda.synchronize()
    move_bytes(arrays, [(0, 17), (3, 18), (3, 19)])
    move_bytes(arrays, [(s, d, m) for s, d, m in zip(src, dst, n) if 0 <= s < 20 and d < 20])
    for a, t in zip(arrays, (cache.k_codes, cache.k_scales, cache.v_codes, cache.v_scales)):
        assert_bytes_equal(to_host(t), a, "pages")


@pytest.mark.parametrize("seed", range(6))
def test_fork_free_compact(seed):
    note("kv fork, free, compact %d" % seed)
    rng = np.random.default_rng(50 + seed)
    page = int(rng.choice([16, 32]))
    fmt = ["nvfp4", "mxfp4"][seed % 2]
    seqs, cols, forks = 9, 7, 12
    pages = [70, 36, 2500, 64, 41, 300][seed]  # 36, 41: too few for every fork
    arrays = pool(rng, 2, pages, 3, page, fmt, 64)
    table, lens, refs = sequences(rng, seqs, cols, page, pages, forks)
    cache = pool_cache(arrays, fmt)
    # one unit stride past the columns: rows of a wider table
    wide = torch.full((seqs + forks, cols + 2), 99, dtype=torch.int32, device=DEV)
    wide[:, :cols] = ints(table)
    tab, ln, rf = wide[:, :cols], ints(lens), ints(refs)

    def same(what):
        torch.cuda.synchronize()
        assert np.array_equal(to_host(tab), table), what
        assert np.array_equal(to_host(ln), lens), what
        assert np.array_equal(to_host(rf), refs), what
        assert torch.all(wide[:, cols:] == 99)
        for a, t in zip(arrays, (cache.k_codes, cache.k_scales, cache.v_codes, cache.v_scales)):
            assert_bytes_equal(to_host(t), a, what)

    window, sinks = int(rng.integers(1, 4 * page)), int(rng.integers(0, 2 * page))
    fp4.kv_free(tab, ln, rf, ints([0, 3]), page, window=window, sinks=sinks)
    kv_ref.free(table, lens, refs, [0, 3], page, window, sinks)
    same("trim")
    parents = [int(x) for x in rng.integers(0, seqs, forks)]
    children = [seqs + int(x) for x in rng.permutation(forks)]
    failed = fp4.kv_fork(cache, tab, ln, rf, ints(parents), ints(children))
    moves, bad = kv_ref.fork(table, lens, refs, parents, children, page)
    move_bytes(arrays, moves)
    same("fork")
    assert int(failed.item()) == bad
    gone = [1, 2, 5, children[0], children[3]]
    fp4.kv_free(tab, ln, rf, ints(gone), page)
    kv_ref.free(table, lens, refs, gone, page, 0, 0)
    same("free")
    place, used = fp4.kv_compact(cache, tab, rf)
    moves, want, n = kv_ref.compact(table, refs)
    move_bytes(arrays, moves)
    same("compact")
    assert int(used.item()) == n and np.array_equal(to_host(place), want)
    before = [t.clone() for t in (cache.k_codes, cache.v_scales)]
    fp4.kv_compact(cache, tab, rf)  # packed already: nothing moves
    same("compact again")
    assert torch.equal(before[0], cache.k_codes) and torch.equal(before[1], cache.v_scales)


def test_many_forks_and_pages():
    """More forks and pages than the list kernel has threads."""
    note("kv many forks")
    rng = np.random.default_rng(60)
    page, seqs, cols, forks, pages = 16, 40, 6, 1500, 5003
    arrays = pool(rng, 1, pages, 1, page, "mxfp4", 64)
    table, lens, refs = sequences(rng, seqs, cols, page, pages, forks)
    cache = pool_cache(arrays, "mxfp4")
    tab, ln, rf = ints(table), ints(lens), ints(refs)
    parents = [int(x) for x in rng.integers(0, seqs, forks)]
    children = list(range(seqs, seqs + forks))
    fp4.kv_fork(cache, tab, ln, rf, ints(parents), ints(children))
    moves, _ = kv_ref.fork(table, lens, refs, parents, children, page)
    move_bytes(arrays, moves)
    fp4.kv_free(tab, ln, rf, ints(children[::2]), page)
    kv_ref.free(table, lens, refs, children[::2], page, 0, 0)
    place, used = fp4.kv_compact(cache, tab, rf)
    moves, want, n = kv_ref.compact(table, refs)
    move_bytes(arrays, moves)
    torch.cuda.synchronize()
    assert np.array_equal(to_host(tab), table) and np.array_equal(to_host(rf), refs)
    assert np.array_equal(to_host(ln), lens) and np.array_equal(to_host(place), want)
    assert_bytes_equal(to_host(cache.k_codes), arrays[0], "codes")


def test_no_work():
    note("kv empty calls")
    cache = fp4.new_kv_cache(4, 16, 1, 64, "mxfp4")
    none = torch.empty(0, 1, 64, dtype=torch.bfloat16, device=DEV)
    batch = fp4.KVBatch(torch.empty(0, 3, dtype=torch.int32, device=DEV), ints([]), ints([0]), 1)
    fp4.kv_append(cache, none, none, batch)
    fp4.kv_gather(cache, batch, 0)
    fp4.kv_attention(none, cache, batch)
    fp4.kv_copy_pages(cache, ints([]), ints([]))
    table, lens, refs = ints(np.zeros((0, 3))), ints([]), ints([0, 0, 0, 0])
    assert int(fp4.kv_fork(cache, table, lens, refs, ints([]), ints([])).item()) == 0
    fp4.kv_free(table, lens, refs, ints([]), 16)
    place, used = fp4.kv_compact(cache, table, refs)
    torch.cuda.synchronize()
    assert int(used.item()) == 0 and torch.all(place == -1)
    # a batch whose table has no columns: nothing is held
    q = torch.randn(2, 4, 64, device=DEV).to(torch.bfloat16)
    b = fp4.KVBatch(torch.empty(2, 0, dtype=torch.int32, device=DEV), ints([5, 0]), ints([0, 1, 2]), 1)
    assert torch.all(fp4.kv_attention(q, cache, b) == 0)


def test_refusals():
    note("kv refusals")
    cache = fp4.new_kv_cache(8, 16, 2, 64, "nvfp4")
    c = kv_ref.Case("nvfp4", 64, 16, 2, [5], 1)
    batch = device_batch(c, [1])
    x = torch.zeros(1, 2, 64, dtype=torch.bfloat16, device=DEV)
    q = torch.zeros(1, 4, 64, dtype=torch.bfloat16, device=DEV)
    with pytest.raises(fp4.FP4Error):
        fp4.kv_append(cache, x, x, batch, layer=1)
    with pytest.raises(ValueError):
        fp4.kv_append(cache, x[:, :1], x[:, :1], batch)
    with pytest.raises(TypeError):
        fp4.kv_append(cache, x.half(), x.half(), batch)
    odd = torch.zeros(2, 2, 65, dtype=torch.bfloat16, device=DEV)[:, :, :64]
    with pytest.raises(fp4.FP4Error) as e:
        fp4.kv_append(cache, odd, odd, device_batch(c, [2]))
    assert e.value.status == -4
    with pytest.raises(fp4.FP4Error):
        fp4.kv_attention(torch.zeros(1, 3, 64, dtype=torch.bfloat16, device=DEV), cache, batch)
    with pytest.raises(TypeError):
        fp4.kv_attention(q.float(), cache, batch)
    with pytest.raises(fp4.FP4Error):
        fp4.kv_attention(q, cache, batch, window=-1)
    with pytest.raises(fp4.FP4Error):
        fp4.kv_attention(q, cache, batch, scale=float("inf"))
    with pytest.raises(ValueError):
        fp4.kv_attention(q, cache, batch._replace(kv_lens=batch.kv_lens.long()))
    with pytest.raises(ValueError):
        fp4.kv_attention(q, cache, batch._replace(cu_q=ints([0, 1, 2])))
    with pytest.raises(ValueError):
        fp4.kv_attention(q, cache, batch, lse=torch.zeros(1, 5, device=DEV))
    with pytest.raises(ValueError):
        fp4.new_kv_cache(8, 24, 2, 64)
    with pytest.raises(ValueError):
        fp4.new_kv_cache(8, 16, 2, 96)
    with pytest.raises(ValueError):
        fp4.new_kv_cache(8, 16, 2, 64, "hif4")
    # a split call with a workspace that is too small
    long = kv_ref.Case("nvfp4", 64, 16, 2, [4000], 1)
    lb = device_batch(long, [1])
    lc = fp4.new_kv_cache(long.pages, 16, 2, 64, "nvfp4")
    need = fp4.kv_attention_workspace_bytes(lc, lb, 4, 1)
    assert need > 0
    with pytest.raises(fp4.FP4Error) as e:
        fp4.kv_attention(q, lc, lb, workspace=torch.empty(need - 16, dtype=torch.uint8, device=DEV))
    assert e.value.status == -6
    with pytest.raises(ValueError):
        fp4.kv_fork(cache, ints([[0]]), ints([1]), ints([1]), ints([0]), ints([0]))
    with pytest.raises(fp4.FP4Error):
        fp4.kv_free(ints([[0]]), ints([1]), ints([1]), ints([0]), 24)
