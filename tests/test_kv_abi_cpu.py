"""The cache's entry points refuse bad arguments on the host, before any HIP
call, with the status that include/fp4.h states.  No computing call is made."""
import os

import numpy as np
import pytest
import torch

import block_scaled_bit_fp4_amd as fp4
from block_scaled_bit_fp4_amd import kv

# Fake device pointers: validation must reject these calls before touching them.
A = 1 << 20          # 16-byte aligned
MIS = (1 << 20) + 4  # misaligned
NULL, FORMAT, SHAPE, ALIGN, DTYPE, WORKSPACE = -1, -2, -3, -4, -5, -6


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(fp4.LIB_PATH):
        from block_scaled_bit_fp4_amd import build
        build.build()
    return fp4.load()


def cache(fmt=0, layers=2, heads=8, dim=128, page=64, rht=0, seed=0, pages=16, kc=A, ks=A, vc=A, vs=A,
          kf=A, vf=A):
    return kv._CACHE.pack(fmt, layers, heads, dim, page, rht, seed, pages, kc, ks, vc, vs, kf, vf)


def batch(table=A, ld=4, lens=A, cu=A, size=3, columns=4, max_q=1, max_kv=0):
    return kv._BATCH.pack(table, ld, lens, cu, size, columns, max_q, max_kv)


# what every call on a layer and a batch refuses
COMMON = [
    (dict(c=None), NULL), (dict(b=None), NULL),
    (dict(c=cache(fmt=2)), FORMAT), (dict(c=cache(fmt=4)), FORMAT), (dict(c=cache(rht=2)), FORMAT),
    (dict(c=cache(dim=96)), SHAPE), (dict(c=cache(page=8)), SHAPE), (dict(c=cache(page=48)), SHAPE),
    (dict(c=cache(page=512)), SHAPE), (dict(c=cache(heads=0)), SHAPE), (dict(c=cache(heads=1025)), SHAPE),
    (dict(c=cache(layers=0)), SHAPE), (dict(c=cache(pages=0)), SHAPE), (dict(c=cache(pages=2**31)), SHAPE),
    (dict(layer=2), SHAPE), (dict(layer=-1), SHAPE),
    (dict(b=batch(size=-1)), SHAPE), (dict(b=batch(size=65536)), SHAPE), (dict(b=batch(columns=5)), SHAPE),
    (dict(b=batch(columns=-1)), SHAPE), (dict(b=batch(max_q=-1)), SHAPE), (dict(b=batch(max_kv=-1)), SHAPE),
    (dict(b=batch(columns=2**26, ld=2**26)), SHAPE),  # positions past 31 bits
    (dict(tokens=-1), SHAPE), (dict(tokens=2**31), SHAPE),
    (dict(b=batch(table=0)), NULL), (dict(b=batch(lens=0)), NULL), (dict(b=batch(cu=0)), NULL),
    (dict(b=batch(table=A + 2)), ALIGN), (dict(b=batch(lens=A + 1)), ALIGN), (dict(b=batch(cu=A + 2)), ALIGN),
    (dict(c=cache(kc=0)), NULL), (dict(c=cache(vs=0)), NULL), (dict(c=cache(kf=0)), NULL),
    (dict(c=cache(vf=0)), NULL), (dict(c=cache(kc=MIS)), ALIGN), (dict(c=cache(ks=MIS)), ALIGN),
    (dict(c=cache(vc=MIS)), ALIGN), (dict(c=cache(kf=A + 2)), ALIGN),
]


def append(lib, c=cache(), layer=0, b=batch(), k=A, kt=1024, kh=128, v=A, vt=1024, vh=128, dt=0, tokens=3):
    return lib.fp4_kv_append(c, layer, b, k, kt, kh, v, vt, vh, dt, tokens, None)


def gather(lib, c=cache(), layer=0, b=batch(), k=A, v=A, ot=1024, oh=128, dt=0, tokens=3):
    return lib.fp4_kv_gather(c, layer, b, k, v, ot, oh, dt, tokens, None)


def attention(lib, c=cache(), layer=0, b=batch(), q=A, qt=4096, qh=128, heads=32, tokens=3, scale=0.1,
              window=0, sinks=0, out=A, odt=0, ot=4096, oh=128, lse=0, ws=A, nws=1 << 30):
    return lib.fp4_kv_attention(c, layer, b, q, qt, qh, heads, tokens, scale, window, sinks, out, odt, ot,
                                oh, lse, ws, nws, None)


@pytest.mark.parametrize("call", [append, gather, attention])
def test_common(lib, call):
    for args, status in COMMON:
        assert call(lib, **args) == status, args
    assert call(lib, c=cache(fmt=1, kf=0, vf=0), b=batch(size=0), tokens=3) == 0  # no sequence: nothing to do
    assert call(lib, tokens=0) == 0


def test_append(lib):
    for args, status in [(dict(dt=2), DTYPE), (dict(k=0), NULL), (dict(v=0), NULL), (dict(k=MIS), ALIGN),
                         (dict(v=MIS), ALIGN), (dict(kt=1025), ALIGN), (dict(vh=132), ALIGN),
                         (dict(dt=1, kh=130), ALIGN),
                         (dict(b=batch(max_q=2**30), tokens=2**30), SHAPE)]:  # pieces past 31 bits
        assert append(lib, **args) == status, args


def test_gather(lib):
    for args, status in [(dict(dt=7), DTYPE), (dict(k=0), NULL), (dict(v=0), NULL), (dict(v=MIS), ALIGN),
                         (dict(ot=1028), ALIGN), (dict(dt=1, oh=130), ALIGN),
                         (dict(b=batch(max_q=2**30), tokens=2**30), SHAPE)]:
        assert gather(lib, **args) == status, args


def test_attention(lib):
    for args, status in [
            (dict(odt=3), DTYPE), (dict(scale=float("inf")), SHAPE), (dict(scale=float("nan")), SHAPE),
            (dict(heads=0), SHAPE), (dict(heads=12), SHAPE), (dict(heads=1 << 20), SHAPE),
            (dict(window=-1), SHAPE), (dict(sinks=-1), SHAPE), (dict(q=0), NULL), (dict(out=0), NULL),
            (dict(q=MIS), ALIGN), (dict(qt=4100), ALIGN), (dict(out=MIS), ALIGN), (dict(oh=130), ALIGN),
            (dict(lse=A + 2), ALIGN)]:
        assert attention(lib, **args) == status, args
    # a call that is split needs its workspace
    long = batch(columns=512, ld=512)
    need = lib.fp4_kv_attention_workspace_bytes(cache(), long, 32, 3, 0, 0)
    assert need > 0
    assert attention(lib, b=long, ws=0) == WORKSPACE
    assert attention(lib, b=long, nws=need - 1) == WORKSPACE
    assert attention(lib, b=long, ws=MIS) == ALIGN
    assert attention(lib, b=batch(max_q=2**20), tokens=2**20, heads=65536) == SHAPE


def test_workspace_bytes(lib):
    size = lib.fp4_kv_attention_workspace_bytes
    assert size(cache(), batch(), 32, 3, 0, 0) == 0          # a short table: one workgroup to a key head
    assert size(None, batch(), 32, 3, 0, 0) == 0
    assert size(cache(dim=96), batch(), 32, 3, 0, 0) == 0
    long = batch(columns=4096, ld=4096)
    # a window bounds the keys that are seen, and so does max_kv
    assert size(cache(), long, 32, 3, 0, 0) > size(cache(), long, 32, 3, 128, 4) == 0
    assert size(cache(), batch(columns=4096, ld=4096, max_kv=300), 32, 3, 0, 0) == 0
    # equal runs: more row tiles than workgroups at once
    many = batch(size=200, columns=4096, ld=4096)
    assert size(cache(), many, 8, 200, 0, 0) == 768 * 2 * 16 * (128 * 4 + 8) + 201 * 4


def test_pages(lib):
    copy = lambda c=cache(), s=A, d=A, t=0, n=2: lib.fp4_kv_copy_pages(c, s, d, t, n, None)
    for args, status in [(dict(c=None), NULL), (dict(c=cache(page=8)), SHAPE), (dict(n=-1), SHAPE),
                         (dict(s=0), NULL), (dict(d=0), NULL), (dict(t=A + 2), ALIGN), (dict(c=cache(kc=0)), NULL),
                         (dict(n=0), 0)]:
        assert copy(**args) == status, args

    def fork(c=cache(), table=A, ld=4, seqs=4, cols=4, lens=A, refs=A, par=A, chi=A, n=2, failed=A, ws=A, nws=32):
        return lib.fp4_kv_fork(c, table, ld, seqs, cols, lens, refs, par, chi, n, failed, ws, nws, None)
    for args, status in [(dict(c=None), NULL), (dict(ld=3), SHAPE), (dict(seqs=-1), SHAPE), (dict(n=-1), SHAPE),
                         (dict(refs=0), NULL), (dict(table=0), NULL), (dict(failed=0), NULL), (dict(lens=0), NULL),
                         (dict(par=0), NULL), (dict(chi=0), NULL), (dict(chi=A + 2), ALIGN), (dict(ws=0), WORKSPACE),
                         (dict(nws=31), WORKSPACE), (dict(cols=2**26, ld=2**26), SHAPE)]:
        assert fork(**args) == status, args

    def free(table=A, ld=4, seqs=4, cols=4, lens=A, refs=A, pages=16, page=64, ids=A, n=2, window=0, sinks=0):
        return lib.fp4_kv_free(table, ld, seqs, cols, lens, refs, pages, page, ids, n, window, sinks, None)
    for args, status in [(dict(page=24), SHAPE), (dict(pages=0), SHAPE), (dict(window=-1), SHAPE), (dict(n=-1), SHAPE),
                         (dict(ld=2), SHAPE), (dict(refs=0), NULL), (dict(lens=0), NULL), (dict(ids=0), NULL),
                         (dict(lens=A + 1), ALIGN), (dict(n=0), 0), (dict(seqs=0), 0)]:
        assert free(**args) == status, args

    def compact(c=cache(), table=A, ld=4, seqs=4, cols=4, refs=A, place=A, used=A, ws=A, nws=76):
        return lib.fp4_kv_compact(c, table, ld, seqs, cols, refs, place, used, ws, nws, None)
    for args, status in [(dict(c=None), NULL), (dict(place=0), NULL), (dict(used=0), NULL), (dict(refs=0), NULL),
                         (dict(used=A + 2), ALIGN), (dict(ws=0), WORKSPACE), (dict(nws=75), WORKSPACE),
                         (dict(ld=1), SHAPE)]:
        assert compact(**args) == status, args


def test_binding_refuses_host_tensors():
    """Wrong places, types and sizes are told apart before the library is called."""
    c = kv.new_kv_cache(4, 16, 2, 64, "mxfp4", device="cpu")
    ids = torch.zeros(1, 2, dtype=torch.int32)
    b = kv.KVBatch(ids, torch.ones(1, dtype=torch.int32), torch.tensor([0, 1], dtype=torch.int32), 1)
    x = torch.zeros(1, 2, 64, dtype=torch.bfloat16)
    for call in (lambda: kv.kv_append(c, x, x, b), lambda: kv.kv_gather(c, b, 1), lambda: kv.kv_attention(x, c, b),
                 lambda: kv.kv_copy_pages(c, ids[0], ids[0]),
                 lambda: kv.kv_free(ids, ids[0], ids[0], ids[0], 16)):
        with pytest.raises(ValueError):
            call()
    for bad in (dict(fmt="hif4"), dict(page_size=24), dict(head_dim=96)):
        with pytest.raises(ValueError):
            kv.new_kv_cache(**{**dict(pages=4, page_size=16, heads=2, head_dim=64, device="cpu"), **bad})
    with pytest.raises(ValueError):  # a size that its field does not hold
        kv._pack(kv._BATCH, A, 4, A, A, 3, 4, 2**31, 0)


def test_new_cache_shapes():
    for fmt, block in (("nvfp4", 16), ("mxfp4", 32), ("mxfp4_oas", 32)):
        c = kv.new_kv_cache(5, 32, 3, 128, fmt, layers=2, device="cpu", k_scale=[0.5, 0.25] if block == 16 else 1.0)
        assert c.k_codes.shape == c.v_codes.shape == (2, 5, 3, 32, 64)
        assert c.k_scales.shape == c.v_scales.shape == (2, 5, 3, 32, 128 // block)
        if block == 16:
            assert np.array_equal(c.k_scale.numpy(), np.float32([0.5, 0.25]))
            assert np.array_equal(c.v_scale.numpy(), np.float32([1 / 448] * 2))
        else:
            assert c.k_scale is None and c.v_scale is None
