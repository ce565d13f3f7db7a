"""The three ways in which the work of few rows is dealt to workgroups: one
piece of each row tile's keys, equal pieces of them, equal runs of the keys of
all sequences.  The host chooses by what the table could hold, the kernels go
by the lengths, so short sequences in a wide table take every way cheaply.
Bounds and inputs as in test_gpu_kv.py."""
import numpy as np
import pytest
import torch

import block_scaled_bit_fp4_amd as fp4
from tests import kv_ref
from tests.gpu_util import note
from tests.test_gpu_kv import check_attention, device_batch, device_cache

pytestmark = pytest.mark.gpu


def lengths(rng, n, most):
    lens = [int(x) for x in rng.integers(0, most, n)]
    lens[0], lens[1], lens[n // 2], lens[-1] = 0, most, 0, 0  # nothing at either end
    return lens


@pytest.mark.parametrize("fmt,rht", [("nvfp4", True), ("mxfp4", True), ("mxfp4_oas", False)])
@pytest.mark.parametrize("dim,heads,group,q_len,batch", [
    (64, 16, 1, 1, 50), (128, 16, 2, 1, 49), (256, 32, 1, 1, 17), (64, 12, 5, 6, 65), (256, 16, 4, 5, 18)])
def test_equal_runs(fmt, rht, dim, heads, group, q_len, batch):
    """More row tiles than workgroups and a table for 8192 keys.  Sequences
    without keys stand first, last and between the others."""
    note("kv equal runs %s dim %d heads %d group %d q %d" % (fmt, dim, heads, group, q_len))
    rng = np.random.default_rng(70)
    lens = lengths(rng, batch, 90)
    lens[2] = 400
    c = kv_ref.Case(fmt, dim, 64, heads, lens, 71, rht=rht, columns=128).fill()
    q_lens = [int(x) for x in rng.integers(0, q_len + 1, batch)]
    q_lens[0] = q_lens[1] = q_lens[2] = q_len
    a = check_attention(c, q_lens, group)
    assert torch.equal(a, check_attention(c, q_lens, group))
    check_attention(c, q_lens, group, out_dtype=torch.float32)


@pytest.mark.parametrize("fmt,rht", [("nvfp4", True), ("mxfp4", True), ("mxfp4", False)])
@pytest.mark.parametrize("dim,heads,group,q_lens", [
    (64, 2, 8, [1, 1, 1, 1, 0]), (128, 1, 4, [1, 1, 1, 1, 1]), (128, 2, 5, [4, 1, 6, 3, 2]),
    (256, 1, 4, [5, 5, 2, 1, 1])])
def test_equal_pieces(fmt, rht, dim, heads, group, q_lens):
    """A table for some ten pieces, sequences of fewer tiles than pieces, of as
    many and of none."""
    note("kv equal pieces %s dim %d heads %d group %d" % (fmt, dim, heads, group))
    lens = [1100, 40, 0, 700, 129]
    c = kv_ref.Case(fmt, dim, 32, heads, lens, 72, rht=rht, columns=140).fill()
    cache, batch = device_cache(c), device_batch(c, q_lens)
    assert fp4.kv_attention_workspace_bytes(cache, batch, heads * group, sum(q_lens)) > 0
    a = check_attention(c, q_lens, group)
    assert torch.equal(a, check_attention(c, q_lens, group))
    check_attention(c, q_lens, group, window=300, sinks=40)


@pytest.mark.parametrize("fmt,rht", [("nvfp4", True), ("mxfp4", True)])
@pytest.mark.parametrize("dim", [64, 128, 256])
def test_one_piece(fmt, rht, dim):
    """Tables of up to some twenty tiles need no workspace and no second launch."""
    note("kv one piece %s dim %d" % (fmt, dim))
    lens = [0, 500, 1, 31, 33, 0]
    c = kv_ref.Case(fmt, dim, 16, 3, lens, 73, rht=rht).fill()
    cache, batch = device_cache(c), device_batch(c, [1] * 6)
    assert fp4.kv_attention_workspace_bytes(cache, batch, 6, 6) == 0
    check_attention(c, [1] * 6, 2)
    check_attention(c, [2, 3, 1, 1, 4, 0], 2, out_dtype=torch.float32)
