"""Refusals of the packed-batch entry points on a machine without a GPU: no call here
reaches a launch."""

import ctypes

import pytest
import torch

from test_abi_host import FAKE, hq, make_cache  # noqa: F401  (hq: the fixture)


def span(hq, n=4, rows=4, T=512, seq_lens=None, cu=None):
    return hq.SpanStruct(seq_lens, cu, T, n, rows)


def rows(hq, ptr=FAKE, dtype=1, rs=1024, hs=128):
    return hq.RowsStruct(ptr, dtype, rs, hs)


def write(hq, cs=None, k="", v="", src=None, src_rows=4, sp=None, U=FAKE):
    k = rows(hq) if k == "" else k
    v = rows(hq) if v == "" else v
    return hq.lib().headq_cache_write_ragged(cs or make_cache(hq), k, v, src_rows, src, sp or span(hq), U, None)


def test_write_refusals(hq):
    assert hq.lib().headq_cache_write_ragged(None, rows(hq), None, 4, None, span(hq), FAKE, None) == 1
    assert hq.lib().headq_cache_write_ragged(make_cache(hq), rows(hq), None, 4, None, None, FAKE, None) == 1
    assert write(hq, make_cache(hq, kmode=1)) == 2          # sealed key blocks
    assert write(hq, make_cache(hq, d=48)) == 2
    assert write(hq, make_cache(hq, B=70000), sp=span(hq, n=0)) == 2
    assert write(hq, k=None) == 1
    assert write(hq, k=rows(hq, ptr=FAKE + 8)) == 1
    assert write(hq, k=rows(hq, rs=1028)) == 1
    assert write(hq, k=rows(hq, hs=-128)) == 1
    assert write(hq, k=rows(hq, dtype=7)) == 1
    assert write(hq, v=rows(hq, dtype=0)) == 1              # another dtype than k
    assert write(hq, src_rows=3) == 1                       # without src: the rows themselves
    assert write(hq, src=FAKE + 4) == 1
    assert write(hq, U=None) == 1
    assert write(hq, sp=span(hq, T=2048)) == 1              # past the capacity
    assert write(hq, sp=span(hq, n=5)) == 1                 # B * n rows are needed without cu
    assert write(hq, sp=span(hq, n=-1)) == 1
    assert write(hq, sp=span(hq, cu=FAKE + 4)) == 1
    assert write(hq, sp=span(hq, n=0)) == 0                 # nothing to do


def read(hq, cs=None, sp=None, U=FAKE, corr=1, k="", v="", ws=None):
    k = rows(hq) if k == "" else k
    v = rows(hq) if v == "" else v
    return hq.lib().headq_cache_read(cs or make_cache(hq), sp or span(hq), U, corr, k, v, ws, None)


def test_read_refusals(hq):
    assert read(hq, corr=2) == 1
    assert read(hq, k=None, v=None) == 1
    assert read(hq, U=None) == 1
    assert read(hq, v=rows(hq, rs=12)) == 1
    assert read(hq, ws=FAKE + 8) == 1
    assert read(hq, sp=span(hq, rows=3)) == 1
    assert read(hq, sp=span(hq, rows=0, n=0)) == 0


def tree(hq, cs=None, q="", Hq=4, mask=None, ms=0, sp=None, U=FAKE, corr=1, out="", lse=None,
         ws=FAKE, nb=1 << 40):
    q = rows(hq) if q == "" else q
    out = rows(hq) if out == "" else out
    return hq.lib().headq_tree_attn(cs or make_cache(hq), q, Hq, mask, ms, sp or span(hq), U, 0.1, corr,
                                    out, lse, ws, nb, None)


def test_tree_refusals(hq):
    assert tree(hq, make_cache(hq, kmode=1)) == 2
    assert tree(hq, Hq=3) == 1
    assert tree(hq, Hq=0) == 1
    assert tree(hq, corr=-2) == 1
    assert tree(hq, mask=FAKE, ms=15) == 1                  # shorter than n * n
    assert tree(hq, out=rows(hq, dtype=0)) == 1             # another dtype than q
    assert tree(hq, lse=FAKE + 4) == 1
    assert tree(hq, q=None) == 1
    assert tree(hq, U=None) == 1
    assert tree(hq, ws=None) == 3
    assert tree(hq, nb=128) == 3
    assert tree(hq, sp=span(hq, n=1 << 23, rows=1 << 23)) == 2
    assert tree(hq, sp=span(hq, n=0)) == 0


def test_tree_workspace(hq):
    L = hq.lib()
    assert L.headq_tree_workspace_bytes(None, 4, 1, 512) == 0
    assert L.headq_tree_workspace_bytes(make_cache(hq), 3, 1, 512) == 0
    assert L.headq_tree_workspace_bytes(make_cache(hq), 4, 0, 512) >= 256
    a = L.headq_tree_workspace_bytes(make_cache(hq), 4, 8, 512)
    assert a >= 256 and L.headq_tree_workspace_bytes(make_cache(hq), 4, 8, 0) <= a


def test_binding_refuses_what_is_not_on_a_gpu(hq):
    t = torch.zeros(2, 2, 128)
    with pytest.raises(ValueError):
        hq._rows(t, "k", 2, 128)
    with pytest.raises(ValueError):
        hq.HeadQCache.from_planes(torch.zeros(1, 2, 16, 32, dtype=torch.uint8), torch.zeros(1, 2, 16, 4),
                                  torch.zeros(1, 2, 16, 4), v=torch.zeros(1, 2, 16, 128))
    with pytest.raises(ValueError):
        hq.HeadQCache.from_planes(torch.zeros(1, 2, 16, 32, dtype=torch.uint8), torch.zeros(1, 2, 16, 4),
                                  torch.zeros(1, 2, 16, 4))   # no values


def test_sizes_past_the_kernels_indices(hq):
    """More than 2^30 packed rows, or lengths, are refused; n may be any bound of n_b."""
    big = make_cache(hq, T_cap=(1 << 30) + 64)
    for sp, want in [(span(hq, n=1, rows=(1 << 30) + 1), 2), (span(hq, n=4, T=(1 << 30) + 16), 2)]:
        assert write(hq, big, src=FAKE, sp=sp) == want
        assert read(hq, big, sp=sp) == want
    far = (1 << 31) - 1
    assert write(hq, sp=span(hq, n=far, rows=0, cu=FAKE), src_rows=0) == 0
    assert read(hq, sp=span(hq, n=far, rows=0, cu=FAKE)) == 0
