"""Overlapping arrays of an eviction, refused on the host before any CUDA call (the pointers are never dereferenced)."""
import pytest
import torch

ARG, WORKSPACE = 1, 5
P = 1 << 40


@pytest.fixture(scope="module")
def g():
    import causal_head_latent_b200 as mod
    return mod


def evict(g, r0=P, b0=1024, d0=P, r1=None, b1=0, d1=None, s=2 * P, ds=2 * P, pos=None, dpos=None, B=2, n=20, dn=20, L=20,
          lens=None, keep=8, new=3 * P, index=4 * P, ws=5 * P, nbytes=None):
    if nbytes is None:
        nbytes = g.gmla_cache_evict_workspace_size(B, L, keep)
    return g.lib.gmla_cache_evict(r0, b0, d0, r1, b1, d1, s, ds, pos, dpos, B, n, dn, L, lens, keep, 0, 0, new, index, ws,
                                  nbytes, None)


@pytest.mark.parametrize("B,n,b0", [(1 << 15, 1 << 33, 1 << 16), (1 << 14, 1 << 35, 1 << 15), (1 << 13, 1 << 34, 1 << 16),
                                    (65535, 1 << 40, 65536)])
def test_extents_past_64_bits_still_overlap(g, B, n, b0):
    """B * cache_len_max * row_bytes of 2^63, 2^64 and nearly 2^72 bytes: no room between a source and a destination
    1 MB behind it, or before it.  Without a workspace a call that passes the check ends there."""
    assert evict(g, B=B, n=n, b0=b0, d0=P + (1 << 20), s=1 << 60, ds=1 << 62, ws=None) == ARG
    assert evict(g, B=B, n=n, b0=b0, d0=P - (1 << 20), s=1 << 60, ds=1 << 62, ws=None) == ARG


def test_arrays_side_by_side_do_not_overlap(g):
    assert evict(g, d0=P + 2 * 20 * 1024, ds=3 * P, ws=None) == WORKSPACE
    assert evict(g, d0=P - 2 * 8 * 1024, dn=8, ds=3 * P, ws=None) == WORKSPACE


ROWS = 2 * 20 * 1024  # bytes of a row array here


def passes(g, **kw):
    """Whether the call gets past every check of its arguments: to the device (there is none here)."""
    return evict(g, **kw) not in (ARG, WORKSPACE)


@pytest.mark.skipif(torch.cuda.is_available(), reason="a call that passes would run")
@pytest.mark.parametrize("kw", [dict(), dict(d0=6 * P, ds=7 * P), dict(r1=8 * P, d1=8 * P, b1=32),
                                dict(r1=8 * P, d1=9 * P, b1=32, d0=6 * P, ds=7 * P), dict(lens=3 * P), dict(lens=8 * P),
                                dict(r1=P, d1=P, b1=1024), dict(r1=P, d1=6 * P, b1=1024, d0=6 * P, ds=7 * P),
                                dict(r1=P + ROWS, d1=6 * P + ROWS, b1=1024, d0=6 * P, ds=7 * P),
                                dict(r1=P + 1024, d1=9 * P, b1=1024, d0=6 * P, ds=7 * P)])  # sources may overlap
def test_arrays_apart_pass(g, kw):
    assert passes(g, **kw)


TWO = dict(r1=8 * P, d1=9 * P, b1=1024, d0=6 * P, ds=7 * P)


@pytest.mark.parametrize("kw", [dict(TWO, d0=8 * P, d1=P),  # swapped: each destination is the other's source
                                dict(TWO, d1=P), dict(TWO, d0=8 * P + 1024), dict(TWO, d1=6 * P), dict(TWO, d1=6 * P + 16),
                                dict(TWO, ds=P + 4), dict(TWO, ds=6 * P + 4096), dict(TWO, pos=10 * P, dpos=7 * P),
                                dict(TWO, pos=10 * P, dpos=2 * P), dict(TWO, d0=2 * P - 1024),
                                dict(r1=P + 1024, d1=P + 1024, b1=1024), dict(r1=P, d1=P, b1=512),
                                dict(s=P, ds=P), dict(s=2 * P, ds=2 * P, pos=2 * P, dpos=2 * P),
                                dict(new=P), dict(new=2 * P + 156), dict(new=4 * P + 60), dict(new=5 * P + 16), dict(index=P + 512),
                                dict(index=3 * P - 60), dict(index=2 * P), dict(index=5 * P), dict(ws=P), dict(ws=2 * P), dict(ws=3 * P),
                                dict(lens=3 * P + 4), dict(lens=4 * P), dict(lens=P), dict(lens=5 * P)])
def test_what_a_call_writes_overlaps_nothing_else(g, kw):
    assert evict(g, **kw) == ARG
