"""Overlapping arrays of an eviction, refused on the host before any CUDA call (the pointers are never dereferenced)."""
import pytest

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
