"""Refusals of the compact-cache calls, on the CPU: every bad argument is turned away on the host before any CUDA
call (the pointers below are never dereferenced)."""
import math

import pytest
import torch

OK, ARG, UNSUPPORTED, CUDA, WORKSPACE = 0, 1, 2, 3, 5
P = 0x10000
BIG = 1 << 62


@pytest.fixture(scope="module")
def g():
    import causal_head_latent_b200 as mod
    return mod


def quantize(g, C=P, B=2, src=10, src0=0, rows=10, dc=512, s=1.0, codes=P, scales=P, n=20, row0=0, at=None):
    return g.lib.gmla_cache_quantize_fp4(C, B, src, src0, rows, dc, s, codes, scales, n, row0, at, None)


def dequantize(g, codes=P, scales=P, B=2, n=20, row0=0, rows=10, dc=512, s=1.0, C=P, dst=10, dst0=0):
    return g.lib.gmla_cache_dequantize_fp4(codes, scales, B, n, row0, rows, dc, s, C, dst, dst0, None)


BAD_SCALES = [0.0, -1.0, 3.0, 0.75, math.inf, math.nan, 2.0 ** 65, 2.0 ** -65]


@pytest.mark.parametrize("kw", [dict(C=None), dict(codes=None), dict(scales=None), dict(C=P + 2), dict(codes=P + 8),
                                dict(scales=P + 4), dict(at=P + 2), dict(B=0), dict(dc=0), dict(rows=0), dict(rows=11),
                                dict(src0=1), dict(src0=-1, rows=5), dict(row0=11), dict(row0=-1), dict(src=0),
                                dict(n=9), dict(rows=BIG, src0=5)] + [dict(s=s) for s in BAD_SCALES])
def test_quantize_refuses(g, kw):
    assert quantize(g, **kw) == ARG


@pytest.mark.parametrize("kw", [dict(dc=96), dict(dc=576), dict(B=65536), dict(rows=1 << 25, src=1 << 26, n=1 << 26)])
def test_quantize_unsupported(g, kw):
    assert quantize(g, **kw) == UNSUPPORTED


@pytest.mark.parametrize("kw", [dict(C=None), dict(codes=None), dict(scales=None), dict(C=P + 8), dict(codes=P + 4),
                                dict(B=-1), dict(rows=0), dict(rows=21, dst=30), dict(row0=11), dict(row0=-1),
                                dict(dst0=1), dict(dst0=-1), dict(dst=9)] + [dict(s=s) for s in BAD_SCALES])
def test_dequantize_refuses(g, kw):
    assert dequantize(g, **kw) == ARG


def test_dequantize_unsupported(g):
    assert dequantize(g, dc=40) == UNSUPPORTED and dequantize(g, B=1 << 20) == UNSUPPORTED


def decode(g, Q=P, codes=P, scales=P, cs=1.0, B=2, n=20, L=20, lens=None, H=4, D=128, dc=512, Wk=P, Wv=P, G=None, O=P,
           ws=P, nbytes=None):
    if nbytes is None:
        nbytes = g.gmla_attend_decode_fp4_workspace_size(B, L, H, dc)
    return g.lib.gmla_attend_decode_fp4(Q, codes, scales, cs, B, n, L, lens, H, D, dc, Wk, Wv, 0.0, G, O, ws, nbytes, None)


@pytest.mark.parametrize("kw", [dict(Q=None), dict(codes=None), dict(scales=None), dict(Wk=None), dict(Wv=None),
                                dict(O=None), dict(Q=P + 2), dict(O=P + 8), dict(G=P + 8), dict(ws=P + 8), dict(lens=P + 1),
                                dict(L=0), dict(L=21), dict(B=0), dict(H=0), dict(dc=-64), dict(D=0), dict(cs=3.0),
                                dict(cs=math.nan)])
def test_decode_refuses(g, kw):
    assert decode(g, **kw) == ARG


@pytest.mark.parametrize("kw", [dict(D=64), dict(dc=96), dict(dc=576), dict(H=97), dict(B=65536),
                                dict(L=0x7fffff80, n=0x7fffff80)])
def test_decode_unsupported(g, kw):
    assert decode(g, **kw) == UNSUPPORTED


def test_decode_workspace(g):
    need = g.gmla_attend_decode_fp4_workspace_size(2, 20, 4, 512)
    assert decode(g, ws=None) == WORKSPACE and decode(g, nbytes=need - 1) == WORKSPACE and decode(g, nbytes=0) == WORKSPACE
    assert g.gmla_attend_decode_fp4_workspace_size(0, 20, 4, 512) == 0
    assert g.gmla_attend_decode_fp4_workspace_size(2, -1, 4, 512) == 0


def score(g, Q=P, C=P, B=2, n=20, L=20, lens=None, H=4, D=128, dc=512, Wk=P, decay=1.0, out=P, ws=P, nbytes=None):
    if nbytes is None:
        nbytes = g.gmla_cache_score_workspace_size(B, L, H, dc)
    return g.lib.gmla_cache_score(Q, C, B, n, L, lens, H, D, dc, Wk, 0.0, decay, out, ws, nbytes, None)


@pytest.mark.parametrize("kw", [dict(Q=None), dict(C=None), dict(Wk=None), dict(out=None), dict(Q=P + 2), dict(C=P + 8),
                                dict(out=P + 2), dict(ws=P + 8), dict(lens=P + 2), dict(L=0), dict(L=21), dict(B=0),
                                dict(H=0), dict(dc=0), dict(decay=math.nan), dict(decay=math.inf)])
def test_score_refuses(g, kw):
    assert score(g, **kw) == ARG


@pytest.mark.parametrize("kw", [dict(D=64), dict(dc=96), dict(dc=576), dict(H=97), dict(B=65536)])
def test_score_unsupported(g, kw):
    assert score(g, **kw) == UNSUPPORTED


def test_score_workspace(g):
    need = g.gmla_cache_score_workspace_size(2, 20, 4, 512)
    assert score(g, ws=None) == WORKSPACE and score(g, nbytes=need - 1) == WORKSPACE
    assert g.gmla_cache_score_workspace_size(2, 20, 0, 512) == 0


def evict(g, r0=P, b0=1024, d0=P, r1=None, b1=0, d1=None, s=P + (1 << 20), ds=P + (1 << 20), pos=None, dpos=None, B=2,
          n=20, dn=20, L=20, lens=None, keep=8, sink=0, recent=0, new=P, index=P, ws=P, nbytes=None):
    if nbytes is None:
        nbytes = g.gmla_cache_evict_workspace_size(B, L, keep)
    return g.lib.gmla_cache_evict(r0, b0, d0, r1, b1, d1, s, ds, pos, dpos, B, n, dn, L, lens, keep, sink, recent, new,
                                  index, ws, nbytes, None)


FAR = P + (1 << 30)


@pytest.mark.parametrize("kw", [dict(r0=None), dict(d0=None), dict(s=None), dict(ds=None), dict(new=None), dict(index=None),
                                dict(r1=P, b1=16), dict(d1=P, b1=16), dict(pos=P), dict(dpos=P), dict(B=0), dict(L=0),
                                dict(L=21), dict(keep=0), dict(sink=-1), dict(recent=-1), dict(sink=5, recent=4),
                                dict(sink=9), dict(sink=BIG, recent=BIG), dict(b0=0), dict(b0=6), dict(b0=65540),
                                dict(r1=P, d1=P, b1=2), dict(r0=P + 4, d0=P + 4), dict(s=P + 2, ds=P + 2),
                                dict(lens=P + 2), dict(ws=P + 4), dict(dn=19),  # in place needs one length
                                dict(d0=FAR),  # one in place, one not
                                dict(d0=FAR, ds=FAR, dn=7),  # too short for what is kept
                                dict(d0=P + 1024, ds=FAR), dict(r0=FAR + 1024, d0=FAR, ds=FAR + (1 << 20))])  # overlap
def test_evict_refuses(g, kw):
    assert evict(g, **kw) == ARG


def test_evict_unsupported_and_workspace(g):
    assert evict(g, B=65536) == UNSUPPORTED
    assert evict(g, L=0x7fffff80, n=0x7fffff80, dn=0x7fffff80) == UNSUPPORTED
    need = g.gmla_cache_evict_workspace_size(2, 20, 8)
    assert evict(g, ws=None) == WORKSPACE and evict(g, nbytes=need - 1) == WORKSPACE
    assert g.gmla_cache_evict_workspace_size(2, 20, 0) == 0


def test_binding_refuses(g, monkeypatch):
    """Types, shapes, strides and devices are the binding's to check: the C calls see addresses only."""
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    C, codes, scales = torch.zeros(2, 4, 128, dtype=torch.bfloat16), *(torch.zeros(2, 9, w, dtype=torch.uint8) for w in (64, 8))
    for bad in (dict(C=C.float()), dict(codes=codes.char()), dict(scales=scales[:, :, :4]), dict(scales=scales[:1])):
        a = {**dict(C=C, codes=codes, scales=scales), **bad}
        with pytest.raises((TypeError, ValueError)):
            g.gmla_cache_quantize_fp4(a["C"], a["codes"], a["scales"])
    with pytest.raises(ValueError, match="contiguous"):
        g.gmla_cache_quantize_fp4(torch.zeros(2, 128, 4, dtype=torch.bfloat16).transpose(1, 2), codes, scales)
    with pytest.raises(ValueError, match="current CUDA device"):
        g.gmla_cache_dequantize_fp4(codes, scales, C)
    with pytest.raises(ValueError, match="dimensions"):
        g.gmla_cache_dequantize_fp4(codes, scales, C[0])
    with pytest.raises(ValueError, match="divide"):
        g._head_width(256, 3)
    with pytest.raises(ValueError, match="one or two"):
        g.gmla_cache_evict([], torch.zeros(2, 4), 4, 2, None, None)
    with pytest.raises(ValueError, match="go with dst"):
        g.gmla_cache_evict([C], torch.zeros(2, 4), 4, 2, None, None, dst_score=torch.zeros(2, 4))
    with pytest.raises(ValueError, match="must match"):
        g.gmla_cache_evict([C], torch.zeros(2, 4), 4, 2, None, None, dst=[C])


def test_binding_refuses_workspaces(g, monkeypatch):
    """A workspace elsewhere would be written through by the kernels."""
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    ws = torch.zeros(1 << 16, dtype=torch.uint8)
    Q, C, W = (torch.zeros(*s, dtype=torch.bfloat16) for s in ((2, 128), (2, 9, 128), (128, 128)))
    codes, scales = (torch.zeros(2, 9, w, dtype=torch.uint8) for w in (64, 8))
    score, index, lens = torch.zeros(2, 9), torch.zeros(2, 4, dtype=torch.int32), torch.zeros(2, dtype=torch.int32)
    for call in (lambda: g.gmla_attend_decode_fp4(Q, codes, scales, 9, W, W, Q, 1, workspace=ws),
                 lambda: g.gmla_cache_score(Q, C, 9, W, score, 1, workspace=ws)):
        with pytest.raises(ValueError, match="workspace must live"):
            call()
    monkeypatch.setattr(torch.cuda, "current_device", lambda: -1)  # the device of tensors on the CPU, as far as the checks go
    with pytest.raises(ValueError, match="workspace must be contiguous"):
        g.gmla_cache_evict([C], score, 9, 4, index, lens, workspace=ws[::2])
    monkeypatch.undo()
    assert g._workspace(None, 0) == (None, 0) and g._workspace(ws, -1) == (ws.data_ptr(), 1 << 16)
