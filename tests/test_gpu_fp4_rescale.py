"""Decode over 4-bit rows where a head's maximum grows by more than the kernel's lazy threshold (8 in base 2) inside a
CTA's share, so that what has been accumulated is scaled down.

The shares of the launch and the growth in each are worked out here from the lengths, and the tests assert that several
tiles fall to a CTA, that maxima grow after a piece's first tile, and that they do for some groups of 32 heads and
not for others.  Rows that are scaled down carry values large enough to matter: without the scaling, or with another
head's, the result would be off by far more than the tolerance (test_gpu_fp4.py's: queries and scores are held
exactly but for a part of a few units)."""
import numpy as np
import pytest
import torch

from tests import fp4_ref
from tests.gpu_util import f64
from tests.test_gpu_fp4 import REL, empty_cache, plain_decode, rand_rows

pytestmark = pytest.mark.gpu
TILE, EMPTY, SHARES, THRESHOLD = 48, 3, 148, 8.0
LEVELS = np.array([0.0, 9.0, 18.0, 9.0, 27.0])  # of a tile's scores, by turns


@pytest.fixture(scope="module")
def g():
    import causal_head_latent_b200 as mod
    return mod


def pieces(lens, L):
    """(share, sequence, first tile, tiles) of every piece of the launch."""
    tiles = [-(-n // TILE) for n in lens]
    places = [(b, t) for b, n in enumerate(tiles) if n for t in range(-EMPTY, n)]
    G = min(SHARES, len(lens) * (-(-L // TILE) + EMPTY), len(places))
    out = []
    for i in range(G):
        mine = places[i * len(places) // G:(i + 1) * len(places) // G]
        for b in sorted({b for b, t in mine}):
            ts = [t for c, t in mine if c == b and t >= 0]
            if ts:
                out.append((i, b, ts[0], len(ts)))
    return out


def growth(z, first, n, rows):
    """[n, H]: whether a head's kept maximum is replaced at each tile of a piece but the first."""
    asked, m = np.zeros((n, z.shape[0]), bool), None
    for j in range(n):
        top = z[:, (first + j) * TILE:min((first + j + 1) * TILE, rows)].max(1)
        if m is None:
            m = top
            continue
        asked[j] = top > m + THRESHOLD
        m = np.where(asked[j], top, m)
    return asked


@pytest.mark.parametrize("B,L,lens", [(1, 30000, None), (8, 6000, [6000, 0, 48, 5999, 3000, 1, 49, 5000]), (40, 900, None)])
@pytest.mark.parametrize("H,d_c", [(96, 512), (7, 64), (33, 320), (64, 128), (96, 192)])
def test_maxima_that_grow_inside_a_share(g, B, L, lens, H, d_c):
    rng = np.random.default_rng(B + H)
    vis = [L] * B if lens is None else lens
    # channel 0 drives the scores; channels 16..31 carry what scaled-down rows weigh in with; the rest is noise
    level = LEVELS[(np.arange(L) // TILE) % len(LEVELS)]
    rows = rng.standard_normal((B, L, d_c))
    rows[:, :, 0] = level
    rows[:, :, 1:16] *= 0.25
    rows[:, :, 16:32] *= 2.0 ** ((27 - level) / 3)[None, :, None]
    gain = np.array([(1.0, 0.0, 0.5, 1.0)[h % 4] if h < 32 else 0.0 if h < 64 else 0.5 for h in range(H)])
    W_k = 0.5 * rng.standard_normal((H, 128, d_c)) * d_c ** -0.5
    W_k[:, 0], W_k[:, :, 0], W_k[:, :, 16:32] = 0, 0, 0
    W_k[:, 0, 0] = gain
    Q = 0.125 * rng.standard_normal((B, H, 128))
    Q[:, :, 0] = 1
    dev = lambda x: torch.from_numpy(x.astype(np.float32)).to(torch.bfloat16).cuda()
    Q, W_k, W_v = dev(Q.reshape(B, H * 128)), dev(W_k.reshape(H * 128, d_c)), rand_rows(rng, H * 128, d_c) * d_c ** -0.5
    codes, scales = empty_cache(B, L, d_c)
    g.gmla_cache_quantize_fp4(dev(rows), codes, scales)
    held = fp4_ref.values(codes.cpu().numpy(), scales.cpu().numpy())
    scale = float(np.float32(np.log(2.0)))  # scores in base 2

    # what the launch meets
    work = pieces(vis, L)
    q = np.einsum("bhd,hdc->bhc", f64(Q).reshape(B, H, 128), f64(W_k).reshape(H, 128, d_c))
    z = [q[b] @ held[b, :vis[b]].T for b in range(B)]
    asked = [growth(z[b], first, n, vis[b]) for i, b, first, n in work]
    assert max(n for _, _, _, n in work) >= 3
    assert sum(a[1:].any() for a in asked) >= 20
    if H > 32:  # in one tile some groups of 32 heads ask and others do not
        groups = np.concatenate([[a[:, h:h + 32].any(1) for h in range(0, H, 32)] for a in asked], axis=1)
        assert (groups.any(0) & ~groups.all(0)).sum() >= 20
    if B > 8:
        assert len(work) > len({i for i, _, _, _ in work})  # several pieces to a CTA

    O = torch.full((B, H * 128), float("nan"), dtype=torch.bfloat16, device="cuda")
    ws = torch.full((g.gmla_attend_decode_fp4_workspace_size(B, L, H, d_c),), 0xFF, dtype=torch.uint8, device="cuda")
    dl = None if lens is None else torch.tensor(lens, dtype=torch.int32, device="cuda")
    g.gmla_attend_decode_fp4(Q, codes, scales, L, W_k, W_v, O, H, lens=dl, scale=scale, workspace=ws)
    g.gmla_get_device_status()
    ref, got = plain_decode(f64(Q), held, vis, f64(W_k), f64(W_v), H, scale=scale), f64(O)
    for b, n in enumerate(vis):
        for h in range(H):
            at = slice(128 * h, 128 * (h + 1))
            assert np.linalg.norm(got[b, at] - ref[b, at]) <= REL * np.linalg.norm(ref[b, at]), (b, h)
