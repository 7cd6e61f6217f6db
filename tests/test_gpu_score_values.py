"""Accumulated attention weights where values are not finite.  A NaN among what a head attends to leaves no weight of
that head defined, wherever the row stands and however the work is cut."""
import numpy as np
import pytest
import torch

from tests.gpu_util import f64
from tests.test_gpu_score import REL, plain, rand

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def g():
    import causal_head_latent_b200 as mod
    return mod


def score(g, Q, C, L, W_k, H, lens=None, scale=0.0, decay=0.0, before=None):
    B, Lmax, d_c = C.shape
    out = torch.full((B, Lmax), 5.0, device="cuda") if before is None else before.clone()
    ws = torch.full((g.gmla_cache_score_workspace_size(B, L, H, d_c),), 0xFF, dtype=torch.uint8, device="cuda")
    dl = None if lens is None else torch.tensor(lens, dtype=torch.int32, device="cuda")
    g.gmla_cache_score(Q, C, L, W_k, out, H, lens=dl, scale=scale, decay=decay, workspace=ws)
    g.gmla_get_device_status()
    return f64(out)


# rows with a NaN: one, some, the last, all, and (tiles are 128 rows) whole tiles, so that pieces of the work hold nothing else
NAN_ROWS = [slice(17, 18), slice(0, 300), slice(-1, None), slice(None), slice(0, 128), slice(256, 512)]
SHAPES = [(96, 512, 2000), (1, 64, 2000), (33, 192, 1000), (96, 128, 40000)]


@pytest.mark.parametrize("H,d_c,L,rows", [(*s, r) for s in SHAPES for r in NAN_ROWS] + [(96, 128, 40000, slice(2560, 7680))])
def test_a_nan_row_leaves_no_weight_of_its_sequence_defined(g, rows, H, d_c, L):
    rng = np.random.default_rng(L + H)
    B = 4
    C, Q, W_k = rand(rng, B, L + 2, d_c), rand(rng, B, H * 128), rand(rng, H * 128, d_c) * d_c ** -0.5
    lens = [L, L, 0, L - 1]
    want = plain(f64(Q), f64(C), lens, W_k=f64(W_k), H=H)
    C[1, :L][rows, d_c // 2] = float("nan")
    C[0, L:], C[3, L - 1:] = float("nan"), float("nan")  # behind the last row: not seen
    got = score(g, Q, C, L, W_k, H, lens)
    assert np.isnan(got[1, :L]).all()
    for b in (0, 3):
        n = lens[b]
        assert np.linalg.norm(got[b, :n] - want[b, :n]) <= REL * np.linalg.norm(want[b, :n])
    for b, n in enumerate(lens):
        assert (got[b, n:] == 5).all()


@pytest.mark.parametrize("value", [float("inf"), float("-inf"), float("nan")])
@pytest.mark.parametrize("H", [5, 64, 96])
def test_a_query_that_is_not_finite(g, value, H):
    """One head without defined weights, so no sum over the heads of that sequence."""
    rng = np.random.default_rng(H)
    B, L, d_c = 2, 1500, 256
    C, Q, W_k = rand(rng, B, L, d_c), rand(rng, B, H * 128), rand(rng, H * 128, d_c) * d_c ** -0.5
    want = plain(f64(Q), f64(C), [L, L], f64(W_k), H)
    Q[0, 128 * (H - 1) + 3] = value
    got = score(g, Q, C, L, W_k, H)
    assert np.isnan(got[0]).all()
    assert np.linalg.norm(got[1] - want[1]) <= REL * np.linalg.norm(want[1])
