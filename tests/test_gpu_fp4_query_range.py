"""Decode over 4-bit rows with queries outside float16's range: the absorbed query is held in float16 under a power
of two of its own for every sequence and head, so its size does not matter, and what is not finite stays so.

Tolerances as in test_gpu_fp4.py: every rounding there is relative to the largest element of an absorbed query.
"""
import numpy as np
import pytest
import torch

from tests import fp4_ref
from tests.gpu_util import f64
from tests.test_gpu_fp4 import REL, empty_cache, plain_decode, rand_rows

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def g():
    import causal_head_latent_b200 as mod
    return mod


def decode(g, Q, rows, W_k, W_v, H, lens=None, cache_scale=1.0, scale=0.0):
    B, L, d_c = rows.shape
    codes, scales = empty_cache(B, L, d_c)
    g.gmla_cache_quantize_fp4(rows, codes, scales, cache_scale=cache_scale)
    O = torch.full((B, H * 128), 3.0, dtype=torch.bfloat16, device="cuda")
    ws = torch.full((g.gmla_attend_decode_fp4_workspace_size(B, L, H, d_c),), 0xFF, dtype=torch.uint8, device="cuda")
    dl = None if lens is None else torch.tensor(lens, dtype=torch.int32, device="cuda")
    g.gmla_attend_decode_fp4(Q, codes, scales, L, W_k, W_v, O, H, cache_scale=cache_scale, lens=dl, scale=scale, workspace=ws)
    g.gmla_get_device_status()
    ref = plain_decode(f64(Q), fp4_ref.values(codes.cpu().numpy(), scales.cpu().numpy(), cache_scale),
                       [L] * B if lens is None else lens, f64(W_k), f64(W_v), H, scale=scale)
    return O, ref


@pytest.mark.parametrize("value", [float("inf"), float("-inf"), float("nan")])
@pytest.mark.parametrize("H,d_c,L", [(96, 512, 700), (5, 64, 3), (33, 320, 20000)])
def test_a_query_that_is_not_finite_gives_nan_for_its_head_alone(g, value, H, d_c, L):
    rng = np.random.default_rng(H)
    B = 3
    Q = rand_rows(rng, B, H * 128)
    W_k, W_v = (rand_rows(rng, H * 128, d_c) * d_c ** -0.5 for _ in range(2))
    rows = rand_rows(rng, B, L, d_c)
    lens = [L, 0, L]
    want = decode(g, Q, rows, W_k, W_v, H, lens)[1]
    bad = Q.clone()
    bad[0, 128 * (H - 2) + 77] = value
    bad[1, 5] = value  # of a sequence without rows: still zero
    O, _ = decode(g, bad, rows, W_k, W_v, H, lens)
    got = f64(O).reshape(B, H, 128)
    want = want.reshape(B, H, 128)
    assert np.isnan(got[0, H - 2]).all()
    assert (got[1] == 0).all()
    got[0, H - 2] = want[0, H - 2] = 0
    for b in (0, 2):
        assert np.linalg.norm(got[b] - want[b]) <= REL * np.linalg.norm(want[b])


def test_a_large_cache_scale_does_not_clamp_the_query(g):
    """q~ = (3, 1) * 2^20 * log2(e) / sqrt(128): both above 65504.  The first row's score is 3 * 2^11, the second's
    1.5 * 2^11 (times 1 / sqrt(128)), so the output is the first row's to e^-271; with both parts clamped to 65504 the
    second would win."""
    s, d_c = 2.0 ** 20, 64
    rows = torch.zeros(1, 2, d_c, dtype=torch.bfloat16, device="cuda")
    rows[0, 0, 0] = s * 2.0 ** -9
    rows[0, 1, 1] = s * 1.5 * 2.0 ** -9
    Q = torch.zeros(1, 128, dtype=torch.bfloat16, device="cuda")
    Q[0, 0], Q[0, 1] = 3.0, 1.0
    W_k, W_v = (torch.zeros(128, d_c, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    W_k[0, 0] = W_k[1, 1] = W_v[0, 0] = W_v[1, 1] = 1.0
    O, ref = decode(g, Q, rows, W_k, W_v, 1, cache_scale=s)
    assert ref[0, 0] == 2048.0 and ref[0, 1] < 1e-100
    assert np.array_equal(f64(O), np.where(ref < 1e-100, 0.0, ref))


@pytest.mark.parametrize("up", [-90, -40, 18, 60, 100])
@pytest.mark.parametrize("H,d_c,L", [(96, 512, 1001), (7, 192, 5000)])
def test_the_size_of_the_key_weights_does_not_matter(g, up, H, d_c, L):
    """Weights 2^up times larger under a score scale 2^up times smaller: the same scores.  Half the heads the other way
    round, by their queries, so that exponents of their own are needed."""
    rng = np.random.default_rng(1000 + up)
    Q = rand_rows(rng, 2, H * 128)
    W_k, W_v = (rand_rows(rng, H * 128, d_c) * d_c ** -0.5 for _ in range(2))
    rows = rand_rows(rng, 2, L, d_c)
    same, ref = decode(g, Q, rows, W_k, W_v, H)
    W_up = W_k * 2.0 ** up
    odd = torch.arange(H, device="cuda").repeat_interleave(128) % 2 == 1
    W_up[odd] *= 2.0 ** -12
    Q_up = torch.where(odd, Q * 2.0 ** 12, Q)
    O, _ = decode(g, Q_up, rows, W_up, W_v, H, scale=128 ** -0.5 * 2.0 ** -up)
    assert np.linalg.norm(f64(O) - ref) <= REL * np.linalg.norm(ref)
    assert np.linalg.norm(f64(same) - ref) <= REL * np.linalg.norm(ref)


@pytest.mark.parametrize("H,d_c", [(96, 512), (16, 128)])
def test_loud_rows_under_a_small_cache_scale(g, H, d_c):
    """Rows near the format's upper end (s = 448), so that q~ times the cache's scale is far below 1."""
    rng = np.random.default_rng(d_c)
    Q = rand_rows(rng, 2, H * 128)
    W_k, W_v = (rand_rows(rng, H * 128, d_c) * d_c ** -0.5 for _ in range(2))
    rows = rand_rows(rng, 2, 900, d_c)
    O, ref = decode(g, Q, rows, W_k, W_v, H, cache_scale=2.0 ** -9)
    assert np.linalg.norm(f64(O) - ref) <= REL * np.linalg.norm(ref)


def test_scores_that_all_overflow_are_not_an_empty_sequence(g):
    """Every score -inf in float32: NaN, as a softmax in float32 gives, not the zeros of a sequence without rows."""
    d_c = 64
    rows = torch.full((2, 70, d_c), 100.0, dtype=torch.bfloat16, device="cuda")
    Q = torch.zeros(2, 128, dtype=torch.bfloat16, device="cuda")
    Q[0, 0], Q[1, 0] = -3e38, -1.0
    W = torch.zeros(128, d_c, dtype=torch.bfloat16, device="cuda")
    W[0] = 1.0
    codes, scales = empty_cache(2, 70, d_c)
    g.gmla_cache_quantize_fp4(rows, codes, scales)
    O = torch.zeros(2, 128, dtype=torch.bfloat16, device="cuda")
    ws = torch.empty(g.gmla_attend_decode_fp4_workspace_size(2, 70, 1, d_c), dtype=torch.uint8, device="cuda")
    g.gmla_attend_decode_fp4(Q, codes, scales, 70, W, W, O, 1, workspace=ws)
    got = f64(O)
    held = fp4_ref.values(codes.cpu().numpy(), scales.cpu().numpy())[1, 0].sum()
    assert np.isnan(got[0]).all()
    assert abs(got[1, 0] - held) <= 2.0 ** -8 * held and (got[1, 1:] == 0).all()


@pytest.mark.parametrize("scale", [float("inf"), float("nan")])
def test_a_score_scale_that_is_not_finite(g, scale):
    rng = np.random.default_rng(9)
    Q, rows = rand_rows(rng, 2, 256), rand_rows(rng, 2, 100, 64)
    W_k, W_v = (rand_rows(rng, 256, 64) for _ in range(2))
    codes, scales = empty_cache(2, 100, 64)
    g.gmla_cache_quantize_fp4(rows, codes, scales)
    O = torch.zeros(2, 256, dtype=torch.bfloat16, device="cuda")
    ws = torch.empty(g.gmla_attend_decode_fp4_workspace_size(2, 100, 2, 64), dtype=torch.uint8, device="cuda")
    g.gmla_attend_decode_fp4(Q, codes, scales, 100, W_k, W_v, O, 2, scale=scale, workspace=ws)
    assert torch.isnan(O).all()
