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


# ---- Sums that are exact, or nearly: queries that the parts of q~ hold exactly, the same in every head, so that no
# error averages out.  A score scale of ln 2 makes scores base 2: the factor on q~ is exactly 1.
LN2 = float(np.float32(np.log(2.0)))

# Relative error of a row's weight where its score S is exact: float32 rounds S - lse (below 32 in size: 2^-20 at most) and
# lse (below 16: 2^-21), log2f is off by a step (below 8: 2^-21), times ln 2; ex2 twice 2^-22; float32 sums of the heads
# (8 roundings deep) and of the rows (24) 2^-24 each: 1.4e-6 + 5e-7 + 1.9e-6.
EXACT = 4e-6


def same_heads(H, d_c, w, q=(1.0,)):
    """Q [1, H*128] and W_k [H*128, d_c] with q~ = sum_i q[i] w[i] in every head."""
    Q, W = torch.zeros(1, H, 128), torch.zeros(H, 128, d_c)
    for i, x in enumerate(q):
        Q[:, :, i], W[:, i] = x, torch.from_numpy(w[i].astype(np.float32))
    return Q.view(1, -1).to(torch.bfloat16).cuda(), W.view(H * 128, d_c).to(torch.bfloat16).cuda()


def bf16(x):
    return torch.from_numpy(np.asarray(x, np.float32)).to(torch.bfloat16).float().numpy().astype(np.float64)


def weights_of(g, Q, rows, W_k, H):
    C = torch.from_numpy(rows.astype(np.float32)).to(torch.bfloat16).cuda()[None]
    got = score(g, Q, C, C.shape[1], W_k, H, scale=LN2)[0]
    return got, plain(f64(Q), f64(C), [C.shape[1]], f64(W_k), H, LN2)[0]


@pytest.mark.parametrize("H,d_c", [(96, 512), (65, 320), (96, 64), (64, 512), (33, 448), (7, 128), (1, 512)])
def test_scores_of_one_channel_are_exact(g, H, d_c):
    """One non-zero channel a row, scores from -10 to 10: nothing is rounded in a sum of one product, so the weights are
    exact to float32 however large the score."""
    rng = np.random.default_rng(d_c)
    L = 700
    w = bf16(rng.uniform(0.5, 2, d_c) * rng.choice([-1, 1], d_c))
    Q, W_k = same_heads(H, d_c, [w])
    rows, at = np.zeros((L, d_c)), rng.integers(0, d_c, L)
    rows[np.arange(L), at] = bf16(rng.uniform(-10, 10, L) / w[at])
    got, want = weights_of(g, Q, rows, W_k, H)
    assert (np.abs(got - want) <= EXACT * want).all()


@pytest.mark.parametrize("pattern", ["loud last", "loud first", "cancelling", "second half zero", "even"])
@pytest.mark.parametrize("H,d_c", [(96, 512), (96, 256), (65, 64), (64, 512), (32, 384), (1, 512)])
def test_sums_grow_in_any_order(g, H, d_c, pattern):
    """Bound: each of the d_c / 16 additions to a sum cuts off less than a step of it, at most 2^-23 of the largest partial
    sum or product, and as much again where 16 products meet; a row's weight moves by ln 2 times its score's error and
    the log-sum-exp's, which is no more than the largest."""
    rng = np.random.default_rng(d_c + H)
    L = 900
    w = bf16(rng.uniform(0.5, 2, d_c))
    Q, W_k = same_heads(H, d_c, [w])
    rows = rng.standard_normal((L, d_c))
    size = np.ones(d_c)
    if pattern == "loud last":
        size[:-8] = 1 / 64
    if pattern == "loud first":
        size[8:] = 1 / 64
    if pattern == "second half zero":
        size[d_c // 2:] = 0
    rows = rows * size
    if pattern == "cancelling":  # what the first half adds up to, the second takes away, but for a few units
        rows = np.abs(rows) * np.where(np.arange(d_c) < d_c // 2, 1, -1)
    target = rng.uniform(-6, 6, L)
    rows[:, -1] += (target - rows @ w) / w[-1] if pattern == "cancelling" else 0
    if pattern != "cancelling":
        rows *= (target / (rows @ w))[:, None].clip(-4, 4)
    rows = bf16(rows)
    keep = np.abs(rows @ w) < 10
    rows = rows[keep]
    got, want = weights_of(g, Q, rows, W_k, H)
    products = rows * w
    largest = max(np.abs(np.cumsum(products, 1)).max(), np.abs(np.cumsum(products[:, d_c // 2:], 1)).max(), np.abs(products).max())
    off = d_c / 16 * 2 * 2.0 ** -23 * largest
    assert (np.abs(got - want) <= (EXACT + 2 * np.log(2) * off) * want).all()


@pytest.mark.parametrize("H,d_c", [(1, 512), (16, 512), (32, 64), (33, 448), (64, 512), (65, 256), (96, 256), (96, 192), (96, 64)])
def test_a_query_of_24_bits_is_whole(g, H, d_c):
    """q~ = 1 + a 2^-10 + b 2^-19, a and b in [1, 2), and rows that take the difference of two channels with the same a: the
    scores are 4 (b - b'), all from the third part.  Sums are exact (a product cancels its pair's within one MMA)."""
    rng = np.random.default_rng(d_c + H)
    L = 800
    a = np.repeat(1 + rng.integers(0, 128, d_c // 2) / 128, 2)
    b = 1 + rng.integers(0, 8, d_c) / 8
    Q, W_k = same_heads(H, d_c, [np.ones(d_c), a, b], (1.0, 2.0 ** -10, 2.0 ** -19))
    rows, at = np.zeros((L, d_c)), 2 * rng.integers(0, d_c // 2, L)
    rows[np.arange(L), at], rows[np.arange(L), at + 1] = 2.0 ** 21, -2.0 ** 21
    got, want = weights_of(g, Q, rows, W_k, H)
    assert want.max() > 3 * want.min()
    assert (np.abs(got - want) <= EXACT * want).all()


@pytest.mark.parametrize("H,d_c", [(1, 512), (64, 512), (65, 448), (96, 512), (96, 320), (96, 256), (96, 64)])
def test_a_query_of_17_bits_is_whole(g, H, d_c):
    """The same with q~ = 1 + a 2^-10 and scores 4 (a - a'), all from the second part."""
    rng = np.random.default_rng(d_c + H)
    L = 800
    a = 1 + rng.integers(0, 128, d_c) / 128
    Q, W_k = same_heads(H, d_c, [np.ones(d_c), a], (1.0, 2.0 ** -10))
    rows, at = np.zeros((L, d_c)), 2 * rng.integers(0, d_c // 2, L)
    rows[np.arange(L), at], rows[np.arange(L), at + 1] = 2.0 ** 12, -2.0 ** 12
    got, want = weights_of(g, Q, rows, W_k, H)
    assert want.max() > 3 * want.min()
    assert (np.abs(got - want) <= EXACT * want).all()
