"""Accumulated attention weights on the GPU against the definition in float64.

Tolerance (relative L2 of what a call adds): q~ = hi + lo keeps 16 bits, so an element is off by 2^-17 of itself
at most and a score z (base 2) by |z| 2^-17 in the worst case (all errors of one sign); its float32 sum of 2 * 512
products by about 2^-20 |z|; ex2 and the sums over rows and heads add a few 2^-22.  A weight moves by ln 2 times
its score's error, the scores here stay below 16 in size: 16 * 2^-17 * ln 2 + 2^-19 < 1e-4 in the worst case,
and, the 512 roundings being independent, about 1/sqrt(512) of it: 2e-5 is used, as float32 outputs elsewhere.
"""
import numpy as np
import pytest
import torch

from tests.gpu_util import f64

pytestmark = pytest.mark.gpu
REL = 2e-5


@pytest.fixture(scope="module")
def g():
    import causal_head_latent_b200 as mod
    return mod


def rand(rng, *shape):
    return torch.from_numpy(rng.standard_normal(shape).astype(np.float32)).to(torch.bfloat16).cuda()


def plain(Q, C, lens, W_k, H, scale=0.0):
    B, d = Q.shape
    D, dc = d // H, C.shape[-1]
    q = np.einsum("bhd,hdc->bhc", Q.reshape(B, H, D), W_k.reshape(H, D, dc)) * (scale if scale > 0 else D ** -0.5)
    out = np.zeros(C.shape[:2])
    for b, n in enumerate(lens):
        if n:
            z = q[b] @ C[b, :n].T
            a = np.exp(z - z.max(-1, keepdims=True))
            out[b, :n] = (a / a.sum(-1, keepdims=True)).sum(0)
    return out


def run(g, B, L, Lmax, H, d_c, lens=None, scale=0.0, decay=1.0, seed=0):
    rng = np.random.default_rng(seed + 31 * B + L)
    C = rand(rng, B, Lmax, d_c)
    vis = [L] * B if lens is None else [min(max(n, 0), L) for n in lens]
    for b, n in enumerate(vis):
        C[b, n:] = float("nan")  # rows nobody stored
    Q = rand(rng, B, H * 128)
    W_k = rand(rng, H * 128, d_c) * d_c ** -0.5
    before = torch.from_numpy(rng.random((B, Lmax)).astype(np.float32)).cuda()
    score = before.clone()
    dl = None if lens is None else torch.tensor(lens, dtype=torch.int32, device="cuda")
    ws = torch.full((g.gmla_cache_score_workspace_size(B, L, H, d_c),), 0xFF, dtype=torch.uint8, device="cuda")
    g.gmla_cache_score(Q, C, L, W_k, score, H, lens=dl, scale=scale, decay=decay, workspace=ws)
    g.gmla_get_device_status()
    add = plain(f64(Q), np.nan_to_num(f64(C)), vis, f64(W_k), H, scale)
    got, old = f64(score), f64(before)
    for b, n in enumerate(vis):
        assert np.array_equal(got[b, n:], old[b, n:])  # rows behind the last one are left as they were
        if n:
            want = decay * old[b, :n] + add[b, :n]
            # the sum itself is rounded to float32 once: half a step of each score
            err = np.abs(got[b, :n] - want) - np.abs(want) * 2.0 ** -24
            assert np.linalg.norm(np.maximum(err, 0)) <= REL * np.linalg.norm(add[b, :n]), (b, n)
            assert abs((got[b, :n] - decay * old[b, :n]).sum() - H) <= 1e-3 * H  # every head's weights sum to 1
    return score


@pytest.mark.parametrize("B,L,H,d_c", [(1, 1, 1, 64), (1, 127, 96, 512), (2, 128, 7, 128), (1, 129, 96, 320),
                                       (3, 500, 33, 192), (2, 1001, 96, 512), (33, 130, 16, 256), (1, 30000, 96, 512)])
def test_one_length(g, B, L, H, d_c):
    run(g, B, L, L + 3, H, d_c)


@pytest.mark.parametrize("lens", [[0], [1, 0, 3], [300, 1, 0, 128, 129, 0, 0, 257], [0, 0, 0, 0], [9000, 2, 2, 2],
                                  [-4, 9999999, 128]])
def test_ragged(g, lens):
    run(g, len(lens), 9000, 9003, 96, 512, lens=lens)


def test_many_short_sequences(g):
    rng = np.random.default_rng(11)
    run(g, 301, 300, 300, 8, 128, lens=rng.integers(0, 301, 301).tolist())


@pytest.mark.parametrize("scale,decay", [(0.02, 1.0), (0.0, 0.5), (0.0, 0.0)])
def test_scale_and_decay(g, scale, decay):
    run(g, 2, 333, 400, 48, 512, scale=scale, decay=decay)


def test_several_groups_of_sequences(g):
    """More sequences than pass through the workspace at once (512 MB: 21 of 65536 rows at 96 heads)."""
    run(g, 23, 65536, 65536, 96, 64, lens=[65536] + [1000 * k + 7 for k in range(21)] + [0])


def test_several_groups_with_few_heads(g):
    """The same where q~ has three parts (512 MB: 32 sequences of 65536 rows at 33 to 64 heads)."""
    run(g, 34, 65536, 65536, 33, 64, lens=[70] * 31 + [65536, 0, 4001])


def test_accumulates_over_captured_steps(g):
    rng = np.random.default_rng(4)
    B, L, H, d_c = 3, 600, 96, 512
    C, Q = rand(rng, B, L, d_c), rand(rng, B, H * 128)
    W_k = rand(rng, H * 128, d_c) * d_c ** -0.5
    score = torch.zeros(B, L, device="cuda")
    lens = torch.tensor([10, 599, 0], dtype=torch.int32, device="cuda")
    ws = torch.empty(g.gmla_cache_score_workspace_size(B, L, H, d_c), dtype=torch.uint8, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        g.gmla_cache_score(Q, C, L, W_k, score, H, lens=lens, workspace=ws)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            lens.add_(1)
            g.gmla_cache_score(Q, C, L, W_k, score, H, lens=lens, workspace=ws)
    torch.cuda.current_stream().wait_stream(side)
    want = plain(f64(Q), f64(C), [10, 599, 0], f64(W_k), H)
    for step in range(1, 3):
        graph.replay()
        want += plain(f64(Q), f64(C), [10 + step, min(599 + step, L), step], f64(W_k), H)
    got = f64(score)
    for b in range(B):
        assert np.linalg.norm(got[b] - want[b]) <= (REL + 2.0 ** -23) * np.linalg.norm(want[b])


def test_twice_gives_the_same_bits(g):
    a = run(g, 4, 2500, 2500, 96, 512, lens=[2500, 1, 900, 64])
    assert torch.equal(a, run(g, 4, 2500, 2500, 96, 512, lens=[2500, 1, 900, 64]))


def test_no_decay_overwrites_what_nobody_initialised(g):
    rng = np.random.default_rng(8)
    C, Q = rand(rng, 2, 200, 128), rand(rng, 2, 512)
    W_k = rand(rng, 512, 128) * 128 ** -0.5
    score = torch.full((2, 200), float("nan"), device="cuda")
    ws = torch.empty(g.gmla_cache_score_workspace_size(2, 150, 4, 128), dtype=torch.uint8, device="cuda")
    g.gmla_cache_score(Q, C, 150, W_k, score, 4, decay=0.0, workspace=ws)
    add = plain(f64(Q), f64(C), [150, 150], f64(W_k), 4)
    assert np.linalg.norm(f64(score)[:, :150] - add[:, :150]) <= REL * np.linalg.norm(add)
    assert torch.isnan(score[:, 150:]).all()


@pytest.mark.parametrize("H,d_c", [(1, 512), (1, 64), (7, 320), (16, 512), (31, 448), (32, 512), (33, 512), (48, 192),
                                   (63, 512), (64, 512), (64, 384)])
@pytest.mark.parametrize("B,L", [(1, 4100), (5, 700)])
def test_few_heads_keep_the_whole_query(g, H, d_c, B, L):
    """With few heads nothing averages out, so q~ has 24 bits and its parts' sums are kept apart.

    Left are the accumulators: each of the d_c / 16 additions to hi's sum (half of them up to 32 heads) truncates it,
    by half a step (2^-22 where the sum is between 2 and 4, as for the rows that weigh most) on average, all of one
    sign; a weight moves by ln 2 times that."""
    rng = np.random.default_rng(H + d_c + L)
    C, Q = rand(rng, B, L, d_c), rand(rng, B, H * 128)
    W_k = rand(rng, H * 128, d_c) * d_c ** -0.5
    score = torch.empty(B, L, device="cuda")
    lens = [L - 37 * b for b in range(B)]
    dl = torch.tensor(lens, dtype=torch.int32, device="cuda")
    ws = torch.full((g.gmla_cache_score_workspace_size(B, L, H, d_c),), 0xFF, dtype=torch.uint8, device="cuda")
    g.gmla_cache_score(Q, C, L, W_k, score, H, lens=dl, decay=0.0, workspace=ws)
    want, got = plain(f64(Q), f64(C), lens, f64(W_k), H), f64(score)
    adds = max(16, d_c // 16) // (2 if H <= 32 else 1)  # at least 16: float32 itself leaves 16 * 2^-24
    for b, n in enumerate(lens):
        assert np.linalg.norm(got[b, :n] - want[b, :n]) <= adds * 2.0 ** -22 * np.log(2) * np.linalg.norm(want[b, :n])
