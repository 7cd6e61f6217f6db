"""Latent rows in 4 bits on the GPU: storing, reading back, decode over them.

Codes and scales are compared byte for byte with the definition in float64 (tests/fp4_ref.py);
reading back is exact.  Decode outputs are compared with the plain definition in float64 over the
rows that the bytes stand for: keys and values rebuilt, softmax, gate.

Tolerance of the decode (relative L2): the output's bfloat16 rounding is at most 2^-8 of a value; q~ is
rounded to float16 (2^-12 of an element at most, so a score of a few units moves by about 2^-12 and a weight
by as much relatively, bounded here by 2^-10) and P to float16 (2^-11 of a weight); c^ enters W_v with 16 bits.
2^-8 + 2^-10 + 2^-11 + 2^-15 < 5.5e-3, the worst case of every rounding at once.
"""
import numpy as np
import pytest
import torch

from tests import fp4_ref
from tests.gpu_util import f64

pytestmark = pytest.mark.gpu
REL = 2.0 ** -8 + 2.0 ** -10 + 2.0 ** -11 + 2.0 ** -15


@pytest.fixture(scope="module")
def g():
    import causal_head_latent_b200 as mod
    return mod


def rand_rows(rng, *shape):
    return torch.from_numpy(rng.standard_normal(shape).astype(np.float32)).to(torch.bfloat16).cuda()


def empty_cache(B, Lmax, d_c, fill=0xA5):
    return (torch.full((B, Lmax, d_c // 2), fill, dtype=torch.uint8, device="cuda"),
            torch.full((B, Lmax, d_c // 16), fill, dtype=torch.uint8, device="cuda"))


@pytest.mark.parametrize("B,rows,d_c,log2", [(1, 1, 64, 0), (3, 37, 192, 0), (2, 1000, 512, -3), (5, 129, 448, 20),
                                             (32, 1, 512, 0)])
def test_store_bytes(g, B, rows, d_c, log2):
    rng = np.random.default_rng(B * 1000 + rows)
    scale = 2.0 ** log2
    C = rand_rows(rng, B, rows + 5, d_c) * scale
    C[:, ::3] *= 100.0  # other magnitudes
    C[:, 1::4] *= 2.0 ** -12  # down to the smallest scale
    codes, scales = empty_cache(B, rows + 9, d_c)
    g.gmla_cache_quantize_fp4(C, codes, scales, src_row0=2, rows=rows, row0=4, cache_scale=scale)
    want_c, want_s = fp4_ref.quantize(f64(C)[:, 2:2 + rows], scale)
    assert np.array_equal(codes.cpu().numpy()[:, 4:4 + rows], want_c)
    assert np.array_equal(scales.cpu().numpy()[:, 4:4 + rows], want_s)
    for t in (codes, scales):  # the other rows are left as they were
        assert (t[:, :4] == 0xA5).all() and (t[:, 4 + rows:] == 0xA5).all()


def test_store_ties_and_special_values(g):
    """Every half-way point of every scale, zeros of both signs, NaN, infinities, the range's ends."""
    rows = []
    for e in range(-12, 13):
        for m in (1.0, 1.125, 1.5, 1.875):
            s = m * 2.0 ** e  # the group's scale, where 6 s is the largest value
            half = [6, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5]
            rows.append([s * v for v in half] + [-s * v for v in half])
            rows.append([s * 6] + [s * v * (1 + d) for v in half[1:] for d in (-1 / 128, 1 / 128)] + [-0.0])
    rows.append([float("nan"), 1.0, -1.0] + [0.0] * 13)
    rows.append([float("inf"), float("-inf"), 3.0] + [-0.0] * 13)
    rows.append([float("nan")] * 16)
    rows.append([3e38, 2688.0, -2689.0, 448.0] + [1.0] * 12)
    rows.append([2.0 ** -133] + [0.0] * 15)
    x = torch.tensor(rows, dtype=torch.float64).to(torch.bfloat16)
    x = torch.cat([x, torch.zeros(-len(rows) % 4, 16, dtype=torch.bfloat16)]).view(1, -1, 64).cuda()
    codes, scales = empty_cache(1, x.shape[1], 64)
    g.gmla_cache_quantize_fp4(x, codes, scales)
    want_c, want_s = fp4_ref.quantize(f64(x))
    assert np.array_equal(scales.cpu().numpy(), want_s)
    assert np.array_equal(codes.cpu().numpy(), want_c)


def test_store_rows_at_each_sequences_own_length(g):
    rng = np.random.default_rng(5)
    B, Lmax, d_c = 6, 20, 128
    C = rand_rows(rng, B, 3, d_c)
    at = torch.tensor([0, 17, 18, -1, -7, 25], dtype=torch.int32, device="cuda")
    codes, scales = empty_cache(B, Lmax, d_c)
    g.gmla_cache_quantize_fp4(C, codes, scales, row_of=at)
    want_c, want_s = fp4_ref.quantize(f64(C))
    exp_c, exp_s = np.full((B, Lmax, d_c // 2), 0xA5, np.uint8), np.full((B, Lmax, d_c // 16), 0xA5, np.uint8)
    for b, a in enumerate(at.tolist()):
        for t in range(3):
            if 0 <= a + t < Lmax:  # rows outside the cache are dropped
                exp_c[b, a + t], exp_s[b, a + t] = want_c[b, t], want_s[b, t]
    assert np.array_equal(codes.cpu().numpy(), exp_c) and np.array_equal(scales.cpu().numpy(), exp_s)


@pytest.mark.parametrize("B,rows,d_c,log2", [(1, 1, 64, 0), (3, 50, 320, 5), (2, 700, 512, -7)])
def test_read_back_is_exact(g, B, rows, d_c, log2):
    rng = np.random.default_rng(rows)
    codes = torch.from_numpy(rng.integers(0, 256, (B, rows + 3, d_c // 2), dtype=np.uint8)).cuda()
    scales = torch.from_numpy(rng.integers(0, 127, (B, rows + 3, d_c // 16), dtype=np.uint8)).cuda()
    C = torch.full((B, rows + 6, d_c), 7.0, dtype=torch.bfloat16, device="cuda")
    g.gmla_cache_dequantize_fp4(codes, scales, C, row0=1, rows=rows, dst_row0=5, cache_scale=2.0 ** log2)
    want = fp4_ref.values(codes.cpu().numpy(), scales.cpu().numpy(), 2.0 ** log2)
    assert np.array_equal(f64(C)[:, 5:5 + rows], want[:, 1:1 + rows])
    assert (C[:, :5] == 7).all() and (C[:, 5 + rows:] == 7).all()


def plain_decode(Q, rows, lens, W_k, W_v, H, G=None, scale=0.0):
    """float64 definition: keys and values rebuilt from the rows of each sequence."""
    B, d = Q.shape
    D = d // H
    dc = rows.shape[-1]
    Wk, Wv = W_k.reshape(H, D, dc), W_v.reshape(H, D, dc)
    out = np.zeros((B, d))
    for b in range(B):
        n = lens[b]
        if n == 0:
            continue
        c = rows[b, :n]
        z = np.einsum("hd,hdc,sc->hs", Q[b].reshape(H, D), Wk, c, optimize=True) * (scale if scale > 0 else D ** -0.5)
        a = np.exp(z - z.max(-1, keepdims=True))
        a /= a.sum(-1, keepdims=True)
        out[b] = np.einsum("hdc,hc->hd", Wv, a @ c).reshape(d)
    if G is not None:
        out /= 1 + np.exp(-G)
    return out


def decode_case(g, B, L, Lmax, H, d_c, lens=None, gate=True, log2=0, scale=0.0, loud=1.0, seed=0):
    rng = np.random.default_rng(seed + 7 * B + L)
    s = 2.0 ** log2
    codes, scales = empty_cache(B, Lmax, d_c, fill=0xFF)  # rows nobody stored: NaN scales
    n_max = L if lens is None else max(1, min(L, max(lens)))
    g.gmla_cache_quantize_fp4(rand_rows(rng, B, n_max, d_c) * s * loud, codes, scales, cache_scale=s)
    vis = [L] * B if lens is None else [min(max(x, 0), L) for x in lens]
    for b, n in enumerate(vis):
        codes[b, n:], scales[b, n:] = 0xFF, 0xFF
    Q = rand_rows(rng, B, H * 128)
    W_k, W_v = (rand_rows(rng, H * 128, d_c) * d_c ** -0.5 for _ in range(2))
    W_k /= s
    G = rand_rows(rng, B, H * 128) if gate else None
    O = torch.full((B, H * 128), float("nan"), dtype=torch.bfloat16, device="cuda")
    ws = torch.full((g.gmla_attend_decode_fp4_workspace_size(B, L, H, d_c),), 0xFF, dtype=torch.uint8, device="cuda")
    dl = None if lens is None else torch.tensor(lens, dtype=torch.int32, device="cuda")
    g.gmla_attend_decode_fp4(Q, codes, scales, L, W_k, W_v, O, H, cache_scale=s, lens=dl, scale=scale, G=G, workspace=ws)
    g.gmla_get_device_status()
    v = fp4_ref.values(codes.cpu().numpy(), np.minimum(scales.cpu().numpy(), 126), s)
    ref = plain_decode(f64(Q), v, vis, f64(W_k), f64(W_v), H, None if G is None else f64(G), scale)
    return O, ref, vis


def check(O, ref, vis):
    got = f64(O)
    assert np.isfinite(got).all()
    for b, n in enumerate(vis):
        if n == 0:
            assert (got[b] == 0).all()
        else:
            assert np.linalg.norm(got[b] - ref[b]) <= REL * np.linalg.norm(ref[b]), (b, n)


@pytest.mark.parametrize("B,L,H,d_c", [(1, 1, 1, 64), (1, 63, 96, 512), (2, 64, 7, 128), (1, 65, 96, 320),
                                       (3, 200, 33, 192), (2, 1001, 96, 512), (33, 130, 16, 256), (1, 20000, 96, 512)])
def test_decode_one_length(g, B, L, H, d_c):
    check(*decode_case(g, B, L, L + 3, H, d_c))


@pytest.mark.parametrize("lens", [[0], [1, 0, 3], [300, 1, 0, 64, 65, 0, 0, 129], [0, 0, 0, 0], [5000, 2, 2, 2], [4999, 5000], [900, 1700, 0, 5000, 333],
                                  [-4, 9999999, 128]])
def test_decode_ragged(g, lens):
    """Lengths of zero and one, lengths outside 0..L clamped, stored rows past a length never read (NaN scales there)."""
    check(*decode_case(g, len(lens), 5000, 5003, 96, 512, lens=lens))


def test_decode_many_short_sequences(g):
    rng = np.random.default_rng(11)
    lens = rng.integers(0, 200, 301).tolist()
    check(*decode_case(g, 301, 200, 200, 8, 128, lens=lens, gate=False))


@pytest.mark.parametrize("log2,scale", [(0, 0.05), (-10, 0.0), (14, 0.0)])
def test_decode_scales(g, log2, scale):
    check(*decode_case(g, 2, 333, 333, 48, 512, log2=log2, scale=scale))


def test_decode_growing_maximum(g):
    """Keys louder and louder: the running maximum grows in almost every tile (the accumulator is rescaled)."""
    rng = np.random.default_rng(3)
    B, L, H, d_c = 1, 3000, 96, 512
    rows = rand_rows(rng, B, L, d_c) * torch.linspace(0.05, 6, L, device="cuda").view(1, L, 1).to(torch.bfloat16)
    codes, scales = empty_cache(B, L, d_c)
    g.gmla_cache_quantize_fp4(rows, codes, scales)
    Q = rand_rows(rng, B, H * 128)
    W_k, W_v = (rand_rows(rng, H * 128, d_c) * d_c ** -0.5 for _ in range(2))
    O = torch.empty(B, H * 128, dtype=torch.bfloat16, device="cuda")
    ws = torch.empty(g.gmla_attend_decode_fp4_workspace_size(B, L, H, d_c), dtype=torch.uint8, device="cuda")
    g.gmla_attend_decode_fp4(Q, codes, scales, L, W_k, W_v, O, H, workspace=ws)
    ref = plain_decode(f64(Q), fp4_ref.values(codes.cpu().numpy(), scales.cpu().numpy()), [L], f64(W_k), f64(W_v), H)
    # scores reach about 25 in base 2: a relative rounding of 2^-12 of q~ moves them by 25 * 2^-12 at most
    tol = REL + 25 * 2.0 ** -12
    assert np.linalg.norm(f64(O) - ref) <= tol * np.linalg.norm(ref)


def test_decode_many_light_keys(g):
    """One key about 2^24 times heavier than each of 60000 others: the others must not vanish from P."""
    B, L, H, d_c = 1, 60001, 1, 64
    rows = torch.zeros(B, L, d_c, dtype=torch.bfloat16, device="cuda")
    rows[:, :, 0] = 1.0
    rows[:, 7, 1] = 6.0
    rows[:, 7, 0] = 0.0
    W_k = torch.zeros(128, d_c, dtype=torch.bfloat16, device="cuda")
    W_k[0, 1] = 1.0
    W_v = torch.zeros(128, d_c, dtype=torch.bfloat16, device="cuda")
    W_v[0, 0] = 1.0
    W_v[1, 1] = 1.0
    Q = torch.zeros(B, 128, dtype=torch.bfloat16, device="cuda")
    Q[0, 0] = 1.0
    codes, scales = empty_cache(B, L, d_c)
    g.gmla_cache_quantize_fp4(rows, codes, scales)
    O = torch.empty(B, 128, dtype=torch.bfloat16, device="cuda")
    ws = torch.empty(g.gmla_attend_decode_fp4_workspace_size(B, L, H, d_c), dtype=torch.uint8, device="cuda")
    scale = 24 * np.log(2) / 6
    g.gmla_attend_decode_fp4(Q, codes, scales, L, W_k, W_v, O, H, scale=scale, workspace=ws)
    light = (L - 1) * 2.0 ** -24
    v = fp4_ref.values(codes[:, :8].cpu().numpy(), scales[:, :8].cpu().numpy())[0]  # 1 is held as 6 * 0.171875
    assert v[0, 0] == 1.03125 and v[7, 1] == 6.0
    want = np.array([light * v[0, 0] / (1 + light), v[7, 1] / (1 + light)])
    # a score of 24 in base 2 is off by 24 * 2^-12 at most (q~ in float16), its weight by ln 2 of that
    assert np.allclose(f64(O)[0, :2], want, rtol=2.0 ** -8 + 24 * 2.0 ** -12 * np.log(2) + 2.0 ** -11)


def test_decode_on_another_stream_and_captured(g):
    """A captured call follows the lengths and the cache as they are at each replay."""
    rng = np.random.default_rng(21)
    B, L, H, d_c = 4, 700, 96, 512
    codes, scales = empty_cache(B, L, d_c, fill=0)
    g.gmla_cache_quantize_fp4(rand_rows(rng, B, L, d_c), codes, scales)
    Q, G = rand_rows(rng, B, H * 128), rand_rows(rng, B, H * 128)
    W_k, W_v = (rand_rows(rng, H * 128, d_c) * d_c ** -0.5 for _ in range(2))
    new = rand_rows(rng, B, 1, d_c)
    lens = torch.tensor([10, 100, 699, 0], dtype=torch.int32, device="cuda")
    O = torch.empty(B, H * 128, dtype=torch.bfloat16, device="cuda")
    ws = torch.empty(g.gmla_attend_decode_fp4_workspace_size(B, L, H, d_c), dtype=torch.uint8, device="cuda")

    def step():
        g.gmla_cache_quantize_fp4(new, codes, scales, row_of=lens)
        lens.add_(1)
        g.gmla_attend_decode_fp4(Q, codes, scales, L, W_k, W_v, O, H, lens=lens, G=G, workspace=ws)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            step()
    torch.cuda.current_stream().wait_stream(side)
    want_lens = [11, 101, 700, 1]
    for _ in range(3):
        graph.replay()
        new.copy_(rand_rows(rng, B, 1, d_c))
        torch.cuda.synchronize()
        want_lens = [n + 1 for n in want_lens]
        vis = [min(n, L) for n in want_lens]
        v = fp4_ref.values(codes.cpu().numpy(), scales.cpu().numpy())
        check(O, plain_decode(f64(Q), v, vis, f64(W_k), f64(W_v), H, f64(G)), vis)
    g.gmla_get_device_status()


def test_decode_matches_bf16_decode_over_the_same_rows(g):
    """Store, read back, and run the bfloat16 decode over the rows read back: the same sequence of calls a
    prefill that continues a 4-bit cache makes."""
    rng = np.random.default_rng(31)
    B, L, H, d_c = 3, 900, 96, 512
    codes, scales = empty_cache(B, L, d_c)
    g.gmla_cache_quantize_fp4(rand_rows(rng, B, L, d_c), codes, scales)
    C = torch.empty(B, L, d_c, dtype=torch.bfloat16, device="cuda")
    g.gmla_cache_dequantize_fp4(codes, scales, C)
    Q = rand_rows(rng, B, H * 128)
    W_k, W_v = (rand_rows(rng, H * 128, d_c) * d_c ** -0.5 for _ in range(2))
    O4, O16 = (torch.empty(B, H * 128, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    g.gmla_attend_decode_fp4(Q, codes, scales, L, W_k, W_v, O4, H, workspace=torch.empty(
        g.gmla_attend_decode_fp4_workspace_size(B, L, H, d_c), dtype=torch.uint8, device="cuda"))
    g.gmla_attend_decode(Q, C, L, W_k, W_v, O16, H, workspace=torch.empty(
        g.gmla_attend_decode_workspace_size(B, L, H, d_c), dtype=torch.uint8, device="cuda"))
    d = np.linalg.norm(f64(O4) - f64(O16)) / np.linalg.norm(f64(O16))
    assert d <= REL + 5e-3  # each side's own bar


def test_decode_twice_gives_the_same_bits(g):
    a, _, _ = decode_case(g, 5, 2500, 2500, 96, 512, lens=[2500, 1, 900, 64, 2400])
    b, _, _ = decode_case(g, 5, 2500, 2500, 96, 512, lens=[2500, 1, 900, 64, 2400])
    assert torch.equal(a, b)
