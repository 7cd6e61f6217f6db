"""The compact-cache calls together, as a serving loop makes them, next to the layer's own calls.

Reference: the same loop in float64 over the values that the library itself stored (bfloat16 queries and latents as
gmla_latent_project wrote them), so every step is compared on equal inputs and errors do not pile up.
"""
import numpy as np
import pytest
import torch

from tests import fp4_ref
from tests.gpu_util import assert_parity, f64
from tests.test_gpu_fp4 import REL, plain_decode
from tests.test_gpu_score import REL as SCORE_REL, plain as plain_score

pytestmark = pytest.mark.gpu
H, D, DC = 4, 128, 128
DM = H * D


@pytest.fixture(scope="module")
def g():
    import causal_head_latent_b200 as mod
    return mod


@pytest.fixture(scope="module")
def weights():
    rng = np.random.default_rng(100)
    def w(o, i):
        return torch.from_numpy((rng.standard_normal((o, i)) * i ** -0.5).astype(np.float32)).to(torch.bfloat16).cuda()
    return dict(W_q=w(DM, DM), W_g=w(DM, DM), W_c=w(DC, DM), W_k=w(DM, DC), W_v=w(DM, DC), W_o=w(DM, DM))


def hidden(rng, B, T):
    return torch.from_numpy(rng.standard_normal((B, T, DM)).astype(np.float32)).to(torch.bfloat16).cuda()


def ws(n):
    return torch.empty(max(16, n), dtype=torch.uint8, device="cuda")


def test_decode_loop_over_a_bounded_bf16_cache(g, weights):
    """Prompts, then decode steps that append, attend, accumulate weights and evict back to a budget in place."""
    rng = np.random.default_rng(0)
    B, prompt, budget, steps = 3, 90, 60, 12
    Lmax = prompt + 1
    w = weights
    C = torch.zeros(B, Lmax, DC, dtype=torch.bfloat16, device="cuda")
    score = torch.zeros(B, Lmax, device="cuda")
    pos = torch.zeros(B, Lmax, dtype=torch.int32, device="cuda")
    pos[:, :prompt] = torch.arange(prompt)
    X = hidden(rng, B, prompt)
    g.gmla_latent_project(X, None, None, w["W_c"], None, None, C=C, cache_len_max=Lmax)
    index = torch.empty(B, budget, dtype=torch.int32, device="cuda")
    lens = torch.empty(B, dtype=torch.int32, device="cuda")
    sw, ew = ws(g.gmla_cache_score_workspace_size(B, Lmax, H, DC)), ws(g.gmla_cache_evict_workspace_size(B, Lmax, budget))
    n, live = prompt, [list(range(prompt)) for _ in range(B)]
    want_score = np.zeros((B, prompt + steps))  # by position
    for t in range(steps):
        at = prompt + t  # position of the new token; its latent goes to row n
        x = hidden(rng, B, 1)
        Q, G = (torch.empty(B, 1, DM, dtype=torch.bfloat16, device="cuda") for _ in range(2))
        g.gmla_latent_project(x, w["W_q"], w["W_g"], w["W_c"], None, None, Q=Q, G=G, C=C, cache_len_max=Lmax, cache_pos=n)
        pos[:, n] = at
        score[:, n] = 0.0
        for b in range(B):
            live[b].append(at)
        n += 1
        O = torch.empty(B, DM, dtype=torch.bfloat16, device="cuda")
        g.gmla_attend_decode(Q[:, 0], C, n, w["W_k"], w["W_v"], O, H, G=G[:, 0].contiguous(),
                             workspace=ws(g.gmla_attend_decode_workspace_size(B, n, H, DC)))
        ref = plain_decode(f64(Q)[:, 0], f64(C), [n] * B, f64(w["W_k"]), f64(w["W_v"]), H, f64(G)[:, 0])
        assert_parity(f64(O), ref, f"decode step {t}")
        before = f64(score)
        g.gmla_cache_score(Q[:, 0].contiguous(), C, n, w["W_k"], score, H, workspace=sw)
        add = plain_score(f64(Q)[:, 0], f64(C), [n] * B, f64(w["W_k"]), H)
        assert np.linalg.norm(f64(score) - before - add) <= (SCORE_REL + 2.0 ** -22) * np.linalg.norm(before + add)
        if n > budget:
            s, p = f64(score), pos.cpu().numpy()
            g.gmla_cache_evict([C], score, n, budget, index, lens, pos=pos, sink=2, recent=8, workspace=ew)
            assert lens.tolist() == [budget] * B
            for b in range(B):
                order = sorted(range(n), key=lambda r: (not (p[b, r] < 2 or p[b, r] > at - 8), -s[b, r], r))
                live[b] = sorted(int(p[b, r]) for r in order[:budget])
                assert sorted(pos[b, :budget].tolist()) == live[b]
            n = budget
    g.gmla_get_device_status()


def test_decode_over_an_evicted_4_bit_cache(g, weights):
    """Prompts of different lengths stored in 4 bits, cut to a budget in a smaller cache, one token appended per
    sequence at its own length, attended to; then the cached rows expanded for a chunk that continues them."""
    rng = np.random.default_rng(1)
    B, Lmax, budget = 4, 200, 64
    w = weights
    lens0 = [200, 37, 64, 130]
    X = hidden(rng, B, Lmax)
    C = torch.empty(B, Lmax, DC, dtype=torch.bfloat16, device="cuda")
    g.gmla_latent_project(X, None, None, w["W_c"], None, None, C=C, cache_len_max=Lmax)
    codes = torch.full((B, Lmax, DC // 2), 0xFF, dtype=torch.uint8, device="cuda")
    scales = torch.full((B, Lmax, DC // 16), 0xFF, dtype=torch.uint8, device="cuda")
    g.gmla_cache_quantize_fp4(C, codes, scales)
    # weights of the last prompt token's query go by the rows as they are held
    held = torch.empty_like(C)
    g.gmla_cache_dequantize_fp4(codes, scales, held)
    Q = torch.empty(B, 1, DM, dtype=torch.bfloat16, device="cuda")
    g.gmla_latent_project(hidden(rng, B, 1), w["W_q"], None, None, None, None, Q=Q)
    lens = torch.tensor(lens0, dtype=torch.int32, device="cuda")
    score = torch.zeros(B, Lmax, device="cuda")
    g.gmla_cache_score(Q[:, 0].contiguous(), held, Lmax, w["W_k"], score, H, lens=lens,
                       workspace=ws(g.gmla_cache_score_workspace_size(B, Lmax, H, DC)))
    room = budget + 8
    small = [torch.full((B, room, t.shape[2]), 0xFF, dtype=torch.uint8, device="cuda") for t in (codes, scales)]
    s2 = torch.zeros(B, room, device="cuda")
    index = torch.empty(B, budget, dtype=torch.int32, device="cuda")
    sc = f64(score)
    g.gmla_cache_evict([codes, scales], score, Lmax, budget, index, lens, lens=lens, sink=1, recent=4, dst=small,
                       dst_score=s2, workspace=ws(g.gmla_cache_evict_workspace_size(B, Lmax, budget)))
    n = [min(x, budget) for x in lens0]
    assert lens.tolist() == n
    src_c, src_s = codes.cpu().numpy(), scales.cpu().numpy()
    for b in range(B):
        idx = index[b, :n[b]].tolist()
        order = sorted(range(lens0[b]), key=lambda r: (not (r < 1 or r > lens0[b] - 1 - 4), -sc[b, r], r))
        assert sorted(idx) == sorted(order[:n[b]])
        assert np.array_equal(small[0][b, :n[b]].cpu().numpy(), src_c[b, idx])
        assert np.array_equal(small[1][b, :n[b]].cpu().numpy(), src_s[b, idx])
    # one decode step: append at each sequence's own length, then attend
    x = hidden(rng, B, 1)
    G, c_new = torch.empty_like(Q), torch.empty(B, 1, DC, dtype=torch.bfloat16, device="cuda")
    g.gmla_latent_project(x, w["W_q"], w["W_g"], w["W_c"], None, None, Q=Q, G=G, C=c_new, cache_len_max=1)
    g.gmla_cache_quantize_fp4(c_new, small[0], small[1], row_of=lens)
    lens.add_(1)
    O = torch.empty(B, DM, dtype=torch.bfloat16, device="cuda")
    g.gmla_attend_decode_fp4(Q[:, 0].contiguous(), small[0], small[1], room, w["W_k"], w["W_v"], O, H, lens=lens,
                             G=G[:, 0].contiguous(),
                             workspace=ws(g.gmla_attend_decode_fp4_workspace_size(B, room, H, DC)))
    v = fp4_ref.values(small[0].cpu().numpy(), np.minimum(small[1].cpu().numpy(), 126))
    ref = plain_decode(f64(Q)[:, 0], v, [k + 1 for k in n], f64(w["W_k"]), f64(w["W_v"]), H, f64(G)[:, 0])
    for b in range(B):
        assert np.linalg.norm(f64(O)[b] - ref[b]) <= REL * np.linalg.norm(ref[b])
    # a chunk that continues sequence 0 needs its cached rows as bfloat16 keys and values
    m = n[0] + 1
    back = torch.empty(B, m, DC, dtype=torch.bfloat16, device="cuda")
    g.gmla_cache_dequantize_fp4(small[0], small[1], back, rows=m)
    K, V = (torch.empty(1, m, DM, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    g.gmla_expand_kv(back[:1].contiguous(), 0, m, W_k=w["W_k"], W_v=w["W_v"], K=K, V=V)
    assert_parity(f64(K)[0], v[0, :m] @ f64(w["W_k"]).T, "keys")
    assert_parity(f64(V)[0], v[0, :m] @ f64(w["W_v"]).T, "values")
    g.gmla_get_device_status()


def test_two_sequences_of_calls_at_once(g, weights):
    """Two streams, a workspace each: the same results as one after the other."""
    rng = np.random.default_rng(2)
    B, L = 8, 3000
    sides, outs = [torch.cuda.Stream() for _ in range(2)], []
    state = []
    for k in range(2):
        C = torch.from_numpy(rng.standard_normal((B, L, DC)).astype(np.float32)).to(torch.bfloat16).cuda()
        Q = torch.from_numpy(rng.standard_normal((B, DM)).astype(np.float32)).to(torch.bfloat16).cuda()
        codes = torch.zeros(B, L, DC // 2, dtype=torch.uint8, device="cuda")
        scales = torch.zeros(B, L, DC // 16, dtype=torch.uint8, device="cuda")
        state.append((C, Q, codes, scales, ws(g.gmla_attend_decode_fp4_workspace_size(B, L, H, DC)),
                      ws(g.gmla_cache_score_workspace_size(B, L, H, DC))))

    def work(k):
        C, Q, codes, scales, w1, w2 = state[k]
        O = torch.empty(B, DM, dtype=torch.bfloat16, device="cuda")
        score = torch.zeros(B, L, device="cuda")
        g.gmla_cache_quantize_fp4(C, codes, scales)
        for _ in range(5):
            g.gmla_attend_decode_fp4(Q, codes, scales, L, weights["W_k"], weights["W_v"], O, H, workspace=w1)
            g.gmla_cache_score(Q, C, L, weights["W_k"], score, H, workspace=w2)
        return O, score

    alone = [work(k) for k in range(2)]
    torch.cuda.synchronize()
    for _ in range(3):
        outs = []
        for k in range(2):
            with torch.cuda.stream(sides[k]):
                outs.append(work(k))
        torch.cuda.synchronize()
        for a, o in zip(alone, outs):
            assert torch.equal(a[0], o[0]) and torch.equal(a[1], o[1])
    g.gmla_get_device_status()
