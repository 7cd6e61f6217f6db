"""Eviction by score on the GPU: the choice, its order and the moved rows, all exact, against plain Python."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def g():
    import causal_head_latent_b200 as mod
    return mod


def choose(score, pos, n_rows, keep, sink, recent):
    """index list of one sequence, from the definition."""
    n = min(keep, n_rows)
    if n_rows == 0:
        return []
    newest = max(int(p) for p in pos[:n_rows])

    def rank(s):
        safe = pos[s] < sink or pos[s] > newest - recent
        x = float(score[s])
        return (0 if safe else 1, 0.0 if safe else (np.inf if x != x else -x), 1 if x != x and not safe else 0, s)
    kept = set(sorted(range(n_rows), key=rank)[:n])
    tails = sorted(s for s in kept if s >= n)
    return [j if j in kept else tails.pop(0) for j in range(n)]


def check(g, B, L, Lmax, keep, lens=None, sink=0, recent=0, inplace=True, fp4=False, with_pos=True, scores=None, seed=0,
          positions=None):
    rng = np.random.default_rng(seed + L + 3 * B)
    score = rng.random((B, Lmax)).astype(np.float32) if scores is None else np.array(scores, np.float32)
    pos = np.tile(np.arange(Lmax, dtype=np.int32), (B, 1)) if positions is None else np.array(positions, np.int32)
    widths = [64, 8] if fp4 else [136]
    rows = [torch.from_numpy(rng.integers(0, 256, (B, Lmax, w), dtype=np.uint8)).cuda() for w in widths]
    if not fp4:
        rows = [rows[0].view(torch.bfloat16)]
    ts, tp = torch.from_numpy(score.copy()).cuda(), torch.from_numpy(pos.copy()).cuda() if with_pos else None
    src = [r.view(torch.uint8).cpu().numpy().copy() for r in rows]
    Dmax = Lmax if inplace else min(keep, L) + 2
    more = {}
    if not inplace:
        more = dict(dst=[torch.full((B, Dmax, r.shape[2]), 7, dtype=torch.uint8, device="cuda").view(r.dtype)
                         if r.dtype == torch.uint8 else torch.full((B, Dmax, r.shape[2]), 7.0, dtype=r.dtype, device="cuda")
                         for r in rows],
                    dst_score=torch.full((B, Dmax), -5.0, device="cuda"),
                    dst_pos=torch.full((B, Dmax), -5, dtype=torch.int32, device="cuda") if with_pos else None)
    out_rows = more["dst"] if more else rows
    out_score, out_pos = (more["dst_score"], more["dst_pos"]) if more else (ts, tp)
    before = [t.clone() for t in out_rows], out_score.clone(), None if out_pos is None else out_pos.clone()
    tl = None if lens is None else torch.tensor(lens, dtype=torch.int32, device="cuda")
    index = torch.full((B, keep), 77, dtype=torch.int32, device="cuda")
    new_lens = torch.full((B,), 77, dtype=torch.int32, device="cuda") if tl is None else tl  # lens is written over
    ws = torch.full((g.gmla_cache_evict_workspace_size(B, L, keep),), 0xFF, dtype=torch.uint8, device="cuda")
    g.gmla_cache_evict(rows, ts, L, keep, index, new_lens, pos=tp, lens=tl, sink=sink, recent=recent, workspace=ws, **more)
    torch.cuda.synchronize()
    for b in range(B):
        n_rows = L if lens is None else min(max(lens[b], 0), L)
        want = choose(score[b], pos[b] if with_pos else np.arange(Lmax), n_rows, keep, sink, recent)
        n = len(want)
        assert int(new_lens[b]) == n
        assert index[b].tolist() == want + [-1] * (keep - n), b
        for t, s, old in zip(out_rows, src, before[0]):
            assert np.array_equal(t.view(torch.uint8)[b, :n].cpu().numpy(), s[b][np.array(want, int)])
            assert torch.equal(t.view(torch.uint8)[b, n:], old.view(torch.uint8)[b, n:])  # left as they were
        assert np.array_equal(out_score[b, :n].cpu().numpy(), score[b][np.array(want, int)], equal_nan=True)
        assert np.array_equal(out_score[b, n:].cpu().numpy(), before[1][b, n:].cpu().numpy(), equal_nan=True)
        if out_pos is not None:
            assert np.array_equal(out_pos[b, :n].cpu().numpy(), pos[b][np.array(want, int)])
            assert torch.equal(out_pos[b, n:], before[2][b, n:])


@pytest.mark.parametrize("inplace", [True, False])
@pytest.mark.parametrize("B,L,keep", [(1, 1, 1), (1, 2, 1), (2, 33, 32), (3, 100, 7), (1, 100, 100), (2, 100, 130),
                                      (2, 4097, 4096), (5, 999, 500), (1, 8193, 100), (2, 20001, 19000),
                                      (1, 300000, 100000), (1, 400000, 1000)])
def test_uniform(g, B, L, keep, inplace):
    check(g, B, L, L + 3, keep, sink=min(4, keep // 4), recent=min(64, keep // 2), inplace=inplace, fp4=B == 2)


@pytest.mark.parametrize("inplace", [True, False])
@pytest.mark.parametrize("lens", [[0, 1, 5, 6], [400, 0, 37, 32, -3, 5000], [9000, 3, 8999]])
def test_ragged(g, lens, inplace):
    check(g, len(lens), 9000, 9001, 32, lens=lens, sink=2, recent=10, inplace=inplace)


@pytest.mark.parametrize("L", [600, 20000])
@pytest.mark.parametrize("kind", ["equal", "two", "special", "negative", "sorted", "reversed"])
def test_ties_and_special_scores(g, kind, L):
    rng = np.random.default_rng(L)
    x = {"equal": np.full(L, 0.25), "two": rng.integers(0, 2, L).astype(float), "negative": -rng.random(L),
         "sorted": np.arange(L) * 1e-3, "reversed": -np.arange(L) * 1e-3,
         "special": rng.choice([np.nan, np.inf, -np.inf, 0.0, -0.0, 1e-45, -1e-45, 3e38, 1.0], L)}[kind]
    for keep in (1, L // 3, L - 1):
        check(g, 1, L, L, keep, scores=x[None])
    check(g, 1, L, L, L // 2, scores=x[None], sink=10, recent=20, inplace=False)


@pytest.mark.parametrize("L", [300000, 400000])
def test_ties_over_many_rows_per_warp(g, L):
    """More than 1024 rows per warp, some tied ones kept: ranks carry from one 1024 to the next."""
    rng = np.random.default_rng(L)
    x = rng.integers(0, 2, (1, L)).astype(float)
    check(g, 1, L, L, L // 3, scores=x, sink=3, recent=7)
    check(g, 1, L, L, 3 * L // 4, scores=x, inplace=False)


def test_protected_rows_after_earlier_evictions(g):
    """Positions out of order (rows filled holes earlier): protection goes by position, not by place."""
    rng = np.random.default_rng(9)
    L = 500
    pos = rng.permutation(2000)[:L][None]
    check(g, 1, L, L, 200, sink=50, recent=100, positions=pos)
    check(g, 1, L, L, 200, sink=50, recent=100, positions=pos, inplace=False, fp4=True)


def test_more_protected_than_kept(g):
    """Positions given twice can protect more rows than are kept: the lowest rows among them stay."""
    pos = np.zeros((1, 300), np.int32)
    check(g, 1, 300, 300, 20, sink=5, recent=5, positions=pos)


@pytest.mark.parametrize("L", [700, 9000])
def test_positions_at_the_ends_of_their_type(g, L):
    """Differences of 32-bit positions pass 32 bits."""
    rng = np.random.default_rng(L)
    ends = np.array([-2 ** 31, -2 ** 31 + 1, -1, 0, 5, 2 ** 31 - 2, 2 ** 31 - 1])
    for top in (7, 5, 2, 1):  # with and without large positions: the recent ones reach below the lowest
        pos = rng.choice(ends[:top], (2, L))
        for sink, recent in ((0, 0), (0, 3), (5, 0), (2, 100)):
            check(g, 2, L, L, 300, sink=sink, recent=recent, positions=pos, seed=top)


def test_without_positions(g):
    check(g, 2, 700, 720, 300, sink=4, recent=32, with_pos=False)


def test_repeated_steps_keep_the_best(g):
    """Decode loop: one row appended, one evicted, captured once and replayed; the survivors are those of a
    single choice, since scores do not change."""
    rng = np.random.default_rng(2)
    B, keep, extra = 3, 64, 40
    Lmax = keep + 1
    all_scores = rng.permutation(B * (keep + extra)).reshape(B, -1).astype(np.float32)
    C = torch.zeros(B, Lmax, 64, dtype=torch.bfloat16, device="cuda")
    score, pos = torch.zeros(B, Lmax, device="cuda"), torch.zeros(B, Lmax, dtype=torch.int32, device="cuda")
    score[:, :keep] = torch.from_numpy(all_scores[:, :keep])
    pos[:, :keep] = torch.arange(keep)
    C[:, :keep, 0] = pos[:, :keep].to(torch.bfloat16)
    index = torch.empty(B, keep, dtype=torch.int32, device="cuda")
    lens = torch.full((B,), Lmax, dtype=torch.int32, device="cuda")
    new_lens = torch.empty(B, dtype=torch.int32, device="cuda")
    ws = torch.empty(g.gmla_cache_evict_workspace_size(B, Lmax, keep), dtype=torch.uint8, device="cuda")
    args = dict(pos=pos, lens=lens, recent=1, workspace=ws)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    for step in range(extra):
        t = keep + step
        score[:, keep] = torch.from_numpy(all_scores[:, t]).cuda()
        pos[:, keep] = t
        C[:, keep, 0] = float(t)
        torch.cuda.synchronize()
        if step == 0:
            with torch.cuda.stream(side):
                g.gmla_cache_evict([C], score, Lmax, keep, index, new_lens, **args)
        elif step == 1:
            with torch.cuda.graph(graph, stream=side):
                g.gmla_cache_evict([C], score, Lmax, keep, index, new_lens, **args)
            graph.replay()
        else:
            graph.replay()
        torch.cuda.synchronize()
        assert new_lens.tolist() == [keep] * B
    for b in range(B):
        # replay the rule on the host
        live = list(range(keep))
        for t in range(keep, keep + extra):
            live.append(t)
            live.remove(min(live[:-1], key=lambda s: all_scores[b, s]))
        assert sorted(pos[b, :keep].tolist()) == live
        assert torch.equal(C[b, :keep, 0].float(), pos[b, :keep].to(torch.bfloat16).float())
        assert score[b, :keep].tolist() == [all_scores[b, p] for p in pos[b, :keep].tolist()]
