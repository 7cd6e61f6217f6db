"""Workloads of the compact latent cache: rows held in 4 bits, decode attention over
them, accumulated attention weights per cached row, and eviction by those weights.

``listed()`` names the cases, ``draw(rng)`` gives more of the same ranges, ``run``
is one pass: the operators in plain torch where ``own`` is false, the library's
calls where it is true.  ``exact`` is the definition in 64 bits.

The 4-bit row.  A latent row of d_c channels is cut into groups of 16.  A group
holds 16 four-bit codes e (sign, then magnitude 0, 0.5, 1, 1.5, 2, 3, 4, 6; the
even channel in the low half of a byte) and one 8-bit scale s (float8 e4m3):
c = cache_scale * s * e, with cache_scale a power of two for the whole cache.
"""
import math

import torch

own = False

HEAD = 128  # head width of the layer
GRID = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
SCALE_MIN = 2.0 ** -9  # smallest positive e4m3 number
SCALE_MAX = 448.0


def listed():
    return [
        # one new token per sequence, its latent stored at each sequence's own length
        dict(name="store_step", op="store", B=32, rows=1, d_c=512, scale_log2=0),
        # the latents of eight long prompts stored after their prefill
        dict(name="store_prompts", op="store", B=8, rows=65536, d_c=512, scale_log2=0),
        # cached rows expanded again for a prefill chunk that continues two short sequences
        dict(name="expand_chunk", op="expand", B=2, rows=4099, d_c=512, scale_log2=-1),
        # the same for one long cached context
        dict(name="expand_long", op="expand", B=1, rows=131072, d_c=512, scale_log2=0),
        # one short sequence: latency
        dict(name="decode_short", op="decode", B=1, L=1001, H=96, d_c=512, ragged=False, gate=True),
        # a batch of sequences of different lengths
        dict(name="decode_ragged", op="decode", B=8, L=16384, H=96, d_c=512, ragged=True, gate=True),
        # the largest decode: 32 sequences of 128K cached tokens
        dict(name="decode_long", op="decode", B=32, L=131072, H=96, d_c=512, ragged=False, gate=True),
        # accumulated weights of the same three shapes, over a bfloat16 cache
        dict(name="score_short", op="score", B=1, L=1001, H=96, d_c=512, ragged=False),
        dict(name="score_ragged", op="score", B=8, L=16384, H=96, d_c=512, ragged=True),
        dict(name="score_long", op="score", B=32, L=131072, H=96, d_c=512, ragged=False),
        # a decode step at a full budget: one row too many per sequence, evicted in place (4-bit rows)
        dict(name="evict_step", op="evict", B=32, L=4097, keep=4096, d_c=512, ragged=False, inplace=True, fp4=True),
        # long prompts cut down to a budget in another cache (bfloat16 rows)
        dict(name="evict_prompts", op="evict", B=8, L=131072, keep=8192, d_c=512, ragged=True, inplace=False, fp4=False),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["store", "expand", "decode", "decode", "score", "score", "evict", "evict"])
    d_c = rng.choice([64, 128, 192, 256, 320, 384, 448, 512, 512, 512])
    B = _log_int(rng, 1, 40)
    if op in ("store", "expand"):
        rows = _log_int(rng, 1, max(1, 131072 // B))
        return dict(op=op, B=B, rows=rows, d_c=d_c, scale_log2=rng.randint(-3, 3))
    L = _log_int(rng, 1, max(1, min(131072, 1500000 // B)))
    if op in ("decode", "score"):
        case = dict(op=op, B=B, L=L, H=rng.choice([1, 7, 16, 33, 64, 95, 96, 96]), d_c=d_c, ragged=rng.random() < 0.6)
        return dict(case, gate=rng.random() < 0.7) if op == "decode" else case
    return dict(op=op, B=B, L=L, keep=_log_int(rng, 1, L + 3), d_c=d_c, ragged=rng.random() < 0.6,
                inplace=rng.random() < 0.5, fp4=rng.random() < 0.5)


# ----------------------------------------------------------------------------- inputs

def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _latents(shape, g):
    """bfloat16 latents as a trained projection gives them: unit normal, a few channels louder."""
    *lead, d_c = shape
    loud = 0.5 + torch.rand(d_c, generator=g, device="cuda") + 4.0 * (torch.rand(d_c, generator=g, device="cuda") < 0.02)
    out = torch.empty(*lead, d_c, dtype=torch.bfloat16, device="cuda")
    flat = out.view(-1, d_c)
    for r in range(0, flat.shape[0], 1 << 18):
        part = flat[r:r + (1 << 18)]
        part.copy_(torch.randn(part.shape, generator=g, device="cuda") * loud)
    return out


def _lengths(case, g):
    B, L = case["B"], case["L"]
    if not case["ragged"]:
        return None
    share = torch.rand(B, generator=g, device="cuda")
    lens = (1 + share * share * (L - 1)).long().clamp(1, L)  # many short, few long
    lens[0] = L
    return lens.to(torch.int32)


def _weights(H, d_c, g):
    return (torch.randn(H * HEAD, d_c, generator=g, device="cuda") / math.sqrt(d_c)).to(torch.bfloat16)


def prepare(case, seed):
    g = _generator(seed)
    B, d_c, op = case["B"], case["d_c"], case["op"]
    s = dict(case)
    if op in ("store", "expand"):
        rows = case["rows"]
        s["cache_scale"] = 2.0 ** case["scale_log2"]
        C = _latents((B, rows, d_c), g) * s["cache_scale"]
        if op == "expand":
            s["codes"], s["scales"] = _quantize(C, s["cache_scale"])
            s["out"] = torch.empty_like(C)
            return s
        room = rows + 7
        s.update(C=C, room=room, at=torch.randint(0, 8, (B,), generator=g, device="cuda", dtype=torch.int32),
                 codes=torch.zeros(B, room, d_c // 2, dtype=torch.uint8, device="cuda"),
                 scales=torch.zeros(B, room, d_c // 16, dtype=torch.uint8, device="cuda"),
                 out=torch.empty(B, room, d_c, dtype=torch.bfloat16, device="cuda"))
        return s
    L = case["L"]
    s["lens"] = _lengths(case, g)
    if op in ("decode", "score"):
        H = case["H"]
        s["Q"] = torch.randn(B, H * HEAD, generator=g, device="cuda").to(torch.bfloat16)
        s["W_k"] = _weights(H, d_c, g)
        if op == "decode":
            s["W_v"] = _weights(H, d_c, g)
            s["G"] = torch.randn(B, H * HEAD, generator=g, device="cuda").to(torch.bfloat16) if case["gate"] else None
            s["codes"], s["scales"] = _quantize(_latents((B, L, d_c), g), 1.0)
            s["cache_scale"] = 1.0
            s["O"] = torch.empty(B, H * HEAD, dtype=torch.bfloat16, device="cuda")
        else:
            s["C"] = _latents((B, L, d_c), g)
            s["score"] = torch.rand(B, L, generator=g, device="cuda") * (H / L)  # one earlier step's worth
    else:
        s["score"] = torch.rand(B, L, generator=g, device="cuda").pow(4)
        s["pos"] = torch.arange(L, dtype=torch.int32, device="cuda").repeat(B, 1)
        s["sink"], s["recent"] = min(4, case["keep"] // 4), min(64, case["keep"] // 2)
        C = _latents((B, L, d_c), g)
        s["rows"] = list(_quantize(C, 1.0)) if case["fp4"] else [C]
        if not case["inplace"]:
            n = case["keep"]
            s["dst"] = [torch.zeros(B, n, r.shape[2], dtype=r.dtype, device="cuda") for r in s["rows"]]
            s["dst_score"] = torch.zeros(B, n, device="cuda")
            s["dst_pos"] = torch.zeros(B, n, dtype=torch.int32, device="cuda")
        s["index"] = torch.empty(B, case["keep"], dtype=torch.int32, device="cuda")
        s["new_lens"] = torch.empty(B, dtype=torch.int32, device="cuda")
    if own:
        import causal_head_latent_b200 as gmla
        size = {"decode": gmla.gmla_attend_decode_fp4_workspace_size,
                "score": gmla.gmla_cache_score_workspace_size}.get(op)
        n = size(B, L, case["H"], d_c) if size else gmla.gmla_cache_evict_workspace_size(B, L, case["keep"])
        s["workspace"] = torch.empty(max(16, n), dtype=torch.uint8, device="cuda")
    return s


# ----------------------------------------------------------------------------- plain forms

def _quantize(C, cache_scale):
    """Packed codes and scale bytes of bfloat16 rows, piece by piece for long ones."""
    *lead, d_c = C.shape
    flat = C.reshape(-1, d_c)
    codes = torch.empty(flat.shape[0], d_c // 2, dtype=torch.uint8, device=C.device)
    scales = torch.empty(flat.shape[0], d_c // 16, dtype=torch.uint8, device=C.device)
    for r in range(0, flat.shape[0], 1 << 18):
        x = flat[r:r + (1 << 18)].float().view(-1, d_c // 16, 16) / cache_scale
        x = torch.nan_to_num(x, nan=0.0)
        a = x.abs()
        top = a.amax(-1).clamp(max=6 * SCALE_MAX)
        s = (top / 6).clamp(min=SCALE_MIN).to(torch.float8_e4m3fn)
        sf = s.float().unsqueeze(-1)
        # half-way points between neighbouring magnitudes; a tie goes to the even code
        mag = (a > 0.25 * sf).to(torch.uint8)
        for half, even_up in ((0.75, True), (1.25, False), (1.75, True), (2.5, False), (3.5, True), (5.0, False)):
            mag += (a >= half * sf) if even_up else (a > half * sf)
        code = torch.where((x < 0) & (mag > 0), mag + 8, mag).view(-1, d_c)
        codes[r:r + (1 << 18)] = code[:, 0::2] | (code[:, 1::2] << 4)
        scales[r:r + (1 << 18)] = s.view(torch.uint8)
    return codes.view(*lead, d_c // 2), scales.view(*lead, d_c // 16)


def _values(codes, scales, cache_scale):
    """float32 rows that packed codes and scales stand for."""
    *lead, half = codes.shape
    grid = torch.tensor(GRID + tuple(-v for v in GRID), device=codes.device)
    e = torch.stack((grid[(codes & 15).int()], grid[(codes >> 4).int()]), -1).view(*lead, half // 8, 16)
    s = scales.view(torch.float8_e4m3fn).float().unsqueeze(-1)
    return (e * (s * cache_scale)).view(*lead, half * 2)


def _visible(s):
    if s["lens"] is None:
        return None
    return torch.arange(s["L"], device="cuda")[None, :] < s["lens"][:, None]


def _probabilities(Q, W_k, C, H, seen):
    """Softmax over the visible cached rows of one query per sequence: [B, H, L], float32."""
    B, d_c = Q.shape[0], C.shape[-1]
    q = torch.einsum("bhd,hdc->bhc", Q.float().view(B, H, HEAD), W_k.float().view(H, HEAD, d_c))
    z = torch.matmul(q / math.sqrt(HEAD), C.transpose(1, 2))
    if seen is not None:
        z.masked_fill_(~seen[:, None, :], -math.inf)
    z -= z.amax(-1, keepdim=True)
    z.exp_()
    z /= z.sum(-1, keepdim=True)
    return z


def _store(s):
    codes, scales = _quantize(s["C"], s["cache_scale"])
    at = s["at"].long()[:, None] + torch.arange(s["rows"], device="cuda")
    b = torch.arange(s["B"], device="cuda")[:, None]
    s["codes"][b, at] = codes
    s["scales"][b, at] = scales
    return _values(s["codes"], s["scales"], s["cache_scale"]).to(torch.bfloat16)


def _decode(s):
    B, H, d_c = s["B"], s["H"], s["d_c"]
    C = _values(s["codes"], s["scales"], s["cache_scale"])
    p = _probabilities(s["Q"], s["W_k"], C, H, _visible(s))
    ctx = torch.matmul(p, C)
    o = torch.einsum("bhc,hdc->bhd", ctx, s["W_v"].float().view(H, HEAD, d_c)).reshape(B, H * HEAD)
    if s["G"] is not None:
        o = o * torch.sigmoid(s["G"].float())
    return o.to(torch.bfloat16)


def _score(s):
    s["score"] += _probabilities(s["Q"], s["W_k"], s["C"].float(), s["H"], _visible(s)).sum(1)
    return s["score"]


def _evict(s):
    B, L, keep = s["B"], s["L"], s["keep"]
    at = torch.arange(L, device="cuda")[None, :]
    lens = s["lens"][:, None].long() if s["lens"] is not None else torch.full((B, 1), L, device="cuda")
    seen = at < lens
    n = lens.clamp(max=keep)
    newest = torch.where(seen, s["pos"], -1).amax(1, keepdim=True)
    safe = (s["pos"] < s["sink"]) | (s["pos"] > newest - s["recent"])
    x = s["score"].double()
    x = torch.where(torch.isnan(x), -math.inf, x.clamp(-1e300, 1e300))
    x = torch.where(safe, math.inf, x)
    x = torch.where(seen, x, -math.inf)
    rank = torch.sort(x, dim=1, descending=True, stable=True).indices
    kept = torch.zeros(B, L, dtype=torch.bool, device="cuda")
    kept.scatter_(1, rank, at.expand(B, L) < n)
    front = at < n
    hole, tail = front & ~kept, kept & ~front
    tails = torch.sort(tail.to(torch.uint8), dim=1, descending=True, stable=True).indices  # tail rows first, ascending
    from_row = torch.where(hole, tails.gather(1, (hole.cumsum(1) - 1).clamp(min=0)), at.expand(B, L))
    width = min(keep, L)
    idx = torch.where(front, from_row, -1)[:, :width]
    s["index"].fill_(-1)
    s["index"][:, :width] = idx.to(torch.int32)
    s["new_lens"].copy_(n[:, 0])
    pick = idx.clamp(min=0)
    live = idx >= 0
    out = [s["index"], s["new_lens"]]
    if s["inplace"]:
        pairs = [(r, r) for r in s["rows"]] + [(s["score"], s["score"]), (s["pos"], s["pos"])]
    else:
        pairs = list(zip(s["rows"], s["dst"])) + [(s["score"], s["dst_score"]), (s["pos"], s["dst_pos"])]
    for src, dst in pairs:
        wide = src.dim() == 3
        take = pick[..., None].expand(-1, -1, src.shape[2]) if wide else pick
        got = src.gather(1, take)
        m = live[..., None] if wide else live
        dst[:, :width] = torch.where(m, got, dst[:, :width])
        out.append(dst)
    return out


# ----------------------------------------------------------------------------- one pass

def _answer(out, s):
    """Evicted caches as what they stand for: 4-bit codes as whole bytes, scales as float8."""
    if not s["fp4"]:
        return out
    return out[:3] + [out[3].view(torch.float8_e4m3fn)] + out[4:]


def run(s):
    op = s["op"]
    if not own:
        if op == "store":
            return _store(s)
        if op == "expand":
            return _values(s["codes"], s["scales"], s["cache_scale"]).to(torch.bfloat16)
        if op == "decode":
            return _decode(s)
        if op == "score":
            return _score(s)
        return _answer(_evict(s), s)
    import causal_head_latent_b200 as gmla
    if op == "store":
        gmla.gmla_cache_quantize_fp4(s["C"], s["codes"], s["scales"], cache_scale=s["cache_scale"], row_of=s["at"])
        gmla.gmla_cache_dequantize_fp4(s["codes"], s["scales"], s["out"], cache_scale=s["cache_scale"])
        return s["out"]
    if op == "expand":
        gmla.gmla_cache_dequantize_fp4(s["codes"], s["scales"], s["out"], cache_scale=s["cache_scale"])
        return s["out"]
    if op == "decode":
        gmla.gmla_attend_decode_fp4(s["Q"], s["codes"], s["scales"], s["L"], s["W_k"], s["W_v"], s["O"], s["H"],
                                    cache_scale=s["cache_scale"], lens=s["lens"], G=s["G"], workspace=s["workspace"])
        return s["O"]
    if op == "score":
        gmla.gmla_cache_score(s["Q"], s["C"], s["L"], s["W_k"], s["score"], s["H"], lens=s["lens"],
                              workspace=s["workspace"])
        return s["score"]
    more = {} if s["inplace"] else dict(dst=s["dst"], dst_score=s["dst_score"], dst_pos=s["dst_pos"])
    gmla.gmla_cache_evict(s["rows"], s["score"], s["L"], s["keep"], s["index"], s["new_lens"], pos=s["pos"],
                          lens=s["lens"], sink=s["sink"], recent=s["recent"], workspace=s["workspace"], **more)
    out = s["rows"] + [s["score"], s["pos"]] if s["inplace"] else s["dst"] + [s["dst_score"], s["dst_pos"]]
    return _answer([s["index"], s["new_lens"]] + out, s)


# ----------------------------------------------------------------------------- what a pass cannot do without

def work(case):
    B, d_c, op = case["B"], case["d_c"], case["op"]
    packed, wide = d_c // 2 + d_c // 16, 2 * d_c
    if op == "store":  # rows in, packed rows out, and the whole small cache read back as bfloat16
        return dict(bytes=B * (case["rows"] * (wide + packed) + (case["rows"] + 7) * (packed + wide)), flops=0)
    if op == "expand":
        return dict(bytes=B * case["rows"] * (packed + wide), flops=0)
    L = case["L"]
    # a ragged batch holds one full sequence, and a third of the length on average in the others
    rows = L + (B - 1) * (L + 2) / 3 if case["ragged"] else B * L
    if op in ("decode", "score"):
        H = case["H"]
        side = 2 * H * HEAD * (d_c + B)  # W_k and Q
        if op == "decode":
            return dict(bytes=rows * packed + 2 * side + 2 * B * H * HEAD * (1 if case["gate"] else 0),
                        flops=rows * H * d_c * 4 + 4 * B * H * HEAD * d_c)
        return dict(bytes=rows * (wide + 8) + side, flops=rows * H * d_c * 2 + 2 * B * H * HEAD * d_c)
    row = (packed if case["fp4"] else wide) + 8
    n = min(case["keep"], L)
    # in place only the kept rows behind the budget move; elsewhere every kept row does
    moved = n * (L - n) / L if case["inplace"] else n
    share = rows / (B * L)
    return dict(bytes=rows * 8 + B * 4 * (case["keep"] + 1) + 2 * B * moved * share * row, flops=0)


# ----------------------------------------------------------------------------- definition in 64 bits

def _nearest64(x, grid):
    """Nearest magnitude of an ascending grid, a tie to the even entry."""
    hi = torch.searchsorted(grid, x.contiguous()).clamp(1, grid.numel() - 1)
    lo = hi - 1
    below, above = x - grid[lo], grid[hi] - x
    up = (above < below) | ((above == below) & (hi % 2 == 0))
    return grid[torch.where(up, hi, lo)]


def _rounded64(C, cache_scale):
    """What the rows C stand for once they are held in 4 bits."""
    e4m3 = sorted({(m / 8 + (1 if e else 0)) * 2.0 ** (max(e, 1) - 7) for e in range(16) for m in range(8)
                   if (e, m) not in ((0, 0), (15, 7))})
    # an even e4m3 number has an even last bit: zero in front keeps that parity
    scale_grid = torch.tensor([0.0] + e4m3, dtype=torch.float64, device=C.device)
    grid = torch.tensor(GRID, dtype=torch.float64, device=C.device)
    x = C.double().unflatten(-1, (-1, 16)) / cache_scale
    s = _nearest64((x.abs().amax(-1) / 6).clamp(SCALE_MIN, SCALE_MAX), scale_grid).unsqueeze(-1)
    return (torch.sign(x) * _nearest64((x.abs() / s).clamp(max=6), grid) * s * cache_scale).flatten(-2)


def _unpacked64(codes, scales, cache_scale):
    """Rows from packed bytes, by the bits: value = (-1)^s 2^(e-1) (1 + m/2), or m/2 for e = 0."""
    low, high = codes.int() & 15, codes.int() >> 4
    n = torch.stack((low, high), -1).flatten(-2)
    e, m = (n >> 1) & 3, n & 1
    mag = torch.where(e == 0, 0.5 * m, torch.ldexp(1.0 + 0.5 * m.double(), e - 1)).double()
    sb = scales.int()
    se, sm = (sb >> 3) & 15, sb & 7
    s = torch.where(se == 0, sm.double() * 2.0 ** -9, torch.ldexp(1.0 + sm.double() / 8, se - 7)).double()
    return torch.where(n >= 8, -mag, mag) * s.repeat_interleave(16, -1) * cache_scale


def exact(case, seed):
    op = case["op"]
    if op == "evict":
        return None  # a choice and copies: whole numbers and rows as they are
    s = prepare(case, seed)
    if op == "store":
        out = torch.zeros(s["B"], s["room"], s["d_c"], dtype=torch.float64, device="cuda")
        for b in range(s["B"]):
            a = int(s["at"][b])
            for r in range(0, s["rows"], 1 << 15):
                part = s["C"][b, r:r + (1 << 15)]
                out[b, a + r:a + r + part.shape[0]] = _rounded64(part, s["cache_scale"])
        return out
    if op == "expand":
        return _unpacked64(s["codes"], s["scales"], s["cache_scale"])
    B, H, L, d_c = s["B"], s["H"], s["L"], s["d_c"]
    Wk = s["W_k"].double().view(H, HEAD, d_c)
    out = []
    for b in range(B):
        n = int(s["lens"][b]) if s["lens"] is not None else L
        q = s["Q"][b].double().view(H, HEAD, 1)
        c = _unpacked64(s["codes"][b, :n], s["scales"][b, :n], 1.0) if op == "decode" else s["C"][b, :n].double()
        z = torch.empty(H, n, dtype=torch.float64, device="cuda")
        for r in range(0, n, 1 << 14):  # keys rebuilt from the latents, head by head
            part = c[r:r + (1 << 14)]
            keys = torch.matmul(Wk, part.t())  # [H, HEAD, rows]
            z[:, r:r + part.shape[0]] = (keys * q).sum(1)
        a = torch.softmax(z / math.sqrt(HEAD), dim=-1)
        if op == "score":
            add = s["score"][b].double().clone()
            add[:n] += a.sum(0)
            out.append(add)
            continue
        o = torch.matmul(s["W_v"].double().view(H, HEAD, d_c), torch.matmul(a, c).unsqueeze(-1)).reshape(-1)
        out.append(o / (1 + torch.exp(-s["G"][b].double())) if s["G"] is not None else o)
    return torch.stack(out)
