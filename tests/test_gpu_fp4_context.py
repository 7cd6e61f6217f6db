"""Decode over 4-bit rows: the context c^ enters the value product with 16 bits, not rounded once to bfloat16."""
import numpy as np
import pytest
import torch

from tests.gpu_util import f64
from tests.test_gpu_fp4 import empty_cache

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def g():
    import causal_head_latent_b200 as mod
    return mod


@pytest.mark.parametrize("B", [1, 2, 3, 7, 12, 40])  # sixteen warps to a sequence down to one
@pytest.mark.parametrize("H,d_c", [(1, 64), (96, 512), (5, 320)])
def test_a_small_difference_of_large_contexts_is_kept(g, B, H, d_c):
    """Two rows of equal weight hold 768 and 3 in channel a, 768 and 0 in channel b (all held exactly): c^ is 385.5 and 384,
    and a value that takes their difference is 1.5.  With c^ in bfloat16 (steps of 2 there) it would be 2 or 0."""
    a, b = 0, d_c - 1
    rows = torch.zeros(B, 2, d_c, dtype=torch.bfloat16, device="cuda")
    rows[:, 0, a] = rows[:, 0, b] = 768.0
    rows[:, 1, a] = 3.0
    codes, scales = empty_cache(B, 2, d_c)
    g.gmla_cache_quantize_fp4(rows, codes, scales)
    Q = torch.zeros(B, H * 128, dtype=torch.bfloat16, device="cuda")
    W_k = torch.ones(H * 128, d_c, dtype=torch.bfloat16, device="cuda")
    W_v = torch.zeros(H * 128, d_c, dtype=torch.bfloat16, device="cuda")
    W_v[:, a], W_v[:, b] = 1.0, -1.0
    O = torch.empty(B, H * 128, dtype=torch.bfloat16, device="cuda")
    ws = torch.empty(g.gmla_attend_decode_fp4_workspace_size(B, 2, H, d_c), dtype=torch.uint8, device="cuda")
    g.gmla_attend_decode_fp4(Q, codes, scales, 2, W_k, W_v, O, H, workspace=ws)
    assert np.array_equal(f64(O), np.full((B, H * 128), 1.5))
