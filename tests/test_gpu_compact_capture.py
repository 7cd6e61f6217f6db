"""The compact-cache calls as the first use of the library in a process, inside a graph capture, replayed."""
import subprocess
import sys

import pytest

from tests.conftest import ROOT

pytestmark = pytest.mark.gpu

CHILD = r"""
import torch
import causal_head_latent_b200 as g
torch.manual_seed(0)
B, L, H, dc = 3, 10000, 8, 128
dev = "cuda"
C = torch.randn(B, L, dc, device=dev).bfloat16()
codes = torch.zeros(B, L, dc // 2, dtype=torch.uint8, device=dev)
scales = torch.zeros(B, L, dc // 16, dtype=torch.uint8, device=dev)
back = torch.zeros_like(C)
Q = torch.randn(B, H * 128, device=dev).bfloat16()
W = torch.randn(H * 128, dc, device=dev).mul_(dc ** -0.5).bfloat16()
O = torch.zeros(B, H * 128, dtype=torch.bfloat16, device=dev)
score = torch.zeros(B, L, device=dev)
index = torch.zeros(B, 64, dtype=torch.int32, device=dev)
n = torch.zeros(B, dtype=torch.int32, device=dev)
dst = [torch.zeros(B, 64, dc, dtype=torch.bfloat16, device=dev)]
ds = torch.zeros(B, 64, device=dev)
def ws(k): return torch.empty(k, dtype=torch.uint8, device=dev)
w1, w2 = ws(g.gmla_attend_decode_fp4_workspace_size(B, L, H, dc)), ws(g.gmla_cache_score_workspace_size(B, L, H, dc))
w3 = ws(g.gmla_cache_evict_workspace_size(B, L, 64))
def run():
    g.gmla_cache_quantize_fp4(C, codes, scales)
    g.gmla_cache_dequantize_fp4(codes, scales, back)
    g.gmla_attend_decode_fp4(Q, codes, scales, L, W, W, O, H, workspace=w1)
    g.gmla_cache_score(Q, back, L, W, score, H, decay=0.0, workspace=w2)
    g.gmla_cache_evict([back], score, L, 64, index, n, dst=dst, dst_score=ds, workspace=w3)
    return [t.clone() for t in (codes, scales, back, O, score, index, n, dst[0], ds)]
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    got = run()
graph.replay()
torch.cuda.synchronize()
want = run()
g.gmla_get_device_status()
assert all(torch.equal(a, b) for a, b in zip(got, want))
assert float(score.sum()) > 0
print("same")
"""


def test_first_calls_are_captured():
    r = subprocess.run([sys.executable, "-c", CHILD], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "same" in r.stdout, r.stdout + r.stderr
