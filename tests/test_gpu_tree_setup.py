"""A handle's first attention over a 4-bit cache, which sets its kernel up, inside a captured graph."""
import os
import subprocess
import sys

import pytest
import torch

from test_gpu_tree import tree  # noqa: F401

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

FIRST = """
import torch
from serial_draft_head_gb300 import KVCache, Tree
torch.manual_seed(1)
T, cap, layout = {T}, {cap}, {layout!r}
cache = KVCache.zeros(40, 16, 2, 64, torch.uint8)
if layout == "slots":
    cache = KVCache(*(x.contiguous() for x in (cache.k, cache.v, cache.k_scale, cache.v_scale)))
for x in (cache.k, cache.v):
    x.copy_(torch.randint(0, 256, x.shape, device="cuda").to(torch.uint8))
for x in (cache.k_scale, cache.v_scale):
    x.copy_(torch.randint(90, 110, x.shape, device="cuda").to(torch.uint8))
pages = torch.randperm(40, device="cuda").int().view(2, 20)
length = torch.tensor([200, 33], dtype=torch.int32, device="cuda")
first = torch.tensor([0, T, 2 * T], dtype=torch.int32, device="cuda")
q = torch.randn(2 * T, 8, 64, device="cuda").bfloat16()
a, b = (Tree(8, 2, 64, max_requests=2, max_nodes=T) for _ in range(2))
out, lse = torch.zeros_like(q), torch.zeros(2 * T, 8, device="cuda")
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    a.attend(q, cache, pages, length, first, softcap=cap, out=out, lse=lse)
graph.replay()
got, got_lse = b.attend(q, cache, pages, length, first, softcap=cap)
assert a.status() == 0 and b.status() == 0
assert torch.isfinite(out).all() and out.abs().max() > 0
assert torch.equal(out, got) and torch.equal(lse, got_lse)
print("right")
"""


@pytest.mark.parametrize("T,cap,layout", [(1, 0.0, "heads"), (1, 2.0, "heads"), (4, 0.0, "slots"), (8, 0.0, "heads"),
                                          (30, 0.0, "heads")])
def test_first_attention_over_4_bits_in_a_graph(tree, T, cap, layout):  # noqa: F811
    """In a process of its own, where nothing has loaded the kernel before."""
    res = subprocess.run([sys.executable, "-c", FIRST.format(T=T, cap=cap, layout=layout)], cwd=ROOT,
                         capture_output=True, text=True, timeout=300)
    assert res.returncode == 0 and res.stdout.strip() == "right", res.stderr[-2000:]
