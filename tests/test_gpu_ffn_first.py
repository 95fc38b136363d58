"""The feed-forward kernels are set up by their own first launch (on the GPU): not by the first
product of a program that uses none of them, and inside a capture too.  Each case is a process of
its own, whose first calls these are."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

HEAD = """
import sys
import torch
import dense_fp16_tensor_gemm_gb300 as gnt
g = torch.Generator("cuda").manual_seed(1)
def normal(*s):
    return torch.randn(*s, generator=g, device="cuda").bfloat16()
a, out = normal(128, 64), torch.empty(128, 128, device="cuda")
torch.cuda.synchronize()
gnt.load()
free = torch.cuda.mem_get_info()[0]
gnt.gemm_nt(a, a, out=out)
torch.cuda.synchronize()
"""

MEMORY = HEAD + """
print((free - torch.cuda.mem_get_info()[0]) / 2 ** 20)
"""

CAPTURE = HEAD + """
tokens = int(sys.argv[1])
x, w = normal(tokens, 512), normal(600, 512) / 16
codes = torch.randint(0, 256, (600, 256), generator=g, device="cuda", dtype=torch.uint8)
scales = torch.rand(600, 4, generator=g, device="cuda").bfloat16() / 64
def run():
    h, gu = gnt.gated_linear(x, w, "gelu", keep=True)
    q, s = gnt.quantize_w4(w)
    return (h, gu, *gnt.gated_linear_backward(h, gu, x, w), q, s, gnt.linear_w4(x, codes, scales),
            gnt.gated_linear_w4(x, codes, scales))
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    captured = run()
graph.replay()
want = run()
gnt.gemm_nt_check()
assert all(torch.equal(a.contiguous().view(torch.uint8), b.contiguous().view(torch.uint8)) for a, b in zip(captured, want))
print("same")
"""


def child(code, *args):
    r = subprocess.run([sys.executable, "-c", code, *args], cwd=ROOT, capture_output=True, text=True, timeout=300,
                       env={**os.environ, "CUDA_MODULE_LOADING": "LAZY"})
    assert r.returncode == 0, r.stderr[-2000:]
    return r.stdout.split()[-1]


def test_the_first_product_brings_in_its_own_kernels():
    # 8 MB of device memory; with the feed-forward kernels, which it does not launch, 14
    assert float(child(MEMORY)) < 11


@pytest.mark.parametrize("tokens", [1, 12, 40, 100, 300])
def test_first_launches_inside_a_capture(tokens):
    assert child(CAPTURE, str(tokens)) == "same"
