"""GPU test of a process whose first call of the library is captured into a CUDA
graph: what the library sets up once per device (status word, memory pool,
kernel attributes) is set up within the capture.
"""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

PROGRAM = """
import sys
import torch
import linear_attention_sequence_gated_gb300 as gdn

op, mode = sys.argv[1:]
gen = torch.Generator(device="cuda")
gen.manual_seed(1)
B, Hkv, n, d, page = 2, 2, 5000, 128, 64
pages = -(-n // page)
cache = torch.zeros((B * pages, Hkv, page // 16, 18 * d), dtype=torch.uint8, device="cuda")
table = torch.arange(B * pages, dtype=torch.int32, device="cuda").reshape(B, pages)
lens = torch.tensor([n, 77], dtype=torch.int32, device="cuda")
k, v = (torch.randn((B, Hkv, n, d), generator=gen, device="cuda").bfloat16() for _ in range(2))
q = torch.randn((B, 8, 1, d), generator=gen, device="cuda").bfloat16()
x = torch.randn((1, 128, 2, 256), generator=gen, device="cuda").bfloat16()
g = torch.zeros((1, 128, 2), device="cuda")


def call():
    if op == "cache":
        gdn.kv4_write(k, v, cache, table, lens, lens)
        return gdn.flash_attn_kv4(q, cache, table, lens)
    return gdn.forward(x, x, x, g, torch.full_like(g, 0.5), l2norm_qk=True)[0]


torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph, capture_error_mode=mode):
    out = call()
graph.replay()
torch.cuda.synchronize()
assert torch.isfinite(out).all() and torch.equal(out, call()) and gdn.device_status() == gdn.OK
"""


@pytest.mark.parametrize("mode", ["global", "thread_local"])
@pytest.mark.parametrize("op", ["cache", "forward"])
def test_the_first_call_of_a_process_can_be_captured(op, mode):
    """Both calls take their workspace from the library."""
    from linear_attention_sequence_gated_gb300 import _build
    _build.build()
    r = subprocess.run([sys.executable, "-c", PROGRAM, op, mode], cwd=ROOT, capture_output=True, text=True, timeout=300,
                       env=dict(os.environ, PYTHONPATH=ROOT))
    assert r.returncode == 0, r.stderr[-2000:]
