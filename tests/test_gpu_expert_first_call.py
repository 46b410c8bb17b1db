"""The first expert call of a process may be one that a graph captures, in either kernel family."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

CHILD = """
import sys
import torch
import combine_warp_top_router_b200 as md
from test_gpu_experts import groups, ints, owned

op, pairs = sys.argv[1], sys.argv[2] == "pairs"
counts, K, N = ([70, 0, 300, 5] * 24, 72, 528) if pairs else ([7, 0, 30, 1], 200, 144)
E = len(counts)
off, cnt, rows, _ = groups(counts)
x, dy = ints(1, rows, K, hi=1), ints(2, rows, N, hi=1)
w = ints(3, *((E, K, N) if op == "kn" else (E, N, K)), hi=1)
call = {"nk": lambda: md.md_expert_gemm(x, w, off, cnt), "kn": lambda: md.md_expert_gemm(x, w, off, cnt, md.MD_W_KN),
        "gated": lambda: md.md_expert_gated(x, w, off, cnt), "wgrad": lambda: md.md_expert_wgrad(dy, x, off, cnt)}[op]
assert md.lib().md_launch_count() == 0  # nothing of the library has run
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    out = call()
assert md.lib().md_launch_count() == 1
# other rows, another split of them among the experts
x.copy_(ints(7, rows, K, hi=1))
off2, cnt2, _, spans = groups(counts[::-1], seed=3)
off.copy_(off2)
cnt.copy_(cnt2)
out.fill_(9)
for _ in range(2):
    graph.replay()
torch.cuda.synchronize()
for e, o, c in spans:
    rows_of = x[o:o + c].double()
    if op == "wgrad":
        assert torch.equal(out[e].double(), dy[o:o + c].double().t() @ rows_of)
        continue
    h = rows_of @ (w[e].double() if op == "kn" else w[e].double().t())
    if op == "gated":  # exact sums; the activation's float32 steps (14 * 2^-24) and one rounding
        g, u = h.chunk(2, 1)
        want = g * torch.sigmoid(g) * u
        assert bool(((out[o:o + c].double() - want).abs() <= (2.0 ** -8 + 14 * 2.0 ** -24) * want.abs() + 1e-37).all())
    else:
        assert torch.equal(out[o:o + c].double(), h)
if op == "wgrad":
    assert not bool(out[cnt == 0].any())
print("first call captured")
"""


@pytest.mark.parametrize("op,form", [("nk", "few"), ("nk", "pairs"), ("kn", "few"), ("kn", "pairs"), ("gated", "few"),
                                     ("gated", "pairs"), ("wgrad", "pairs")])
def test_first_call_of_a_process_is_captured(op, form):
    env = dict(os.environ, PYTHONPATH=os.pathsep.join([ROOT, os.path.join(ROOT, "tests")]))
    r = subprocess.run([sys.executable, "-c", CHILD, op, form], env=env, cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "first call captured" in r.stdout, r.stdout + r.stderr
