"""Each call's first use in a process inside a stream capture, in a process of its own: the results of every call, whichever kernel
the sizes choose, are those of a replay alone."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

CODE = """
import torch
from hybrid_gated_deltanet_gb300 import binding as gb
bf, dev = torch.bfloat16, "cuda"
t = lambda *s: torch.ones(s, dtype=bf, device=dev)
i32 = lambda v: torch.tensor(v, dtype=torch.int32, device=dev)
w, a, b = t(256, 64), t(2, 16, 64), t(2, 256, 16)
ffn, lora, one = gb.Ffn(w, w, w.view(64, 256)), gb.Lora(a, b), i32([1])
cases = []
for n, heads in ((3, 2), (40000, 2), (40000, 1)):  # few tokens; many; many, one head
    x, cu, pos = t(n, 64), i32([0, n]), torch.arange(n, dtype=torch.int32, device=dev)
    wide, gated, out, rows, turned = (torch.full(s, 7.0, dtype=bf, device=dev)
                                      for s in ((n, 256), (n, 256), (n, 64), (n, heads, 64), (n, heads, 64)))
    rows[:] = torch.arange(64, device=dev) / 64
    ws = [torch.empty(size, dtype=torch.uint8, device=dev) for size in (gb.gdn_proj_lora_workspace_size(n, 256, 64, 16, 1),
                                                                        gb.gdn_ffn_workspace_size(n, 64, 256))]
    cases.append((x, cu, pos, wide, gated, out, rows, turned, ws))
plan = gb.gdn_rope_plan(gb.RopeConfig(64, 32))
def calls():
    for x, cu, pos, wide, gated, out, rows, turned, ws in cases:
        gb.gdn_rope(plan, pos, rows, None, turned)
        gb.gdn_proj_lora(x, w, lora, cu, one, wide, ws[0])
        gb.gdn_proj_gated(x, w, w, gated)
        gb.gdn_ffn(ffn, x, out, ws[1])
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    calls()
torch.cuda.synchronize()
for case in cases:
    for got in case[3:6] + case[7:8]:
        assert (got == 7).all()  # a capture runs nothing
graph.replay()
torch.cuda.synchronize()
replayed = []
for x, cu, pos, wide, gated, out, rows, turned, ws in cases:
    assert (wide == 64 + 16 * 64).all(), wide
    # a gate of 64 is silu(64) = 64 to 2^-20, its value 64: 4096, and 256 of those 2^20, each a number of bf16
    assert (gated == 4096).all() and (out == 2 ** 20).all(), (gated, out)
    assert (turned[..., 32:] == rows[..., 32:]).all() and (turned[0] == rows[0]).all() and (turned[1:, :, :32] != 7).all()
    replayed.append([v.clone() for v in (wide, gated, out, turned)])
    for v in (wide, gated, out, turned):
        v.fill_(7.0)
calls()
torch.cuda.synchronize()
for (x, cu, pos, wide, gated, out, rows, turned, ws), was in zip(cases, replayed):
    for v, r in zip((wide, gated, out, turned), was):
        assert torch.equal(v, r)
assert gb.gdn_device_status() == 0
"""


def test_first_calls_are_captured():
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    subprocess.run([sys.executable, "-c", CODE], check=True, cwd=root, timeout=120)
