"""The workspace of gdn_attn_tree may be a dense tensor of any type and shape, as that of every other call."""
import pytest
import torch

import test_tree_attn
from hybrid_gated_deltanet_gb300 import binding as gb

pytestmark = pytest.mark.gpu


def call(c, ws, o):
    d = c.dev
    gb.gdn_attn_tree(c.cfg, d["q"], d["k"], d["v"], d["kp"], d["vp"], d["table"], d["cu"], d["parents"], d["ctx"],
                     c.max_nodes, c.max_ctx, o, ws)
    return o


def test_any_dense_tensor_will_do():
    c = test_tree_attn.Case(16, 4, 256, 16, [(2000, 9), (700, 3)], 51)
    want = c.call()
    n = c.ws.numel()
    assert n % 64 == 0
    for ws in (torch.empty(n // 4, device="cuda"), torch.empty(2, n // 2, dtype=torch.int8, device="cuda"),
               torch.empty(4, n // 64, 8, dtype=torch.bfloat16, device="cuda")):
        assert torch.equal(call(c, ws, torch.zeros_like(want)), want)
    with pytest.raises(gb.GdnError, match="required"):
        call(c, torch.empty(n // 4 - 4, device="cuda"), want)
    with pytest.raises(ValueError, match="workspace: libgdn takes dense"):
        call(c, torch.empty(n // 4, 2, device="cuda")[:, 0], want)
    with pytest.raises(ValueError, match="workspace: found a tensor on cpu"):
        call(c, torch.empty(n), want)
