"""The binding's checks of device tensors in the rotary, adapter and feed-forward calls."""
import pytest
import torch

from hybrid_gated_deltanet_gb300 import binding as gb

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


def _t(*shape, dtype=BF):
    return torch.zeros(shape, dtype=dtype, device="cuda")


def test_rope_binding_refusals():
    plan, pos = gb.gdn_rope_plan(gb.RopeConfig(64, 32)), _t(3, dtype=torch.int32)
    q = _t(3, 4, 64)
    for bad, match in ((_t(3, 4, 64, dtype=torch.float32), "q: found torch.float32"), (_t(2, 4, 64), r"q: found torch.bfloat16 \(2, 4"),
                       (_t(3, 4, 32), "q: found"), (_t(12, 64), "q: found"), (_t(4, 3, 64).transpose(0, 1), "q: found strides"),
                       (_t(3, 4, 128)[..., ::2], "q: found strides"), (_t(1, 4, 64).expand(3, 4, 64), "q: found strides"),
                       (q.cpu(), "q: found a tensor on cpu")):
        with pytest.raises(ValueError, match=match):
            gb.gdn_rope(plan, pos, bad, None)
    with pytest.raises(ValueError, match="q_out: found 2 heads, required 4"):
        gb.gdn_rope(plan, pos, q, None, _t(3, 2, 64))
    with pytest.raises(ValueError, match="k_out: found 4 heads, required None without k"):
        gb.gdn_rope(plan, pos, q, None, None, q)
    with pytest.raises(ValueError, match="positions"):
        gb.gdn_rope(plan, pos.long(), q, None)
    with pytest.raises(gb.GdnError, match="q: found address"):
        gb.gdn_rope(plan, pos, _t(3, 5 * 64)[:, 4:260].unflatten(1, (4, 64)), None)


def test_projection_binding_refusals():
    x, w, out = _t(4, 64), _t(72, 64), _t(4, 72)
    with pytest.raises(ValueError, match="w_up: found"):
        gb.gdn_proj_gated(x, w, _t(71, 64), out)
    with pytest.raises(ValueError, match="w_gate: found"):
        gb.gdn_proj_gated(x, _t(72, 32), w, out)
    with pytest.raises(ValueError, match="out: found"):
        gb.gdn_proj_gated(x, w, w, _t(3, 72))
    with pytest.raises(ValueError, match="act: libgdn takes dense"):
        gb.gdn_proj_gated(_t(4, 128)[:, :64], w, w, out)
    with pytest.raises(gb.GdnError, match="ld_out: found 64"):
        gb.gdn_proj_gated(x, w, w, _t(4, 64))
    ffn, ws = gb.Ffn(w, w, _t(64, 72)), _t(4 * 72 * 2, dtype=torch.uint8)
    with pytest.raises(ValueError, match="out: found"):
        gb.gdn_ffn(ffn, x, out, ws)
    with pytest.raises(ValueError, match="ffn.w_down: found"):
        gb.gdn_ffn(gb.Ffn(w, w, w), x, _t(4, 64), ws)
    with pytest.raises(gb.GdnError, match="workspace: found 575 bytes, required 576"):
        gb.gdn_ffn(ffn, x, _t(4, 64), ws[:575])
    with pytest.raises(gb.GdnError, match="workspace: found NULL"):
        gb.gdn_ffn(ffn, x, _t(4, 64))
    gb.gdn_ffn(ffn, x, _t(4, 64), _t(144, dtype=torch.float32))  # a workspace of any type
    cu, idx = _t(3, dtype=torch.int32), _t(2, dtype=torch.int32)
    good = gb.Lora(_t(5, 8, 64), _t(5, 72, 8))
    lws = _t(gb.gdn_proj_lora_workspace_size(4, 72, 64, 8, 2), dtype=torch.uint8)
    for bad, match in ((gb.Lora(_t(5, 8, 32), good.b), "lora.a: found"), (gb.Lora(good.a, _t(5, 8, 72)), "lora.b: found"),
                       (gb.Lora(good.a, _t(4, 72, 8)), "lora.b: found"), (gb.Lora(_t(8, 64), good.b), "lora.a: found"),
                       (gb.Lora(good.a, good.b, _t(5)), "lora.scale: found")):
        with pytest.raises(ValueError, match=match):
            gb.gdn_proj_lora(x, w, bad, cu, idx, out, lws)
    with pytest.raises(ValueError, match="cu_rows: found"):
        gb.gdn_proj_lora(x, w, good, idx, idx, out, lws)
    with pytest.raises(gb.GdnError, match="workspace"):
        gb.gdn_proj_lora(x, w, good, cu, idx, out, lws[:-1])
    gb.gdn_proj_lora(x, w, good, cu, idx, out, lws)
    torch.cuda.synchronize()
