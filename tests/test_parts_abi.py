"""Refusals of the rotary, adapter and feed-forward calls, on the host without a GPU: status and message at the C boundary, and
the binding's checks.  No call here reaches a launch."""
import ctypes
import math

import pytest
import torch

from hybrid_gated_deltanet_gb300 import binding as gb
from hybrid_gated_deltanet_gb300 import build as gbuild
from parts_cases import frequencies

FAKE = 0x100000  # an aligned address that is never dereferenced on the host


@pytest.fixture(scope="module")
def lib():
    gbuild.build()
    return gb.load()


def _refused(lib, status, got, needle):
    err = lib.gdn_last_error().decode()
    assert got == status and needle in err, (got, err)


@pytest.mark.parametrize("kw", [dict(theta=1e4), dict(theta=1e7, factor=8.0), dict(theta=1e6, factor=4.0, orig_len=32768),
                                dict(theta=5e5, factor=16.0, orig_len=8192, beta_fast=8.0, beta_slow=2.0),
                                dict(theta=1e4, factor=2.0, orig_len=5)])
def test_plan_frequencies(lib, kw):
    """turns 2^-64 2 pi is the frequency, to the 53 bits of a double (the sums of a ramp cost a few more)."""
    plan = gb.gdn_rope_plan(gb.RopeConfig(128, 96, **kw))
    want = frequencies(96, **kw)
    for i in range(48):
        got = plan.turns[i] / 2.0 ** 64 * 2 * math.pi
        assert abs(got - float(want[i])) <= 2.0 ** -50 * float(want[i]) + 2.0 ** -60
    assert all(plan.turns[i] == 0 for i in range(48, 128))
    m = 0.1 * math.log(kw["factor"]) + 1 if "orig_len" in kw else 1.0
    assert abs(plan.mscale - m) <= 2.0 ** -24 * m
    assert abs(gb.gdn_rope_plan(gb.RopeConfig(128, 96, mscale=0.25, **kw)).mscale - 0.25) == 0


@pytest.mark.parametrize("kw", [dict(theta=1e4, factor=1e-6), dict(theta=1e4, factor=0.07), dict(theta=1e4, factor=0.15),
                                dict(theta=5e5, factor=1e-3, orig_len=64)])
def test_plan_frequencies_above_a_turn(lib, kw):
    """A factor far below 1 gives frequencies of whole turns and more per position, of which only the rest counts."""
    plan = gb.gdn_rope_plan(gb.RopeConfig(64, 64, **kw))
    for i, f in enumerate(frequencies(64, **{**kw, "factor": float(torch.tensor(kw["factor"], dtype=torch.float32))})):
        turns = float(f) / (2 * math.pi)
        off = (plan.turns[i] / 2.0 ** 64 - turns) % 1.0
        assert min(off, 1 - off) <= 2.0 ** -50 * turns + 2.0 ** -52


@pytest.mark.parametrize("kw,status,needle", [
    (dict(head_dim=12), -2, "cfg.head_dim: found 12"), (dict(head_dim=264), -2, "cfg.head_dim: found 264"),
    (dict(rotary_dim=24), -2, "cfg.rotary_dim: found 24"), (dict(rotary_dim=0), -2, "cfg.rotary_dim: found 0"),
    (dict(rotary_dim=144), -2, "required a multiple of 16, 16..head_dim = 128"), (dict(layout=2), -2, "cfg.layout: found 2"),
    (dict(act_dtype=2), -3, "cfg.act_dtype: found 2"), (dict(theta=1.0), -5, "cfg.theta: found 1"),
    (dict(theta=float("nan")), -5, "cfg.theta: found nan"), (dict(theta=float("inf")), -5, "cfg.theta: found inf"),
    (dict(factor=0.0), -5, "cfg.factor: found 0"), (dict(factor=-2.0), -5, "cfg.factor: found -2"),
    (dict(orig_len=-1), -5, "cfg.orig_len: found -1"), (dict(orig_len=9, beta_fast=0.0), -5, "cfg.beta_fast/beta_slow: found 0/1"),
    (dict(mscale=-1.0), -5, "cfg.mscale: found -1"), (dict(mscale=float("nan")), -5, "cfg.mscale: found nan")])
def test_rope_plan_refusals(lib, kw, status, needle):
    cfg = gb.RopeConfig(**{**dict(head_dim=128, rotary_dim=64), **kw})
    plan = gb.CRopePlan()
    _refused(lib, status, lib.gdn_rope_plan_init(ctypes.byref(cfg.c()), ctypes.byref(plan)), needle)
    with pytest.raises(gb.GdnError):
        gb.gdn_rope_plan(cfg)


def test_rope_plan_refuses_null(lib):
    _refused(lib, -1, lib.gdn_rope_plan_init(None, ctypes.byref(gb.CRopePlan())), "cfg: found NULL")
    _refused(lib, -1, lib.gdn_rope_plan_init(ctypes.byref(gb.RopeConfig(128, 64).c()), None), "plan: found NULL")


def _rope(lib, plan="made", **kw):
    a = dict(positions=FAKE, n=5, q=FAKE, ldq=1024, hq=8, qo=FAKE, ldqo=1024, k=FAKE, ldk=256, hkv=2, ko=FAKE, ldko=256)
    a.update(kw)
    if plan == "made":
        plan = ctypes.byref(gb.gdn_rope_plan(gb.RopeConfig(128, 64)))
    return lib.gdn_rope(plan, *a.values(), None)


def test_rope_refusals(lib):
    _refused(lib, -1, _rope(lib, None), "plan: found NULL")
    _refused(lib, -2, _rope(lib, ctypes.byref(gb.CRopePlan())), "plan.head_dim: found 0")  # a plan that nothing filled
    _refused(lib, -5, _rope(lib, n=-1), "n_tok: found -1")
    _refused(lib, -5, _rope(lib, n=1 << 31), "n_tok: found 2147483648")
    _refused(lib, -5, _rope(lib, hq=-1), "n_q_heads/n_kv_heads: found -1/2")
    _refused(lib, -5, _rope(lib, hkv=5000), "found 8/5000")
    _refused(lib, -2, _rope(lib, ldq=1016), "ld_q: found 1016, required >= 1024")
    _refused(lib, -2, _rope(lib, ldqo=1025), "ld_q_out: found 1025")
    _refused(lib, -2, _rope(lib, ldk=252), "ld_k: found 252")
    _refused(lib, -2, _rope(lib, ldko=8), "ld_k_out: found 8")
    _refused(lib, -2, _rope(lib, ldqo=2048), "ld_q_out: found 2048, required ld_q = 1024 in place")
    _refused(lib, -2, _rope(lib, ldko=512), "ld_k_out: found 512, required ld_k = 256 in place")
    for name, needle in (("positions", "positions"), ("q", "q"), ("qo", "q_out"), ("k", "k"), ("ko", "k_out")):
        _refused(lib, -1, _rope(lib, **{name: None}), f"{needle}: found NULL")
    _refused(lib, -4, _rope(lib, q=FAKE + 8), "q: found address")
    _refused(lib, -4, _rope(lib, positions=FAKE + 2), "positions: found address")
    assert _rope(lib, n=0) == 0 and _rope(lib, hq=0, hkv=0, q=None, k=None) == 0


def _gated(lib, **kw):
    a = dict(x=FAKE, g=FAKE, u=FAKE, out=FAKE, n=5, n_out=64, k=64, ld=64)
    a.update(kw)
    return lib.gdn_proj_gated(*a.values(), None)


def test_gated_refusals(lib):
    _refused(lib, -5, _gated(lib, n=-1), "n_tok: found -1")
    _refused(lib, -5, _gated(lib, n=(1 << 22) + 1), "n_tok: found 4194305")
    _refused(lib, -2, _gated(lib, n_out=0), "n_out: found 0")
    _refused(lib, -2, _gated(lib, k=12), "k: found 12")
    _refused(lib, -2, _gated(lib, k=0), "k: found 0")
    for k in (2 ** 24 + 8, 2 ** 31 - 8):  # (beyond what a plan's costs are counted in)
        _refused(lib, -2, _gated(lib, k=k), f"k: found {k}")
        assert lib.gdn_proj_lora_workspace_size(5, 64, k, 16, 1) == 0
    _refused(lib, -2, _gated(lib, ld=56), "ld_out: found 56")
    _refused(lib, -2, _gated(lib, ld=68), "ld_out: found 68")
    for name, needle in (("x", "act"), ("g", "w_gate"), ("u", "w_up"), ("out", "out")):
        _refused(lib, -1, _gated(lib, **{name: None}), f"{needle}: found NULL")
        _refused(lib, -4, _gated(lib, **{name: FAKE + 8}), f"{needle}: found address")
    assert _gated(lib, n=0, x=None, out=None) == 0


def _ffn(lib, weights=(FAKE, FAKE, FAKE, 64, 128), **kw):
    a = dict(h=FAKE, n=5, out=FAKE, ws=FAKE, nws=1 << 20)
    a.update(kw)
    return lib.gdn_ffn(None if weights is None else ctypes.byref(gb.CFfn(*weights)), *a.values(), None)


def test_ffn_refusals(lib):
    _refused(lib, -1, _ffn(lib, None), "ffn: found NULL")
    _refused(lib, -2, _ffn(lib, (FAKE, FAKE, FAKE, 60, 128)), "hidden/inter: found 60/128")
    _refused(lib, -2, _ffn(lib, (FAKE, FAKE, FAKE, 64, 0)), "hidden/inter: found 64/0")
    for i, name in enumerate(("w_gate", "w_up", "w_down")):
        w = [FAKE, FAKE, FAKE, 64, 128]
        w[i] = None
        _refused(lib, -1, _ffn(lib, w), f"ffn.{name}: found NULL")
    _refused(lib, -5, _ffn(lib, n=-3), "n_tok: found -3")
    for name, needle in (("h", "h"), ("out", "out"), ("ws", "workspace")):
        _refused(lib, -1, _ffn(lib, **{name: None}), f"{needle}: found NULL")
        _refused(lib, -4, _ffn(lib, **{name: FAKE + 4}), f"{needle}: found address")
    assert lib.gdn_ffn_workspace_size(5, 64, 128) == 5 * 128 * 2 and lib.gdn_last_error() == b""
    _refused(lib, -6, _ffn(lib, nws=1279), "found 1279 bytes, required 1280 bytes")
    assert lib.gdn_ffn_workspace_size(5, 63, 128) == 0 and b"hidden/inter" in lib.gdn_last_error()
    with pytest.raises(gb.GdnError, match="hidden/inter"):
        gb.gdn_ffn_workspace_size(5, 64, 4)
    assert _ffn(lib, n=0, h=None, out=None, ws=None) == 0


def _lora(lib, lora=(FAKE, FAKE, None, 3, 16), **kw):
    a = dict(x=FAKE, w=FAKE, lora=None if lora is None else ctypes.byref(gb.CLora(*lora)), cu=FAKE, idx=FAKE, n_seg=2,
             out=FAKE, n=5, n_out=60, k=64, ld=64, ws=FAKE, nws=1 << 20)
    a.update(kw)
    return lib.gdn_proj_lora(*a.values(), None)


def test_lora_refusals(lib):
    _refused(lib, -1, _lora(lib, None), "lora: found NULL")
    for rank in (0, 12, 136, -8):
        _refused(lib, -2, _lora(lib, (FAKE, FAKE, None, 3, rank)), f"lora.rank: found {rank}")
    _refused(lib, -5, _lora(lib, (FAKE, FAKE, None, 0, 16)), "lora.n_adapters: found 0")
    _refused(lib, -1, _lora(lib, (None, FAKE, None, 3, 16)), "lora.a: found NULL")
    _refused(lib, -1, _lora(lib, (FAKE, None, None, 3, 16)), "lora.b: found NULL")
    _refused(lib, -4, _lora(lib, (FAKE, FAKE, FAKE + 2, 3, 16)), "lora.scale: found address")
    _refused(lib, -5, _lora(lib, n_seg=-1), "n_seg: found -1")
    _refused(lib, -5, _lora(lib, n=-1), "n_tok: found -1")
    _refused(lib, -2, _lora(lib, n_out=0), "n_out: found 0")
    _refused(lib, -2, _lora(lib, k=4), "k: found 4")
    _refused(lib, -2, _lora(lib, ld=60), "ld_out: found 60")
    for name, needle in (("x", "act"), ("w", "w"), ("cu", "cu_rows"), ("idx", "adapter_idx"), ("out", "out"), ("ws", "workspace")):
        _refused(lib, -1, _lora(lib, **{name: None}), f"{needle}: found NULL")
        _refused(lib, -4, _lora(lib, **{name: FAKE + 2}), f"{needle}: found address")
    need = lib.gdn_proj_lora_workspace_size(5, 60, 64, 16, 2)
    assert need > 0
    _refused(lib, -6, _lora(lib, nws=need - 1), f"required {need} bytes")
    assert lib.gdn_proj_lora_workspace_size(5, 60, 64, 9, 2) == 0 and b"lora.rank" in lib.gdn_last_error()
    with pytest.raises(gb.GdnError, match="n_seg"):
        gb.gdn_proj_lora_workspace_size(5, 60, 64, 16, -2)
    assert _lora(lib, n=0, x=None, out=None, ws=None, cu=None, idx=None) == 0


def test_binding_refuses_host_tensors(lib):
    bf, plan = torch.bfloat16, gb.gdn_rope_plan(gb.RopeConfig(64, 32))
    x, pos = torch.zeros((3, 2, 64), dtype=bf), torch.zeros(3, dtype=torch.int32)
    with pytest.raises(ValueError, match="positions: found a tensor on cpu"):
        gb.gdn_rope(plan, pos, x, None)
    with pytest.raises(ValueError, match="act: found a tensor on cpu"):
        gb.gdn_proj_gated(x[:, 0], x[:, 0], x[:, 0], x[:, 0])
    with pytest.raises(ValueError, match="h: found a tensor on cpu"):
        gb.gdn_ffn(gb.Ffn(x[:, 0], x[:, 0], x[:, 0]), x[:, 0], x[:, 0])
    with pytest.raises(ValueError, match="act: found a tensor on cpu"):
        gb.gdn_proj_lora(x[:, 0], x[:, 0], gb.Lora(x, x), pos, pos, x[:, 0])
