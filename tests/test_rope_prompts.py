"""gdn_rope over prompts: the form in which a thread walks over all heads of a token (a captured call's kernel name says so),
and more tokens than one launch takes.  Tolerances as in the other tests of rotary positions: half a step of the type and fp32
arithmetic on a pair, 2^-21 of m (|a| + |b|); the 64-bit form runs on the GPU."""
import pytest
import torch

from hybrid_gated_deltanet_gb300 import binding as gb
from launches import kernels
from parts_cases import HALF, frequencies

pytestmark = pytest.mark.gpu
ACT = {"bf16": (torch.bfloat16, gb.BF16), "fp32": (torch.float32, gb.F32)}
ALL_HEADS = "Lb1EEE"  # k_rope<T, true>


def _check(got, x, positions, freq, half, m=1.0):
    """As parts_cases.rope, on the device and in place of a copy to the host: 64-bit angles of positions up to 2^20 are off by
    2^-33 radians, which is left out."""
    n = freq.numel()
    angle = positions.double()[:, None] * freq.to(x.device)
    c, s = (m * torch.cos(angle))[:, None], (m * torch.sin(angle))[:, None]
    first = slice(0, n) if half else slice(0, 2 * n, 2)
    second = slice(n, 2 * n) if half else slice(1, 2 * n, 2)
    a, b = x[..., first].double(), x[..., second].double()
    slack = 2.0 ** -21 * m * (a.abs() + b.abs())
    for part, want in ((first, a * c - b * s), (second, b * c + a * s)):
        off = (got[..., part].double() - want).abs() - HALF[got.dtype] * (want.abs() + slack) - slack
        assert bool((off <= 0).all()), float(off.max())
    assert torch.equal(got[..., 2 * n:], x[..., 2 * n:])


def _rows(gen, n, heads, D, dtype):
    return torch.randn((n, heads, D), generator=gen, device="cuda").to(dtype)


@pytest.mark.parametrize("layout", [gb.ROPE_HALF, gb.ROPE_INTERLEAVED])
@pytest.mark.parametrize("act", ["bf16", "fp32"])
@pytest.mark.parametrize("n,hq,hkv,D,rot", [(9001, 4, 1, 128, 96), (12345, 1, 0, 256, 64), (5001, 6, 3, 256, 256), (40003, 0, 2, 24, 16),
                                            (3, 1, 0, 40, 32)])
def test_rope_many_tokens(n, hq, hkv, D, rot, act, layout):
    gen = torch.Generator(device="cuda").manual_seed(n)
    dtype, code = ACT[act]
    plan, freq = gb.gdn_rope_plan(gb.RopeConfig(D, rot, 1e6, layout, code)), frequencies(rot, 1e6)
    pos = torch.randint(-(1 << 20), 1 << 20, (n,), generator=gen, device="cuda", dtype=torch.int32)
    q, k = (None if h == 0 else _rows(gen, n, h, D, dtype) for h in (hq, hkv))
    outs = [None if x is None else torch.full_like(x, 7.0) for x in (q, k)]
    keep = [None if x is None else x.clone() for x in (q, k)]
    names = kernels(lambda s: gb.gdn_rope(plan, pos, q, k, *outs, stream=s))
    assert len(names) == 1 and ALL_HEADS in names[0], names
    gb.gdn_rope(plan, pos, q, k, *outs)
    for x, was, out in zip((q, k), keep, outs):
        if x is not None:
            assert torch.equal(x, was)
            _check(out, x, pos, freq, layout == gb.ROPE_HALF)
    gb.gdn_rope(plan, pos, q, k)  # in place: the same bits
    for x, out in zip((q, k), outs):
        assert x is None or torch.equal(x, out)


@pytest.mark.parametrize("act", ["bf16", "fp32"])
def test_rope_many_tokens_in_joint_rows_one_in_place(act):
    """Rows [q | k | v], q copied out of them and k where it lies; what is not rotated stays."""
    gen = torch.Generator(device="cuda").manual_seed(4)
    dtype, code = ACT[act]
    n, hq, hkv, D, rot = 16001, 6, 2, 128, 64
    plan, freq = gb.gdn_rope_plan(gb.RopeConfig(D, rot, 1e4, act_dtype=code, factor=4.0, orig_len=2048)), frequencies(rot, 1e4, 4.0, 2048)
    joint = _rows(gen, n, hq + 2 * hkv, D, dtype)
    was, pos = joint.clone(), torch.arange(n, dtype=torch.int32, device="cuda")
    out = torch.full((n, hq + 1, D), 5.0, dtype=dtype, device="cuda")
    call = lambda s=None: gb.gdn_rope(plan, pos, joint[:, :hq], joint[:, hq:hq + hkv], out[:, :hq], None, stream=s)  # noqa: E731
    assert ALL_HEADS in kernels(call)[0]
    call()
    assert torch.equal(joint[:, :hq], was[:, :hq]) and torch.equal(joint[:, hq + hkv:], was[:, hq + hkv:]) and (out[:, hq:] == 5).all()
    _check(out[:, :hq], was[:, :hq], pos, freq, True, plan.mscale)
    _check(joint[:, hq:hq + hkv], was[:, hq:hq + hkv], pos, freq, True, plan.mscale)


def test_rope_more_tokens_than_a_launch_takes():
    n, D = (1 << 22) + 5, 16
    gen = torch.Generator(device="cuda").manual_seed(5)
    plan, freq = gb.gdn_rope_plan(gb.RopeConfig(D, D, 1e4)), frequencies(D, 1e4)
    q, k = (_rows(gen, n, 1, D, torch.bfloat16) for _ in range(2))
    pos = torch.randint(0, 1 << 20, (n,), generator=gen, device="cuda", dtype=torch.int32)
    k_out = torch.zeros_like(k)
    was = q.clone()
    names = kernels(lambda s: gb.gdn_rope(plan, pos, q, k, None, k_out, stream=s))
    assert len(names) == 2 and ALL_HEADS in names[0] and ALL_HEADS not in names[1], names
    gb.gdn_rope(plan, pos, q, k, None, k_out)
    _check(q, was, pos, freq, True)
    _check(k_out, k, pos, freq, True)
