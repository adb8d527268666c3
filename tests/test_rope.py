"""Rotary positions (gdn_rope) against the 64-bit form.

Tolerance of an element: half a step of its type, plus fp32 arithmetic on a pair: sine and cosine to 2^-22 (sincospif:
2 ulp, and the angle to 2^-32 of a turn), each product and the sum to 2^-24 -- together below 2^-21 of m (|a| + |b|)."""
import pytest
import torch

from hybrid_gated_deltanet_gb300 import binding as gb
from parts_cases import HALF, bf16, check, frequencies, i32, rope

pytestmark = pytest.mark.gpu
ACT = {"bf16": (torch.bfloat16, gb.BF16), "fp32": (torch.float32, gb.F32)}


def _rows(gen, n, heads, D, dtype):
    return torch.randn((n, heads, D), generator=gen, dtype=torch.float64).to(dtype)


def _check(plan_cfg, x, positions, got, freq, m=1.0, angle_err=0.0):
    want, size = rope(x.cpu().double(), positions.cpu(), freq, plan_cfg.layout == gb.ROPE_HALF, m)
    check(got, want, (2.0 ** -21 + angle_err) * size, "rope")


@pytest.mark.parametrize("layout", [gb.ROPE_HALF, gb.ROPE_INTERLEAVED])
@pytest.mark.parametrize("act", ["bf16", "fp32"])
@pytest.mark.parametrize("n,hq,hkv,D,rot", [(1, 16, 4, 256, 64), (2, 1, 1, 16, 16), (37, 24, 2, 256, 256),
                                            (300, 3, 5, 96, 48), (5, 4, 0, 128, 96), (5, 0, 3, 128, 32), (3, 2, 2, 24, 16),
                                            (7, 2, 1, 40, 32), (2500, 4, 2, 64, 64)])
def test_rope_shapes(n, hq, hkv, D, rot, act, layout):
    gen = torch.Generator().manual_seed(n + D)
    dtype, code = ACT[act]
    cfg = gb.RopeConfig(D, rot, 1e6, layout, code)
    plan, freq = gb.gdn_rope_plan(cfg), frequencies(rot, 1e6)
    pos = torch.randint(0, 1 << 20, (n,), generator=gen, dtype=torch.int32).cuda()
    q, k = (None if h == 0 else _rows(gen, n, h, D, dtype).cuda() for h in (hq, hkv))
    outs = [None if x is None else torch.full_like(x, 7.0) for x in (q, k)]
    keep = [None if x is None else x.clone() for x in (q, k)]
    gb.gdn_rope(plan, pos, q, k, *outs)
    for x, was, out in zip((q, k), keep, outs):
        if x is not None:
            assert torch.equal(x, was)
            _check(cfg, x, pos, out, freq)
            assert torch.equal(out[..., rot:], x[..., rot:])
    gb.gdn_rope(plan, pos, q, k)  # in place: the same bits
    for x, out in zip((q, k), outs):
        assert x is None or torch.equal(x, out)
    assert gb.gdn_device_status() == 0


@pytest.mark.parametrize("layout", [gb.ROPE_HALF, gb.ROPE_INTERLEAVED])
def test_rope_rows_inside_wider_ones(layout):
    """q and k as parts of [q | k | v] rows: in place, nothing else is touched; and out of them into other rows."""
    gen = torch.Generator().manual_seed(3)
    n, hq, hkv, D, rot = 65, 6, 2, 128, 64
    joint = _rows(gen, n, hq + 2 * hkv, D, torch.bfloat16).cuda()
    was, pos = joint.clone(), torch.arange(100, 100 + n, dtype=torch.int32, device="cuda")
    cfg = gb.RopeConfig(D, rot, 1e4, layout)
    plan, freq = gb.gdn_rope_plan(cfg), frequencies(rot, 1e4)
    wide = torch.full((n, 3 * hq, D), 5.0, dtype=torch.bfloat16, device="cuda")
    gb.gdn_rope(plan, pos, joint[:, :hq], joint[:, hq:hq + hkv], wide[:, hq:2 * hq], None)
    assert torch.equal(joint[:, :hq], was[:, :hq]) and torch.equal(joint[:, hq + hkv:], was[:, hq + hkv:])
    assert (wide[:, :hq] == 5).all() and (wide[:, 2 * hq:] == 5).all()
    _check(cfg, was[:, :hq], pos, wide[:, hq:2 * hq], freq)
    _check(cfg, was[:, hq:hq + hkv], pos, joint[:, hq:hq + hkv], freq)


@pytest.mark.parametrize("positions,turn_err", [([0, 1, -1, 1 << 20, -(1 << 20)], 2.0 ** -32),
                                                ([2 ** 31 - 1, -2 ** 31, 10 ** 9, -10 ** 9 + 7], 2.0 ** -22)])
def test_rope_far_and_negative_positions(positions, turn_err):
    """The stated exactness of the angles; the 64-bit angle itself is off by 2^-53 of its value, below 2^-22 radians."""
    gen = torch.Generator().manual_seed(5)
    cfg = gb.RopeConfig(128, 128, 1e4, gb.ROPE_HALF, gb.F32)
    x = _rows(gen, len(positions), 3, 128, torch.float32).cuda()
    out = torch.empty_like(x)
    gb.gdn_rope(gb.gdn_rope_plan(cfg), i32(positions), x, None, out)
    _check(cfg, x, i32(positions), out, frequencies(128, 1e4), angle_err=2 * 3.15 * turn_err + (2.0 ** -22 if turn_err > 1e-8 else 0))


@pytest.mark.parametrize("kw,m", [(dict(factor=8.0), 1.0), (dict(factor=4.0, orig_len=32768), 1.1386294361119891),
                                  (dict(factor=40.0, orig_len=4096), 1.3688879454113936),
                                  (dict(factor=0.5, orig_len=4096), 1.0), (dict(factor=4.0, orig_len=100), 1.1386294361119891),
                                  (dict(factor=16.0, orig_len=8192, beta_fast=8.0, beta_slow=2.0, mscale=0.7), 0.7)])
def test_rope_scaled_for_long_contexts(kw, m):
    gen = torch.Generator().manual_seed(6)
    cfg = gb.RopeConfig(128, 64, 5e5, gb.ROPE_INTERLEAVED, gb.F32, **kw)
    freq = frequencies(64, 5e5, **{k: v for k, v in kw.items() if k != "mscale"})
    x = _rows(gen, 50, 2, 128, torch.float32).cuda()
    pos = torch.randint(0, 1 << 17, (50,), generator=gen, dtype=torch.int32).cuda()
    out = torch.empty_like(x)
    gb.gdn_rope(gb.gdn_rope_plan(cfg), pos, None, x, None, out)
    # (mscale is a float: 2^-24 more)
    _check(cfg, x, pos, out, freq, m, 2.0 ** -24)


def test_rope_gradient_is_the_rotation_back():
    """d/dx of <g, rope(x)> is rope at the negated positions: against the transpose and against differences."""
    gen = torch.Generator().manual_seed(7)
    cfg = gb.RopeConfig(64, 32, 1e4, gb.ROPE_HALF, gb.F32, factor=4.0, orig_len=2048)
    plan, freq, m = gb.gdn_rope_plan(cfg), frequencies(32, 1e4, 4.0, 2048), 1.1386294361119891
    x, g = (_rows(gen, 9, 2, 64, torch.float32) for _ in range(2))
    pos = torch.randint(0, 9000, (9,), generator=gen, dtype=torch.int32)
    dx = torch.empty_like(x).cuda()
    gb.gdn_rope(plan, -pos.cuda(), g.cuda(), None, dx)
    x64 = x.double().requires_grad_()
    rope(x64, pos, freq, True, m)[0].backward(g.double())
    _, size = rope(g.double(), -pos, freq, True, m)
    check(dx, x64.grad, 2.0 ** -20 * size)
    # differences of the 64-bit form (linear in x, so any step is exact to rounding)
    for at in [(0, 0, 0), (4, 1, 17), (8, 0, 31), (3, 1, 50)]:
        e = torch.zeros_like(x, dtype=torch.float64)
        e[at] = 1.0
        slope = ((rope(x.double() + e, pos, freq, True, m)[0] - rope(x.double() - e, pos, freq, True, m)[0]) * g.double()).sum() / 2
        assert abs(float(dx[at]) - float(slope)) <= 2.0 ** -20 * float(size[at]) + HALF[torch.float32] * abs(float(slope)) + 1e-12


def test_rope_not_numbers_stay_in_their_pair():
    cfg = gb.RopeConfig(64, 32, 1e4, gb.ROPE_HALF)
    x = torch.ones((4, 2, 64), dtype=torch.bfloat16, device="cuda")
    x[1, 0, 3], x[2, 1, 40], x[3, 0, 20] = float("nan"), float("inf"), -float("inf")
    gb.gdn_rope(gb.gdn_rope_plan(cfg), i32([5, 6, 7, 8]), x, None)
    bad = ~torch.isfinite(x)
    want = torch.zeros_like(bad)
    want[1, 0, 3] = want[1, 0, 19] = want[2, 1, 40] = want[3, 0, 4] = want[3, 0, 20] = True
    assert torch.equal(bad, want)


def test_rope_rows_past_2_to_the_32_bytes():
    n, ld = 4100, 1 << 20  # 8.6 GB between the first and the last row
    big = torch.empty((n, ld // 64, 64), dtype=torch.bfloat16, device="cuda")
    rows = [0, 1, 2047, 2048, 4095, 4099]
    big[:, 8:10] = 0
    gen = torch.Generator().manual_seed(8)
    x = _rows(gen, len(rows), 2, 64, torch.bfloat16).cuda()
    big[rows, 8:10] = x
    cfg = gb.RopeConfig(64, 64, 1e4, gb.ROPE_HALF)
    pos = torch.arange(n, dtype=torch.int32, device="cuda")
    gb.gdn_rope(gb.gdn_rope_plan(cfg), pos, big[:, 8:10], None)
    _check(cfg, x, pos[rows], big[rows, 8:10], frequencies(64, 1e4))


def test_rope_empty_captured_and_on_another_stream():
    cfg = gb.RopeConfig(128, 64, 1e6)
    plan, freq = gb.gdn_rope_plan(cfg), frequencies(64, 1e6)
    gb.gdn_rope(plan, i32([]), torch.empty((0, 4, 128), dtype=torch.bfloat16, device="cuda"), None)
    gb.gdn_rope(plan, i32([1, 2]), None, None)
    gen = torch.Generator().manual_seed(9)
    x = _rows(gen, 33, 4, 128, torch.bfloat16).cuda()
    pos, out, out2 = torch.arange(33, dtype=torch.int32, device="cuda"), torch.zeros_like(x), torch.zeros_like(x)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    gb.gdn_rope(plan, pos, x, None, out2, stream=side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        with torch.cuda.graph(graph, stream=side):
            gb.gdn_rope(plan, pos, x, None, out)
    pos += 1000
    graph.replay()
    torch.cuda.synchronize()
    _check(cfg, x, pos, out, freq)
    _check(cfg, x, pos - 1000, out2, freq)


def test_rope_in_place_beside_a_copy():
    """q where it lies and k copied: of q only the rotated elements are touched."""
    gen = torch.Generator().manual_seed(10)
    cfg = gb.RopeConfig(128, 32, 1e4)
    q, k = (_rows(gen, 20, h, 128, torch.bfloat16).cuda() for h in (3, 2))
    was, pos, k_out = q.clone(), torch.arange(20, dtype=torch.int32, device="cuda"), torch.zeros_like(k)
    gb.gdn_rope(gb.gdn_rope_plan(cfg), pos, q, k, None, k_out)
    freq = frequencies(32, 1e4)
    _check(cfg, was, pos, q, freq)
    _check(cfg, k, pos, k_out, freq)
    assert torch.equal(q[..., 32:], was[..., 32:]) and torch.equal(k_out[..., 32:], k[..., 32:])
