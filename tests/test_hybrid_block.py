"""An attention layer and its feed-forward block, the calls together as a server makes them: the joint projection with each
request's adapter, rotary positions on its rows, attention over the paged cache, the out-projection with adapters, the
feed-forward block -- for the prompts, then for a decoding step on what they left.  Against 64 bits, with every tensor
that passes between two calls rounded to bf16 there as well."""
import math
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

from oracle import attention as at
from hybrid_gated_deltanet_gb300 import binding as gb
from parts_cases import bf16, cumulative, frequencies, gated, i32, lora, product, rope

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


def test_prompts_then_a_decoding_step():
    gen = torch.Generator().manual_seed(31)
    Hq, Hkv, D, page, hidden, inter, rank, pool = 8, 2, 128, 16, 264, 520, 16, 3
    lens, which = [40, 150, 7], [1, -1, 2]
    B, n, width = len(lens), sum(lens), (Hq + 2 * Hkv) * D
    w = lambda o, i: bf16(gen, o, i, std=i ** -0.5)  # noqa: E731
    w_qkv, w_o, g, u, d = w(width, hidden), w(hidden, Hq * D), w(inter, hidden), w(inter, hidden), w(hidden, inter)
    qa, qb = bf16(gen, pool, rank, hidden, std=hidden ** -0.5), bf16(gen, pool, width, rank, std=0.3 * rank ** -0.5)
    oa, ob = bf16(gen, pool, rank, Hq * D, std=(Hq * D) ** -0.5), bf16(gen, pool, hidden, rank, std=0.3 * rank ** -0.5)
    scale = torch.tensor([1.0, 2.0, 0.5])
    rcfg = gb.RopeConfig(D, 64, 1e6, gb.ROPE_HALF)
    plan, freq, acfg = gb.gdn_rope_plan(rcfg), frequencies(64, 1e6), gb.AttnConfig(Hq, Hkv, D, page)
    max_pages = 12
    table = torch.randperm(B * max_pages, generator=gen).to(torch.int32).view(B, max_pages).cuda()
    kp, vp = (torch.zeros((B * max_pages, Hkv, page, D), dtype=BF, device="cuda") for _ in range(2))
    dw = [t.cuda() for t in (w_qkv, w_o)]
    ffn = gb.Ffn(g.cuda(), u.cuda(), d.cuda())
    lq, lo = gb.Lora(qa.cuda(), qb.cuda(), scale.cuda()), gb.Lora(oa.cuda(), ob.cuda(), scale.cuda())
    idx = i32(which)

    def ws(size):
        return torch.empty(size, dtype=torch.uint8, device="cuda") if size else None

    def layer(h, cu, positions, attention):
        m = h.shape[0]
        qkv = torch.empty((m, width), dtype=BF, device="cuda")
        gb.gdn_proj_lora(h, dw[0], lq, cu, idx, qkv, ws(gb.gdn_proj_lora_workspace_size(m, width, hidden, rank, B)))
        rows = qkv.view(m, Hq + 2 * Hkv, D)
        gb.gdn_rope(plan, positions, rows[:, :Hq], rows[:, Hq:Hq + Hkv])
        q, k, v = (t.contiguous() for t in rows.split([Hq, Hkv, Hkv], 1))
        o = torch.empty((m, Hq, D), dtype=BF, device="cuda")
        attention(q, k, v, o)
        r = torch.empty((m, hidden), dtype=BF, device="cuda")
        gb.gdn_proj_lora(o.view(m, Hq * D), dw[1], lo, cu, idx, r, ws(gb.gdn_proj_lora_workspace_size(m, hidden, Hq * D, rank, B)))
        out = torch.empty_like(r)
        gb.gdn_ffn(ffn, r, out, ws(gb.gdn_ffn_workspace_size(m, hidden, inter)))
        return out

    h, h1 = bf16(gen, n, hidden), bf16(gen, B, hidden)
    cu, ctx0 = i32(cumulative(lens)), i32([0] * B)
    pos = i32([i for m in lens for i in range(m)])
    out = layer(h.cuda(), cu, pos, lambda q, k, v, o: gb.gdn_attn_prefill(acfg, q, k, v, kp, vp, table, cu, ctx0, o))
    seq = i32(lens)
    most = max(lens) + 1
    aws = ws(gb.gdn_attn_workspace_size(acfg, B, most))
    one = layer(h1.cuda(), i32([0, 1, 2, 3]), seq,
                lambda q, k, v, o: gb.gdn_attn_decode(acfg, q, k, v, kp, vp, table, seq, most, o, aws))
    torch.cuda.synchronize()
    assert gb.gdn_device_status() == 0

    # 64 bits, rounded where the calls hand over
    r16 = lambda t: t.to(BF).double()  # noqa: E731
    f64 = [t.double() for t in (w_qkv, w_o, g, u, d, qa, qb, oa, ob)]

    def before(x, cu64, p):
        y = r16(lora(x.double(), f64[0], f64[5], f64[6], scale.tolist(), cu64, which)[0]).view(-1, Hq + 2 * Hkv, D)
        q, k = (r16(rope(t.contiguous(), p, freq, True)[0]) for t in (y[:, :Hq], y[:, Hq:Hq + Hkv]))
        return q.numpy(), k.numpy(), y[:, Hq + Hkv:].numpy()

    def after(o, cu64):
        r = r16(lora(r16(torch.from_numpy(o)).reshape(-1, Hq * D), f64[1], f64[7], f64[8], scale.tolist(), cu64, which)[0])
        return product(r16(gated(r, f64[2], f64[3])[0]), f64[4])[0]

    c64 = cumulative(lens)
    q, k, v = before(h, c64, pos.cpu())
    o = np.concatenate([at.prefill_attention(q[a:b], k[a:b], v[a:b], 0, 1 / math.sqrt(D)) for a, b in zip(c64, c64[1:])])
    want = after(o, c64)
    q1, k1, v1 = before(h1, [0, 1, 2, 3], seq.cpu())
    o1 = np.stack([at.decode_attention(q1[s], np.concatenate([k[a:b], k1[s:s + 1]]), np.concatenate([v[a:b], v1[s:s + 1]]),
                                       1 / math.sqrt(D)) for s, (a, b) in enumerate(zip(c64, c64[1:]))])
    want1 = after(o1, [0, 1, 2, 3])
    # five tensors pass between calls, each a rounding that the next values inherit (2^-8 / sqrt(3) in the mean square where
    # kernel and oracle round to different sides, twice that for the gate's slope and the product), and the softmax's weights and the result are
    # rounded: 8 of them in quadrature, 2^-8 sqrt(8 / 3) 1.5 < 1e-2
    for got, ref in ((out, want), (one, want1)):
        assert torch.isfinite(got).all()
        assert float((got.cpu().double() - ref).norm() / ref.norm()) <= 1e-2


def test_first_calls_under_capture():
    """Each call's first use in a process may be inside a stream capture, whichever kernel the sizes choose."""
    code = """
import torch
from hybrid_gated_deltanet_gb300 import binding as gb
bf, dev = torch.bfloat16, "cuda"
t = lambda *s: torch.ones(s, dtype=bf, device=dev)
i32 = lambda v: torch.tensor(v, dtype=torch.int32, device=dev)
plan = gb.gdn_rope_plan(gb.RopeConfig(64, 32))
rows, pos, w, a, b = t(3, 2, 64), i32([1, 2, 3]), t(256, 64), t(2, 16, 64), t(2, 256, 16)
cases = []
for n in (3, 40000):
    ws = torch.empty(max(gb.gdn_proj_lora_workspace_size(n, 256, 64, 16, 1), gb.gdn_ffn_workspace_size(n, 64, 256)), dtype=torch.uint8, device=dev)
    cases.append((t(n, 64), t(n, 256), t(n, 64), i32([0, n]), ws))
one = i32([1])
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    gb.gdn_rope(plan, pos, rows, None)
    for x, wide, out, cu, ws in cases:
        gb.gdn_proj_lora(x, w, gb.Lora(a, b), cu, one, wide, ws)
        gb.gdn_ffn(gb.Ffn(w, w, w.view(64, 256)), x, out, ws)
graph.replay()
torch.cuda.synchronize()
for x, wide, out, cu, ws in cases:
    assert (wide == 64 + 16 * 64).all(), wide
assert gb.gdn_device_status() == 0
"""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    subprocess.run([sys.executable, "-c", code], check=True, cwd=root, timeout=120)
