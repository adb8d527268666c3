"""One serving step over drafted trees, the calls together as a server makes them: verify through the
DeltaNet layer and the attention layer, pages for the accepted paths, K and V appended, states
committed; then a plain decode step continues from what they left.  Every part is checked against the oracle on the tokens
that a sequence ends up with."""
import math

import numpy as np
import pytest
import torch

import oracle
from oracle import attention as at
from hybrid_gated_deltanet_gb300 import binding as gb
from hybrid_gated_deltanet_gb300 import synth
from gdn_cases import config, dev, host, oracle_kwargs, params_dev, rel_fro
from tree_cases import cumulative, gather, i32, line, make_tree

pytestmark = pytest.mark.gpu


def test_draft_verify_accept_commit_decode():
    r = synth.rng_for(73, 1)
    geom, act = synth.Geometry(2, 4, 128, 128, 4), synth.BF16
    Hq, Hkv, D, page = 16, 4, 256, 16
    acfg, cfg = gb.AttnConfig(Hq, Hkv, D, page), config(geom, act)
    p = synth.make_params(geom, r, act)
    prm, kw = params_dev(p), oracle_kwargs(p)
    ctx, nodes = [70, 0, 31, 48], [12, 5, 20, 1]
    B, N, cu = len(ctx), sum(nodes), cumulative(nodes)
    n_pages = 24
    pages = r.permutation(n_pages).astype(np.int32)
    table = np.full((B, 8), -1, np.int32)
    used = 0
    for b in range(B):
        m = math.ceil(ctx[b] / page)
        table[b, :m], used = pages[used:used + m], used + m
    trees = [make_tree(r, n, "tree") for n in nodes]
    bf = lambda *s: synth.store(r.standard_normal(s), synth.BF16)  # noqa: E731
    kp, vp, q, k, v = bf(n_pages, Hkv, page, D), bf(n_pages, Hkv, page, D), bf(N + B, Hq, D), bf(N + B, Hkv, D), bf(N + B, Hkv, D)
    tok = synth.make_tokens(geom, N + B, r, act)  # the last B rows: the decode step after
    S, CS = synth.make_state(geom, B, r), synth.make_conv_state(geom, B, r, act)
    d = {n: dev(t) for n, t in tok.items()}
    kpd, vpd, qd, kd, vd, Sd, Cd, td = dev(kp), dev(vp), dev(q), dev(k), dev(v), dev(S), dev(CS), i32(table)
    cud, par, ctxd, slots = i32(cu), i32([x for t in trees for x in t]), i32(ctx), i32(range(B))
    # verify
    y = torch.empty((N, geom.value_dim), dtype=torch.bfloat16, device="cuda")
    gb.gdn_verify_tree(cfg, prm, d["x"][:N], d["z"][:N], d["a"][:N], d["b"][:N], Cd, Sd, slots, cud, par, max(nodes), y)
    o = torch.empty((N, Hq, D), dtype=torch.bfloat16, device="cuda")
    ws = torch.empty(gb.gdn_attn_tree_workspace_size(acfg, B, max(nodes), max(ctx)), dtype=torch.uint8, device="cuda")
    gb.gdn_attn_tree(acfg, qd[:N], kd[:N], vd[:N], kpd, vpd, td, cud, par, ctxd, max(nodes), max(ctx), o, ws)
    # accept the line of one node of each sequence, nothing of the second
    paths = [line(trees[0], 11), [], line(trees[2], 17), [0]]
    width = max(len(x) for x in paths)
    path = np.full((B, width), -1, np.int32)
    for b, x in enumerate(paths):
        path[b, :len(x)] = x
    newd = i32([len(x) for x in paths])
    cap = B * width
    cu_rows, slot_map, src = i32([0] * (B + 1)), torch.zeros(cap, dtype=torch.int64, device="cuda"), i32([0] * cap)
    head = i32([0])
    gb.gdn_page_tables(page, n_pages, ctxd, newd, i32(pages[used:]), i32([0]), td, cu_rows, slot_map, head, i32(path),
                       cud, src)
    gb.gdn_attn_append(acfg, kd[:N], vd[:N], slot_map, kpd, vpd, src)
    gb.gdn_commit_tree(cfg, prm, d["x"][:N], d["a"][:N], d["b"][:N], Cd, Sd, slots, cu_rows, src, width)
    # the next plain step, on what the commits left; its own page comes from the same call
    ctx2 = ctxd + (cu_rows[1:] - cu_rows[:-1])
    one, cu2 = i32([1] * B), i32([0] * (B + 1))
    gb.gdn_page_tables(page, n_pages, ctx2, one, i32(pages[used:]), head, td, cu2,
                       torch.zeros(B, dtype=torch.int64, device="cuda"), i32([0]))
    y2 = torch.empty((B, geom.value_dim), dtype=torch.bfloat16, device="cuda")
    gb.gdn_decode_step(cfg, prm, d["x"][N:], d["z"][N:], d["a"][N:], d["b"][N:], Cd, Sd, slots, y2)
    o2 = torch.empty((B, Hq, D), dtype=torch.bfloat16, device="cuda")
    most = max(ctx) + width + 1
    nws = gb.gdn_attn_workspace_size(acfg, B, most)
    gb.gdn_attn_decode(acfg, qd[N:], kd[N:], vd[N:], kpd, vpd, td, ctx2, most, o2,
                       torch.empty(nws, dtype=torch.uint8, device="cuda") if nws else None)
    torch.cuda.synchronize()
    assert gb.gdn_device_status() == 0
    q64, k64, v64 = q.f64[:], k.f64[:], v.f64[:]
    for b in range(B):
        K0, _ = gather(kp.f64[:], table[b], page, n_pages, ctx[b])
        V0, _ = gather(vp.f64[:], table[b], page, n_pages, ctx[b])

        def layer(rows):
            return oracle.run_sequence(geom, *(tok[n].f64[np.asarray(rows)] for n in ("x", "z", "a", "b")),
                                       s0=S.f64[b], conv0=CS.f64[b], heads=list(range(4)), **kw)["y"][-1]

        def attention(rows):
            return at.decode_attention(q64[rows[-1]], np.concatenate([K0, k64[rows]]), np.concatenate([V0, v64[rows]]),
                                       1 / math.sqrt(D))

        # y: bf16 rounding 2^-8 and 11-bit operands; o: weights and o rounded to bf16, 2 x 2^-8
        for i in range(nodes[b]):
            rows = [int(cu[b]) + a for a in line(trees[b], i)]
            assert rel_fro(host(y)[cu[b] + i], layer(rows)) <= 7.8e-3
            assert rel_fro(host(o)[cu[b] + i], attention(rows)) <= 8e-3
        rows = [int(cu[b]) + a for a in paths[b]] + [N + b]
        assert rel_fro(host(y2)[b], layer(rows)) <= 7.8e-3
        assert rel_fro(host(o2)[b], attention(rows)) <= 8e-3
