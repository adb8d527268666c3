"""The operators of speculative decoding over trees of drafted tokens, as measured cases.

A serving step of the hybrid model that drafts a tree per sequence runs, in order:

  attn_tree    gdn_attn_tree      every node attends to its sequence's paged cache, its ancestors and itself
  verify_tree  gdn_verify_tree    every node's Gated DeltaNet output from its parent's state (no state written)
  page_tables  gdn_page_tables    pages and row maps for the accepted tokens (or for the prompts of a prefill)
  append       gdn_attn_append    K and V rows into the cache by a slot map
  commit_tree  gdn_commit_tree    the accepted path applied to the recurrent and conv states in place

run() computes each either in its plain form (elementary torch operations in 32 bits) or, where `own` is
true, by the framework's calls.  Trees are parent lists: node i of a sequence hangs off node parents[i] < i,
or off the end of the cached sequence (-1).
"""
import math

import torch

own = False

DEV = "cuda"
NO_PAGE = -1


# ---- the cases -----------------------------------------------------------------------------------
def listed():
    return [
        # one interactive user, a short context and a small tree: the latency of one attention layer
        dict(name="attn_tree 1x300, 8 nodes", op="attn_tree", B=1, ctx=300, nodes=8, hq=16, hkv=4, d=256, page=16,
             shape="tree"),
        # a batch of ragged contexts at d = 128 and wide groups
        dict(name="attn_tree 16x8192, 24 nodes", op="attn_tree", B=16, ctx=8192, nodes=24, hq=32, hkv=4, d=128,
             page=64, shape="tree"),
        # long contexts and the largest tree, 12 query heads to a kv-head, pages of 528
        dict(name="attn_tree 4x32768, 64 nodes", op="attn_tree", B=4, ctx=32768, nodes=64, hq=24, hkv=2, d=256,
             page=528, shape="tree"),
        # one user's small tree through one DeltaNet layer
        dict(name="verify_tree 1x8 nodes", op="verify_tree", B=1, nodes=8, hk=16, hv=32, d=128, k=4, act="bf16",
             shape="tree"),
        # a full batch of ragged trees
        dict(name="verify_tree 64x32 nodes", op="verify_tree", B=64, nodes=32, hk=16, hv=32, d=128, k=4, act="bf16",
             shape="tree"),
        # fp32 activations, a drafted chain instead of a tree
        dict(name="verify_tree fp32 8x20 chain", op="verify_tree", B=8, nodes=20, hk=16, hv=48, d=128, k=4, act="fp32",
             shape="chain"),
        # the accepted paths of a batch, wide value heads
        dict(name="commit_tree 64x6 rows", op="commit_tree", B=64, rows=6, hk=16, hv=48, d=128, k=4, act="bf16"),
        # one user's accepted path
        dict(name="commit_tree 1x3 rows", op="commit_tree", B=1, rows=3, hk=16, hv=32, d=128, k=4, act="bf16"),
        # pages and maps for the accepted tokens of a batch
        dict(name="page_tables 64 paths", op="page_tables", B=64, ctx=8192, new=8, page=16, paths=True),
        # pages and maps for a batch of prompts
        dict(name="page_tables 20 prompts", op="page_tables", B=20, ctx=0, new=30000, page=16, paths=False),
        # the accepted rows of a batch gathered into the cache
        dict(name="append 300 gathered rows", op="append", rows=300, hkv=4, d=256, page=16, gathered=True),
        # a prompt's K and V into the cache
        dict(name="append 65536 rows", op="append", rows=65536, hkv=2, d=256, page=528, gathered=False),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["attn_tree", "attn_tree", "verify_tree", "verify_tree", "commit_tree", "page_tables", "append"])
    heads = rng.choice([(16, 32), (16, 48), (4, 4), (2, 8)])
    shape = rng.choice(["tree", "tree", "chain"])
    if op == "attn_tree":
        hq, hkv, d, page = rng.choice([(16, 4, 256, 16), (24, 2, 256, 528), (32, 4, 128, 64), (8, 8, 128, 8),
                                       (4, 2, 128, 32), (32, 1, 128, 24), (16, 4, 256, 40)])
        B, nodes = _log_int(rng, 1, 32), _log_int(rng, 1, 64)
        ctx = _log_int(rng, 1, max(1, min(32768, 131072 // B)))
        return dict(op=op, B=B, ctx=ctx, nodes=nodes, hq=hq, hkv=hkv, d=d, page=page, shape=shape)
    if op == "verify_tree":
        act, d = rng.choice([("bf16", 128), ("bf16", 128), ("bf16", 128), ("bf16", 64), ("fp32", 128), ("fp32", 32)])
        B, nodes = _log_int(rng, 1, 64), _log_int(rng, 1, 64)
        nodes = max(1, min(nodes, 2048 // B))
        return dict(op=op, B=B, nodes=nodes, hk=heads[0], hv=heads[1], d=d, k=rng.choice([2, 3, 4, 4]), act=act,
                    shape=shape)
    if op == "commit_tree":
        act, d = rng.choice([("bf16", 128), ("bf16", 128), ("bf16", 64), ("fp32", 128), ("fp32", 32)])
        return dict(op=op, B=_log_int(rng, 1, 64), rows=_log_int(rng, 1, 20), hk=heads[0], hv=heads[1], d=d,
                    k=rng.choice([2, 3, 4, 4]), act=act)
    if op == "page_tables":
        page, paths = rng.choice([8, 16, 40, 64, 528]), rng.random() < 0.5
        B = _log_int(rng, 1, 512)
        new = _log_int(rng, 1, 24 if paths else max(1, min(30000, 300000 // B)))
        return dict(op=op, B=B, ctx=rng.choice([0, _log_int(rng, 1, 8192)]), new=new, page=page, paths=paths)
    hkv, d, page = rng.choice([(4, 256, 16), (2, 256, 528), (4, 128, 64), (8, 128, 8), (1, 128, 24)])
    return dict(op=op, rows=_log_int(rng, 1, 65536), hkv=hkv, d=d, page=page, gathered=rng.random() < 0.5)


# ---- sizes that follow from a case alone ----------------------------------------------------------
def _spread(n, lo, hi):
    """n whole numbers over [lo, hi], the first of them hi (a golden-ratio sequence)."""
    return [hi] + [lo + int((hi - lo + 1) * ((i * 0.6180339887498949) % 1.0)) for i in range(1, n)]


def _ctx_of(c):
    lens = _spread(c["B"], c["ctx"] // 4, c["ctx"])
    if c["B"] >= 4:
        lens[-1] = 0  # a sequence that has just begun
    return lens


def _nodes_of(c):
    nodes = _spread(c["B"], 1, c["nodes"])
    if c["B"] >= 8:
        nodes[-2] = 0  # a sequence without a draft in this step
    return nodes


def _rows_of(c):
    rows = _spread(c["B"], 1, c["rows"])
    if c["B"] >= 8:
        rows[-2] = 0  # nothing accepted
    return rows


def _new_of(c):
    new = _spread(c["B"], 1, c["new"])
    if c["B"] >= 8:
        new[-2] = 0
    return new


def work(c):
    if c["op"] == "attn_tree":
        ctx, nodes = _ctx_of(c), _nodes_of(c)
        n = sum(nodes)
        kv = sum(x for x, m in zip(ctx, nodes) if m > 0)
        pairs = sum(m * (x + 1) for x, m in zip(ctx, nodes))
        return {"bytes": 4 * c["d"] * c["hkv"] * (kv + n) + 4 * n * c["hq"] * c["d"],
                "flops": 4 * pairs * c["hq"] * c["d"]}
    if c["op"] in ("verify_tree", "commit_tree"):
        verify = c["op"] == "verify_tree"
        per = _nodes_of(c) if verify else _rows_of(c)
        n, live = sum(per), sum(m > 0 for m in per)
        e = 2 if c["act"] == "bf16" else 4
        ch, vd = (2 * c["hk"] + c["hv"]) * c["d"], c["hv"] * c["d"]
        slot = c["hv"] * c["d"] * c["d"] * 4 + (c["k"] - 1) * ch * e
        row = (ch + 2 * c["hv"]) * e + (2 * vd * e if verify else 0)
        return {"bytes": live * slot * (1 if verify else 2) + n * row + ch * c["k"] * e,
                "flops": n * c["hv"] * c["d"] * c["d"] * (4 if verify else 6)}
    if c["op"] == "page_tables":
        ctx, new, p = _ctx_of(c), _new_of(c), c["page"]
        rows = sum(new)
        pages = sum((x + m + p - 1) // p - (x + p - 1) // p for x, m in zip(ctx, new))
        return {"bytes": 12 * c["B"] + 8 * pages + 8 * rows + (8 * rows if c["paths"] else 0), "flops": rows}
    return {"bytes": c["rows"] * (8 * c["hkv"] * c["d"] + 8 + (4 if c["gathered"] else 0)), "flops": 0}


# ---- inputs ----------------------------------------------------------------------------------------
class _Rand:
    def __init__(self, seed):
        self.g = torch.Generator(device=DEV).manual_seed(seed)
        self.h = torch.Generator().manual_seed(seed)

    def normal(self, shape, dtype, std=1.0):
        return (torch.randn(shape, generator=self.g, device=DEV) * std).to(dtype)

    def uniform(self, shape, dtype, lo, hi):
        return (torch.rand(shape, generator=self.g, device=DEV) * (hi - lo) + lo).to(dtype)

    def perm(self, n):
        return torch.randperm(n, generator=self.h)

    def unit(self):
        return float(torch.rand((), generator=self.h))


def _i32(v):
    return torch.as_tensor(v, dtype=torch.int32).to(DEV)


def _cumulative(v):
    return [sum(v[:i]) for i in range(len(v) + 1)]


def _shuffled(r, *lists):
    order = r.perm(len(lists[0])).tolist()
    return [[v[i] for i in order] for v in lists]


def _tree(r, n, shape):
    """Parents of n nodes: a chain, or nodes that mostly hang off recent ones (several roots are possible)."""
    if shape == "chain":
        return [i - 1 for i in range(n)]
    return [int(r.unit() ** 0.5 * (i + 1)) - 1 for i in range(n)]


def _paged(r, lens, page, extra):
    """A block table that holds `lens` tokens on scattered pages of a pool with some pages to spare."""
    need = [(x + page - 1) // page for x in lens]
    n_pages = sum(need) + extra
    perm = r.perm(n_pages)
    table = torch.full((len(lens), max(1, max(need))), NO_PAGE, dtype=torch.int32)
    at = 0
    for b, m in enumerate(need):
        table[b, :m] = perm[at:at + m].to(torch.int32)
        at += m
    return table, n_pages, perm[at:]


def prepare(case, seed):
    c, r = case, _Rand(seed)
    s = {"case": c}
    if c["op"] == "attn_tree":
        ctx, nodes = _shuffled(r, _ctx_of(c), _nodes_of(c))
        n = sum(nodes)
        table, n_pages, _ = _paged(r, ctx, c["page"], 3)
        bf = torch.bfloat16
        s.update(q=r.normal((n, c["hq"], c["d"]), bf), k_new=r.normal((n, c["hkv"], c["d"]), bf),
                 v_new=r.normal((n, c["hkv"], c["d"]), bf),
                 k_pool=r.normal((n_pages, c["hkv"], c["page"], c["d"]), bf),
                 v_pool=r.normal((n_pages, c["hkv"], c["page"], c["d"]), bf), block_table=table.to(DEV),
                 cu_nodes=_i32(_cumulative(nodes)), parents=_i32([p for m in nodes for p in _tree(r, m, c["shape"])]),
                 ctx_lens=_i32(ctx), o=torch.zeros((n, c["hq"], c["d"]), dtype=bf, device=DEV))
        if own:
            from hybrid_gated_deltanet_gb300 import binding as gb
            s["cfg"] = gb.AttnConfig(c["hq"], c["hkv"], c["d"], c["page"])
            ws = gb.gdn_attn_tree_workspace_size(s["cfg"], c["B"], c["nodes"], c["ctx"])
            s["ws"] = torch.empty(ws, dtype=torch.uint8, device=DEV) if ws else None
    elif c["op"] in ("verify_tree", "commit_tree"):
        verify = c["op"] == "verify_tree"
        act = torch.bfloat16 if c["act"] == "bf16" else torch.float32
        ch, vd, hv, d, B = (2 * c["hk"] + c["hv"]) * c["d"], c["hv"] * c["d"], c["hv"], c["d"], c["B"]
        (per,) = _shuffled(r, _nodes_of(c) if verify else _rows_of(c))
        # a commit takes its rows out of the trees that were verified
        nodes = per if verify else [2 * m + 1 for m in per]
        n, n_slots = sum(nodes), B + 3
        s.update(x=r.normal((n, ch), act), a=r.normal((n, hv), act), b=r.normal((n, hv), act),
                 conv_w=r.uniform((ch, c["k"]), act, -0.5, 0.5), A_log=r.uniform((hv,), torch.float32, 0, math.log(16)),
                 norm_w=r.normal((d,), torch.float32, 0.1).add(1).to(act),
                 conv_pool=r.normal((n_slots, c["k"] - 1, ch), act, 0.1),
                 state_pool=r.normal((n_slots, hv, d, d), torch.float32, 0.1), slot_idx=_i32(r.perm(n_slots)[:B]),
                 cu_nodes=_i32(_cumulative(nodes)))
        if verify:
            s.update(z=r.normal((n, vd), act), parents=_i32([p for m in nodes for p in _tree(r, m, c["shape"])]),
                     y=torch.zeros((n, vd), dtype=act, device=DEV))
        else:
            first = _cumulative(nodes)
            rows = [first[b] + j for b in range(B) for j in sorted(r.perm(nodes[b])[:per[b]].tolist())]
            s.update(cu_rows=_i32(_cumulative(per)), src_rows=_i32(rows))
        if own:
            from hybrid_gated_deltanet_gb300 import binding as gb
            s["cfg"] = gb.Config(c["hk"], hv, d, d, c["k"], 64, gb.BF16 if c["act"] == "bf16" else gb.F32)
            s["prm"] = gb.Params(conv_w=s["conv_w"], A_log=s["A_log"], norm_w=s["norm_w"])
    elif c["op"] == "page_tables":
        ctx, new = _shuffled(r, _ctx_of(c), _new_of(c))
        p = c["page"]
        total = [x + m for x, m in zip(ctx, new)]
        table, n_pages, spare = _paged(r, ctx, p, sum((t + p - 1) // p for t in total) + 2)
        wide = torch.full((c["B"], max((t + p - 1) // p for t in total) + 1), NO_PAGE, dtype=torch.int32)
        m = min(wide.shape[1], table.shape[1])
        wide[:, :m] = table[:, :m]
        rows = sum(new)
        s.update(n_pages=n_pages, ctx_lens=_i32(ctx), new_lens=_i32(new), free_pages=_i32(spare), head=_i32([1]),
                 block_table=wide.to(DEV), cu_rows=_i32([0] * (c["B"] + 1)),
                 slot_map=torch.zeros(rows + 5, dtype=torch.int64, device=DEV), head_out=_i32([0]),
                 path=None, cu_nodes=None, src_rows=None)
        if c["paths"]:
            nodes = [2 * k + 1 for k in new]
            path = torch.full((c["B"], max(new) + 1), -1, dtype=torch.int32)
            for b, k in enumerate(new):
                path[b, :k] = torch.sort(r.perm(nodes[b])[:k]).values.to(torch.int32)
            s.update(path=path.to(DEV), cu_nodes=_i32(_cumulative(nodes)), src_rows=_i32([0] * (rows + 5)))
    else:
        n, bf = c["rows"], torch.bfloat16
        src = 2 * n if c["gathered"] else n
        n_pages = (n + c["page"] - 1) // c["page"] + 4
        shape = (n_pages, c["hkv"], c["page"], c["d"])
        # whole pages in random order, as a prompt's pages lie; one row in 64 goes nowhere
        pages = r.perm(n_pages).to(DEV)
        at = torch.arange(n, device=DEV)
        slots = pages[at // c["page"]] * c["page"] + at % c["page"]
        slots[at % 64 == 63] = -1
        s.update(k_new=r.normal((src, c["hkv"], c["d"]), bf), v_new=r.normal((src, c["hkv"], c["d"]), bf),
                 k_pool=r.normal(shape, bf), v_pool=r.normal(shape, bf), slot_map=slots,
                 src_rows=torch.sort(r.perm(src)[:n]).values.to(torch.int32).to(DEV) if c["gathered"] else None)
        if own:
            from hybrid_gated_deltanet_gb300 import binding as gb
            s["cfg"] = gb.AttnConfig(c["hkv"], c["hkv"], c["d"], c["page"])
    return s


def run(s):
    if own:
        return _own(s)
    return {"attn_tree": _plain_attn, "verify_tree": _plain_verify, "commit_tree": _plain_commit,
            "page_tables": _plain_tables, "append": _plain_append}[s["case"]["op"]](s)


# ---- the framework's calls -------------------------------------------------------------------------
def _own(s):
    from hybrid_gated_deltanet_gb300 import binding as gb
    c = s["case"]
    if c["op"] == "attn_tree":
        gb.gdn_attn_tree(s["cfg"], s["q"], s["k_new"], s["v_new"], s["k_pool"], s["v_pool"], s["block_table"],
                         s["cu_nodes"], s["parents"], s["ctx_lens"], c["nodes"], c["ctx"], s["o"], s["ws"])
        return s["o"]
    if c["op"] == "verify_tree":
        gb.gdn_verify_tree(s["cfg"], s["prm"], s["x"], s["z"], s["a"], s["b"], s["conv_pool"], s["state_pool"],
                           s["slot_idx"], s["cu_nodes"], s["parents"], c["nodes"], s["y"])
        return s["y"]
    if c["op"] == "commit_tree":
        gb.gdn_commit_tree(s["cfg"], s["prm"], s["x"], s["a"], s["b"], s["conv_pool"], s["state_pool"], s["slot_idx"],
                           s["cu_rows"], s["src_rows"], c["rows"])
        return s["state_pool"], s["conv_pool"]
    if c["op"] == "page_tables":
        gb.gdn_page_tables(c["page"], s["n_pages"], s["ctx_lens"], s["new_lens"], s["free_pages"], s["head"],
                           s["block_table"], s["cu_rows"], s["slot_map"], s["head_out"], s["path"], s["cu_nodes"],
                           s["src_rows"])
        out = [s["block_table"], s["cu_rows"], s["slot_map"], s["head_out"]]
        return out + [s["src_rows"]] if c["paths"] else out
    gb.gdn_attn_append(s["cfg"], s["k_new"], s["v_new"], s["slot_map"], s["k_pool"], s["v_pool"], s["src_rows"])
    return s["k_pool"], s["v_pool"]


# ---- the plain forms -------------------------------------------------------------------------------
def _padded(cu, width):
    """Rows of a ragged batch as a rectangle: row index [B, width] (clamped) and which of them exist."""
    at = cu[:-1, None].long() + torch.arange(width, device=cu.device)
    there = at < cu[1:, None].long()
    return torch.where(there, at, 0), there


def _reach(parents, there):
    """Ancestor-or-self matrix [B, n, n] of the trees: powers of (1 + parent matrix), doubled each time."""
    n = parents.shape[1]
    eye = torch.eye(n, device=parents.device)
    up = (parents[:, :, None] == torch.arange(n, device=parents.device)).float() * there[:, :, None]
    reach = eye + up
    for _ in range(max(1, (n - 1).bit_length())):
        reach = ((reach @ reach) > 0).float()
    return reach > 0


def _plain_attn(s):
    c = s["case"]
    G, D, width = c["hq"] // c["hkv"], c["d"], c["nodes"]
    rows, there = _padded(s["cu_nodes"], width)
    B = rows.shape[0]
    parents = torch.where(there, s["parents"][rows].long(), -1)
    table = s["block_table"].long()
    L = table.shape[1] * c["page"]
    held = torch.arange(L, device=table.device) < s["ctx_lens"][:, None]

    def keys(pool, new):  # [B, hkv, L + width, D]
        old = pool[table.clamp(min=0)].permute(0, 2, 1, 3, 4).reshape(B, c["hkv"], L, D).float()
        return torch.cat([old, new[rows].permute(0, 2, 1, 3).float()], 2)

    q = s["q"][rows].float().view(B, width, c["hkv"], G, D).permute(0, 2, 1, 3, 4).reshape(B, c["hkv"], width * G, D)
    scores = (q @ keys(s["k_pool"], s["k_new"]).transpose(2, 3)).view(B, c["hkv"], width, G, L + width) / math.sqrt(D)
    seen = torch.cat([held[:, None, :].expand(B, width, L), _reach(parents, there)], 2)
    scores = torch.where(seen[:, None, :, None, :], scores, -math.inf)
    p = torch.exp(scores - scores.amax(-1, keepdim=True))
    p = (p / p.sum(-1, keepdim=True)).view(B, c["hkv"], width * G, L + width)
    v = keys(s["v_pool"], s["v_new"])
    v = torch.where(torch.cat([held, there], 1)[:, None, :, None], v, 0.0)
    o = (p @ v).view(B, c["hkv"], width, G, D).permute(0, 2, 1, 3, 4).reshape(B, width, c["hq"], D)
    out = s["o"].clone()
    out[rows[there]] = o[there].to(out.dtype)
    return out


def _sigmoid(x):
    return 1.0 / (1.0 + torch.exp(-x))


def _layer_inputs(c, s, taps):
    """q, k [B, n, hv, d] (normalised), v [B, n, hv, d] from the conv's taps [B, n, K, channels], oldest first."""
    u = (taps * s["conv_w"].float().t()).sum(2)
    u = u * _sigmoid(u)
    B, n, hk, hv, d = u.shape[0], u.shape[1], c["hk"], c["hv"], c["d"]
    q, k, v = u[..., :hk * d].view(B, n, hk, d), u[..., hk * d:2 * hk * d].view(B, n, hk, d), u[..., 2 * hk * d:]
    q = q / torch.sqrt((q * q).sum(-1, keepdim=True) + 1e-6)
    k = k / torch.sqrt((k * k).sum(-1, keepdim=True) + 1e-6)
    return (q.repeat_interleave(hv // hk, 2), k.repeat_interleave(hv // hk, 2), v.reshape(B, n, hv, d))


def _gates(s, rows):
    """log of the decay and beta, [B, n, hv]."""
    a, b = s["a"][rows].float(), s["b"][rows].float()
    soft = torch.clamp(a, min=0) + torch.log1p(torch.exp(-a.abs()))
    return -torch.exp(s["A_log"]) * soft, _sigmoid(b)


def _plain_verify(s):
    c = s["case"]
    n, K, hv, d = c["nodes"], c["k"], c["hv"], c["d"]
    rows, there = _padded(s["cu_nodes"], n)
    B = rows.shape[0]
    parents = torch.where(there, s["parents"][rows].long(), -1)
    reach = _reach(parents, there)
    slots = s["slot_idx"].long()
    # taps of a node: itself, its parent, ..., then the conv state backwards from its newest row
    hist = torch.cat([s["conv_pool"][slots].float(), s["x"][rows].float()], 1)  # [B, K-1 + n, channels]
    step = torch.cat([torch.arange(K - 1, device=rows.device).sub(1).clamp(min=0).expand(B, K - 1),
                      torch.where(parents >= 0, parents + K - 1, K - 2)], 1)  # the entry before each entry
    at = torch.arange(n, device=rows.device).expand(B, n) + K - 1
    order = [at]
    for _ in range(K - 1):
        order.append(torch.gather(step, 1, order[-1]))
    taps = torch.stack([torch.gather(hist, 1, i[:, :, None].expand(B, n, hist.shape[2])) for i in order[::-1]], 2)
    q, k, v = _layer_inputs(c, s, taps)
    g, beta = _gates(s, rows)
    g = torch.where(there[:, :, None], g, 0.0)
    total = reach.float() @ g  # log decay from the cached state to the node, the node's own included
    decay = torch.exp(torch.where(reach[..., None], total[:, :, None] - total[:, None], -math.inf))  # [B, i, j, hv]
    decay = decay.permute(0, 3, 1, 2)
    q, k, v, beta, first = (t.transpose(1, 2) for t in (q, k, v, beta[..., None], torch.exp(total)[..., None]))
    S = s["state_pool"][slots]
    from_k, from_q = k @ S.transpose(2, 3), q @ S.transpose(2, 3)  # [B, hv, n, d_v]
    pair_k = decay * (k @ k.transpose(2, 3)) * (1 - torch.eye(n, device=k.device))
    pair_q = decay * (q @ k.transpose(2, 3))
    # u_i = beta_i (v_i - first_i S k_i - sum over proper ancestors decay_ij (k_i . k_j) u_j)
    u = beta * (v - first * from_k)
    for i in range(1, n):
        u[:, :, i] -= beta[:, :, i] * (pair_k[:, :, i, :i, None] * u[:, :, :i]).sum(2)
    o = (first * from_q + pair_q @ u).transpose(1, 2)  # [B, n, hv, d]
    z = s["z"][rows].float().view(B, n, hv, d)
    y = o / torch.sqrt((o * o).mean(-1, keepdim=True) + 1e-6) * s["norm_w"].float() * z * _sigmoid(z)
    out = s["y"].clone()
    out[rows[there]] = y.reshape(B, n, hv * d)[there].to(out.dtype)
    return out


def _plain_commit(s):
    c = s["case"]
    n, K = c["rows"], c["k"]
    at, there = _padded(s["cu_rows"], n)
    rows = torch.where(there, s["src_rows"][at].long(), 0)
    slots = s["slot_idx"].long()
    hist = torch.cat([s["conv_pool"][slots], s["x"][rows]], 1)  # [B, K-1 + n, channels]
    taps = torch.stack([hist[:, m:m + n].float() for m in range(K)], 2)
    _, k, v = _layer_inputs(c, s, taps)
    g, beta = _gates(s, rows)
    S = s["state_pool"][slots]
    for i in range(n):
        alpha = torch.exp(g[:, i])[..., None, None]
        e = v[:, i, :, :, None] - alpha * (S * k[:, i, :, None, :]).sum(-1, keepdim=True)
        new = alpha * S + beta[:, i, :, None, None] * e * k[:, i, :, None, :]
        S = torch.where(there[:, i, None, None, None], new, S)
    s["state_pool"][slots] = S
    count = there.sum(1)
    keep = count[:, None] + torch.arange(K - 1, device=at.device)
    s["conv_pool"][slots] = torch.gather(hist, 1, keep[:, :, None].expand(-1, -1, hist.shape[2]))
    return s["state_pool"], s["conv_pool"]


def _plain_tables(s):
    c, p = s["case"], s["case"]["page"]
    ctx, new = s["ctx_lens"].long(), s["new_lens"].long()
    table, cap = s["block_table"].clone(), s["slot_map"].numel()
    dev = ctx.device
    room = s["free_pages"].numel() - s["head"].long()
    fits = (ctx >= 0) & (new >= 0) & (ctx + new <= table.shape[1] * p)
    old_pages = (ctx + p - 1) // p
    need = torch.where(fits, (ctx + new + p - 1) // p - old_pages, 0)
    taken, asked = torch.cumsum(need, 0), torch.cumsum(torch.where(fits, new, 0), 0)
    granted = fits & ((need == 0) | (taken <= room)) & ((new == 0) | (asked <= cap))
    rows, pages = torch.where(granted, new, 0), torch.where(granted, need, 0)
    cu = torch.cat([torch.zeros(1, dtype=torch.long, device=dev), torch.cumsum(rows, 0)])
    column = torch.arange(table.shape[1], device=dev)
    fresh = (column >= old_pages[:, None]) & (column < (old_pages + pages)[:, None])
    source = s["head"].long() + (taken - need)[:, None] + column - old_pages[:, None]
    table = torch.where(fresh, s["free_pages"][torch.where(fresh, source, 0)], table)
    at = torch.arange(cap, device=dev)
    b = (at[:, None] >= cu[1:]).sum(1) if cap * c["B"] < 1 << 24 else torch.bucketize(at, cu[1:], right=True)
    live = b < c["B"]
    b = torch.where(live, b, 0)
    i = at - cu[b]
    pos = torch.where(live, ctx[b] + i, 0)
    page = table[b, pos // p].long()
    slot = torch.where(live & (page >= 0) & (page < s["n_pages"]), page * p + pos % p, -1)
    out = [table, cu.int(), slot, (s["head"].long() + torch.where(granted, taken, 0).amax()).int()]
    if c["paths"]:
        node = s["path"][b, torch.where(live, i, 0)].long()
        n = (s["cu_nodes"][1:] - s["cu_nodes"][:-1]).long()[b]
        out.append(torch.where(live & (node >= 0) & (node < n), s["cu_nodes"].long()[b] + node, -1).int())
    return out


def _plain_append(s):
    page = s["case"]["page"]
    keep = s["slot_map"] >= 0
    slot = s["slot_map"][keep]
    src = (s["src_rows"].long() if s["src_rows"] is not None else torch.arange(keep.numel(), device=keep.device))[keep]
    s["k_pool"][slot // page, :, slot % page] = s["k_new"][src]
    s["v_pool"][slot // page, :, slot % page] = s["v_new"][src]
    return s["k_pool"], s["v_pool"]


# ---- from the definitions, in 64 bits ----------------------------------------------------------------
def exact(case, seed):
    s = prepare(case, seed)
    with torch.no_grad():
        return {"attn_tree": _exact_attn, "verify_tree": _exact_verify, "commit_tree": _exact_commit,
                "page_tables": _exact_tables, "append": _exact_append}[case["op"]](s)


def _line(parents, i):
    """Node i and its ancestors, from the root down."""
    line = []
    while i >= 0:
        line.append(i)
        i = parents[i]
    return line[::-1]


def _exact_attn(s):
    c = s["case"]
    D, G = c["d"], c["hq"] // c["hkv"]
    cu, ctx, parents = s["cu_nodes"].tolist(), s["ctx_lens"].tolist(), s["parents"].tolist()
    out = s["o"].double()
    for b in range(c["B"]):
        n = cu[b + 1] - cu[b]
        if n == 0:
            continue
        pos = torch.arange(ctx[b], device=DEV)
        page = s["block_table"][b].long()[pos // c["page"]]
        mine = parents[cu[b]:cu[b + 1]]
        mask = torch.zeros((n, n), dtype=torch.bool)
        for i in range(n):
            mask[i, _line(mine, i)] = True
        mask = torch.cat([torch.ones((n, ctx[b]), dtype=torch.bool), mask], 1).to(DEV)
        for h in range(c["hkv"]):
            K = torch.cat([s["k_pool"][page, h, pos % c["page"]], s["k_new"][cu[b]:cu[b + 1], h]]).double()
            V = torch.cat([s["v_pool"][page, h, pos % c["page"]], s["v_new"][cu[b]:cu[b + 1], h]]).double()
            for g in range(h * G, (h + 1) * G):
                w = torch.softmax((s["q"][cu[b]:cu[b + 1], g].double() @ K.T / D ** 0.5).masked_fill(~mask, -math.inf), 1)
                out[cu[b]:cu[b + 1], g] = w @ V
    return out


def _token(c, s, window, row, S):
    """One token of the layer after the raw inputs `window` (oldest first, the token's own last): new state, output o."""
    hk, hv, d = c["hk"], c["hv"], c["d"]
    u = (torch.stack(window).T * s["conv_w"].double()).sum(1)
    u = u / (1 + torch.exp(-u))
    q, k, v = u[:hk * d].view(hk, d), u[hk * d:2 * hk * d].view(hk, d), u[2 * hk * d:].view(hv, d)
    q, k = (t / torch.sqrt((t ** 2).sum(1, keepdim=True) + 1e-6) for t in (q, k))
    head = torch.arange(hv, device=u.device) // (hv // hk)
    q, k = q[head], k[head]
    alpha = torch.exp(-torch.exp(s["A_log"].double()) * torch.logaddexp(s["a"][row].double(), torch.zeros((), dtype=torch.float64, device=u.device)))
    beta = torch.sigmoid(s["b"][row].double())
    S = alpha[:, None, None] * S
    S = S + (beta[:, None] * (v - torch.einsum("hvk,hk->hv", S, k)))[:, :, None] * k[:, None, :]
    return S, torch.einsum("hvk,hk->hv", S, q)


def _exact_verify(s):
    c, K = s["case"], s["case"]["k"]
    cu, parents, slots = s["cu_nodes"].tolist(), s["parents"].tolist(), s["slot_idx"].tolist()
    out = s["y"].double()
    x = s["x"].double()
    for b in range(c["B"]):
        states, n = {-1: s["state_pool"][slots[b]].double()}, cu[b + 1] - cu[b]
        before = list(s["conv_pool"][slots[b]].double())
        mine = parents[cu[b]:cu[b + 1]]
        for i in range(n):
            window = (before + [x[cu[b] + j] for j in _line(mine, i)])[-K:]
            states[i], o = _token(c, s, window, cu[b] + i, states[mine[i]])
            z = s["z"][cu[b] + i].double().view(c["hv"], c["d"])
            y = o / torch.sqrt((o ** 2).mean(1, keepdim=True) + 1e-6) * s["norm_w"].double() * z / (1 + torch.exp(-z))
            out[cu[b] + i] = y.reshape(-1)
    return out


def _exact_commit(s):
    c, K = s["case"], s["case"]["k"]
    cu, src, slots = s["cu_rows"].tolist(), s["src_rows"].tolist(), s["slot_idx"].tolist()
    state, conv, x = s["state_pool"].double(), s["conv_pool"].double(), s["x"].double()
    for b in range(c["B"]):
        S, hist = state[slots[b]], list(conv[slots[b]])
        for row in src[cu[b]:cu[b + 1]]:
            hist = hist + [x[row]]
            S, _ = _token(c, s, hist[-K:], row, S)
        state[slots[b]] = S
        conv[slots[b]] = torch.stack(hist[-(K - 1):])
    return state, conv


def _exact_tables(s):
    c, p = s["case"], s["case"]["page"]
    ctx, new, table = s["ctx_lens"].tolist(), s["new_lens"].tolist(), s["block_table"].cpu().clone()
    free, at, cap = s["free_pages"].tolist(), s["head"].tolist()[0], s["slot_map"].numel()
    cu, slots, src = [0], [], []
    for b in range(c["B"]):  # the lists are long enough here for every sequence to get its pages
        have, want = -(-ctx[b] // p), -(-(ctx[b] + new[b]) // p)
        table[b, have:want] = torch.tensor(free[at:at + want - have], dtype=torch.int32)
        at += want - have
        held = table[b].tolist()
        slots += [held[t // p] * p + t % p for t in range(ctx[b], ctx[b] + new[b])]
        if c["paths"]:
            first = int(s["cu_nodes"][b])
            src += [first + j for j in s["path"][b, :new[b]].tolist()]
        cu.append(cu[-1] + new[b])
    out = [table, torch.tensor(cu, dtype=torch.int32), torch.tensor(slots + [-1] * (cap - len(slots))),
           torch.tensor([at], dtype=torch.int32)]
    return out + [torch.tensor(src + [-1] * (cap - len(src)), dtype=torch.int32)] if c["paths"] else out


def _exact_append(s):
    page = s["case"]["page"]
    slots = s["slot_map"].cpu()
    src = s["src_rows"].cpu().long() if s["src_rows"] is not None else torch.arange(slots.numel())
    out = []
    for pool, new in ((s["k_pool"], s["k_new"]), (s["v_pool"], s["v_new"])):
        rows = pool.transpose(1, 2).reshape(-1, pool.shape[1], pool.shape[3]).double()  # one row a slot
        rows[slots[slots >= 0].to(DEV)] = new[src[slots >= 0].to(DEV)].double()
        out.append(rows.view(pool.shape[0], page, pool.shape[1], pool.shape[3]).transpose(1, 2).contiguous())
    return tuple(out)
