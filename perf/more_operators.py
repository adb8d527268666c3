"""What a hybrid model's layer needs around its attention and its projections, as measured cases.

  rope    gdn_rope         rotary positions of an attention layer's queries and keys, before gdn_attn_decode,
                           gdn_attn_prefill or gdn_attn_tree takes them
  lora    gdn_proj_lora    a projection that every request shares, and beside it the low-rank adapter of each request
  gated   gdn_proj_gated   the gated half of the feed-forward block: both projections, SiLU and the product
  ffn     gdn_ffn          the whole block: the gated half and the projection back to the model width

run() computes each either in its plain form (elementary torch operations in 32 bits) or, where `own` is
true, by the framework's calls.
"""
import math

import torch

own = False

DEV = "cuda"


# ---- the cases -----------------------------------------------------------------------------------
def listed():
    return [
        # one user's next token, a quarter of each head rotated, in place: pure latency
        dict(name="rope 1 token", op="rope", n=1, hq=16, hkv=4, d=256, rot=64, layout="half", act="bf16", theta=1e7,
             factor=1.0, orig=0, far=8192, place="in"),
        # a decoding batch far beyond the trained length: interleaved pairs, frequencies scaled by parts
        dict(name="rope 300 tokens, scaled", op="rope", n=300, hq=24, hkv=2, d=256, rot=128, layout="interleaved",
             act="bf16", theta=1e6, factor=4.0, orig=32768, far=131072, place="out"),
        # prompts of a prefill, whole heads, q and k taken out of one joint projection's rows
        dict(name="rope 65536 tokens", op="rope", n=65536, hq=32, hkv=4, d=128, rot=128, layout="half", act="bf16",
             theta=1e6, factor=1.0, orig=0, far=65536, place="joint"),
        # one user with an adapter
        dict(name="lora 1 token", op="lora", prompts=0, longest=0, singles=1, k=2560, n_out=12352, rank=16, pool=8),
        # a decoding batch in which every request has its own adapter
        dict(name="lora 64 tokens, 64 requests", op="lora", prompts=0, longest=0, singles=64, k=2560, n_out=12352,
             rank=16, pool=64),
        # a step that mixes pieces of prompts with decoding requests, the out-projection
        dict(name="lora mixed step", op="lora", prompts=3, longest=1000, singles=41, k=4096, n_out=2560, rank=32,
             pool=24),
        # ragged prompts of ten requests, large adapters
        dict(name="lora prompts", op="lora", prompts=10, longest=1500, singles=0, k=2560, n_out=12352, rank=64, pool=6),
        # the gated half alone, where the projection back carries adapters: a prompt of an odd length
        dict(name="gated 4099 tokens", op="gated", n=4099, k=2560, inter=9216),
        # and a small model's decoding batch
        dict(name="gated 24 tokens", op="gated", n=24, k=1024, inter=3584),
        # one user's token through a feed-forward block
        dict(name="ffn 1 token", op="ffn", n=1, k=2560, inter=9216),
        # a decoding batch
        dict(name="ffn 64 tokens", op="ffn", n=64, k=2560, inter=9216),
        # a prompt
        dict(name="ffn 8192 tokens", op="ffn", n=8192, k=2560, inter=9216),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _log_8(rng, lo, hi):
    return 8 * _log_int(rng, lo // 8, hi // 8)


def draw(rng):
    op = rng.choice(["rope", "rope", "lora", "lora", "gated", "ffn"])
    if op == "rope":
        hq, hkv, d = rng.choice([(16, 4, 256), (24, 2, 256), (32, 4, 128), (8, 8, 128), (4, 1, 64), (6, 2, 128),
                                 (12, 3, 96)])
        rot = rng.choice([r for r in (16, 32, 48, 64, 96, 128, 256) if r <= d])
        act = rng.choice(["bf16", "bf16", "bf16", "fp32"])
        factor, orig = rng.choice([(1.0, 0), (1.0, 0), (8.0, 0), (4.0, 32768), (40.0, 4096)])
        most = 65536 * 36 * 128 * 2 // ((hq + hkv) * d * (2 if act == "bf16" else 4))
        return dict(op=op, n=_log_int(rng, 1, min(65536, most)), hq=hq, hkv=hkv, d=d, rot=rot,
                    layout=rng.choice(["half", "interleaved"]), act=act, theta=rng.choice([1e4, 5e5, 1e6, 1e7]),
                    factor=factor, orig=orig, far=_log_int(rng, 16, 1 << 20),
                    place=rng.choice(["in", "out", "joint"] if orig == 0 else ["out"]))
    if op == "lora":
        k, n_out = rng.choice([(2560, 12352), (4096, 2560), (_log_8(rng, 64, 2560), _log_8(rng, 64, 12352))])
        kind = rng.choice(["decode", "mixed", "prompts"])
        return dict(op=op, prompts=0 if kind == "decode" else rng.randint(1, 8),
                    longest=0 if kind == "decode" else _log_int(rng, 2, 1500),
                    singles=0 if kind == "prompts" else _log_int(rng, 1, 200 if kind == "decode" else 60), k=k,
                    n_out=n_out, rank=rng.choice([8, 16, 16, 24, 32, 64]), pool=_log_int(rng, 1, 64))
    return dict(op=op, n=_log_int(rng, 1, 8192 if op == "ffn" else 4099), k=rng.choice([2560, _log_8(rng, 64, 2560)]),
                inter=rng.choice([9216, _log_8(rng, 64, 9216)]))


# ---- sizes that follow from a case alone ----------------------------------------------------------
def _segments(c):
    """Lengths of a batch's requests: pieces of prompts over [longest / 4, longest], then single tokens."""
    P, L = c["prompts"], c["longest"]
    lens = [max(1, L - int((L - L // 4) * ((i * 0.6180339887498949) % 1.0))) for i in range(P)]
    return lens + [1] * c["singles"]


def _adapters(c):
    """An adapter for each request: every eighth has none, the others take the pool's in turn."""
    n = c["prompts"] + c["singles"]
    return [-1 if i % 8 == 5 else i % c["pool"] for i in range(n)]


def work(c):
    if c["op"] == "rope":
        e = 2 if c["act"] == "bf16" else 4
        width = c["rot"] if c["place"] != "out" else c["d"]  # a copy moves the rest of the head too
        elements = c["n"] * (c["hq"] + c["hkv"])
        return {"bytes": 2 * e * elements * width + 4 * c["n"], "flops": 3 * elements * c["rot"]}
    if c["op"] == "lora":
        lens, which = _segments(c), _adapters(c)
        n, served = sum(lens), sum(m for m, a in zip(lens, which) if a >= 0)
        used = len({a for a in which if a >= 0})
        k, n_out, r = c["k"], c["n_out"], c["rank"]
        return {"bytes": 2 * (n_out * k + n * (k + n_out) + used * r * (k + n_out)) + 8 * len(lens),
                "flops": 2 * n * k * n_out + 2 * served * r * (k + n_out)}
    n, k, m = c["n"], c["k"], c["inter"]
    if c["op"] == "gated":
        return {"bytes": 2 * (2 * k * m + n * (k + m)), "flops": 4 * n * k * m}
    return {"bytes": 2 * (3 * k * m + 2 * n * k), "flops": 6 * n * k * m}


# ---- inputs ----------------------------------------------------------------------------------------
class _Rand:
    def __init__(self, seed):
        self.g = torch.Generator(device=DEV).manual_seed(seed)
        self.h = torch.Generator().manual_seed(seed)

    def normal(self, shape, dtype, std=1.0):
        return (torch.randn(shape, generator=self.g, device=DEV) * std).to(dtype)

    def perm(self, n):
        return torch.randperm(n, generator=self.h).tolist()


def prepare(case, seed):
    c, r, bf = case, _Rand(seed), torch.bfloat16
    s = {"case": c}
    if c["op"] == "rope":
        act = bf if c["act"] == "bf16" else torch.float32
        n, hq, hkv, d = c["n"], c["hq"], c["hkv"], c["d"]
        if c["place"] == "joint":  # rows [q | k | v] of one projection, rotated where they lie
            rows = r.normal((n, hq + 2 * hkv, d), act)
            s.update(q=rows[:, :hq], k=rows[:, hq:hq + hkv])
        else:
            s.update(q=r.normal((n, hq, d), act), k=r.normal((n, hkv, d), act))
        s.update(q_out=torch.zeros_like(s["q"]) if c["place"] == "out" else None,
                 k_out=torch.zeros_like(s["k"]) if c["place"] == "out" else None)
        # a few sequences, each with its run of positions
        starts = torch.randint(0, c["far"], (max(1, min(8, n // 2)),), generator=r.h)
        at = torch.arange(n)
        piece = (n + len(starts) - 1) // len(starts)
        s["positions"] = (starts[at // piece] + at % piece).to(torch.int32).to(DEV)
        s["inv_freq"] = _inv_freq(c).to(DEV)
        if own:
            from hybrid_gated_deltanet_gb300 import binding as gb
            s["plan"] = gb.gdn_rope_plan(gb.RopeConfig(
                head_dim=d, rotary_dim=c["rot"], theta=c["theta"],
                layout=gb.ROPE_HALF if c["layout"] == "half" else gb.ROPE_INTERLEAVED,
                act_dtype=gb.BF16 if c["act"] == "bf16" else gb.F32, factor=c["factor"], orig_len=c["orig"]))
    elif c["op"] == "lora":
        lens, which = _segments(c), _adapters(c)
        order, names = r.perm(len(lens)), r.perm(c["pool"])
        lens, which = [lens[i] for i in order], [names[which[i]] if which[i] >= 0 else -1 for i in order]
        n, k, n_out, rank, pool = sum(lens), c["k"], c["n_out"], c["rank"], c["pool"]
        cu = [sum(lens[:i]) for i in range(len(lens) + 1)]
        s.update(x=r.normal((n, k), bf), w=r.normal((n_out, k), bf, k ** -0.5),
                 a=r.normal((pool, rank, k), bf, k ** -0.5), b=r.normal((pool, n_out, rank), bf, 0.3 * rank ** -0.5),
                 scale=r.normal((pool,), torch.float32, 0.2).add(1.5), out=torch.zeros((n, n_out), dtype=bf, device=DEV),
                 cu_rows=torch.tensor(cu, dtype=torch.int32).to(DEV),
                 adapter_idx=torch.tensor(which, dtype=torch.int32).to(DEV),
                 requests=[(cu[i], cu[i + 1], which[i]) for i in range(len(lens))])
        if own:
            from hybrid_gated_deltanet_gb300 import binding as gb
            s["lora"] = gb.Lora(s["a"], s["b"], s["scale"])
            ws = gb.gdn_proj_lora_workspace_size(n, n_out, k, rank, len(lens))
            s["ws"] = torch.empty(ws, dtype=torch.uint8, device=DEV) if ws else None
    else:
        n, k, m = c["n"], c["k"], c["inter"]
        s.update(h=r.normal((n, k), bf), w_gate=r.normal((m, k), bf, k ** -0.5), w_up=r.normal((m, k), bf, k ** -0.5))
        if c["op"] == "gated":
            s["out"] = torch.zeros((n, m), dtype=bf, device=DEV)
        else:
            s.update(w_down=r.normal((k, m), bf, m ** -0.5), out=torch.zeros((n, k), dtype=bf, device=DEV))
            if own:
                from hybrid_gated_deltanet_gb300 import binding as gb
                s["ffn"] = gb.Ffn(s["w_gate"], s["w_up"], s["w_down"])
                ws = gb.gdn_ffn_workspace_size(n, k, m)
                s["ws"] = torch.empty(ws, dtype=torch.uint8, device=DEV) if ws else None
    return s


def run(s):
    if own:
        return _own(s)
    return {"rope": _plain_rope, "lora": _plain_lora, "gated": _plain_gated, "ffn": _plain_ffn}[s["case"]["op"]](s)


# ---- the framework's calls -------------------------------------------------------------------------
def _own(s):
    from hybrid_gated_deltanet_gb300 import binding as gb
    op = s["case"]["op"]
    if op == "rope":
        gb.gdn_rope(s["plan"], s["positions"], s["q"], s["k"], s["q_out"], s["k_out"])
        return (s["q"], s["k"]) if s["q_out"] is None else (s["q_out"], s["k_out"])
    if op == "lora":
        gb.gdn_proj_lora(s["x"], s["w"], s["lora"], s["cu_rows"], s["adapter_idx"], s["out"], s["ws"])
    elif op == "gated":
        gb.gdn_proj_gated(s["h"], s["w_gate"], s["w_up"], s["out"])
    else:
        gb.gdn_ffn(s["ffn"], s["h"], s["out"], s["ws"])
    return s["out"]


# ---- the plain forms -------------------------------------------------------------------------------
def _inv_freq(c):
    """Angle of a pair per position, in radians: theta^(-2i/rot), scaled for a context `factor` times as long."""
    rot, theta, factor, orig = c["rot"], c["theta"], c["factor"], c["orig"]
    i = torch.arange(rot // 2, dtype=torch.float64)
    inv = theta ** (-2.0 * i / rot)
    if orig == 0:
        return inv / factor
    # by parts: pairs that turn more than 32 times within the trained length keep their frequency, those
    # that turn less than once are slowed down by the factor, and a ramp joins them
    turns = lambda t: rot * math.log(orig / (t * 2 * math.pi)) / (2 * math.log(theta))
    low, high = max(math.floor(turns(32.0)), 0), min(math.ceil(turns(1.0)), rot - 1)
    ramp = ((i - low) / max(high - low, 0.001)).clamp(0, 1)
    return inv * (1 - ramp) + inv / factor * ramp


def _magnitude(c):
    return 0.1 * math.log(c["factor"]) + 1 if c["orig"] > 0 and c["factor"] > 1 else 1.0


def _plain_rope(s):
    c, rot = s["case"], s["case"]["rot"]
    angle = s["positions"].double()[:, None] * s["inv_freq"]
    cos = (torch.cos(angle) * _magnitude(c)).float()[:, None]
    sin = (torch.sin(angle) * _magnitude(c)).float()[:, None]
    outs = []
    for x, out in ((s["q"], s["q_out"]), (s["k"], s["k_out"])):
        if out is None:
            out = x
        turn = x[..., :rot].float()
        if c["layout"] == "half":
            a, b = turn[..., :rot // 2], turn[..., rot // 2:]
            new = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
        else:
            a, b = turn[..., 0::2], turn[..., 1::2]
            new = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
        out[..., :rot] = new.to(out.dtype)
        if out is not x:
            out[..., rot:] = x[..., rot:]
        outs.append(out)
    return tuple(outs)


def _plain_lora(s):
    x = s["x"].float()
    y = x @ s["w"].float().t()
    for first, last, adapter in s["requests"]:
        if adapter >= 0:
            low = x[first:last] @ s["a"][adapter].float().t()
            y[first:last] += s["scale"][adapter] * (low @ s["b"][adapter].float().t())
    return y.to(torch.bfloat16)


def _half(s):
    h = s["h"].float()
    gate, up = h @ s["w_gate"].float().t(), h @ s["w_up"].float().t()
    return gate / (1 + torch.exp(-gate)) * up


def _plain_gated(s):
    return _half(s).to(torch.bfloat16)


def _plain_ffn(s):
    return (_half(s) @ s["w_down"].float().t()).to(torch.bfloat16)


# ---- from the definitions, in 64 bits ----------------------------------------------------------------
def exact(case, seed):
    s = prepare(case, seed)
    return {"rope": _exact_rope, "lora": _exact_lora, "gated": _exact_ffn, "ffn": _exact_ffn}[case["op"]](s)


def _exact_rope(s):
    """Each pair as a complex number, multiplied by magnitude e^(i position frequency)."""
    c = s["case"]
    rot, half = c["rot"], c["rot"] // 2
    freq = []
    for i in range(half):
        f = math.pow(c["theta"], -2 * i / rot)
        if c["orig"]:
            edge = [rot * math.log(c["orig"] / (2 * math.pi * t)) / math.log(c["theta"]) / 2 for t in (32, 1)]
            lo, hi = max(0, math.floor(edge[0])), min(rot - 1, math.ceil(edge[1]))
            slow = min(1.0, max(0.0, (i - lo) / max(hi - lo, 0.001)))
            f = f * ((1 - slow) + slow / c["factor"])
        else:
            f = f / c["factor"]
        freq.append(f)
    size = 1 + 0.1 * math.log(c["factor"]) if c["orig"] and c["factor"] > 1 else 1.0
    angle = torch.outer(s["positions"].double(), torch.tensor(freq, dtype=torch.float64, device=DEV))
    turn = torch.polar(torch.full_like(angle, size), angle)[:, None, :]
    index = torch.arange(half, device=DEV)
    first, second = (index, index + half) if c["layout"] == "half" else (2 * index, 2 * index + 1)
    outs = []
    for x in (s["q"], s["k"]):
        y = x.double()
        for at in range(0, x.shape[0], 8192):  # complex numbers of a part of the rows at a time
            part = y[at:at + 8192]
            z = torch.complex(part[..., first], part[..., second]) * turn[at:at + 8192]
            part[..., first], part[..., second] = z.real, z.imag
        outs.append(y)
    return tuple(outs)


def _exact_lora(s):
    y = s["x"].double() @ s["w"].double().T
    for first, last, adapter in s["requests"]:
        if adapter >= 0:
            delta = s["b"][adapter].double() @ (s["a"][adapter].double() @ s["x"][first:last].double().T)
            y[first:last] += float(s["scale"][adapter]) * delta.T
    return y


def _exact_ffn(s):
    h = s["h"].double()
    gate, up = torch.einsum("nk,mk->nm", h, s["w_gate"].double()), torch.einsum("nk,mk->nm", h, s["w_up"].double())
    a = gate * torch.sigmoid(gate) * up
    return a if s["case"]["op"] == "gated" else torch.einsum("nm,km->nk", a, s["w_down"].double())
