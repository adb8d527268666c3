"""Projections of many tokens whose last tiles are split along K (gdn_proj_lora, gdn_ffn): alone and behind whole waves of tiles,
in three parts and in five (four are read together, then the rest), with adapters in the last part.

Each call says itself that it split: the counters in its workspace, behind the tokens' own rows, hold the number of parts.
Tolerances as in the other tests of these calls, from fp32 sums and one rounding; the 64-bit forms run on the GPU."""
import pytest
import torch

from hybrid_gated_deltanet_gb300 import binding as gb
from parts_cases import check, cumulative, gated, i32, lora, product

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


def _rand(gen, *shape, std=1.0):
    return (torch.randn(shape, generator=gen, device="cuda") * std).to(BF)


def _counters(ws, own, tiles):
    """The counters of `tiles` split tiles (8 warps of two CTAs each) behind the call's own bytes."""
    at = (own + 255) // 256 * 256
    return ws[at:at + 32 * tiles].view(torch.int32)


def _low_row(rank):
    return 64 if rank <= 32 else 2 * ((rank + 63) // 64 * 64)


# tokens, requests and their adapters; columns; K; split tiles; parts
MIXED = [1] * 20 + [900, 7, 40] + [1] * 20 + [1453]
LORA = {
    "behind whole waves, mixed requests": (MIXED, 2560, 4096, 24, 3),
    "alone": ([2, 700, 30, 1, 257, 1, 1009], 520, 16392, 24, 3),
    "behind whole waves, five parts": ([1, 1, 300, 14, 1000, 90, 1, 16, 777], 2391, 10248, 14, 5),
}


class _Lora:
    def __init__(self, name, rank, pool=5):
        lens, self.n_out, self.k, self.tiles, self.parts = LORA[name]
        gen = torch.Generator(device="cuda").manual_seed(rank + self.n_out)
        self.n, self.cu, self.which, self.rank = sum(lens), cumulative(lens), [(i * 3) % 7 - 1 for i in range(len(lens))], rank
        self.x, self.w = _rand(gen, self.n, self.k), _rand(gen, self.n_out, self.k, std=self.k ** -0.5)
        self.a, self.b = _rand(gen, pool, rank, self.k, std=self.k ** -0.5), _rand(gen, pool, self.n_out, rank, std=rank ** -0.5)
        self.scale = torch.rand(pool, generator=gen, device="cuda") + 0.5
        self.ad, self.cud, self.idx = gb.Lora(self.a, self.b, self.scale), i32(self.cu), i32(self.which)
        self.size = gb.gdn_proj_lora_workspace_size(self.n, self.n_out, self.k, rank, len(lens))
        self.ld = (self.n_out + 7) // 8 * 8

    def workspace(self):
        return torch.full((self.size,), 255, dtype=torch.uint8, device="cuda")

    def run(self, out, ws, stream=None):
        gb.gdn_proj_lora(self.x, self.w, self.ad, self.cud, self.idx, out, ws, stream=stream)

    def split(self, ws):
        return (_counters(ws, self.n * (_low_row(self.rank) * 2 + 4), self.tiles) == self.parts).all()


@pytest.mark.parametrize("rank", [16, 40, 72, 128])
@pytest.mark.parametrize("name", LORA)
def test_lora(name, rank):
    c = _Lora(name, rank)
    ws, out = c.workspace(), torch.full((c.n + 1, c.ld), 7.0, dtype=BF, device="cuda")
    c.run(out[:c.n], ws)
    assert c.split(ws)
    y, d = lora(c.x.double(), c.w.double(), c.a.double(), c.b.double(), c.scale.double().tolist(), c.cu, c.which)
    check(out[:c.n, :c.n_out], y.cpu(), d.cpu())
    assert (out[c.n:] == 7).all() and (out[:, c.n_out:] == 7).all()
    again = torch.empty_like(out[:c.n])
    c.run(again, ws)  # with the counters that the first call left
    assert torch.equal(again[:, :c.n_out], out[:c.n, :c.n_out]) and c.split(ws)
    assert gb.gdn_device_status() == 0


@pytest.mark.parametrize("name", LORA)
def test_lora_captured_replayed_and_beside_another(name):
    c = _Lora(name, 32)
    ws, ws2 = c.workspace(), c.workspace()
    out, side_out, want, first = (torch.zeros((c.n, c.ld), dtype=BF, device="cuda") for _ in range(4))
    c.run(out, ws)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c.run(first, ws)
        c.run(out, ws)
    side = torch.cuda.Stream()
    for turn in range(3):
        c.which = [(e + 1) % 6 - 1 for e in c.which]
        c.idx.copy_(i32(c.which))
        c.run(want, ws)
        out.zero_()
        torch.cuda.synchronize()
        graph.replay()
        c.run(side_out, ws2, stream=side)
        c.run(side_out, ws2, stream=side)
        torch.cuda.synchronize()
        assert c.split(ws) and c.split(ws2)
        assert torch.equal(out[:, :c.n_out], want[:, :c.n_out]) and torch.equal(side_out[:, :c.n_out], want[:, :c.n_out])
    assert gb.gdn_device_status() == 0


# tokens, hidden, inter; split tiles, parts
FFN = [(2400, 2560, 4096, 24, 3), (2000, 520, 16392, 24, 3), (2200, 2400, 10248, 14, 5), (20002, 264, 8200, 6, 4)]


def _ffn(n, hidden, inter):
    gen = torch.Generator(device="cuda").manual_seed(n + hidden)
    weights = (_rand(gen, inter, hidden, std=hidden ** -0.5), _rand(gen, inter, hidden, std=hidden ** -0.5),
               _rand(gen, hidden, inter, std=inter ** -0.5))
    ws = torch.full((gb.gdn_ffn_workspace_size(n, hidden, inter),), 255, dtype=torch.uint8, device="cuda")
    return gen, weights, ws


@pytest.mark.parametrize("n,hidden,inter,tiles,parts", FFN)
def test_ffn(n, hidden, inter, tiles, parts):
    gen, (g, u, d), ws = _ffn(n, hidden, inter)
    h, out = _rand(gen, n, hidden), torch.full((n + 1, hidden), 7.0, dtype=BF, device="cuda")
    gb.gdn_ffn(gb.Ffn(g, u, d), h, out[:n], ws)
    assert (_counters(ws, n * inter * 2, tiles) == parts).all()
    for rows in torch.arange(n, device="cuda").split(4096):  # (64-bit halves of 20002 tokens at once: 1.3 GB each)
        a, da = gated(h[rows].double(), g.double(), u.double())
        want, slack = product(a, d.double())
        da = da + 2.0 ** -8 * (a.abs() + da)  # the half's rounding
        check(out[rows], want.cpu(), (slack + da @ d.double().abs().T).cpu())
    assert (out[n:] == 7).all()
    again = torch.empty_like(h)
    gb.gdn_ffn(gb.Ffn(g, u, d), h, again, ws)
    assert torch.equal(again, out[:n]) and (_counters(ws, n * inter * 2, tiles) == parts).all()
    assert gb.gdn_device_status() == 0


@pytest.mark.parametrize("n,hidden,inter,tiles,parts", FFN[:1] + FFN[2:3])
def test_ffn_captured_replayed_and_beside_another(n, hidden, inter, tiles, parts):
    gen, weights, ws = _ffn(n, hidden, inter)
    ffn, ws2 = gb.Ffn(*weights), ws.clone()
    h, mid, out, want, side_out = (torch.zeros((n, hidden), dtype=BF, device="cuda") for _ in range(5))
    inputs = [_rand(gen, n, hidden) for _ in range(3)]
    gb.gdn_ffn(ffn, inputs[0], mid, ws)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        gb.gdn_ffn(ffn, h, mid, ws)
        gb.gdn_ffn(ffn, mid, out, ws)
    side = torch.cuda.Stream()
    for x in inputs:
        gb.gdn_ffn(ffn, x, mid, ws)
        gb.gdn_ffn(ffn, mid, want, ws)
        h.copy_(x)
        torch.cuda.synchronize()
        graph.replay()
        gb.gdn_ffn(ffn, x, side_out, ws2, stream=side)
        torch.cuda.synchronize()
        assert torch.equal(out, want) and torch.equal(side_out, mid)
        assert (_counters(ws, n * inter * 2, tiles) == parts).all() and (_counters(ws2, n * inter * 2, tiles) == parts).all()
    assert gb.gdn_device_status() == 0
