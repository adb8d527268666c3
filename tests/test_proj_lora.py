"""A shared projection with each request's low-rank adapter (gdn_proj_lora) against 64 bits.

Tolerance of an element: one bf16 rounding (2^-8) of the sum; fp32 sums on either side of the adapter and in the shared
product; the low-rank activations carried to 2^-16 (parts_cases.lora adds these up through |b|)."""
import pytest
import torch

from hybrid_gated_deltanet_gb300 import binding as gb
from parts_cases import bf16, check, cumulative, i32, lora, product

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


class Case:
    def __init__(self, seed, lens, which, k, n_out, rank, pool, scaled=True, delta=1.0):
        gen = torch.Generator().manual_seed(seed)
        n = sum(lens)
        self.cu, self.which = cumulative(lens), which
        self.x, self.w = bf16(gen, n, k), bf16(gen, n_out, k, std=k ** -0.5)
        self.a, self.b = bf16(gen, pool, rank, k, std=k ** -0.5), bf16(gen, pool, n_out, rank, std=delta * rank ** -0.5)
        self.scale = torch.rand(pool, generator=gen) + 0.5 if scaled else None
        self.n, self.k, self.n_out, self.rank = n, k, n_out, rank

    def run(self, out=None, ws=None, n=None, **kw):
        if out is None:
            out = torch.empty((self.n, (self.n_out + 7) // 8 * 8), dtype=BF, device="cuda")
        if ws is None:
            size = gb.gdn_proj_lora_workspace_size(self.n, self.n_out, self.k, self.rank, len(self.which))
            ws = torch.full((size,), 255, dtype=torch.uint8, device="cuda")  # (NaN, whatever it is read as)
        gb.gdn_proj_lora(self.x.cuda(), self.w.cuda(), gb.Lora(self.a.cuda(), self.b.cuda(),
                         None if self.scale is None else self.scale.cuda()), i32(self.cu), i32(self.which), out, ws, **kw)
        return out

    def exact(self):
        scale = [1.0] * self.a.shape[0] if self.scale is None else self.scale.double().tolist()
        return lora(self.x.double(), self.w.double(), self.a.double(), self.b.double(), scale, self.cu, self.which)

    def check(self, out):
        check(out[:, :self.n_out], *self.exact())


MIXES = {
    "one token": ([1], [0]),
    "decoding": ([1] * 19, [i % 4 for i in range(19)]),
    "decoding, many": ([1] * 150, [(i * 7) % 5 - 1 for i in range(150)]),
    "one prompt": ([300], [2]),
    "prompts": ([40, 129, 3, 256, 17], [1, 0, 3, 1, 2]),
    "mixed": ([1, 1, 700, 1, 1, 1, 90, 1], [0, 1, 2, 3, 2, 1, 0, 3]),
    "empty requests, none served": ([0, 5, 0, 0, 33, 0], [0, -1, 1, 2, -1, 3]),
    "some without an adapter": ([5, 60, 1, 400, 2], [-1, 3, 99, -5, 0]),
    "long prompts": ([1, 2000, 17, 3, 4200, 1, 15, 16, 900], [1, 0, 2, 3, -1, 0, 1, 2, 3]),
    "long prompts, none served": ([3000, 6000], [-1, 4]),
}


@pytest.mark.parametrize("mix", MIXES)
@pytest.mark.parametrize("rank,k,n_out", [(16, 264, 200), (8, 72, 129), (64, 520, 384)])
def test_lora_mixes(mix, rank, k, n_out):
    c = Case(rank + k, *MIXES[mix], k, n_out, rank, 4)
    out = c.run()
    c.check(out)
    assert torch.equal(c.run()[:, :n_out], out[:, :n_out])
    assert gb.gdn_device_status() == 0


@pytest.mark.parametrize("rank", [8, 16, 24, 32, 40, 48, 64, 72, 96, 128])
@pytest.mark.parametrize("lens", [[1] * 9, [2, 200, 100, 1], [2, 4000, 100, 1, 3000]])
def test_lora_ranks(rank, lens):
    """Every rank in steps of 8, adapters whose part is larger than the shared product, and no scale."""
    c = Case(rank, lens, [i % 3 for i in range(len(lens))], 256, 320, rank, 3, scaled=False, delta=20.0)
    c.check(c.run())


@pytest.mark.parametrize("rank", [16, 40, 64, 128])
@pytest.mark.parametrize("lens,n_out,k", [([1, 300, 30, 1, 257], 265, 4104), ([200], 96, 2560), ([5000, 1, 1, 15000], 264, 2560)])
def test_lora_split_along_k(lens, n_out, k, rank):
    """Few tiles of a long K, alone or behind whole waves of tiles: parts of a tile joined through the workspace, the adapters in
    one of them; twice, with the counters that the first call left."""
    c = Case(rank + n_out, lens, [(i * 2) % 5 - 1 for i in range(len(lens))], k, n_out, rank, 4)
    ws = torch.full((gb.gdn_proj_lora_workspace_size(c.n, n_out, k, rank, len(lens)),), 255, dtype=torch.uint8, device="cuda")
    out = c.run(ws=ws)
    c.check(out)
    assert torch.equal(c.run(ws=ws)[:, :n_out], out[:, :n_out])
    assert gb.gdn_device_status() == 0


@pytest.mark.parametrize("n,n_out,k", [(1, 12352, 2560), (64, 2560, 4096), (1, 1, 8), (200, 1, 8), (33, 2000, 1024)])
def test_lora_decoding_sizes(n, n_out, k):
    c = Case(n, [1] * n, [i % 5 for i in range(n)], k, n_out, 16, 5)
    c.check(c.run())


@pytest.mark.parametrize("rank", [16, 72])
@pytest.mark.parametrize("lens", [[1, 2, 1, 3, 1], [1, 150, 1, 400, 2], [1, 3000, 1, 4500, 498]])
def test_lora_not_numbers_stay_with_their_request(lens, rank):
    """NaN and infinities in one adapter reach that adapter's requests only; in a token, that token only."""
    c = Case(11, lens, [0, 1, 2, 3, 1], 136, 200, rank, 4)
    clean = c.run()[:, :200]
    c.check(clean)
    c.a[1, 3, 5], c.b[1, 7, 2], c.b[1, 8, 0] = float("nan"), float("inf"), float("nan")
    bad_token = c.cu[2]  # the request after the first with adapter 1
    c.x[bad_token, 9] = float("inf")
    out = c.run()[:, :200]
    rows = torch.arange(c.n)
    served = torch.zeros(c.n, dtype=torch.bool)
    for s, e in enumerate(c.which):
        if e == 1:
            served |= (rows >= c.cu[s]) & (rows < c.cu[s + 1])
    touched = served | (rows == bad_token)
    assert torch.equal(out[~touched], clean[~touched])
    assert torch.isnan(out[served]).all() and not torch.isfinite(out[bad_token]).any()


def test_lora_tokens_outside_every_request():
    for n, cu in ((30, [4, 4, 9, 21]), (900, [100, 130, 700, 890]), (9000, [100, 107, 7000, 8890]), (9000, [-5, 3000, 3001, 9100])):
        c = Case(12, [n], [0], 136, 96, 24, 4)
        c.cu, c.which = cu, [1, 3, 2]
        out = c.run()
        c.check(out)
        plain = torch.empty((n, 96), dtype=BF, device="cuda")
        size = gb.gdn_proj_workspace_size(n, 96, 136)
        gb.gdn_proj_gemm(c.x.cuda(), c.w.cuda(), plain, torch.empty(size, dtype=torch.uint8, device="cuda") if size else None)
        check(plain, *product(c.x.double(), c.w.double()))


def test_lora_without_requests():
    for n in (3, 700, 20000):
        c = Case(13, [n], [0], 64, 72, 8, 1)
        c.cu, c.which = [0], []
        c.check(c.run())


def test_lora_request_rows_that_are_not_in_order():
    """cu_rows that are not what they should be address nothing outside, and no wait runs out."""
    for n in (40, 800, 20000):
        c = Case(14, [n], [0], 64, 72, 16, 2)
        c.cu, c.which = [-7, -3, 2 ** 31 - 1, -2 ** 31, 5, 9], [0, 1, 0, 7, 1]
        c.run()
        torch.cuda.synchronize()
    assert gb.gdn_device_status() == 0


@pytest.mark.parametrize("lens", [[1] * 10, [1, 300, 30, 1, 257], [1, 6000, 30, 1, 2570]])
def test_lora_out_rows_and_workspace_end(lens):
    """Nothing past the columns, the rows or the workspace's stated size is written."""
    c = Case(15, lens, [i % 3 for i in range(len(lens))], 72, 100, 16, 3)
    size = gb.gdn_proj_lora_workspace_size(c.n, 100, 72, 16, len(lens))
    ws = torch.full((size + 64,), 9, dtype=torch.uint8, device="cuda")
    out = torch.full((c.n + 2, 112), 7.0, dtype=BF, device="cuda")
    c.run(out[:c.n], ws[:size])
    c.check(out[:c.n])
    assert (out[:c.n, 100:] == 7).all() and (out[c.n:] == 7).all() and (ws[size:] == 9).all()


@pytest.mark.parametrize("lens,k", [([1] * 12, 264), ([1, 400, 1, 60], 264), ([1, 6400, 1, 60], 264), ([1, 6400, 1, 60], 4096)])
def test_lora_captured_replayed_and_beside_another(lens, k):
    c = Case(16, lens, [i % 3 for i in range(len(lens))], k, 392, 32, 3)
    x, w, ad = c.x.cuda(), c.w.cuda(), gb.Lora(c.a.cuda(), c.b.cuda(), c.scale.cuda())
    cu, which = i32(c.cu), i32(c.which)
    size = gb.gdn_proj_lora_workspace_size(c.n, 392, k, 32, len(lens))
    ws, ws2 = (torch.empty(size, dtype=torch.uint8, device="cuda") for _ in range(2))
    out, side_out = (torch.zeros((c.n, 392), dtype=BF, device="cuda") for _ in range(2))
    gb.gdn_proj_lora(x, w, ad, cu, which, out, ws)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        gb.gdn_proj_lora(x, w, ad, cu, which, out, ws)
        gb.gdn_proj_lora(x, w, ad, cu, which, out, ws)
    side = torch.cuda.Stream()
    for turn in range(3):
        c.which = [(e + 1) % 4 - 1 for e in c.which]
        which.copy_(i32(c.which))
        side.wait_stream(torch.cuda.current_stream())
        graph.replay()
        gb.gdn_proj_lora(x, w, ad, cu, which, side_out, ws2, stream=side)
        torch.cuda.synchronize()
        c.check(out)
        assert torch.equal(out, side_out)
    assert gb.gdn_device_status() == 0


def test_lora_no_tokens():
    c = Case(17, [2], [0], 64, 72, 8, 1)
    gb.gdn_proj_lora(torch.empty((0, 64), dtype=BF, device="cuda"), c.w.cuda(), gb.Lora(c.a.cuda(), c.b.cuda()), i32([0]), i32([]),
                     torch.empty((0, 72), dtype=BF, device="cuda"))


def test_lora_pool_past_2_to_the_32_bytes():
    """Adapters whose rows lie beyond 4 GB of the pool."""
    gen = torch.Generator().manual_seed(18)
    pool, n_out, rank, k = 2200, 16384, 64, 64  # b: 4.6 GB
    a = torch.zeros((pool, rank, k), dtype=BF, device="cuda")
    b = torch.zeros((pool, n_out, rank), dtype=BF, device="cuda")
    used = [0, 2199, 2100]
    au, bu = bf16(gen, 3, rank, k, std=0.1), bf16(gen, 3, n_out, rank, std=0.1)
    a[used], b[used] = au.cuda(), bu.cuda()
    w = bf16(gen, n_out, k, std=0.1)
    for lens in ([1, 1, 1], [30, 150, 100]):
        n, cu = sum(lens), cumulative(lens)
        x = bf16(gen, n, k)
        out = torch.empty((n, n_out), dtype=BF, device="cuda")
        ws = torch.empty(gb.gdn_proj_lora_workspace_size(n, n_out, k, rank, 3), dtype=torch.uint8, device="cuda")
        gb.gdn_proj_lora(x.cuda(), w.cuda(), gb.Lora(a, b), i32(cu), i32(used), out, ws)
        check(out, *lora(x.double(), w.double(), au.double(), bu.double(), [1.0] * 3, cu, [0, 1, 2]))


@pytest.mark.parametrize("rank", [8, 16, 40])
@pytest.mark.parametrize("lens", [[1] * 6, [3] * 40, [1500, 7, 9000]])
def test_lora_infinite_activations(lens, rank):
    """An infinite element of a token, positive weights: infinity, with ranks that fill their tiles and with others."""
    c = Case(rank, lens, [i % 2 for i in range(len(lens))], 136, 520, rank, 2)
    c.x, c.w, c.a, c.b = c.x.abs(), c.w.abs() + 0.01, c.a.abs() + 0.01, c.b.abs() + 0.01
    clean = c.run()
    c.x[c.n // 2, 7] = float("inf")
    out = c.run()
    assert torch.isposinf(out[c.n // 2]).all()
    rest = torch.arange(c.n) != c.n // 2
    assert torch.equal(out[rest.cuda()], clean[rest.cuda()])
    assert gb.gdn_device_status() == 0
