"""The gated half of a feed-forward block (gdn_proj_gated) and the whole block (gdn_ffn) against 64 bits.

Tolerances: fp32 sums of k bf16 products are off by at most (k + 8) 2^-24 sum |x w|; the result is rounded once (2^-8).
The block rounds its gated half to bf16 as well: 2^-8 of each element, carried through |w_down|; and since the two roundings
are independent and each is off by 2^-8 / sqrt(3) at most in the mean square, the block as a whole by 2^-8 sqrt(2/3) < 3.2e-3."""
import pytest
import torch

from hybrid_gated_deltanet_gb300 import binding as gb
from parts_cases import bf16, check, gated, product

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


def _weights(gen, n, k):
    return bf16(gen, n, k, std=k ** -0.5)


@pytest.mark.parametrize("n,n_out,k", [(1, 1, 8), (1, 65, 72), (2, 64, 64), (16, 200, 136), (17, 63, 520), (33, 640, 256),
                                       (64, 1000, 264), (65, 129, 72), (128, 72, 2560), (129, 136, 64), (257, 385, 136),
                                       (300, 128, 1024), (520, 260, 72), (1000, 1100, 192), (2049, 96, 64), (40001, 136, 136),
                                       (2000, 3001, 264), (30000, 385, 72)])
def test_gated_shapes(n, n_out, k):
    gen = torch.Generator().manual_seed(n + n_out + k)
    x, g, u = bf16(gen, n, k), _weights(gen, n_out, k), _weights(gen, n_out, k)
    ld = (n_out + 7) // 8 * 8 + 8
    out = torch.full((n + 3, ld), 7.0, dtype=BF, device="cuda")
    gb.gdn_proj_gated(x.cuda(), g.cuda(), u.cuda(), out[:n])
    check(out[:n, :n_out], *gated(x.double(), g.double(), u.double()))
    assert (out[:n, n_out:] == 7).all() and (out[n:] == 7).all()  # nothing past the columns or the rows
    again = torch.empty_like(out[:n])
    gb.gdn_proj_gated(x.cuda(), g.cuda(), u.cuda(), again)
    assert torch.equal(again[:, :n_out], out[:n, :n_out])
    assert gb.gdn_device_status() == 0


def test_gated_halves_of_one_matrix_and_large_gates():
    """Gates far out on both sides: silu is the gate itself or zero, and no NaN arises."""
    gen = torch.Generator().manual_seed(1)
    n, m, k = 40, 96, 64
    x, w = bf16(gen, n, k, std=30.0), bf16(gen, 2 * m, k)
    for rows in (n, 700, 50000):
        xs = x.repeat((rows + n - 1) // n, 1)[:rows]
        out = torch.empty((rows, m), dtype=BF, device="cuda")
        wd = w.cuda()
        gb.gdn_proj_gated(xs.cuda(), wd[:m], wd[m:], out)
        assert torch.isfinite(out).all()
        check(out, *gated(xs.double(), w[:m].double(), w[m:].double()))


@pytest.mark.parametrize("n", [3, 100, 600, 40000])
def test_gated_not_numbers_stay_in_their_row_and_column(n):
    gen = torch.Generator().manual_seed(2)
    k, m = 136, 200
    x, g, u = bf16(gen, n, k), _weights(gen, m, k), _weights(gen, m, k)
    x[1, 5], g[7, 9], u[130, 1] = float("nan"), float("inf"), float("nan")
    out = torch.empty((n, m), dtype=BF, device="cuda")
    gb.gdn_proj_gated(x.cuda(), g.cuda(), u.cuda(), out)
    want = torch.zeros((n, m), dtype=torch.bool)
    want[1] = want[:, 130] = True
    bad = ~torch.isfinite(out).cpu()
    bad[:, 7] = want[:, 7]  # (an infinite gate: silu is infinite on one side, 0 or NaN on the other)
    assert torch.equal(bad, want)


@pytest.mark.parametrize("n,hidden,inter", [(1, 8, 8), (1, 2560, 1000), (5, 136, 1096), (64, 256, 640), (70, 72, 8),
                                            (129, 264, 520), (300, 128, 384), (1025, 320, 200),
                                            # few tiles of a long K, and a few behind whole waves of them: split along K
                                            (300, 264, 2600), (513, 520, 4104), (2000, 520, 16392), (20000, 264, 2560)])
def test_ffn_shapes(n, hidden, inter):
    gen = torch.Generator().manual_seed(n + hidden + inter)
    h, g, u, d = bf16(gen, n, hidden), _weights(gen, inter, hidden), _weights(gen, inter, hidden), _weights(gen, hidden, inter)
    ws = torch.empty(gb.gdn_ffn_workspace_size(n, hidden, inter) + 16, dtype=torch.uint8, device="cuda")
    ws[-16:] = 9
    out = torch.full((n + 2, hidden), 7.0, dtype=BF, device="cuda")
    gb.gdn_ffn(gb.Ffn(g.cuda(), u.cuda(), d.cuda()), h.cuda(), out[:n], ws[:-16])
    a, da = gated(h.double(), g.double(), u.double())
    want, slack = product(a, d.double())
    da = da + 2.0 ** -8 * (a.abs() + da)  # the half's rounding
    check(out[:n], want, slack + da @ d.double().abs().T)
    got = out[:n].cpu().double()
    assert (got - want).norm() <= 3.2e-3 * want.norm() or n * hidden < 1000
    assert (out[n:] == 7).all() and (ws[-16:] == 9).all()
    # the two calls in turn give the same bits
    half = torch.empty((n, inter), dtype=BF, device="cuda")
    gb.gdn_proj_gated(h.cuda(), g.cuda(), u.cuda(), half)
    assert torch.equal(half.view(torch.uint8).flatten(), ws[:half.nbytes])
    assert gb.gdn_device_status() == 0


@pytest.mark.parametrize("n,hidden,inter", [(2, 256, 712), (200, 256, 712), (700, 256, 712), (300, 256, 4096), (2000, 520, 16392)])
def test_ffn_captured_replayed_and_beside_another(n, hidden, inter):
    """Two blocks in a row in one graph, replayed with new inputs, while another stream runs the same block with a workspace of
    its own: the results of plain calls."""
    gen = torch.Generator().manual_seed(4)
    ffn = gb.Ffn(*(t.cuda() for t in (_weights(gen, inter, hidden), _weights(gen, inter, hidden), _weights(gen, hidden, inter))))
    size = gb.gdn_ffn_workspace_size(n, hidden, inter)
    new = lambda: torch.empty(size, dtype=torch.uint8, device="cuda")  # noqa: E731
    h, inputs = torch.empty((n, hidden), dtype=BF, device="cuda"), [bf16(gen, n, hidden).cuda() for _ in range(4)]
    mid, out, want, side_out = (torch.zeros_like(h) for _ in range(4))
    ws, ws2 = new(), new()
    gb.gdn_ffn(ffn, inputs[0], mid, ws)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        gb.gdn_ffn(ffn, h, mid, ws)
        gb.gdn_ffn(ffn, mid, out, ws)
    side = torch.cuda.Stream()
    for x in inputs:
        h.copy_(x)
        side.wait_stream(torch.cuda.current_stream())
        graph.replay()
        gb.gdn_ffn(ffn, x, side_out, ws2, stream=side)
        torch.cuda.synchronize()
        got, got_side = out.clone(), side_out.clone()
        gb.gdn_ffn(ffn, x, mid, ws)
        assert torch.equal(got_side, mid)
        gb.gdn_ffn(ffn, mid.clone(), want, ws)
        assert torch.equal(got, want)
    assert gb.gdn_device_status() == 0


@pytest.mark.parametrize("n", [5, 300, 3000])
def test_ffn_in_place(n):
    """The result over the input: the input has been read when the first of it is written."""
    gen = torch.Generator().manual_seed(6)
    hidden, inter = 264, 520
    ffn = gb.Ffn(*(t.cuda() for t in (_weights(gen, inter, hidden), _weights(gen, inter, hidden), _weights(gen, hidden, inter))))
    ws = torch.empty(gb.gdn_ffn_workspace_size(n, hidden, inter), dtype=torch.uint8, device="cuda")
    h = bf16(gen, n, hidden).cuda()
    out = torch.empty_like(h)
    gb.gdn_ffn(ffn, h, out, ws)
    gb.gdn_ffn(ffn, h, h, ws)
    assert torch.equal(h, out)


def test_no_tokens():
    g = torch.zeros((16, 64), dtype=BF, device="cuda")
    empty, out = torch.empty((0, 64), dtype=BF, device="cuda"), torch.empty((0, 16), dtype=BF, device="cuda")
    gb.gdn_proj_gated(empty, g, g, out)
    gb.gdn_ffn(gb.Ffn(g, g, torch.zeros((64, 16), dtype=BF, device="cuda")), empty, torch.empty_like(empty))


def test_gated_result_past_2_to_the_32_bytes():
    """Rows so far apart that the last ones lie beyond 4 GB."""
    gen = torch.Generator().manual_seed(5)
    n, m, k, ld = 2100, 72, 64, 1 << 20
    x, g, u = bf16(gen, n, k), _weights(gen, m, k), _weights(gen, m, k)
    big = torch.empty((n, ld), dtype=BF, device="cuda")
    big[:, m:m + 8] = 7
    gb.gdn_proj_gated(x.cuda(), g.cuda(), u.cuda(), big)
    check(big[:, :m], *gated(x.double(), g.double(), u.double()))
    assert (big[:, m:m + 8] == 7).all()
    few = torch.zeros_like(big[:40])
    gb.gdn_proj_gated(x[:40].cuda(), g.cuda(), u.cuda(), few)
    check(few[:, :m], *gated(x[:40].double(), g.double(), u.double()))
