"""Low-rank activations near the end of fp32's range (gdn_proj_lora): finite ones give finite results in the kernels of few and
of many tokens.  Tolerance as in the other tests of the adapters: fp32 sums, the activations to 2^-16, one rounding."""
import pytest
import torch

from hybrid_gated_deltanet_gb300 import binding as gb
from launches import kernels
from parts_cases import bf16, check, cumulative, i32, lora

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


@pytest.mark.parametrize("rank", [16, 72])
@pytest.mark.parametrize("lens,kernel", [([1, 1, 5], "k_few"), ([3000, 1, 15, 2500, 16], "k_wide")])
def test_activations_between_the_largest_bf16_and_the_largest_float(lens, kernel, rank):
    gen = torch.Generator().manual_seed(rank)
    k, n_out, n, which = 72, 200, sum(lens), [0, 1, 1, 0, 0][:len(lens)]
    x, w = bf16(gen, n, k), bf16(gen, n_out, k, std=k ** -0.5)
    a, b = bf16(gen, 2, rank, k, std=k ** -0.5), bf16(gen, 2, n_out, rank, std=rank ** -0.5)
    # activations 3 and 5 are +-2^127 (1.9921875 + 0.75 2^-7): fp32 holds them, bf16 rounds them to infinity
    x[:, :2], w[:, :2] = 2.0 ** 64, 0.0
    a[:, :, :2] = 0.0
    a[:, 3, 0], a[:, 3, 1] = 2.0 ** 63 * 1.9921875, 2.0 ** 63 * 0.75 * 2.0 ** -7
    a[:, 5] = -a[:, 3]
    a[:, 3, 2:] = a[:, 5, 2:] = 0.0
    b[:, :, 3] = 2.0 ** -120 * bf16(gen, 2, n_out).abs()
    b[:, :, 5] = 0.0
    scale = torch.ones(2)
    big = x.double() @ a[0, 3].double()
    assert (big < torch.finfo(torch.float32).max).all() and torch.isinf(big.to(BF)).all()
    cu = cumulative(lens)
    xd, wd, ad = x.cuda(), w.cuda(), gb.Lora(a.cuda(), b.cuda(), scale.cuda())
    cud, idx, out = i32(cu), i32(which), torch.empty((n, n_out), dtype=BF, device="cuda")
    ws = torch.empty(gb.gdn_proj_lora_workspace_size(n, n_out, k, rank, len(lens)), dtype=torch.uint8, device="cuda")
    run = lambda stream=None: gb.gdn_proj_lora(xd, wd, ad, cud, idx, out, ws, stream=stream)  # noqa: E731
    assert any(kernel in name for name in kernels(run))
    run()
    assert torch.isfinite(out).all()
    check(out, *lora(x.double(), w.double(), a.double(), b.double(), scale.tolist(), cu, which))
    assert gb.gdn_device_status() == 0
