"""The feed-forward block at each token tile of the kernel of few tokens, and with one half by either kernel; a captured call's
kernel names say which.  Tolerances as in the other tests of the block."""
import pytest
import torch

from hybrid_gated_deltanet_gb300 import binding as gb
from launches import kernels
from parts_cases import check, gated, product

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


@pytest.mark.parametrize("n,hidden,inter,half,back", [
    (16, 264, 1096, "k_fewILi16ELi1EE", "k_fewILi16ELi0EE"), (17, 264, 1096, "k_fewILi32ELi1EE", "k_fewILi32ELi0EE"),
    (32, 2560, 712, "k_fewILi32ELi1EE", "k_fewILi32ELi0EE"), (33, 264, 1096, "k_fewILi64ELi1EE", "k_fewILi64ELi0EE"),
    (65, 520, 2600, "k_fewILi128ELi1EE", "k_fewILi128ELi0EE"), (300, 264, 2600, "k_fewILi128ELi1EE", "k_fewILi128ELi0EE"),
    (300, 2560, 9216, "k_wideILi1EE", "k_fewILi128ELi0EE"), (600, 2560, 9216, "k_wideILi1EE", "k_wideILi0EE")])
def test_ffn(n, hidden, inter, half, back):
    gen = torch.Generator(device="cuda").manual_seed(n + hidden)
    rand = lambda *s, std=1.0: (torch.randn(s, generator=gen, device="cuda") * std).to(BF)  # noqa: E731
    h, g, u = rand(n, hidden), rand(inter, hidden, std=hidden ** -0.5), rand(inter, hidden, std=hidden ** -0.5)
    d, out = rand(hidden, inter, std=inter ** -0.5), torch.full((n + 1, hidden), 7.0, dtype=BF, device="cuda")
    ws = torch.full((gb.gdn_ffn_workspace_size(n, hidden, inter),), 255, dtype=torch.uint8, device="cuda")
    call = lambda s=None: gb.gdn_ffn(gb.Ffn(g, u, d), h, out[:n], ws, stream=s)  # noqa: E731
    names = kernels(call)
    assert len(names) == 2 and half in names[0] and back in names[1], names
    call()
    a, da = gated(h.double(), g.double(), u.double())
    want, slack = product(a, d.double())
    da = da + 2.0 ** -8 * (a.abs() + da)  # the half's rounding
    check(out[:n], want.cpu(), (slack + da @ d.double().abs().T).cpu())
    assert (out[n:] == 7).all() and gb.gdn_device_status() == 0
