"""Which of the two kernels a projection runs, at sizes where the other one took much longer: a captured call's kernel names.
The figures are graph replays of both, in us, the kernel of few tokens first."""
import pytest
import torch

from hybrid_gated_deltanet_gb300 import binding as gb
from launches import kernels
from parts_cases import cumulative, i32

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


def _t(*shape):
    return torch.zeros(shape, dtype=BF, device="cuda")


@pytest.mark.parametrize("k,n_out,rank,lens,kernel", [
    (2560, 12352, 16, [1], "k_few"),            # 16 / 29
    (2560, 12352, 16, [1] * 64, "k_few"),       # 23 / 45
    (2560, 12352, 16, [12] * 4, "k_few"),       # 21 / 29: four short requests
    (2560, 12352, 16, [128], "k_wide"),         # 42 / 22
    (2560, 12352, 64, [64], "k_wide"),          # 40 / 22
    (2560, 12352, 128, [16], "k_few"),          # 25.5 / 26.4
    (2560, 12352, 128, [16, 16], "k_wide"),     # 42 / 26
    (2560, 12352, 128, [16] * 4, "k_wide"),     # 70 / 28
    (4096, 2560, 128, [64, 64], "k_wide"),      # 45 / 32
    (4096, 2560, 32, [1] * 300, "k_few"),       # 40 / 169
    (4096, 2560, 32, [32] * 32, "k_wide"),      # 94 / 31
    (1024, 3584, 128, [64], "k_wide"),          # 32 / 15
    (1024, 3584, 128, [32] * 4, "k_wide"),      # 53 / 23
])
def test_projection_with_adapters(k, n_out, rank, lens, kernel):
    n = sum(lens)
    x, w, ad = _t(n, k), _t(n_out, k), gb.Lora(_t(4, rank, k), _t(4, n_out, rank))
    cu, idx, out = i32(cumulative(lens)), i32([i % 4 for i in range(len(lens))]), _t(n, n_out)
    ws = torch.empty(gb.gdn_proj_lora_workspace_size(n, n_out, k, rank, len(lens)), dtype=torch.uint8, device="cuda")
    names = kernels(lambda s: gb.gdn_proj_lora(x, w, ad, cu, idx, out, ws, stream=s))
    assert len(names) == 2 and kernel in names[1], names


@pytest.mark.parametrize("k,n_out,n,kernel", [(2560, 9216, 64, "k_few"), (64, 262144, 64, "k_few"), (1024, 3584, 256, "k_few"),
                                              (2560, 9216, 257, "k_wide"), (1024, 3584, 768, "k_wide")])
def test_gated_half(k, n_out, n, kernel):
    # 20 / 23, 60 / 78, 10.5 / 11.4, 50 / 33, 27 / 17.5
    x, g, out = _t(n, k), _t(n_out, k), _t(n, n_out)
    names = kernels(lambda s: gb.gdn_proj_gated(x, g, g, out, stream=s))
    assert len(names) == 1 and kernel in names[0], names
