"""Forms of gdn_proj_lora that only some sizes reach: every token tile of the kernel of few tokens (with a ring of several
tokens' rows, and of one), more requests than the low side keeps in shared memory, and a token tile of many adapters in the
kernel of many tokens.  A captured call's kernel names say that it is reached.  Tolerances as in the other tests of the adapters;
the 64-bit form runs on the GPU."""
import pytest
import torch

from hybrid_gated_deltanet_gb300 import binding as gb
from launches import kernels
from parts_cases import check, cumulative, i32, lora

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


def _run(lens, which, k, n_out, rank, pool, kernel, spoil=None):
    """Checks the call against 64 bits; then, with NaN in adapter `spoil`, that the other requests' rows are the same bits."""
    gen = torch.Generator(device="cuda").manual_seed(rank + k)
    rand = lambda *s, std=1.0: (torch.randn(s, generator=gen, device="cuda") * std).to(BF)  # noqa: E731
    n, cu = sum(lens), cumulative(lens)
    x, w, scale = rand(n, k), rand(n_out, k, std=k ** -0.5), torch.rand(pool, generator=gen, device="cuda") + 0.5
    a, b = rand(pool, rank, k, std=k ** -0.5), rand(pool, n_out, rank, std=rank ** -0.5)
    ad, cud, idx = gb.Lora(a, b, scale), i32(cu), i32(which)
    out = torch.full((n + 1, (n_out + 7) // 8 * 8), 7.0, dtype=BF, device="cuda")
    ws = torch.full((gb.gdn_proj_lora_workspace_size(n, n_out, k, rank, len(lens)),), 255, dtype=torch.uint8, device="cuda")
    call = lambda s=None: gb.gdn_proj_lora(x, w, ad, cud, idx, out[:n], ws, stream=s)  # noqa: E731
    names = kernels(call)
    assert kernel in names[-1], names
    call()
    y, d = lora(x.double(), w.double(), a.double(), b.double(), scale.double().tolist(), cu, which)
    check(out[:n, :n_out], y.cpu(), d.cpu())
    assert (out[n:] == 7).all() and (out[:, n_out:] == 7).all()
    if spoil is not None:
        clean = out.clone()
        a[spoil, 0, 1], b[spoil, :, rank - 1] = float("nan"), float("inf")
        call()
        hit = torch.zeros(n, dtype=torch.bool)
        for s, e in enumerate(which):
            if e == spoil:
                hit[cu[s]:cu[s + 1]] = True
        hit = hit.cuda()
        assert torch.equal(out[:n][~hit], clean[:n][~hit]) and torch.isnan(out[:n, :n_out][hit]).all()
    assert gb.gdn_device_status() == 0


@pytest.mark.parametrize("n,rank", [(65, 8), (100, 8), (70, 16), (127, 16), (65, 24), (127, 40), (100, 64), (65, 128), (100, 128)])
def test_token_tiles_of_128(n, rank):
    _run([1] * n, [(i * 5) % 7 - 1 for i in range(n)], 2560, 12352, rank, 6, "k_fewILi128ELi2EE", spoil=2)


@pytest.mark.parametrize("lens,n_out,k,rank,tokens", [
    ([1] * 30, 2560, 4096, 32, 16), ([9, 7], 72, 4096, 128, 16), ([5, 1, 10], 12350, 264, 40, 16), ([4] * 12, 2000, 264, 16, 16),
    ([1] * 60, 2560, 4096, 32, 32), ([1] * 30, 5000, 2560, 128, 32), ([1] * 30, 12352, 2560, 72, 32),
    ([1] * 64, 12352, 2560, 16, 64), ([1] * 64, 12352, 2560, 64, 64), ([12] * 4, 12352, 2560, 16, 64), ([1] * 130, 5000, 2560, 96, 64)])
def test_smaller_token_tiles(lens, n_out, k, rank, tokens):
    _run(lens, [(i * 5) % 7 - 1 for i in range(len(lens))], k, n_out, rank, 6, f"k_fewILi{tokens}ELi2EE", spoil=4)


def test_several_token_tiles_of_128():
    lens = [1] * 150 + [3, 0, 2] + [1] * 145
    _run(lens, [(i * 5) % 7 - 1 for i in range(len(lens))], 4096, 2555, 32, 6, "k_fewILi128ELi2EE", spoil=0)


@pytest.mark.parametrize("rank", [16, 72])
def test_more_than_1024_requests_in_a_call_of_many_tokens(rank):
    lens = [[20, 16, 0, 33, 15, 1, 40][i % 7] for i in range(1600)]
    _run(lens, [(i * 3) % 8 - 1 for i in range(1600)], 136, 200, rank, 7, "k_wideILi2EE", spoil=3)


@pytest.mark.parametrize("rank", [8, 16, 40, 72, 128])
def test_a_token_tile_of_many_adapters(rank):
    """100 single tokens, each with an adapter of its own, between two prompts, and a prompt that uses one of them."""
    lens = [1900] + [1] * 100 + [700, 2]
    which = [3] + list(range(100)) + [50, 99]
    _run(lens, which, 136, 520, rank, 100, "k_wideILi2EE", spoil=50)
