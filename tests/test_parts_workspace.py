"""The workspaces of gdn_ffn and gdn_proj_lora, on the host without a GPU: one that was made for the largest call serves the
smaller ones.  What a call needs is read from its refusal of an empty workspace; no call here reaches a launch."""
import ctypes
import re

import pytest

from hybrid_gated_deltanet_gb300 import binding as gb
from hybrid_gated_deltanet_gb300 import build as gbuild

FAKE = 0x100000  # an aligned address that is never dereferenced on the host
TOKENS = list(range(1, 700)) + list(range(700, 6000, 37)) + [8192, 9590, 19456, 19457, 20002, 40000, 1 << 22]


@pytest.fixture(scope="module")
def lib():
    gbuild.build()
    return gb.load()


def _need(lib, status):
    err = lib.gdn_last_error().decode()
    assert status == -6, err
    return int(re.search(r"found 0 bytes, required (\d+) bytes", err).group(1))


def _ffn_need(lib, n, hidden, inter):
    w = gb.CFfn(FAKE, FAKE, FAKE, hidden, inter)
    return _need(lib, lib.gdn_ffn(ctypes.byref(w), FAKE, n, FAKE, FAKE, 0, None))


def _lora_need(lib, n, n_out, k, rank, n_seg):
    c, ld = gb.CLora(FAKE, FAKE, None, 8, rank), (n_out + 7) // 8 * 8
    return _need(lib, lib.gdn_proj_lora(FAKE, FAKE, ctypes.byref(c), FAKE, FAKE, n_seg, FAKE, n, n_out, k, ld, FAKE, 0, None))


@pytest.mark.parametrize("hidden,inter", [(2560, 9216), (1024, 3584), (264, 8200), (520, 16392), (8, 8)])
def test_ffn_workspace_serves_fewer_tokens(lib, hidden, inter):
    had, most = 0, 0
    for n in TOKENS:
        size, most = lib.gdn_ffn_workspace_size(n, hidden, inter), max(most, _ffn_need(lib, n, hidden, inter))
        assert size >= had and size >= most, n
        had = size
    for n in (1, 40, 64):  # decoding steps pay for nothing that only more tokens use
        assert lib.gdn_ffn_workspace_size(n, hidden, inter) == _ffn_need(lib, n, hidden, inter) == n * inter * 2


@pytest.mark.parametrize("n_out,k", [(2560, 4096), (12352, 2560), (264, 8200), (520, 16392), (72, 64)])
def test_lora_workspace_serves_fewer_tokens_lower_ranks_and_any_requests(lib, n_out, k):
    had, most = 0, 0
    for n in TOKENS:
        size = lib.gdn_proj_lora_workspace_size(n, n_out, k, 64, 3)
        for rank, n_seg in ((64, 3), (64, 0), (64, 1 << 20), (64, min(n, 1 << 20)), (8, 1), (32, 8)):
            assert lib.gdn_proj_lora_workspace_size(n, n_out, k, rank, n_seg) <= size
            most = max(most, _lora_need(lib, n, n_out, k, rank, n_seg))
        assert size >= had and size >= most, n
        had = size


def test_a_call_takes_what_it_needs(lib):
    """Sizes whose last tiles are split need more than the tokens' own rows, those that are not do not."""
    assert _ffn_need(lib, 8192, 2560, 9216) > 8192 * 9216 * 2
    assert _ffn_need(lib, 200, 2560, 9216) == 200 * 9216 * 2
    assert _lora_need(lib, 2400, 2560, 4096, 32, 44) > 2400 * (64 * 2 + 4)
    assert _lora_need(lib, 64, 2560, 4096, 32, 64) == 64 * (64 * 2 + 4)
