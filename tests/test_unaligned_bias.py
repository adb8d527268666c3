"""A conv bias that starts at an odd element of a flat buffer of parameters: 2-byte alignment (4 in fp32) is all that
a bias needs.  The results are those of a copy that is aligned, bit for bit."""
import pytest
import torch

import test_tree_gdn
import test_tree_more
from hybrid_gated_deltanet_gb300 import binding as gb
from hybrid_gated_deltanet_gb300 import synth
from gdn_cases import config, dev, params_dev

pytestmark = pytest.mark.gpu


def at_odd_element(t, skip=1):
    flat = torch.zeros(t.numel() + skip, dtype=t.dtype, device=t.device)
    out = flat[skip:].view(t.shape)
    out.copy_(t)
    assert out.data_ptr() % 16 == skip * t.element_size() and out.is_contiguous()
    return out


def shifted(prm, skip):
    return gb.Params(prm.conv_w, prm.A_log, prm.norm_w, at_odd_element(prm.conv_b, skip), prm.dt_bias)


@pytest.mark.parametrize("skip", [1, 2, 3])
@pytest.mark.parametrize("act", [synth.BF16, synth.F32])
@pytest.mark.parametrize("geom", [synth.Geometry(2, 4, 128, 128, 4), synth.Geometry(2, 6, 64, 64, 3)])
def test_trees(geom, act, skip):
    paths = [[0, 2, 5], list(range(20)), [0]]
    one, two = (test_tree_more.Biased([9, 40, 1], geom, act, 33) for _ in range(2))
    two.dev["prm"] = shifted(one.dev["prm"], skip)
    y = one.verify()
    one.check(y, sample=6)
    assert torch.equal(y, two.verify())
    for c in (one, two):
        test_tree_gdn.commit(c, paths)
    assert torch.equal(one.dev["S"], two.dev["S"]) and torch.equal(one.dev["CS"], two.dev["CS"])
