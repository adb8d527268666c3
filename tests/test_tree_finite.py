"""Every output of a tree verify of finite inputs is finite (the worst of a list of errors passes over NaN: here each
row is looked at)."""
import numpy as np
import pytest

from hybrid_gated_deltanet_gb300 import synth
from test_tree_decay import Case

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("act", [synth.BF16, synth.F32])
@pytest.mark.parametrize("shape", ["tree", "chain", "star", "comb"])
@pytest.mark.parametrize("geom", [synth.Geometry(2, 4, 128, 128, 4), synth.Geometry(1, 8, 128, 128, 2),
                                  synth.Geometry(3, 3, 128, 128, 3), synth.Geometry(2, 6, 64, 64, 3),
                                  synth.Geometry(1, 1, 32, 32, 2)])
def test_outputs_are_finite(geom, shape, act):
    c = Case([64, 1, 2, 17, 0, 33, 48, 16, 32], geom, act, 97, shape)
    c.check(c.verify(), sample=2)


@pytest.mark.parametrize("most", [16, 32, 64])
def test_outputs_of_many_trees_are_finite(most):
    """Several waves of CTAs, all v-heads of a k-head in one."""
    r = np.random.default_rng(most)
    c = Case([int(v) for v in r.integers(0, most + 1, 200)], synth.Geometry(2, 6, 128, 128, 4), synth.BF16, 98)
    c.max_nodes = most
    c.check(c.verify(), sample=2, heads=[0, 5])


@pytest.mark.parametrize("nodes", [[8], [1], [8, 3, 8, 0, 5], [9], [8] * 40])
@pytest.mark.parametrize("shape", ["tree", "chain"])
def test_few_small_trees(nodes, shape):
    """bf16, d = 128: trees of up to 8 nodes on either side of the rule between the two forms of the kernel."""
    c = Case(nodes, synth.Geometry(2, 4, 128, 128, 4), synth.BF16, 99, shape)
    c.check(c.verify(), sample=4)
