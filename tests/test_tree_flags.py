"""Each flag of the layer alone, and all together, in gdn_verify_tree and gdn_commit_tree, against the fp64 oracle with
the same flags; and GDN_DEBUG's check of a commit's slots.  Tolerances of test_tree_gdn.py."""
import numpy as np
import pytest
import torch

import test_tree_gdn
from hybrid_gated_deltanet_gb300 import binding as gb
from hybrid_gated_deltanet_gb300 import synth
from gdn_cases import dev
from test_tree_decay import Case

pytestmark = pytest.mark.gpu

FLAGS = [gb.RAW_QKV, gb.NO_L2NORM, gb.GATES_DIRECT, gb.NO_OUTNORM,
         gb.RAW_QKV | gb.NO_L2NORM | gb.GATES_DIRECT | gb.NO_OUTNORM]
FORMS = [(synth.Geometry(2, 4, 128, 128, 4), synth.BF16), (synth.Geometry(2, 4, 128, 128, 4), synth.F32),
         (synth.Geometry(1, 3, 64, 64, 3), synth.F32), (synth.Geometry(2, 2, 32, 32, 2), synth.BF16)]


def flagged(nodes, geom, act, seed, flags):
    """Small inputs, so that keys that are not normalised stay below length 1 (the recurrence then contracts)."""
    c = Case(nodes, geom, act, seed, flags=flags)
    r = np.random.default_rng(seed)
    c.tok["x"] = synth.store(0.05 * r.standard_normal((c.N, geom.conv_channels)), act)
    c.dev["x"] = dev(c.tok["x"])
    if flags & gb.GATES_DIRECT:
        c.gates(-r.uniform(0, 1, (c.N, geom.n_v_heads)), b=r.uniform(0, 1, (c.N, geom.n_v_heads)))
    return c


@pytest.mark.parametrize("geom,act", FORMS)
@pytest.mark.parametrize("flags", FLAGS)
def test_verify_tree_with_flags(geom, act, flags):
    c = flagged([1, 12, 33], geom, act, 91, flags)
    c.check(c.verify(), sample=8)


@pytest.mark.parametrize("geom,act", FORMS)
@pytest.mark.parametrize("flags", FLAGS)
def test_commit_tree_with_flags(geom, act, flags):
    """Paths of one row, of a few, and of more rows than the kernel stages at a time."""
    c = flagged([1, 9, 40], geom, act, 92, flags)
    paths = [[0], [0, 3, 8], list(range(0, 40, 2)) + [39]]
    test_tree_gdn.commit(c, paths)
    test_tree_gdn.check_commit(c, paths)


def test_debug_checks_the_slots_of_a_commit(monkeypatch):
    c = Case([3, 4, 2], synth.Geometry(1, 2, 64, 64, 4), synth.BF16, 93)
    paths, slots = [[0], [0, 1], [1]], c.dev["slots"].clone()
    S, CS = c.dev["S"].clone(), c.dev["CS"].clone()
    gb.gdn_device_status()
    monkeypatch.setenv("GDN_DEBUG", "1")
    for where, value, said in ((2, int(slots[0]), "twice"), (1, c.n_slots, f"found slot {c.n_slots}"),
                               (0, -1, "found slot -1")):
        c.dev["slots"] = slots.clone()
        c.dev["slots"][where] = value
        with pytest.raises(gb.GdnError, match=said):
            test_tree_gdn.commit(c, paths)
        assert gb.gdn_device_status() & 2
    assert torch.equal(c.dev["S"], S) and torch.equal(c.dev["CS"], CS)  # refused before any kernel wrote
    c.dev["slots"] = slots
    test_tree_gdn.commit(c, paths)
    test_tree_gdn.check_commit(c, paths)
