"""Trees whose decays differ along a line: strong ones before weak ones, and states that are erased (alpha = 0).

The decay between a node and an ancestor is the product of the alphas after the ancestor, whatever came
before it.  Against the fp64 oracle with the tolerances of test_tree_gdn.py.  They hold here too: a gate is good
to 6 x 2^-24 of itself (two functions and a product), a decay e^-x that is the sum of such gates to
x e^-x 3.6e-7 <= 1.4e-7 of the term that it scales."""
import numpy as np
import pytest

import oracle
import test_tree_gdn
from hybrid_gated_deltanet_gb300 import binding as gb
from hybrid_gated_deltanet_gb300 import synth
from gdn_cases import dev, host, oracle_kwargs, params_dev

pytestmark = pytest.mark.gpu

GEOMS = [synth.Geometry(2, 4, 128, 128, 4), synth.Geometry(1, 3, 64, 64, 4)]
FORMS = [(g, a) for g in GEOMS for a in (synth.BF16, synth.F32)]


class Case(test_tree_gdn.Case):
    def gates(self, a, A_log=None, b=None):
        """a (and b): a value per node and v-head, or one that is broadcast."""
        for name, v in (("a", a), ("b", b)):
            if v is not None:
                self.tok[name] = synth.store(np.broadcast_to(v, (self.N, self.geom.n_v_heads)), self.act)
                self.dev[name] = dev(self.tok[name])
        if A_log is not None:
            self.p["A_log"] = synth.store(np.broadcast_to(A_log, self.geom.n_v_heads), synth.F32)
            self.dev["prm"] = params_dev(self.p)

    def check(self, y, skipped=(), **kw):
        got = host(y)
        for b in range(len(self.nodes)):
            assert b in skipped or np.isfinite(got[self.cu[b]:self.cu[b + 1]]).all(), b
        return super().check(y, skipped, **kw)

    def run_oracle(self, b, rows, heads):
        at = np.asarray(rows)
        return oracle.run_sequence(self.geom, *(self.tok[k].f64[at] for k in ("x", "z", "a", "b")),
                                   s0=self.S.f64[self.slots[b]], conv0=self.CS.f64[self.slots[b]], heads=heads,
                                   q_scale=self.cfg.q_scale, flags=self.cfg.flags, **oracle_kwargs(self.p))


@pytest.mark.parametrize("geom,act", FORMS)
@pytest.mark.parametrize("shape", ["chain", "tree"])
@pytest.mark.parametrize("strong,weak,A_log", [(8.0, -8.0, np.log(16.0)), (10.0, -12.0, np.log(16.0)), (8.0, -14.0, 10.0)])
def test_weak_decays_after_strong_ones(geom, act, shape, strong, weak, A_log):
    c = Case([64, 20], geom, act, 81, shape)
    a = np.full((c.N, 1), weak)
    a[:10] = a[64:70] = strong
    c.gates(a, A_log)
    c.check(c.verify(), sample=8)


@pytest.mark.parametrize("geom,act", FORMS)
def test_a_gate_that_overflows_erases_the_state(geom, act):
    """exp(A_log) past fp32 on one v-head: log alpha = -inf at every node, alpha = 0."""
    c = Case([30, 3], geom, act, 82)
    A_log = np.zeros(geom.n_v_heads)
    A_log[1] = 90.0
    c.gates(c.tok["a"].f64[:], A_log)
    c.check(c.verify(), sample=8)


@pytest.mark.parametrize("act", [synth.BF16, synth.F32])
@pytest.mark.parametrize("geom", GEOMS)
@pytest.mark.parametrize("shape", ["chain", "tree"])
@pytest.mark.parametrize("lowest", [-np.inf, -3e38, -200.0])
def test_erased_states_with_direct_gates(act, geom, shape, lowest):
    """Some nodes of a tree erase the state (log alpha given): their descendants see what follows, and commits agree."""
    c = Case([33, 9], geom, act, 83, shape, flags=gb.GATES_DIRECT)
    r = np.random.default_rng(84)
    a = -r.uniform(0, 0.5, (c.N, geom.n_v_heads))
    a[5], a[12, 0], a[20], a[33 + 2] = lowest, lowest, lowest, lowest
    c.gates(a, b=r.uniform(0, 1, (c.N, geom.n_v_heads)))
    c.check(c.verify(), sample=12)
    paths = [list(range(0, 25)), [0, 2, 3]]
    test_tree_gdn.commit(c, paths)
    test_tree_gdn.check_commit(c, paths)


def test_decays_of_many_v_heads_in_a_cta():
    """bf16, d = 128, all 5 v-heads of a k-head in one CTA, each with decays of its own."""
    c = Case([40, 20] + [3] * 160, synth.Geometry(1, 5, 128, 128, 4), synth.BF16, 85)
    a = np.full((c.N, 5), -14.0)
    a[:8, 0], a[3:6, 1], a[40:50, 2], a[:, 3], a[5, 4] = 8.0, 8.0, 8.0, 1.0, 12.0
    c.gates(a, np.asarray([10.0, 10.0, 10.0, 0.0, 90.0]))
    c.check(c.verify(), sample=4)
