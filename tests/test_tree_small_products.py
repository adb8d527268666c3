"""Queries almost orthogonal to an ancestor's key: the node's output is a small product times the ancestor's
value, and must be right relative to itself.

The nodes keep nothing of their own (beta ~ 0) over an empty state, so o_i is decay x (q_i . k_0) u_0 with
|q_i . k_0| between 1e-4 and 2e-4 of |q_i| |k_0|.  The norm's epsilon is the larger part of its root here, so that an
error of the product is an error of y.  The product is made in fp32.  Its factors are off by up to 2^-21 (SiLU), each
independently, its sum of 128 terms of up to about |q| |k| / 128 by 2^-24 a step: sqrt(2) 2^-21 x 128^-1/2 = 6e-8 of |q| |k|
as a standard deviation, 6e-4 of the smallest product, and three of them 2e-3.  That is added to the
tolerances of test_tree_gdn.py; operands of 11 bits would be off by 128^-1/2 2^-12 = 2e-5 of |q| |k|, a tenth of the product."""
import numpy as np
import pytest

import test_tree_gdn
from hybrid_gated_deltanet_gb300 import synth
from gdn_cases import dev, params_dev
from test_tree_decay import Case

pytestmark = pytest.mark.gpu


EXTRA = 2e-3


def silu(x):
    return x / (1 + np.exp(-x))


def near_orthogonal(r, k, target=1.5e-4):
    """bf16 inputs x whose silu has a cosine of about `target` with k."""
    x = synth.store(r.standard_normal((8000, 128)) - 0.45, synth.BF16).f64[:]
    q = silu(x)
    cos = np.abs(q @ k) / (np.linalg.norm(q, axis=1) * np.linalg.norm(k))
    best = int(np.argmin(np.abs(cos - target)))
    assert 1e-4 < cos[best] < 2e-4
    return x[best]


@pytest.mark.parametrize("act", [synth.BF16, synth.F32])
@pytest.mark.parametrize("geom,B,n", [(synth.Geometry(1, 2, 128, 128, 4), 1, 9), (synth.Geometry(1, 2, 128, 128, 2), 2, 40),
                                      (synth.Geometry(1, 8, 128, 128, 4), 160, 5), (synth.Geometry(1, 5, 128, 128, 3), 160, 20)])
def test_small_products_with_an_ancestor(act, geom, B, n, monkeypatch):
    c = Case([n] * B, geom, act, 95)
    r = np.random.default_rng(96)
    K, C, Hv = geom.d_conv, geom.conv_channels, geom.n_v_heads
    w = np.zeros((C, K))
    w[:, -1] = 1.0  # u = silu(x)
    c.p["conv_w"] = synth.store(w, act)
    x = synth.store(r.standard_normal((n, C)) - 0.45, synth.BF16).f64[:]
    k0 = silu(x[0, 128:256])
    for i in range(1, n):
        x[i, :128] = near_orthogonal(r, k0)
    c.trees = [[-1] + [0] * (n - 1)] * B
    c.tok["x"] = synth.store(np.tile(x, (B, 1)), act)
    c.S, c.CS = (synth.store(np.zeros(v.shape), v.dtype) for v in (c.S, c.CS))
    c.dev.update({k: dev(v) for k, v in (("x", c.tok["x"]), ("S", c.S), ("CS", c.CS))})
    c.dev["parents"].copy_(c.dev["parents"].new_tensor(c.trees[0] * B))
    b = np.full((n, 1), -30.0)
    b[0] = 4.0
    c.gates(-3.0, np.linspace(-2.0, 1.0, Hv), np.tile(b, (B, 1)))
    monkeypatch.setitem(test_tree_gdn.TOL_Y, act, test_tree_gdn.TOL_Y[act] + EXTRA)
    c.nodes = c.nodes[:2]  # (the other trees are copies)
    y = c.verify()
    c.N = sum(c.nodes)
    c.check(y[:c.N], sample=8)
