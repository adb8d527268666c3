"""GPU parity of gdn_verify_tree and gdn_commit_tree against the fp64 oracle.

A node's output is the oracle's on the node's line of ancestors.  Tolerances (relative
Frobenius): bf16 y is rounded once (2^-8 of each value) and made of sums of products whose
operands are rounded to 11 bits (2^-11 each, truncation 2^-10): 2^-8 + 4 x 2^-10 = 7.8e-3.  fp32
arithmetic throughout: sums of 128 terms, 128 x 2^-24 = 7.6e-6 of the terms' size at most, through
two stages and the norm: 2e-5.  The committed state is fp32 arithmetic whatever the activations:
2e-5.  Conv states are copies: equal bit for bit."""
import numpy as np
import pytest
import torch

import oracle
from hybrid_gated_deltanet_gb300 import binding as gb
from hybrid_gated_deltanet_gb300 import synth
from gdn_cases import config, dev, host, oracle_kwargs, params_dev, rel_fro, sample_heads
from tree_cases import cumulative, i32, line, make_tree

pytestmark = pytest.mark.gpu

TOL_Y = {synth.BF16: 2.0 ** -8 + 4 * 2.0 ** -10, synth.F32: 2e-5}
TOL_S = 2e-5
SMALL = synth.Geometry(2, 4, 128, 128, 4)


class Case:
    def __init__(self, nodes, geom, act, seed, shape="tree", spare_rows=0, q_scale=1.0, flags=0, n_slots=None):
        r = synth.rng_for(71, seed)
        self.geom, self.act, self.nodes = geom, act, nodes
        self.cfg, self.p = config(geom, act, q_scale=q_scale, flags=flags), synth.make_params(geom, r, act)
        self.cu = cumulative(nodes)
        self.N = int(self.cu[-1]) + spare_rows
        self.trees = [make_tree(r, n, shape) for n in nodes]
        self.tok = synth.make_tokens(geom, self.N, r, act)
        B = len(nodes)
        self.n_slots = n_slots or B + 2
        self.S = synth.make_state(geom, self.n_slots, r)
        self.CS = synth.make_conv_state(geom, self.n_slots, r, act)
        self.slots = r.permutation(self.n_slots)[:B].astype(np.int32)
        self.dev = {k: dev(v) for k, v in self.tok.items()}
        self.dev.update(S=dev(self.S), CS=dev(self.CS), prm=params_dev(self.p), slots=i32(self.slots), cu=i32(self.cu),
                        parents=i32([p for t in self.trees for p in t] + [0] * spare_rows))
        self.max_nodes = max(1, max(nodes))

    def verify(self, y=None, stream=None):
        d = self.dev
        if y is None:
            y = torch.full((self.N, self.geom.value_dim), 7.0, dtype=self.cfg.torch_dtype, device="cuda")
        gb.gdn_verify_tree(self.cfg, d["prm"], d["x"], d["z"], d["a"], d["b"], d["CS"], d["S"], d["slots"], d["cu"],
                           d["parents"], self.max_nodes, y, stream)
        return y

    def run_oracle(self, b, rows, heads):
        at = np.asarray(rows)
        return oracle.run_sequence(self.geom, *(self.tok[k].f64[at] for k in ("x", "z", "a", "b")),
                                   s0=self.S.f64[self.slots[b]], conv0=self.CS.f64[self.slots[b]], heads=heads,
                                   q_scale=self.cfg.q_scale, **oracle_kwargs(self.p))

    def check(self, y, skipped=(), heads=None, sample=None):
        torch.cuda.synchronize()
        assert gb.gdn_device_status() == 0
        got, dv = host(y), self.geom.d_v
        heads = heads if heads is not None else list(range(self.geom.n_v_heads))
        cols = np.concatenate([np.arange(h * dv, (h + 1) * dv) for h in heads])
        r = np.random.default_rng(11)
        live = np.zeros(self.N, bool)
        worst = 0.0
        for b, n in enumerate(self.nodes):
            if b in skipped:
                continue
            live[self.cu[b]:self.cu[b + 1]] = True
            some = range(n) if sample is None or n <= sample else sorted({0, n - 1} | set(r.choice(n, sample - 2)))
            for i in some:
                rows = [int(self.cu[b]) + a for a in line(self.trees[b], i)]
                ref = self.run_oracle(b, rows, heads)["y"][-1][cols]
                worst = max(worst, rel_fro(got[self.cu[b] + i][cols], ref))
        assert worst <= TOL_Y[self.act], worst
        assert (got[~live] == 7.0).all()
        return worst


@pytest.mark.parametrize("act", [synth.BF16, synth.F32])
@pytest.mark.parametrize("shape", ["tree", "chain", "star", "comb"])
def test_verify_tree_shapes(act, shape):
    c = Case([1, 2, 5, 17, 0, 33], SMALL, act, 1, shape)
    c.check(c.verify(), sample=8)


@pytest.mark.parametrize("geom", [synth.Geometry(1, 1, 32, 32, 2), synth.Geometry(2, 6, 64, 64, 3),
                                  synth.Geometry(1, 8, 128, 128, 2), synth.Geometry(3, 3, 128, 128, 3)])
@pytest.mark.parametrize("act", [synth.BF16, synth.F32])
def test_verify_tree_geometries(geom, act):
    c = Case([3, 20, 64], geom, act, 2, q_scale=geom.d_k ** -0.5)
    c.check(c.verify(), sample=6)


def test_verify_tree_4b_and_wide():
    for geom in (synth.QWEN35_4B, synth.WIDE_GVA):
        c = Case([16, 64, 7, 48], geom, synth.BF16, 3)
        c.check(c.verify(), heads=sample_heads(geom.n_v_heads, 3), sample=5)


def test_verify_tree_many_sequences():
    r = np.random.default_rng(2)
    c = Case([int(v) for v in r.integers(0, 13, 150)], synth.Geometry(2, 4, 128, 128, 4), synth.BF16, 4)
    c.check(c.verify(), heads=[0, 3], sample=2)


def test_a_chain_equals_verify_rows():
    """A chain through gdn_verify_tree and through gdn_verify_rows_nosnap."""
    B, r = 5, 9
    c = Case([r] * B, synth.QWEN35_4B, synth.BF16, 5, "chain")
    y = c.verify()
    d = c.dev
    want = torch.empty_like(y).view(B, r, -1)
    gb.gdn_verify_rows_nosnap(c.cfg, d["prm"], *(d[k].view(B, r, -1) for k in ("x", "z", "a", "b")), d["CS"], d["S"],
                              d["slots"], want)
    torch.cuda.synchronize()
    assert rel_fro(host(y), host(want).reshape(B * r, -1)) <= TOL_Y[synth.BF16]


def test_verify_tree_writes_nothing_else():
    c = Case([4, 9], SMALL, synth.BF16, 6, spare_rows=3)
    c.check(c.verify())
    assert np.array_equal(host(c.dev["S"]), c.S.f64[:]) and np.array_equal(host(c.dev["CS"]), c.CS.f64[:])


def test_verify_tree_skips():
    """Trees above max_nodes, slots out of range, rows past the arrays; two trees may read one slot."""
    c = Case([4, 9, 3, 6, 2], SMALL, synth.BF16, 7)
    c.max_nodes = 8
    c.slots = np.asarray([2, 0, 99, 2, -1], np.int32)
    c.dev["slots"] = i32(c.slots)
    c.check(c.verify(), skipped=(1, 2, 4))
    c.max_nodes, c.slots = 64, np.asarray([1, 0, 2, 3, 4], np.int32)
    c.dev["slots"], c.dev["cu"] = i32(c.slots), i32([0, 4, 13, 16, 22, 30])
    c.check(c.verify(), skipped=(4,))


def test_verify_tree_parents_out_of_range():
    c = Case([6], SMALL, synth.F32, 8)
    c.trees = [[-5, 0, 7, 3, 1, 4]]
    c.dev["parents"] = i32(c.trees[0])
    c.check(c.verify())


@pytest.mark.parametrize("act", [synth.BF16, synth.F32])
def test_verify_tree_nan_off_the_line(act):
    """NaN inputs of a node reach its descendants and nobody else."""
    c = Case([20], SMALL, act, 9)
    ref = c.verify().clone()
    c.dev["x"][7] = float("nan")
    y = c.verify()
    torch.cuda.synchronize()
    for i in range(20):
        if 7 in line(c.trees[0], i):
            assert torch.isnan(y[i].float()).any()
        else:
            assert torch.equal(y[i], ref[i]), i


def test_verify_tree_slow_and_fast_decay():
    """Decays from almost 1 to almost 0 along a chain of 64."""
    for A_log in (-6.0, 4.0):
        c = Case([64], SMALL, synth.F32, 10, "chain")
        c.p["A_log"] = synth.store(np.full(4, A_log), synth.F32)
        c.dev["prm"] = params_dev(c.p)
        c.check(c.verify(), sample=6)


def test_verify_tree_flags():
    """RAW_QKV, NO_L2NORM, GATES_DIRECT and NO_OUTNORM together: the bare recurrence on given q, k, v, log
    alpha and beta, against a plain loop."""
    n, geom = 12, synth.Geometry(1, 2, 64, 64, 4)
    c = Case([n], geom, synth.F32, 12, flags=15)
    r = np.random.default_rng(8)
    a, b = -r.uniform(0, 1, (n, 2)).astype(np.float32), r.uniform(0, 1, (n, 2)).astype(np.float32)
    x = 0.1 * r.standard_normal((n, geom.conv_channels)).astype(np.float32)
    for k, v in (("a", a), ("b", b), ("x", x)):
        c.dev[k] = torch.from_numpy(v).cuda()
    y = host(c.verify())
    x, S0 = x.astype(np.float64), c.S.f64[c.slots[0]]
    want = np.empty((n, 128))
    for j in range(2):
        states = {}
        for i in range(n):
            q, k, v = x[i, :64], x[i, 64:128], x[i, 128 + 64 * j:192 + 64 * j]
            p = c.trees[0][i]
            S = np.exp(float(a[i, j])) * (states[p] if p >= 0 else S0[j])
            S = S + float(b[i, j]) * np.outer(v - S @ k, k)
            states[i] = S
            want[i, 64 * j:64 * j + 64] = S @ q
    assert rel_fro(y, want) <= TOL_Y[synth.F32]


# ---- commit ---------------------------------------------------------------------------------------


def commit(c, paths, src=True, max_rows=None, stream=None):
    d = c.dev
    rows = [int(c.cu[b]) + i for b, p in enumerate(paths) for i in p]
    cu = i32(cumulative([len(p) for p in paths]))
    gb.gdn_commit_tree(c.cfg, d["prm"], d["x"], d["a"], d["b"], d["CS"], d["S"], d["slots"], cu,
                       i32(rows) if src else None, max_rows or max(1, max(len(p) for p in paths)), stream)


def check_commit(c, paths, heads=None, skipped=()):
    torch.cuda.synchronize()
    assert gb.gdn_device_status() == 0
    S, CS = host(c.dev["S"]), host(c.dev["CS"])
    S0, C0 = c.S.f64[:], c.CS.f64[:]
    heads = heads if heads is not None else list(range(c.geom.n_v_heads))
    for b, p in enumerate(paths):
        s = c.slots[b]
        if b in skipped or not p:
            continue
        ref = c.run_oracle(b, [int(c.cu[b]) + i for i in p], heads)
        assert rel_fro(S[s][heads], ref["S"][heads]) <= TOL_S
        assert np.array_equal(CS[s], ref["conv"])
        S0[s], C0[s] = S[s], CS[s]
    assert np.array_equal(S, S0) and np.array_equal(CS, C0)  # nothing else is written


@pytest.mark.parametrize("act", [synth.BF16, synth.F32])
@pytest.mark.parametrize("geom", [SMALL, synth.Geometry(1, 1, 32, 32, 2), synth.Geometry(2, 6, 64, 64, 3),
                                  synth.Geometry(1, 8, 128, 128, 4)])
def test_commit_tree_paths(geom, act):
    """Paths of one row to 64, none among them: states by the oracle, conv states bit for bit."""
    c = Case([1, 5, 40, 64, 9, 30], geom, act, 21)
    paths = [[0], [0, 3], list(range(2, 35)), list(range(64)), [], list(range(0, 30, 2))]
    commit(c, paths)
    check_commit(c, paths)


def test_commit_tree_without_source_rows():
    c = Case([3, 1, 7], SMALL, synth.BF16, 22)
    paths = [list(range(n)) for n in c.nodes]
    commit(c, paths, src=False)
    check_commit(c, paths)


def test_commit_tree_4b_and_wide():
    for geom in (synth.QWEN35_4B, synth.WIDE_GVA):
        c = Case([9, 4, 20, 12], geom, synth.BF16, 23)
        paths = [[0, 2, 7], [3], list(range(18)), [1, 2, 3, 5, 8]]
        commit(c, paths)
        check_commit(c, paths, heads=sample_heads(geom.n_v_heads, 3))


def test_commit_tree_skips():
    """Rows above max_rows, bad slots and source rows outside the arrays."""
    c = Case([6, 12, 3, 5], SMALL, synth.BF16, 24)
    c.slots = np.asarray([1, 0, 77, 3], np.int32)
    c.dev["slots"] = i32(c.slots)
    paths = [[0, 3], list(range(10)), [0], [1, 4]]
    rows = [int(c.cu[b]) + i for b, p in enumerate(paths) for i in p]
    bad = rows[:1] + [-1] + rows[1:2] + rows[2:13] + [c.N, rows[13], 1 << 30, rows[14]]
    d = c.dev
    gb.gdn_commit_tree(c.cfg, d["prm"], d["x"], d["a"], d["b"], d["CS"], d["S"], d["slots"], i32([0, 3, 13, 14, 18]),
                       i32(bad), 9)
    check_commit(c, paths, skipped=(1, 2))


def test_commit_tree_equals_decode_steps():
    """A committed path and the same tokens one decode step at a time."""
    c = Case([8, 8, 8], synth.QWEN35_4B, synth.BF16, 25)
    path = [0, 2, 3, 6]
    d = c.dev
    S, CS = d["S"].clone(), d["CS"].clone()
    y = torch.empty((3, c.geom.value_dim), dtype=torch.bfloat16, device="cuda")
    for i in path:
        at = torch.tensor([int(v) + i for v in c.cu[:-1]], device="cuda")
        gb.gdn_decode_step(c.cfg, d["prm"], d["x"][at], d["z"][at], d["a"][at], d["b"][at], CS, S, d["slots"], y)
    commit(c, [path] * 3)
    torch.cuda.synchronize()
    assert rel_fro(host(d["S"]), host(S)) <= TOL_S and torch.equal(d["CS"], CS)


def test_verify_then_commit_on_a_stream_and_captured():
    c = Case([10, 30], SMALL, synth.BF16, 26)
    want = c.verify().clone()
    paths = [[0, 1], [0, 4, 9]]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    y = torch.zeros_like(want)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        c.verify(y)
    y.zero_()
    with torch.cuda.stream(s):
        g.replay()
        commit(c, paths)
    check_commit(c, paths)
    assert torch.equal(y, want)
