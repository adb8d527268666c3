"""GPU parity of gdn_attn_tree against the fp64 oracle, element by element.

The tolerance follows from the roundings the call documents.  The weights are rounded to
bf16 (half a step: 2^-8 relative) and divided by the sum of the rounded weights, so
o is off by at most 2^-8 sum_j p_j |v_j - o| (to first order; 1.02 covers the second), its own
rounding adds 2^-8 |o|.  fp32 scores: D products, |s| sums of at most a few hundred, so an
absolute error below D 2^-24 max sum |q k| scale < 1e-4, which moves every weight by 1e-4 relative;
with the fp32 sums of o (2^-24 per term, a few thousand terms) 3e-4 sum_j p_j |v_j| covers both."""
import math

import numpy as np
import pytest
import torch

from oracle import attention as at
from hybrid_gated_deltanet_gb300 import binding as gb
from hybrid_gated_deltanet_gb300 import synth
from gdn_cases import dev, host
from tree_cases import cumulative, gather, i32, line, make_tree, paged

pytestmark = pytest.mark.gpu


def _bf16(r, shape):
    return synth.store(r.standard_normal(shape), synth.BF16)


def _expect(q, K, V, scale):
    """o and the tolerance of every element; q [Hq, D], K, V [L, Hkv, D]."""
    Hq, D = q.shape
    G = Hq // K.shape[1]
    o = at.decode_attention(q, K, V, scale)
    tol = np.empty_like(o)
    for h in range(Hq):
        s = scale * (K[:, h // G] @ q[h])
        p = np.exp(s - s.max())
        p /= p.sum()
        v = V[:, h // G]
        tol[h] = 1.02 * 2.0 ** -8 * (p @ np.abs(v - o[h]) + np.abs(o[h])) + 3e-4 * (p @ np.abs(v)) + 1e-30
    return o, tol


class Case:
    def __init__(self, Hq, Hkv, D, page, seqs, seed, shape="tree", holes=(), scale=0.0, spare_rows=0, max_nodes=None,
                 max_ctx=None):
        """seqs: (cached tokens, nodes) per sequence."""
        r = synth.rng_for(67, seed)
        self.cfg = gb.AttnConfig(Hq, Hkv, D, page, scale)
        self.scale = scale or 1 / math.sqrt(D)
        self.ctx = [c for c, _ in seqs]
        self.nodes = [n for _, n in seqs]
        self.table, self.n_pages, _ = paged(r, self.ctx, page, holes=holes)
        self.cu = cumulative(self.nodes)
        self.N = int(self.cu[-1]) + spare_rows
        self.trees = [make_tree(r, n, shape) for n in self.nodes]
        self.parents = np.asarray([p for t in self.trees for p in t] + [0] * spare_rows, np.int32)
        self.q, self.k, self.v = _bf16(r, (self.N, Hq, D)), _bf16(r, (self.N, Hkv, D)), _bf16(r, (self.N, Hkv, D))
        self.kp, self.vp = _bf16(r, (self.n_pages, Hkv, page, D)), _bf16(r, (self.n_pages, Hkv, page, D))
        self.max_nodes = max_nodes or max(1, max(self.nodes))
        self.max_ctx = max(self.ctx) if max_ctx is None else max_ctx
        self.dev = dict(q=dev(self.q), k=dev(self.k), v=dev(self.v), kp=dev(self.kp), vp=dev(self.vp),
                        table=i32(self.table), cu=i32(self.cu), parents=i32(self.parents), ctx=i32(self.ctx))

    def call(self, o=None, stream=None):
        d = self.dev
        if o is None:
            o = torch.full((self.N, self.cfg.n_q_heads, self.cfg.head_dim), 7.0, dtype=torch.bfloat16, device="cuda")
        nws = gb.gdn_attn_tree_workspace_size(self.cfg, len(self.ctx), self.max_nodes, self.max_ctx)
        self.ws = torch.empty(nws, dtype=torch.uint8, device="cuda") if nws else None
        gb.gdn_attn_tree(self.cfg, d["q"], d["k"], d["v"], d["kp"], d["vp"], d["table"], d["cu"], d["parents"],
                         d["ctx"], self.max_nodes, self.max_ctx, o, self.ws, stream)
        return o

    def check(self, o, skipped=(), sample=None):
        """sample: nodes checked per sequence (all by default)."""
        torch.cuda.synchronize()
        assert gb.gdn_device_status() == 0
        got, cfg = host(o), self.cfg
        q, k, v = host(self.dev["q"]), host(self.dev["k"]), host(self.dev["v"])
        kp, vp = host(self.dev["kp"]), host(self.dev["vp"])
        r = np.random.default_rng(5)
        live = np.zeros(self.N, bool)
        for b, n in enumerate(self.nodes):
            rows = slice(int(self.cu[b]), int(self.cu[b + 1]))
            if b in skipped:
                continue
            live[rows] = True
            K0, there = gather(kp, self.table[b], cfg.page_size, self.n_pages, self.ctx[b])
            V0, _ = gather(vp, self.table[b], cfg.page_size, self.n_pages, self.ctx[b])
            some = range(n) if sample is None or n <= sample else sorted({0, n - 1} | set(r.choice(n, sample - 2)))
            for i in some:
                at_ = [int(self.cu[b]) + a for a in line(self.trees[b], i)]
                ref, tol = _expect(q[rows][i], np.concatenate([K0[there], k[at_]]),
                                   np.concatenate([V0[there], v[at_]]), self.scale)
                err = np.abs(got[rows][i] - ref)
                assert (err <= tol).all(), (b, i, float((err / tol).max()))
        assert (got[~live] == 7.0).all()  # rows of no tree, and of skipped ones, are left as they were


SEQS = [(0, 1), (1, 5), (37, 8), (64, 64), (65, 33), (100, 0), (300, 17), (16, 2)]


@pytest.mark.parametrize("shape", ["tree", "chain", "star", "comb"])
def test_tree_shapes_4b(shape):
    """16 query / 4 kv heads of 256, pages of 16: contexts and trees of odd sizes, none among both."""
    c = Case(16, 4, 256, 16, SEQS, 1, shape)
    c.check(c.call())


@pytest.mark.parametrize("Hq,Hkv,D,page", [(24, 2, 256, 528), (8, 8, 128, 8), (4, 2, 128, 32), (32, 4, 128, 64),
                                           (32, 1, 128, 24), (16, 4, 256, 40), (16, 1, 256, 8), (1, 1, 128, 4096),
                                           (20, 1, 128, 16)])
def test_head_layouts_and_pages(Hq, Hkv, D, page):
    c = Case(Hq, Hkv, D, page, [(0, 3), (130, 64), (529, 21), (63, 1), (1100, 10)], 2)
    c.check(c.call(), sample=6)


def test_long_context_is_split():
    """A few sequences with long contexts: the keys of one are shared out and joined."""
    c = Case(16, 4, 256, 16, [(9000, 20), (4097, 64)], 3)
    c.check(c.call(), sample=4)
    c = Case(32, 4, 128, 64, [(20000, 5)], 4)
    c.check(c.call(), sample=5)


def test_many_sequences():
    r = np.random.default_rng(3)
    c = Case(8, 2, 128, 16, [(int(r.integers(0, 200)), int(r.integers(0, 9))) for _ in range(300)], 5)
    c.check(c.call(), sample=2)


def test_scale_and_spare_rows():
    c = Case(16, 4, 256, 16, [(50, 7), (20, 4)], 6, scale=0.21, spare_rows=9, max_nodes=64, max_ctx=5000)
    c.check(c.call())


def test_pages_outside_the_pool_are_left_out():
    c = Case(16, 4, 256, 16, [(64, 9), (200, 12), (16, 3)], 7, holes=[(0, 1), (1, 0), (1, 12), (2, 0)])
    c.check(c.call())


def test_skipped_sequences():
    """Trees above max_nodes, contexts that are negative, above max_ctx_len or past the block table."""
    c = Case(16, 4, 256, 16, [(40, 9), (30, 20), (33, 5), (48, 6), (47, 3)], 8, max_nodes=9, max_ctx=47)
    c.check(c.call(), skipped=(1, 3))
    c.dev["ctx"] = i32([40, 30, -1, 1000, 47])
    c.max_ctx = 2000
    c.check(c.call(), skipped=(1, 2, 3))
    c.dev["ctx"], c.dev["cu"] = i32(c.ctx), i32([0, 9, 29, 34, 40, 50])  # the last tree runs past the rows
    c.max_nodes = 64
    c.check(c.call(), skipped=(4,))


def test_parents_out_of_range_are_first_nodes():
    c = Case(16, 4, 256, 16, [(20, 6)], 9)
    c.trees = [[-5, 0, 7, 3, 1, 4]]
    c.dev["parents"] = i32(c.trees[0])
    c.check(c.call())


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
def test_what_a_node_does_not_see_does_not_reach_it(bad):
    """NaN and infinities in cache rows past the context, on unused pages, and in nodes off the line."""
    c = Case(16, 4, 256, 16, [(70, 20), (0, 5), (15, 64)], 10)
    ref = c.call().clone()
    for name in ("kp", "vp"):
        pool = c.dev[name]
        used = torch.zeros(c.n_pages, 16, dtype=torch.bool)
        for b, n in enumerate(c.ctx):
            for t in range(n):
                used[c.table[b][t // 16], t % 16] = True
        pool.masked_fill_(~used.cuda()[:, None, :, None], bad)
    assert torch.equal(c.call(), ref)
    # one node of each tree holds `bad`: its own line and its descendants see it, the others keep their values
    hit = [7, 2, 30]
    for b, a in enumerate(hit):
        c.dev["v"][int(c.cu[b]) + a] = bad
        c.dev["k"][int(c.cu[b]) + a, :, 0] = bad
    o = c.call()
    torch.cuda.synchronize()
    for b, n in enumerate(c.nodes):
        for i in range(n):
            row = int(c.cu[b]) + i
            if hit[b] in line(c.trees[b], i):
                assert not torch.isfinite(o[row].float()).all()
            else:
                assert torch.equal(o[row], ref[row]), (b, i)


def test_infinite_values_on_the_line_arrive():
    """An infinite value of a node reaches exactly the same dim of its descendants."""
    c = Case(16, 4, 256, 16, [(30, 12)], 11, "chain")
    ref = c.call().clone()
    c.dev["v"][5, 2, 17] = float("inf")
    o = c.call()
    torch.cuda.synchronize()
    want = ref.clone()
    want[5:, 8:12, 17] = float("inf")
    assert torch.equal(o, want)


def test_captured_calls_with_their_own_workspaces():
    """Two calls captured into one graph each, replayed on two streams, give the eager results."""
    cases = [Case(16, 4, 256, 16, [(3000, 12), (100, 3)], 12), Case(16, 4, 256, 16, [(2500, 64)], 13)]
    want = [c.call().clone() for c in cases]
    graphs, outs, keep = [], [], []
    for c in cases:
        o = torch.zeros_like(want[len(outs)])
        c.call(o)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            c.call(o)
        keep.append(c.ws)
        graphs.append(g)
        outs.append(o)
    for o in outs:
        o.fill_(7.0)
    torch.cuda.synchronize()
    for _ in range(3):
        for g, s in zip(graphs, (torch.cuda.Stream(), torch.cuda.Stream())):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(o, w) for o, w in zip(outs, want))


def test_same_call_twice_is_bitwise_equal():
    c = Case(24, 2, 256, 528, [(6000, 40), (700, 64)], 14)
    assert torch.equal(c.call(), c.call())
