"""More of the operators over trees of drafted tokens: CTAs that take several v-heads, biases, infinities and
NaN in large trees, more lists than SMs, pools past 4 GB, empty calls and two streams at once.  The
tolerances are those of test_tree_gdn.py and test_tree_attn.py; what is only moved must be equal."""
import numpy as np
import pytest
import torch

import oracle
import test_tree_attn
import test_tree_gdn
from hybrid_gated_deltanet_gb300 import binding as gb
from hybrid_gated_deltanet_gb300 import synth
from gdn_cases import dev, host, oracle_kwargs, rel_fro, sample_heads
from tree_cases import i32, line

pytestmark = pytest.mark.gpu

SIZES = [64, 33, 1, 16, 48, 17, 32, 2]


@pytest.mark.parametrize("geom", [synth.Geometry(4, 12, 128, 128, 4), synth.Geometry(2, 16, 128, 128, 3),
                                  synth.Geometry(8, 8, 128, 128, 4)])
def test_verify_tree_all_v_heads_in_a_cta(geom):
    """Enough trees for a CTA per k-head: 3 and 8 v-heads in it, taken in pairs, and one."""
    B = -(-160 // geom.n_k_heads)
    c = test_tree_gdn.Case((SIZES + [3] * B)[:max(B, len(SIZES))], geom, synth.BF16, 31)
    c.check(c.verify(), heads=sample_heads(geom.n_v_heads, 3), sample=3)


@pytest.mark.parametrize("G", [1, 2, 3])
def test_verify_tree_many_small_trees(G):
    """More CTAs than two for each SM, trees of up to 16 nodes: a third one on an SM."""
    r = np.random.default_rng(9)
    c = test_tree_gdn.Case([int(v) for v in r.integers(0, 17, 170)], synth.Geometry(2, 2 * G, 128, 128, 4), synth.BF16, 43)
    c.check(c.verify(), heads=[0, 2 * G - 1], sample=2)


def unreached(c, b, bad):
    return [i for i in range(c.nodes[b]) if bad not in line(c.trees[b], i)]


def check_rows(c, y, b, nodes, heads):
    """The nodes' outputs of these v-heads against the oracle."""
    cols = np.concatenate([np.arange(h * 128, (h + 1) * 128) for h in heads])
    for i in nodes:
        ref = c.run_oracle(b, [int(c.cu[b]) + a for a in line(c.trees[b], i)], heads)["y"][-1][cols]
        assert rel_fro(y[c.cu[b] + i][cols], ref) <= test_tree_gdn.TOL_Y[c.act], i


@pytest.mark.parametrize("nodes", [20, 50])
@pytest.mark.parametrize("many", [False, True])
def test_verify_tree_nan_and_infinities_stay_on_their_lines(nodes, many):
    """A NaN row reaches its descendants alone; an infinity in one channel of v only their v-head."""
    geom = synth.Geometry(4, 12, 128, 128, 4)
    c = test_tree_gdn.Case([nodes, 5] + [2] * (40 if many else 0), geom, synth.BF16, 32)
    bad, x = 3, c.dev["x"].clone()
    free = unreached(c, 0, bad)
    assert 2 < len(free) < nodes - 1
    c.dev["x"][int(c.cu[0]) + bad] = float("nan")
    y = host(c.verify())
    check_rows(c, y, 0, free[-4:], [0, 4, 11])
    check_rows(c, y, 1, range(5), [0, 4, 11])
    down = [i for i in range(nodes) if i not in free]
    assert all(np.isnan(y[c.cu[0] + i]).any() for i in down)
    c.dev["x"] = x
    c.dev["x"][int(c.cu[0]) + bad, 2 * 4 * 128 + 5 * 128 + 9] = float("inf")  # v-head 5, its channel 9
    y = host(c.verify())
    check_rows(c, y, 0, free[-4:], [4, 5, 11])
    check_rows(c, y, 0, down[-4:], [4, 11])
    check_rows(c, y, 1, range(5), [4, 5, 11])
    assert all(not np.isfinite(y[c.cu[0] + i][5 * 128 + 9]) for i in down)


class Biased(test_tree_gdn.Case):
    def __init__(self, *args, **kw):
        super().__init__(*args, **kw)
        r = np.random.default_rng(7)
        self.bias = dict(conv_b=synth.store(0.3 * r.standard_normal(self.geom.conv_channels), self.act),
                         dt_bias=synth.store(r.standard_normal(self.geom.n_v_heads), synth.F32))
        p = self.dev["prm"]
        self.dev["prm"] = gb.Params(p.conv_w, p.A_log, p.norm_w, **{k: dev(v) for k, v in self.bias.items()})

    def run_oracle(self, b, rows, heads):
        at = np.asarray(rows)
        return oracle.run_sequence(self.geom, *(self.tok[k].f64[at] for k in ("x", "z", "a", "b")),
                                   s0=self.S.f64[self.slots[b]], conv0=self.CS.f64[self.slots[b]], heads=heads,
                                   q_scale=self.cfg.q_scale, **oracle_kwargs(self.p),
                                   **{k: v.f64 for k, v in self.bias.items()})


@pytest.mark.parametrize("act", [synth.BF16, synth.F32])
@pytest.mark.parametrize("geom", [synth.Geometry(2, 4, 128, 128, 4), synth.Geometry(2, 6, 64, 64, 3)])
def test_biases(geom, act):
    c = Biased([9, 40, 1], geom, act, 33)
    c.check(c.verify(), sample=6)
    paths = [[0, 2, 5], list(range(20)), [0]]
    test_tree_gdn.commit(c, paths)
    test_tree_gdn.check_commit(c, paths)


@pytest.mark.parametrize("D,page", [(128, 64), (256, 16)])
def test_attention_of_more_lists_than_sms(D, page):
    """Lists laid end to end and cut wherever a worker's share ends."""
    r = np.random.default_rng(8)
    seqs = [(int(r.integers(0, 3000)), int(r.integers(0, 20))) for _ in range(50)]
    c = test_tree_attn.Case(16, 4, D, page, seqs, 34)
    c.check(c.call(), sample=2)


def test_attention_of_many_sequences_in_pieces():
    """More than 32 sequences, fewer lists than SMs: pieces of equal length, some sequences skipped or short."""
    r = np.random.default_rng(10)
    seqs = [(int(r.integers(0, 1500)) if i % 5 else int(r.integers(0, 40)), int(r.integers(0, 20))) for i in range(70)]
    c = test_tree_attn.Case(8, 2, 128, 16, seqs, 44)
    c.check(c.call(), sample=2)
    c = test_tree_attn.Case(4, 1, 256, 32, seqs[:40], 45)
    c.check(c.call(), sample=2)


def past_4gb(small, rows):
    """The rows of `small` as the last ones of a tensor of more than 4 GB, and the first one's place."""
    n = (1 << 32) // (small[0].numel() * small.element_size()) + rows + 3
    big = torch.empty((n, *small.shape[1:]), dtype=small.dtype, device="cuda")
    big[n - rows:] = small
    return big, n - rows


def test_caches_past_4_gb():
    c = test_tree_attn.Case(16, 4, 256, 16, [(700, 9), (40, 3)], 35)
    want = c.call().clone()
    c.dev["kp"], at = past_4gb(c.dev["kp"], c.n_pages)
    c.dev["vp"], _ = past_4gb(c.dev["vp"], c.n_pages)
    c.dev["table"] = torch.where(c.dev["table"] >= 0, c.dev["table"] + at, c.dev["table"])
    assert torch.equal(c.call(), want)
    rows = torch.tensor([(at + 1) * 16 + 5, at * 16, 17], dtype=torch.int64, device="cuda")
    k, v = c.dev["k"][:3].contiguous(), c.dev["v"][:3].contiguous()
    gb.gdn_attn_append(c.cfg, k, v, rows, c.dev["kp"], c.dev["vp"])
    for i, row in enumerate(rows.tolist()):
        assert torch.equal(c.dev["kp"][row // 16, :, row % 16], k[i])
        assert torch.equal(c.dev["vp"][row // 16, :, row % 16], v[i])


@pytest.mark.parametrize("act", [synth.BF16, synth.F32])
def test_states_past_4_gb(act):
    c = test_tree_gdn.Case([9, 30], synth.QWEN35_4B, act, 36)
    paths = [[0, 1], [0, 4, 9]]
    want = c.verify().clone()
    slots = c.dev["slots"].clone()
    S, at = past_4gb(c.dev["S"], c.n_slots)
    CS = torch.empty((S.shape[0], *c.dev["CS"].shape[1:]), dtype=c.dev["CS"].dtype, device="cuda")
    CS[at:] = c.dev["CS"]
    small = c.dev["S"], c.dev["CS"]
    test_tree_gdn.commit(c, paths)
    c.dev["S"], c.dev["CS"], c.dev["slots"] = S, CS, slots + at
    assert torch.equal(c.verify(), want)
    test_tree_gdn.commit(c, paths)
    assert torch.equal(S[at:], small[0]) and torch.equal(CS[at:], small[1])


def test_calls_without_nodes():
    """No node at all: nothing is written, nothing fails."""
    c = test_tree_gdn.Case([0, 0], test_tree_gdn.SMALL, synth.BF16, 37, spare_rows=2)
    c.check(c.verify())
    S = c.dev["S"].clone()
    test_tree_gdn.commit(c, [[], []], max_rows=4)
    assert torch.equal(S, c.dev["S"])
    for spare in (0, 2):
        a = test_tree_attn.Case(16, 4, 256, 16, [(20, 0), (0, 0)], 38, spare_rows=spare)
        a.check(a.call())
    gb.gdn_attn_append(a.cfg, a.dev["k"], a.dev["v"], torch.empty(0, dtype=torch.int64, device="cuda"), a.dev["kp"],
                       a.dev["vp"])
    torch.cuda.synchronize()
    assert gb.gdn_device_status() == 0


def test_two_streams_at_once():
    """Calls of all kinds on two streams, each with its own data: the results of one at a time."""
    g = [test_tree_gdn.Case([12, 40, 3, 64], synth.QWEN35_4B, synth.BF16, 39 + i) for i in range(2)]
    a = [test_tree_attn.Case(16, 4, 256, 16, [(1500, 12), (200, 30), (3000, 5)], 41 + i) for i in range(2)]
    want = [(x.verify().clone(), y.call().clone()) for x, y in zip(g, a)]
    paths = [[0, 1], [0, 4, 9], [2], list(range(20))]
    alone = []
    for x in g:
        S, CS = x.dev["S"].clone(), x.dev["CS"].clone()
        test_tree_gdn.commit(x, paths)
        alone.append((x.dev["S"], x.dev["CS"]))
        x.dev["S"], x.dev["CS"] = S, CS
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream() for _ in range(2)], [[], []]
    for _ in range(8):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append((g[i].verify(), a[i].call()))
    for i, s in enumerate(streams):
        with torch.cuda.stream(s):
            test_tree_gdn.commit(g[i], paths)
    torch.cuda.synchronize()
    assert gb.gdn_device_status() == 0
    for i in range(2):
        assert all(torch.equal(y, want[i][0]) and torch.equal(o, want[i][1]) for y, o in got[i])
        assert torch.equal(g[i].dev["S"], alone[i][0]) and torch.equal(g[i].dev["CS"], alone[i][1])
