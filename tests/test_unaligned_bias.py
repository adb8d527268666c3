"""A conv bias that starts at an odd element of a flat buffer of parameters: 2-byte alignment (4 in fp32) is all that
a bias needs.  The results are those of a copy that is aligned, bit for bit."""
import pytest
import torch

import oracle
import test_tree_gdn
import test_tree_more
from hybrid_gated_deltanet_gb300 import binding as gb
from hybrid_gated_deltanet_gb300 import synth
from gdn_cases import config, dev, host, oracle_kwargs, params_dev, rel_fro, tol_for

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


@pytest.mark.parametrize("skip", [1, 2, 3])
@pytest.mark.parametrize("act", [synth.BF16, synth.F32])
@pytest.mark.parametrize("geom", [synth.Geometry(2, 4, 128, 128, 4), synth.Geometry(2, 6, 64, 64, 3)])
def test_prefill_and_decode(geom, act, skip):
    """150 tokens through the chunked prefill and one decode step after them."""
    T = 150
    r = synth.rng_for(73, skip)
    p, tok = synth.make_params(geom, r, act), synth.make_tokens(geom, T + 1, r, act)
    cfg, prm = config(geom, act), params_dev(p)
    prm.conv_b = dev(synth.store(0.3 * r.standard_normal(geom.conv_channels), act))
    x, z, a, b = (dev(tok[k]) for k in ("x", "z", "a", "b"))
    slots, got = torch.zeros(1, dtype=torch.int32, device="cuda"), []
    for q in (prm, shifted(prm, skip)):
        S = torch.empty((1, geom.n_v_heads, geom.d_v, geom.d_k), device="cuda")
        CS = torch.empty((1, geom.d_conv - 1, geom.conv_channels), dtype=cfg.torch_dtype, device="cuda")
        y = torch.empty((T + 1, geom.value_dim), dtype=cfg.torch_dtype, device="cuda")
        ws = torch.empty(gb.gdn_workspace_size(cfg, gb.OP_CHUNK_PREFILL, T), dtype=torch.uint8, device="cuda")
        gb.gdn_chunk_prefill(cfg, q, x[:T], z[:T], a[:T], b[:T], None, None, S[0], CS[0], y[:T], ws)
        gb.gdn_decode_step(cfg, q, x[T:], z[T:], a[T:], b[T:], CS, S, slots, y[T:])
        got.append((y, S, CS))
    torch.cuda.synchronize()
    want = oracle.run_sequence(geom, *(tok[k].f64 for k in ("x", "z", "a", "b")), conv_b=host(prm.conv_b),
                               **oracle_kwargs(p))
    assert rel_fro(host(got[0][0]), want["y"]) <= tol_for(act)["y"] and rel_fro(host(got[0][1])[0], want["S"]) <= tol_for(act)["S"]
    assert all(torch.equal(u, v) for u, v in zip(*got))
