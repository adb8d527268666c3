"""Refusals of the tree and page-table calls, on the host without a GPU: status and message at the C
boundary, and the binding's checks of dtypes, shapes and devices.  No call here reaches a launch."""
import ctypes

import pytest
import torch

from hybrid_gated_deltanet_gb300 import binding as gb
from hybrid_gated_deltanet_gb300 import build as gbuild

FAKE = 0x100000  # an aligned address that is never dereferenced on the host


@pytest.fixture(scope="module")
def lib():
    gbuild.build()
    return gb.load()


def _err(lib):
    return lib.gdn_last_error().decode()


def _refused(lib, status, got, needle):
    assert got == status and needle in _err(lib), (got, _err(lib))


def _attn(lib, cfg=None, **kw):
    a = dict(q=FAKE, k_new=FAKE, v_new=FAKE, k_pool=FAKE, v_pool=FAKE, block_table=FAKE, cu_nodes=FAKE, parents=FAKE,
             ctx_lens=FAKE, B=2, n_nodes=9, max_nodes=8, max_pages=4, n_pages=8, max_ctx=60, o=FAKE, ws=FAKE,
             nws=1 << 40)
    a.update(kw)
    c = (cfg or gb.AttnConfig(16, 4, 256, 16)).c()
    return lib.gdn_attn_tree(ctypes.byref(c), *a.values(), None)


def test_attn_tree_refusals(lib):
    _refused(lib, -2, _attn(lib, gb.AttnConfig(16, 4, 64, 16)), "cfg.head_dim: found 64")
    _refused(lib, -7, _attn(lib, gb.AttnConfig(12, 4, 128, 16)), "G = n_q_heads / n_kv_heads = 3")
    _refused(lib, -5, _attn(lib, B=-1), "B: found -1")
    _refused(lib, -5, _attn(lib, n_nodes=-1), "n_nodes: found -1")
    _refused(lib, -5, _attn(lib, max_nodes=65), "max_nodes: found 65, required 1..64")
    _refused(lib, -5, _attn(lib, max_nodes=0), "max_nodes: found 0")
    _refused(lib, -5, _attn(lib, max_pages=0), "max_pages/n_pages/max_ctx_len: found 0/8/60")
    _refused(lib, -5, _attn(lib, max_ctx=-1), "found 4/8/-1")
    for name in ("q", "k_new", "v_new", "k_pool", "v_pool", "block_table", "cu_nodes", "parents", "ctx_lens", "o"):
        _refused(lib, -1, _attn(lib, **{name: None}), f"{name}: found NULL")
    _refused(lib, -4, _attn(lib, q=FAKE + 8), "q: found address")
    _refused(lib, -4, _attn(lib, parents=FAKE + 2), "parents: found address")
    assert _attn(lib, B=0) == 0 and _attn(lib, n_nodes=0) == 0 and _err(lib) == ""
    c = gb.AttnConfig(16, 4, 256, 16).c()
    need = lib.gdn_attn_tree_workspace_size(ctypes.byref(c), 4, 64, 32768)
    if need:
        _refused(lib, -6, _attn(lib, B=4, max_nodes=64, max_ctx=32768, nws=need - 1), f"required {need} bytes")
        _refused(lib, -1, _attn(lib, B=4, max_nodes=64, max_ctx=32768, ws=None), "workspace: found NULL")
    assert lib.gdn_attn_tree_workspace_size(ctypes.byref(c), 4, 65, 100) == 0 and "max_nodes" in _err(lib)
    assert lib.gdn_attn_tree_workspace_size(ctypes.byref(c), -1, 4, 100) == 0 and "B/max_ctx_len" in _err(lib)


def _cfg(**kw):
    c = gb.Config(16, 32, 128, 128, 4, 64, gb.BF16)
    for k, v in kw.items():
        setattr(c, k, v)
    return c.c()


def _prm(**kw):
    p = dict(conv_w=FAKE, conv_b=None, A_log=FAKE, dt_bias=None, norm_w=FAKE)
    p.update(kw)
    return gb.CParams(*p.values())


def _verify(lib, cfg=None, prm=None, **kw):
    a = dict(x=FAKE, z=FAKE, a=FAKE, b=FAKE, conv_pool=FAKE, state_pool=FAKE, slot_idx=FAKE, cu_nodes=FAKE,
             parents=FAKE, B=2, n_nodes=9, max_nodes=8, n_slots=4, y=FAKE)
    a.update(kw)
    c, p = cfg or _cfg(), prm or _prm()
    return lib.gdn_verify_tree(ctypes.byref(c), ctypes.byref(p), *a.values(), None)


def test_verify_tree_refusals(lib):
    _refused(lib, -3, _verify(lib, _cfg(act_dtype=4)), "cfg.act_dtype: found 4")
    _refused(lib, -2, _verify(lib, _cfg(d_k=48, d_v=48)), "cfg.d_k: found 48")
    _refused(lib, -5, _verify(lib, B=70000), "B: found 70000")
    _refused(lib, -5, _verify(lib, n_nodes=-4), "n_nodes: found -4")
    _refused(lib, -5, _verify(lib, max_nodes=100), "max_nodes: found 100")
    _refused(lib, -5, _verify(lib, n_slots=0), "n_slots: found 0")
    _refused(lib, -1, _verify(lib, prm=_prm(A_log=None)), "prm.A_log")
    for name in ("x", "z", "a", "b", "conv_pool", "state_pool", "slot_idx", "cu_nodes", "parents", "y"):
        _refused(lib, -1, _verify(lib, **{name: None}), f"{name}: found NULL")
    _refused(lib, -4, _verify(lib, y=FAKE + 2), "y: found address")
    _refused(lib, -4, _verify(lib, a=FAKE + 1), "a: found address")
    assert _verify(lib, B=0) == 0 and _verify(lib, n_nodes=0) == 0


def _commit(lib, cfg=None, **kw):
    a = dict(x=FAKE, a=FAKE, b=FAKE, conv_pool=FAKE, state_pool=FAKE, slot_idx=FAKE, cu_rows=FAKE, src_rows=FAKE, B=2,
             n_rows=5, n_src=9, max_rows=8, n_slots=4)
    a.update(kw)
    c, p = cfg or _cfg(), _prm()
    return lib.gdn_commit_tree(ctypes.byref(c), ctypes.byref(p), *a.values(), None)


def test_commit_tree_refusals(lib):
    _refused(lib, -5, _commit(lib, n_rows=-1), "n_rows/n_src: found -1/9")
    _refused(lib, -5, _commit(lib, n_src=-1), "n_rows/n_src: found 5/-1")
    _refused(lib, -5, _commit(lib, max_rows=65), "max_rows: found 65, required 1..64")
    _refused(lib, -5, _commit(lib, B=-1), "B: found -1")
    _refused(lib, -5, _commit(lib, n_slots=0), "n_slots: found 0")
    for name in ("x", "a", "b", "conv_pool", "state_pool", "slot_idx", "cu_rows"):
        _refused(lib, -1, _commit(lib, **{name: None}), f"{name}: found NULL")
    _refused(lib, -4, _commit(lib, src_rows=FAKE + 2), "src_rows: found address")
    _refused(lib, -4, _commit(lib, state_pool=FAKE + 8), "state_pool: found address")
    assert _commit(lib, B=0) == 0 and _commit(lib, n_rows=0) == 0 and _commit(lib, n_src=0) == 0


def _tables(lib, **kw):
    a = dict(page=16, n_pages=8, ctx=FAKE, new=FAKE, B=2, free=FAKE, n_free=4, head=FAKE, table=FAKE, max_pages=4,
             cu=FAKE, slot_map=FAKE, n_rows=5, head_out=FAKE + 16, path=FAKE, path_len=3, cu_nodes=FAKE, src=FAKE)
    a.update(kw)
    return lib.gdn_page_tables(*a.values(), None)


def test_page_tables_refusals(lib):
    _refused(lib, -5, _tables(lib, page=0), "page_size/n_pages: found 0/8")
    _refused(lib, -5, _tables(lib, page=1 << 30, n_pages=1 << 30), "at most 2^40 rows")
    _refused(lib, -5, _tables(lib, B=-1), "B: found -1")
    _refused(lib, -5, _tables(lib, n_free=-1), "n_free/max_pages/n_rows: found -1/4/5")
    _refused(lib, -5, _tables(lib, n_rows=-1), "found 4/4/-1")
    _refused(lib, -5, _tables(lib, head_out=FAKE), "head_out: found the address of head")
    _refused(lib, -1, _tables(lib, path=None), "required all three or none")
    _refused(lib, -1, _tables(lib, src=None), "required all three or none")
    _refused(lib, -5, _tables(lib, path_len=0), "path_len: found 0")
    for name, said in (("ctx", "ctx_lens"), ("new", "new_lens"), ("free", "free_pages"), ("head", "head"),
                       ("table", "block_table"), ("cu", "cu_rows"), ("slot_map", "slot_map"), ("head_out", "head_out")):
        _refused(lib, -1, _tables(lib, **{name: None}), f"{said}: found NULL")
    _refused(lib, -4, _tables(lib, slot_map=FAKE + 4), "slot_map: found address")


def _append(lib, cfg=None, **kw):
    a = dict(k=FAKE, v=FAKE, n_src=9, slot_map=FAKE, src=FAKE, n_rows=5, kp=FAKE, vp=FAKE, n_pages=8)
    a.update(kw)
    c = (cfg or gb.AttnConfig(16, 4, 256, 16)).c()
    return lib.gdn_attn_append(ctypes.byref(c), *a.values(), None)


def test_append_refusals(lib):
    _refused(lib, -2, _append(lib, gb.AttnConfig(4, 4, 256, 12)), "cfg.page_size: found 12")
    _refused(lib, -5, _append(lib, n_rows=-1), "n_rows/n_src: found -1/9")
    _refused(lib, -5, _append(lib, n_src=1 << 31), "n_rows/n_src")
    _refused(lib, -5, _append(lib, n_pages=0), "n_pages: found 0")
    for name, said in (("k", "k_new"), ("v", "v_new"), ("slot_map", "slot_map"), ("kp", "k_pool"), ("vp", "v_pool")):
        _refused(lib, -1, _append(lib, **{name: None}), f"{said}: found NULL")
    _refused(lib, -4, _append(lib, kp=FAKE + 2), "k_pool: found address")
    assert _append(lib, n_rows=0) == 0 and _append(lib, n_src=0) == 0


def test_binding_refuses_host_tensors():
    """Tensors that are not on a CUDA device never reach the library."""
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    bf = lambda *s: torch.zeros(s, dtype=torch.bfloat16)  # noqa: E731
    cfg = gb.AttnConfig(4, 2, 128, 16)
    with pytest.raises(ValueError, match="required one CUDA device"):
        gb.gdn_attn_tree(cfg, bf(3, 4, 128), bf(3, 2, 128), bf(3, 2, 128), bf(2, 2, 16, 128), bf(2, 2, 16, 128),
                         i32(1, 2), i32(2), i32(3), i32(1), 3, 20, bf(3, 4, 128))
    with pytest.raises(ValueError, match="block_table: found"):
        gb.gdn_attn_tree(cfg, bf(3, 4, 128), bf(3, 2, 128), bf(3, 2, 128), bf(2, 2, 16, 128), bf(2, 2, 16, 128),
                         i32(2), i32(2), i32(3), i32(1), 3, 20, bf(3, 4, 128))
    with pytest.raises(ValueError, match="required one CUDA device"):
        gb.gdn_attn_append(cfg, bf(3, 2, 128), bf(3, 2, 128), torch.zeros(3, dtype=torch.int64), bf(2, 2, 16, 128),
                           bf(2, 2, 16, 128))
    with pytest.raises(ValueError, match="required one CUDA device"):
        gb.gdn_page_tables(16, 4, i32(2), i32(2), i32(4), i32(1), i32(2, 4), i32(3), torch.zeros(5, dtype=torch.int64),
                           i32(1))
    c = gb.Config(2, 4, 32, 32)
    prm = gb.Params(conv_w=bf(256, 4), A_log=torch.zeros(4), norm_w=bf(32))
    with pytest.raises(ValueError, match="required one CUDA device"):
        gb.gdn_verify_tree(c, prm, bf(3, 256), bf(3, 128), bf(3, 4), bf(3, 4), bf(2, 3, 256), torch.zeros(2, 4, 32, 32),
                           i32(1), i32(2), i32(3), 3, bf(3, 128))
    with pytest.raises(ValueError, match="required one CUDA device"):
        gb.gdn_commit_tree(c, prm, bf(3, 256), bf(3, 4), bf(3, 4), bf(2, 3, 256), torch.zeros(2, 4, 32, 32), i32(1),
                           i32(2), None, 3)
