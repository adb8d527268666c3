"""gdn_page_tables and gdn_attn_append on the GPU against plain loops over the definitions (whole
numbers and copies: equal)."""
import numpy as np
import pytest
import torch

from hybrid_gated_deltanet_gb300 import binding as gb
from tree_cases import cumulative, i32

pytestmark = pytest.mark.gpu


def expect(page, n_pages, ctx, new, free, head, table, n_rows, path=None, cu_nodes=None):
    table, cu, slots, src = table.copy(), [0], [], []
    room, pages, rows, at = max(0, len(free) - head) if head >= 0 else 0, 0, 0, 0
    for b in range(len(ctx)):
        c, n = int(ctx[b]), int(new[b])
        fits = c >= 0 and n >= 0 and c + n <= table.shape[1] * page and (path is None or n <= path.shape[1])
        have = -(-c // page)
        need = -(-(c + n) // page) - have if fits else 0
        pages, rows = pages + need, rows + (n if fits else 0)
        granted = fits and n > 0 and (need == 0 or pages <= room) and rows <= n_rows
        if granted:
            table[b, have:have + need] = free[head + at:head + at + need]
            at += need
            for t in range(c, c + n):
                p = int(table[b, t // page])
                slots.append(p * page + t % page if 0 <= p < n_pages else -1)
                if path is not None:
                    i = int(path[b, t - c])
                    src.append(int(cu_nodes[b]) + i if 0 <= i < cu_nodes[b + 1] - cu_nodes[b] else -1)
        cu.append(cu[-1] + (n if granted else 0))
    pad = [-1] * (n_rows - len(slots))
    return table, np.asarray(cu), np.asarray(slots + pad), head + at, np.asarray(src + pad)


def run(page, n_pages, ctx, new, free, head, table, n_rows, path=None, cu_nodes=None):
    B = len(ctx)
    t = i32(table)
    cu, slots = i32([9] * (B + 1)), torch.full((n_rows,), 9, dtype=torch.int64, device="cuda")
    out = i32([9])
    src = i32([9] * n_rows) if path is not None else None
    gb.gdn_page_tables(page, n_pages, i32(ctx), i32(new), i32(free), i32([head]), t, cu, slots, out,
                       None if path is None else i32(path), None if path is None else i32(cu_nodes), src)
    want = expect(page, n_pages, ctx, new, free, head, table, n_rows, path, cu_nodes)
    torch.cuda.synchronize()
    np.testing.assert_array_equal(t.cpu().numpy(), want[0])
    np.testing.assert_array_equal(cu.cpu().numpy(), want[1])
    np.testing.assert_array_equal(slots.cpu().numpy(), want[2])
    assert int(out[0]) == want[3]
    if path is not None:
        np.testing.assert_array_equal(src.cpu().numpy(), want[4])
    return want


def case(seed, B, ctx_max, new_max, page, spare=5, paths=False):
    r = np.random.default_rng(seed)
    ctx, new = r.integers(0, ctx_max + 1, B), r.integers(0, new_max + 1, B)
    have, want = -(-ctx // page), -(-(ctx + new) // page)
    n_pages = int(want.sum()) + spare
    perm = r.permutation(n_pages)
    table = np.full((B, int(want.max()) + 1), -1, np.int64)
    at = 0
    for b in range(B):
        table[b, :have[b]] = perm[at:at + have[b]]
        at += have[b]
    path = cu = None
    if paths:
        nodes = 2 * new + 1
        cu = cumulative(nodes)
        path = np.full((B, max(1, int(new.max()))), -1, np.int64)
        for b in range(B):
            path[b, :new[b]] = np.sort(r.permutation(nodes[b])[:new[b]])
    return n_pages, ctx, new, perm[at:], table, path, cu


@pytest.mark.parametrize("page", [1, 7, 16, 528])
@pytest.mark.parametrize("B", [1, 3, 64, 1024, 1025, 3000])
def test_page_tables_sizes(page, B):
    n_pages, ctx, new, free, table, _, _ = case(B, B, 100, 40, page)
    run(page, n_pages, ctx, new, free, 0, table, int(new.sum()) + 3)


def test_page_tables_paths():
    n_pages, ctx, new, free, table, path, cu = case(5, 77, 900, 9, 16, paths=True)
    run(16, n_pages, ctx, new, free, 0, table, int(new.sum()), path, cu)
    path[3, 0], path[5, :] = 10 ** 6, -4  # nodes outside their trees
    run(16, n_pages, ctx, new, free, 0, table, int(new.sum()) + 40, path, cu)


def test_page_tables_long_prompts():
    n_pages, ctx, new, free, table, _, _ = case(6, 20, 0, 30000, 16)
    run(16, n_pages, ctx, new, free, 0, table, int(new.sum()))


def test_page_tables_list_runs_out():
    n_pages, ctx, new, free, table, _, _ = case(7, 50, 60, 30, 8)
    for room in (0, 1, 17, 60):
        want = run(8, n_pages, ctx, new, free[:room], 0, table, int(new.sum()))
        assert want[3] <= room
    run(8, n_pages, ctx, new, free, len(free) - 4, table, int(new.sum()))
    run(8, n_pages, ctx, new, free, len(free) + 4, table, int(new.sum()))  # a head past the list: nothing left
    run(8, n_pages, ctx, new, free, -3, table, int(new.sum()))
    run(8, n_pages, ctx, new, np.zeros(0, np.int64), 0, table, int(new.sum()))


def test_page_tables_rows_run_out_and_bad_lengths():
    n_pages, ctx, new, free, table, _, _ = case(8, 40, 60, 30, 16)
    for n_rows in (0, 1, 100):
        run(16, n_pages, ctx, new, free, 0, table, n_rows)
    ctx, new = ctx.copy(), new.copy()
    ctx[3], new[5], ctx[9], new[11] = -1, -2, 2 ** 31 - 1, 2 ** 31 - 1
    run(16, n_pages, ctx, new, free, 0, table, 2000)


def test_page_tables_nothing_to_do():
    n_pages, ctx, new, free, table, _, _ = case(9, 5, 60, 0, 16)
    run(16, n_pages, ctx, new, free, 2, table, 4)
    run(16, 3, np.zeros(0, int), np.zeros(0, int), np.zeros(0, int), 0, np.zeros((0, 4), int), 2)


def test_page_tables_pages_outside_the_pool():
    n_pages, ctx, new, free, table, _, _ = case(10, 12, 60, 30, 16)
    free = free.copy()
    free[1], free[2] = n_pages, -5
    table[0, :] = np.where(table[0] >= 0, n_pages + 1, table[0])
    run(16, n_pages, ctx, new, free, 0, table, int(new.sum()))


@pytest.mark.parametrize("Hkv,D,page", [(4, 256, 16), (2, 256, 528), (8, 128, 8), (1, 128, 24), (3, 128, 64)])
@pytest.mark.parametrize("n,gathered", [(1, False), (1, True), (37, True), (700, False), (5000, True)])
def test_append(Hkv, D, page, n, gathered):
    g = torch.Generator().manual_seed(n)
    n_pages = n // page + 3
    src = 2 * n + 3 if gathered else n
    k, v = (torch.randn(src, Hkv, D, generator=g).bfloat16().cuda() for _ in range(2))
    pools = [torch.randn(n_pages, Hkv, page, D, generator=g).bfloat16().cuda() for _ in range(2)]
    slots = torch.randperm(n_pages * page, generator=g)[:n]
    rows = torch.randint(0, src, (n,), generator=g) if gathered else torch.arange(n)
    if n > 10:
        slots[3], slots[5], slots[6] = -1, n_pages * page, 2 ** 40
        if gathered:
            rows[8], rows[9] = -1, src
    want = [p.clone() for p in pools]
    ok = (slots >= 0) & (slots < n_pages * page) & (rows >= 0) & (rows < src)
    s, r = slots[ok].cuda(), rows[ok].cuda()
    for w, new in zip(want, (k, v)):
        w[s // page, :, s % page] = new[r]
    cfg = gb.AttnConfig(Hkv, Hkv, D, page)
    gb.gdn_attn_append(cfg, k, v, slots.cuda(), *pools, rows.int().cuda() if gathered else None)
    torch.cuda.synchronize()
    assert all(torch.equal(p, w) for p, w in zip(pools, want))


def test_append_offsets_past_32_bits():
    """A pool of more than 2^32 bytes and 2^31 elements: rows at its far end."""
    Hkv, D, page, n_pages = 4, 256, 64, 34000
    pool = torch.zeros(n_pages, Hkv, page, D, dtype=torch.bfloat16, device="cuda")
    assert pool.numel() > 1 << 31
    k = torch.randn(3, Hkv, D, device="cuda").bfloat16()
    slots = torch.tensor([n_pages * page - 1, n_pages * page - page, 5], device="cuda")
    other = torch.zeros_like(pool)
    gb.gdn_attn_append(gb.AttnConfig(Hkv, Hkv, D, page), k, -k, slots, pool, other)
    torch.cuda.synchronize()
    assert torch.equal(pool[-1, :, -1], k[0]) and torch.equal(pool[-1, :, 0], k[1]) and torch.equal(pool[0, :, 5], k[2])
    assert torch.equal(other[-1, :, -1], -k[0]) and int((pool != 0).any(-1).sum()) == 3 * Hkv
