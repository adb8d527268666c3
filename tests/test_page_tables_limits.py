"""gdn_page_tables at the ends of its ranges."""
import pytest
import torch

from hybrid_gated_deltanet_gb300 import binding as gb
from tree_cases import i32

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("new", [3, 2 ** 31 - 40000, 2 ** 31 - 1])
def test_as_many_rows_as_a_count_holds(new):
    """2^31 - 1 rows of the map, few or all of them one sequence's, with rows before the map that stay as they were."""
    n_rows, page, pad = 2 ** 31 - 1, 1 << 20, 100000
    pages = -(-new // page)
    buf = torch.full((n_rows + pad,), 7, dtype=torch.int64, device="cuda")
    slots, ids = buf[pad:], torch.randperm(pages, device="cuda").int()
    cu, out, table = i32([9, 9]), i32([9]), torch.full((1, 2048), -1, dtype=torch.int32, device="cuda")
    gb.gdn_page_tables(page, pages, i32([0]), i32([new]), ids, i32([0]), table, cu, slots, out)
    torch.cuda.synchronize()
    assert cu.tolist() == [0, new] and int(out) == pages
    assert torch.equal(table[0, :pages], ids) and bool((table[0, pages:] == -1).all())
    assert bool((buf[:pad] == 7).all()) and bool((slots[new:] == -1).all())
    for at in range(0, new, 1 << 28):  # (in parts: a comparison takes as much memory again)
        pos = torch.arange(at, min(new, at + (1 << 28)), device="cuda")
        assert torch.equal(slots[at:at + len(pos)], ids.long()[pos // page] * page + pos % page), at


def test_as_many_pages_as_a_count_holds():
    """The same of pages: one sequence takes 2^31 - 1 of a list of as many, a row each."""
    n, pad = 2 ** 31 - 1, 100000
    ids = torch.zeros(n, dtype=torch.int32, device="cuda")
    ids[::1000] = 5
    buf = torch.full((n + pad,), 7, dtype=torch.int32, device="cuda")
    table, slots = buf[pad:].view(1, n), torch.full((n,), 9, dtype=torch.int64, device="cuda")
    cu, out = i32([9, 9]), i32([9])
    gb.gdn_page_tables(1, 8, i32([0]), i32([n]), ids, i32([0]), table, cu, slots, out)
    torch.cuda.synchronize()
    assert cu.tolist() == [0, n] and int(out) == n
    assert torch.equal(table[0], ids) and bool((buf[:pad] == 7).all())
    for at in range(0, n, 1 << 28):
        assert torch.equal(slots[at:at + (1 << 28)], ids[at:at + (1 << 28)].long()), at


@pytest.mark.parametrize("B,n_rows", [(0, 0), (0, 5), (3, 0)])
def test_paths_of_nothing(B, n_rows):
    """Paths given to a call without sequences, or without rows to list (torch's empty tensors have no address)."""
    cu, out = i32([9] * (B + 1)), i32([9])
    slots, src = torch.full((n_rows,), 9, dtype=torch.int64, device="cuda"), i32([9] * n_rows)
    table = torch.full((B, 4), -1, dtype=torch.int32, device="cuda")
    gb.gdn_page_tables(16, 8, i32([5] * B), i32([2] * B), i32([3, 1]), i32([1]), table, cu, slots, out,
                       i32([[0, 1]] * B).view(B, 2), i32([3 * i for i in range(B + 1)]), src)
    torch.cuda.synchronize()
    assert cu.tolist() == [0] * (B + 1) and int(out) == 1 and bool((table == -1).all())
    assert slots.tolist() == [-1] * n_rows and src.tolist() == [-1] * n_rows
