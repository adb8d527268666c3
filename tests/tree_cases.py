"""Shared helpers of the tests on trees of drafted tokens: trees as parent lists, their
lines of ancestors, and paged caches."""
from __future__ import annotations

import math

import numpy as np
import torch


def i32(v):
    return torch.as_tensor(np.asarray(v), dtype=torch.int32).cuda()


def cumulative(v):
    return np.concatenate([[0], np.cumsum(v)]).astype(np.int32)


def make_tree(r, n, shape):
    """Parents of n nodes: 'chain', 'star' (every node on its own), 'comb' (a chain with a leaf at each
    node) or 'tree' (random, several first nodes possible)."""
    if shape == "chain":
        return [i - 1 for i in range(n)]
    if shape == "star":
        return [-1] * n
    if shape == "comb":
        return [i - 1 if i % 2 else max(i - 2, -1) for i in range(n)]
    return [int(r.integers(-1, i)) if i else -1 for i in range(n)]


def line(parents, i):
    """Node i and its ancestors, first one first; a parent outside [0, i) is the cached sequence's end."""
    out = [i]
    while 0 <= parents[out[-1]] < out[-1]:
        out.append(parents[out[-1]])
    return out[::-1]


def paged(r, lens, page, spare=2, holes=()):
    """Block table of `lens` tokens on scattered pages, and the number of pages of the pool.  holes:
    (sequence, page) entries that point outside the pool."""
    need = [math.ceil(x / page) for x in lens]
    n_pages = sum(need) + spare
    perm = r.permutation(n_pages).astype(np.int32)
    table = np.full((len(lens), max(1, max(need))), -1, np.int32)
    at = 0
    for b, m in enumerate(need):
        table[b, :m] = perm[at:at + m]
        at += m
    for k, (b, p) in enumerate(holes):
        table[b, p] = n_pages + 5 if k % 2 else -7
    return table, n_pages, perm[at:]


def gather(pool, table, page, n_pages, length):
    """Rows 0 .. length-1 of a sequence from a pool [n_pages, H, page, D], and which of them exist."""
    pos = np.arange(length)
    ids = table[pos // page] if length else np.zeros(0, np.int32)
    there = (ids >= 0) & (ids < n_pages)
    return pool[np.where(there, ids, 0), :, pos % page], there
