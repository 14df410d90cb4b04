"""GPU: fork, reserve and release of shared pages against the page-by-page
oracle: tables, counts and copies must be equal, whatever the sequence of
calls, and a call that is refused changes nothing."""

import numpy as np
import pytest
import torch

import oracle
from draft_util import DEV, i32

pytestmark = pytest.mark.gpu


class Pages:
    """The device state beside the oracle's."""

    def __init__(self, B, per, pages, layers=1, Hkv=1, d=64, seed=0):
        from visual_token_sparsity_gb300 import binding as sv
        self.B, self.per = B, per
        g = torch.Generator().manual_seed(seed)
        self.table = torch.full((B, per), -1, dtype=torch.int32, device=DEV)
        self.pool = sv.PagePool(torch.zeros(pages, dtype=torch.int32, device=DEV), i32([0] * B))
        self.pools = [tuple(torch.randn(pages, Hkv, 16, d, generator=g).to(torch.bfloat16).to(DEV) for _ in range(2))
                      for _ in range(layers)]
        self.layers = [sv.KvLayer(*p) for p in self.pools]
        self.ws = sv.workspace(sv.sv_pages_workspace_bytes(B, per, pages))
        self.book = oracle.PageBook([0] * pages, [[-1] * per] * B, [0] * B)
        self.len = [0] * B
        self.sv = sv

    def seqs(self):
        return self.sv.SeqBatch(self.table, 0, self.per * 16 - 1, i32([0] * self.B), i32(self.len))

    def reserve(self, new):
        before = [tuple(x.clone() for x in p) for p in self.pools]
        T = max(new)
        s = self.sv.SeqBatch(self.table, 0, self.per * 16 - T, i32([0] * self.B), i32(self.len))
        self.sv.sv_pages_reserve(self.pool, self.layers, s, T, self.ws, n_new=i32(new))
        self.book.reserve(self.len, new)
        for old, now in zip(before, self.pools):
            for x, y in zip(old, now):
                for a, b in self.book.copies:
                    x[b] = x[a]
                assert torch.equal(x, y)
        if self.book.ok:
            self.len = [a + b for a, b in zip(self.len, new)]

    def release(self, keep):
        self.sv.sv_pages_release(self.pool, self.seqs(), i32(keep), self.ws)
        self.book.release(keep)
        self.len = [n if k < 0 else min(n, k) for n, k in zip(self.len, keep)]

    def fork(self, parent, child, n_tok=None):
        self.sv.sv_pages_fork(self.pool, self.seqs(), i32(parent), i32(child), self.ws,
                              n_tok=None if n_tok is None else i32(n_tok))
        self.book.fork(parent, child, n_tok)
        for i, (p, c) in enumerate(zip(parent, child)):
            self.len[c] = self.len[p] if n_tok is None else n_tok[i]

    def check(self, status=0):
        assert self.pool.ref.tolist() == self.book.ref
        assert self.pool.n_pages.tolist() == self.book.n
        assert self.table.tolist() == self.book.table
        got = self.sv.sv_read_device_status(self.ws, clear=True)
        assert got == status


@pytest.mark.parametrize("layers,Hkv,d", [(1, 1, 64), (3, 4, 128), (70, 1, 64)])
def test_branches_of_a_conversation(lib, layers, Hkv, d):
    p = Pages(6, 7, 31, layers, Hkv, d)
    p.reserve([40, 33, 0, 0, 0, 0])
    p.check()
    p.fork([0, 0, 1], [2, 3, 5])
    p.check()
    p.reserve([0, 5, 9, 20, 0, 1])          # private last pages, fresh ones behind
    p.check()
    p.fork([2], [4], [17])                  # before the end of the parent's tokens
    p.check()
    p.reserve([0, 0, 1, 0, 30, 0])
    p.check()
    p.release([-1, 0, 3, -1, 64, 16])
    p.check()
    p.reserve([8, 40, 0, 0, 3, 0])
    p.check()
    p.release([0] * 6)
    p.check()
    assert not p.pool.ref.any()


@pytest.mark.parametrize("seed", range(4))
def test_random_calls(lib, seed):
    g = np.random.default_rng(seed)
    B, per = int(g.integers(2, 70)), int(g.integers(1, 50))
    p = Pages(B, per, int(g.integers(1, B * per + 1)), 1, 1, 64, seed)
    for _ in range(40):
        what = int(g.integers(0, 4))
        if what == 0:
            free = [b for b in range(B) if p.book.n[b] == 0]
            kids = [b for b in free if g.random() < 0.5]
            parents = [b for b in range(B) if b not in kids]
            if kids and parents:
                p.fork([int(x) for x in g.choice(parents, len(kids))], kids)
                p.check()
        elif what == 1:
            p.release([int(g.integers(0, p.len[b] + 20)) if g.random() < 0.5 else -1 for b in range(B)])
            p.check()
        else:
            new = [int(g.integers(0, min(60, per * 16 - p.len[b]) + 1)) if g.random() < 0.4 else 0 for b in range(B)]
            if max(new) + max(p.len) > per * 16:
                new = [min(x, per * 16 - max(p.len)) for x in new]
            if max(new) > 0:
                p.reserve(new)
                p.check(0 if p.book.ok else p.sv.SV_DEV_NO_PAGES)


@pytest.mark.parametrize("pages", [20001, 16386, 40000])
def test_free_pages_far_apart(lib, pages):
    """The scan for free pages passes whole chunks that hold none."""
    p = Pages(2, 4, pages)
    p.pool.ref.fill_(1)
    p.pool.ref[[5, 16383, pages - 2, pages - 1]] = 0
    p.book.ref = p.pool.ref.tolist()
    p.reserve([33, 10])
    p.check()
    assert p.table.tolist() == [[5, 16383, pages - 2, -1], [pages - 1, -1, -1, -1]]
    p.reserve([16, 0])                      # no page left
    p.check(p.sv.SV_DEV_NO_PAGES)


def test_refused_forks_change_nothing(lib):
    p = Pages(5, 4, 20)
    p.reserve([20, 9, 0, 0, 0])
    p.check()
    sv, s = p.sv, p.seqs()
    bad = [([0], [5]), ([-1], [2]), ([5], [2]), ([0], [0]), ([2, 0], [3, 2])]
    for parent, child in bad:
        sv.sv_pages_fork(p.pool, s, i32(parent), i32(child), p.ws)
        if len(parent) == 2:                # row 2 is a parent here: only it is refused as a child
            p.book.fork([2], [3])
        p.check(sv.SV_DEV_BAD_INDEX)
    sv.sv_pages_fork(p.pool, s, i32([0]), i32([1]), p.ws)          # holds pages
    p.check(sv.SV_DEV_BAD_LENGTH)
    sv.sv_pages_fork(p.pool, s, i32([0]), i32([2]), p.ws, n_tok=i32([33]))
    p.check(sv.SV_DEV_BAD_LENGTH)
    sv.sv_pages_fork(p.pool, s, i32([0, 1]), i32([2, 2]), p.ws)     # the first pair wins
    p.book.fork([0], [2])
    p.check(sv.SV_DEV_BAD_INDEX)


def test_bad_state_is_reported_and_skipped(lib):
    p = Pages(3, 4, 8)
    p.reserve([20, 20, 0])
    p.check()
    sv = p.sv
    p.pool.n_pages[0] = 5                    # more than the row has
    for call in (lambda: sv.sv_pages_release(p.pool, p.seqs(), i32([0, -1, -1]), p.ws),
                 lambda: sv.sv_pages_reserve(p.pool, p.layers, sv.SeqBatch(p.table, 0, 30), 4, p.ws,
                                             n_new=i32([4, 0, 0]))):
        keep = p.table[0].clone()
        call()
        got = sv.sv_read_device_status(p.ws, clear=True)
        assert got == sv.SV_DEV_BAD_LENGTH
        assert torch.equal(p.table[0], keep)
    # a page without references stays at none
    p.pool.n_pages[0] = 2
    page = int(p.table[0, 0])
    p.pool.ref[page] = 0
    sv.sv_pages_release(p.pool, p.seqs(), i32([0, -1, -1]), p.ws)
    got = sv.sv_read_device_status(p.ws, clear=True)
    assert got == sv.SV_DEV_BAD_BLOCK
    assert (p.pool.ref >= 0).all() and p.table[0].tolist() == [-1] * 4


def test_reserve_without_layers_and_in_a_graph(lib):
    """Bookkeeping alone, captured once: every replay takes its own pages."""
    p = Pages(2, 8, 16)
    s = p.sv.SeqBatch(p.table, 0, 100, i32([0, 0]), length := i32([0, 0]))
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        p.sv.sv_pages_reserve(p.pool, [], s, 20, p.ws)
    for _ in range(3):
        g.replay()
        length += 20
        p.book.reserve(p.len, [20, 20])
        p.len = [x + 20 for x in p.len]
    torch.cuda.synchronize()
    p.check()
