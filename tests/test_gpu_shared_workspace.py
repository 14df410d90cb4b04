"""GPU: one workspace for calls of any kind and shape, one after the other:
every call gives the bits that it gives in a workspace of its own."""

import math

import numpy as np
import pytest
import torch

from draft_util import DEV, Cache, i32, mask64, random_tree
from visual_token_sparsity_gb300 import synth

pytestmark = pytest.mark.gpu


class Batch:
    """A cache of B sequences and the calls over it, each a function of the
    workspace that returns its outputs."""

    def __init__(self, B, H, Hkv, d, n_vis, n_text, T, seed):
        from visual_token_sparsity_gb300 import binding as sv
        self.sv, self.B, self.H, self.Hkv, self.d, self.T, self.n_vis = sv, B, H, Hkv, d, T, n_vis
        c = Cache(B, Hkv, d, n_vis + n_text + T, seed=seed)
        self.n_tok, self.per, self.blocks = n_vis + n_text + T, c.per, c.blocks
        self.layer, self.bt = c.layer(), c.bt.to(DEV)
        self.seqs = sv.SeqBatch(self.bt, n_vis, n_text)
        self.q = synth.normal_bf16((B, T, H, d), seed + 5).to(DEV)
        g = np.random.default_rng(seed)
        self.mask = mask64([random_tree(T, g) for _ in range(B)]) if T <= 64 else None

    def bytes(self):
        sv = self.sv
        return max(sv.sv_attn_workspace_bytes(self.B, self.H, self.Hkv, self.d, self.n_tok),
                   sv.sv_tree_attn_workspace_bytes(self.B, self.T, self.H, self.Hkv, self.d, self.n_tok),
                   sv.sv_retrieve_workspace_bytes(self.B, self.H, self.Hkv, self.d, self.n_vis, 20),
                   sv.sv_pages_workspace_bytes(self.B, self.per, self.blocks))

    def decode(self, ws):
        q = self.q[:, 0].contiguous()
        out, lse = torch.full_like(q, 7.0), torch.full((self.B, self.H), 7.0, device=DEV)
        self.sv.sv_sparse_decode_attn(q, 0.125, self.layer, self.seqs, None, 0, out, lse, ws)
        return out, lse

    def tree(self, ws):
        out, lse = torch.full_like(self.q, 7.0), torch.full((self.B, self.T, self.H), 7.0, device=DEV)
        self.sv.sv_tree_attn(self.q, 0.125, self.layer, self.seqs, None, 0, self.mask, out, lse, ws)
        return out, lse

    def retrieve(self, ws):
        vis = torch.full((self.B, self.Hkv, 20), -7, dtype=torch.int32, device=DEV)
        self.sv.sv_retrieve_topk(self.q[:, :1].contiguous(), self.layer, self.seqs, 20, vis, None, ws)
        return vis,

    def reserve(self, ws):
        table, n_pages = torch.full_like(self.bt, -1), i32([0] * self.B)
        pool = self.sv.PagePool(torch.zeros(self.blocks, dtype=torch.int32, device=DEV), n_pages)
        self.sv.sv_pages_reserve(pool, [], self.sv.SeqBatch(table, self.n_vis, 0), self.T, ws)
        return table, n_pages


def check(calls, nbytes):
    """Every call in its turn over one workspace, twice, and each alone."""
    from visual_token_sparsity_gb300 import binding as sv
    shared = sv.workspace(nbytes)
    for what, call in calls * 2:
        got = call(shared)
        alone = call(sv.workspace(nbytes))
        torch.cuda.synchronize()
        assert sv.sv_read_device_status(shared) == 0
        for i, (x, y) in enumerate(zip(got, alone)):
            assert torch.equal(x, y), f"{what}, output {i}"


@pytest.mark.parametrize("first", ["decode", "tree", "retrieve", "reserve"])
def test_a_small_batch_before_a_larger_one(lib, first):
    """What the small batch's call leaves behind is not taken for the larger
    one's counters (a split or a row that is never the last writes nothing)."""
    one, many = Batch(1, 8, 4, 64, 1500, 40, 20, 1), Batch(32, 8, 4, 64, 700, 30, 8, 2)
    check([(first + " of 1", getattr(one, first)), ("decode of 32", many.decode), ("tree of 32", many.tree),
           ("decode of 1", one.decode), ("retrieve of 1", one.retrieve)], max(one.bytes(), many.bytes()))


@pytest.mark.parametrize("B,H,Hkv", [(4097, 1, 1), (600, 16, 8), (2048, 4, 2)])
def test_as_many_units_as_there_are_counters(lib, B, H, Hkv):
    """More (sequence, KV head) units than counters, and just as many."""
    many, one = Batch(B, H, Hkv, 64, 40, 9, 3, 3), Batch(2, 8, 8, 128, 900, 9, 3, 4)
    check([("decode of many", many.decode), ("decode of 2", one.decode), ("tree of many", many.tree)],
          max(one.bytes(), many.bytes()))


def salience(B, H, N, d, std, seed):
    """std 3: logits so large that units are computed again (the fail list)."""
    from visual_token_sparsity_gb300 import binding as sv
    q, k = (synth.normal_bf16((B, H, N, d), seed + i, std=std).to(DEV) for i in range(2))

    def call(ws):
        sal = torch.full((B, N), 7.0, device=DEV)
        sv.sv_salience_prefill(q, k, 1 / math.sqrt(d), sal, ws)
        return sal,
    return call, sv.sv_salience_workspace_bytes(B, H, N, d)


def test_salience_of_several_shapes_among_other_calls(lib):
    """The list of units to compute again begins empty wherever it lies."""
    one = Batch(1, 28, 4, 128, 3000, 40, 30, 6)
    parts = [salience(2, 3, 300, 64, 1.0, 1), salience(1, 16, 729, 72, 3.0, 2), salience(1, 2, 1500, 80, 3.0, 3),
             salience(3, 2, 200, 128, 1.0, 4)]
    calls = [("tree", one.tree)] + [(f"salience {i}", c) for i, (c, _) in enumerate(parts)] + [("decode", one.decode)]
    check(calls, max([one.bytes()] + [n for _, n in parts]))
