"""GPU: tree attention in every way that its work can be cut: tiles of 128 or
256 query rows, paired and alternating streams in one CTA, units that lie in
several pieces, partial results kept by unit or by CTA.

Each case runs twice.  With random operands, against 64-bit arithmetic and the
bounds of draft_util.  And with queries of zeros, which show one lost or
doubled token whatever the length: every weight is exactly 1, and each token's
V is 1 in one dim and 0 in the others, so that a dim is the share of its
tokens, 10 to 140 of them: one more or less moves it by 0.7 % or more, where
its rounding moves it by 0.4 % at most (2^-8), and every dim that it moves has
T * H rows to show it.  lse is the logarithm of the count: log2 within two last
bits below 16 (2^-20 each) times ln 2, a rounding at the end (2^-21 below 8,
2^-20 below 16), under 3e-6, where one token of 2^16 is 1.5e-5.
"""

import math

import numpy as np
import pytest
import torch

from draft_util import DEV, assert_tree_close, f64, i32, mask64, random_tree, select
from visual_token_sparsity_gb300 import synth

pytestmark = pytest.mark.gpu

# name: H, Hkv, d, B, T, n_vis, k, n_text, mask, ragged | row tile, row tiles, pieces of one, partials by unit
CASES = {
    "draft": (28, 4, 128, 8, 27, 4700, None, 150, "tree", False, 256, 1, 152, True),
    "draft_ragged": (28, 4, 128, 8, 27, 9000, 5200, 200, "tree", True, 256, 1, 152, True),
    "draft_d64": (28, 4, 64, 8, 27, 9000, 5200, 200, "any", True, 256, 1, 152, True),
    "question": (28, 4, 128, 1, 193, 6500, None, 23, "chain", False, 256, 6, 25, True),
    "question_d64": (14, 2, 64, 2, 193, 13000, 6600, 40, "chain", True, 256, 6, 25, True),
    "wide_tree": (16, 1, 64, 9, 64, 5000, None, 77, "tree", False, 256, 4, 38, True),
    "by_cta": (8, 4, 64, 50, 9, 300, None, 40, "tree", False, 128, 1, 152, False),
    "by_cta_ragged": (32, 32, 128, 6, 16, 2000, 700, 128, "tree", True, 128, 1, 152, False),
    "by_cta_paired": (28, 4, 128, 40, 27, 1500, 900, 100, "tree", True, 256, 1, 152, False),
    "by_cta_row_tiles": (16, 4, 64, 20, 75, 850, None, 60, "chain", False, 256, 2, 76, False),
    "by_cta_row_tiles_ragged": (16, 4, 128, 20, 75, 1700, 860, 70, "chain", True, 256, 2, 76, False),
    "by_unit_short": (28, 4, 128, 8, 32, 784, None, 256, "tree", True, 128, 2, 76, True),
    "one_piece_each": (7, 1, 64, 2, 1500, 300, 200, 5, "chain", True, 128, 83, 1, False),
}


class Work:
    def __init__(self, H, Hkv, d, B, T, n_vis, k, n_text, kind, ragged, *_, seed=0):
        self.shape = H, Hkv, d, B, T
        self.n_vis, self.k, self.n_text = n_vis, k, n_text
        g = np.random.default_rng(seed + H + B + T)
        self.nv, self.nt, self.ks, self.tn = [n_vis] * B, [n_text] * B, [k or 0] * B, [T] * B
        if ragged:
            # a third of the sequences: lengths between nothing and half
            few = g.permutation(B)[: (B + 2) // 3]
            for b in few:
                self.nv[b], self.nt[b] = int(g.integers(0, n_vis // 2)), int(g.integers(0, n_text + 1))
                self.ks[b] = int(g.integers(0, min(k or 0, self.nv[b]) + 1))
            for b in g.permutation(B)[: (B + 2) // 3]:
                self.tn[b] = int(g.integers(0, T + 1))
        self.ragged = ragged
        per = synth.blocks_for(n_vis + n_text + T)
        self.blocks = B * per + 3
        self.bt = synth.random_block_table(B, per, self.blocks, seed=seed + 1).to(DEV)
        gen = torch.Generator(device=DEV).manual_seed(seed + 2)
        rand = lambda *s: torch.randn(*s, generator=gen, device=DEV).to(torch.bfloat16)
        self.kp, self.vp = rand(self.blocks, Hkv, 16, d), rand(self.blocks, Hkv, 16, d)
        self.q = rand(B, T, H, d)
        self.gen = gen
        self.vis = None if k is None else select(B, Hkv, self.nv, self.ks, k, seed)
        self.masks = {"chain": None, "tree": [random_tree(T, g) for _ in range(B)] if kind == "tree" else None,
                      "any": [[int(x) for x in g.integers(0, 1 << 63, T, dtype=np.uint64) * np.uint64(2)]
                              for _ in range(B)] if kind == "any" else None}[kind]

    def count_tokens(self):
        """Queries of zeros, and V with a single 1 in each row."""
        self.q.zero_()
        d = self.shape[2]
        dim = torch.randint(0, d, self.vp.shape[:-1], generator=self.gen, device=DEV)
        self.vp.copy_(torch.nn.functional.one_hot(dim, d))

    def run(self):
        from visual_token_sparsity_gb300 import binding as sv
        H, Hkv, d, B, T = self.shape
        lens = (i32(self.nv), i32(self.nt), None if self.k is None else i32(self.ks)) if self.ragged else ()
        seqs = sv.SeqBatch(self.bt, self.n_vis, self.n_text, *lens)
        out = torch.full((B, T, H, d), 7.0, dtype=torch.bfloat16, device=DEV)
        lse = torch.full((B, T, H), 7.0, device=DEV)
        n_tok = (self.n_vis if self.k is None else self.k) + self.n_text + T
        ws = sv.workspace(sv.sv_tree_attn_workspace_bytes(B, T, H, Hkv, d, n_tok))
        sv.sv_tree_attn(self.q, 1 / math.sqrt(d), sv.KvLayer(self.kp, self.vp), seqs,
                        None if self.vis is None else i32(self.vis), self.k or 0,
                        None if self.masks is None else mask64(self.masks), out, lse, ws,
                        n_new=i32(self.tn) if self.ragged else None)
        status = sv.sv_read_device_status(ws)
        for b in range(B):
            assert (out[b, self.tn[b]:] == 7).all() and (lse[b, self.tn[b]:] == 7).all()
        return out, lse, status

    def sees(self, b):
        """bool [T'][T']: which drafted token of sequence b sees which."""
        n = self.tn[b]
        if self.masks is None:
            return torch.ones(n, n, dtype=torch.bool, device=DEV).tril()
        return torch.tensor([[bool((m >> s) & 1) for s in range(n)] for m in self.masks[b][:n]], dtype=torch.bool,
                            device=DEV).view(n, n)

    def units(self):
        """(b, g, logical K and V in 64 bits, seen [T'][tokens]) of every unit."""
        _, Hkv, d, B, _ = self.shape
        for b in range(B):
            n = self.tn[b]
            if n == 0:
                continue
            tail = list(range(self.nv[b], self.nv[b] + self.nt[b] + n))
            drafted = self.sees(b)
            for g in range(Hkv):
                vis = list(range(self.nv[b])) if self.vis is None else [x for x in self.vis[b, g, :self.ks[b]] if x >= 0]
                at = torch.tensor(vis + tail, dtype=torch.long, device=DEV)
                page = self.bt[b][at // 16].long()
                seen = torch.cat([torch.ones(n, len(at) - n, dtype=torch.bool, device=DEV), drafted], 1)
                yield b, g, self.kp[page, g, at % 16].double(), self.vp[page, g, at % 16].double(), seen

    def check(self, out, lse, what):
        H, Hkv, d, B, T = self.shape
        G = H // Hkv
        ref, mag = (np.zeros((B, T, H, d)) for _ in range(2))
        ref_lse = np.full((B, T, H), -np.inf)
        for b, g, K, V, seen in self.units():
            n = self.tn[b]
            q = self.q[b, :n, g * G:(g + 1) * G].double()
            z = torch.einsum("thd,sd->ths", q, K) / math.sqrt(d)
            z = z.masked_fill(~seen[:, None], -math.inf)
            top = z.amax(-1, keepdim=True)
            w = torch.exp(z - torch.where(top == -math.inf, 0.0, top))
            total = w.sum(-1, keepdim=True)
            p = w / torch.where(total == 0, 1.0, total)
            ref[b, :n, g * G:(g + 1) * G] = (p @ V).cpu().numpy()
            mag[b, :n, g * G:(g + 1) * G] = (p @ V.abs()).cpu().numpy()
            ref_lse[b, :n, g * G:(g + 1) * G] = (top + torch.log(total))[..., 0].cpu().numpy()
        for b in range(B):
            n = self.tn[b]
            assert_tree_close(out[b, :n], lse[b, :n], ref[b, :n], ref_lse[b, :n], mag[b, :n], f"{what}, sequence {b}")

    def check_counts(self, out, lse, what):
        H, Hkv, d, B, T = self.shape
        G = H // Hkv
        for b, g, _, V, seen in self.units():
            n = self.tn[b]
            count = seen.double() @ V                                     # [T'][d]
            total = count.sum(-1)
            ref = count / total.clamp(min=1)[:, None]
            got = out[b, :n, g * G:(g + 1) * G].double()
            off = (got - ref[:, None]).abs() > 2.0 ** -8 * ref[:, None] * (1 + 2.0 ** -10)
            assert not off.any(), f"{what}: sequence {b}, KV head {g}, (token, head, dim) {off.nonzero()[0].tolist()}"
            l = lse[b, :n, g * G:(g + 1) * G].double()
            none = total == 0
            assert torch.isneginf(l[none]).all()
            err = (l[~none] - torch.log(total[~none])[:, None]).abs()
            assert err.numel() == 0 or err.max() <= 3e-6, f"{what}: sequence {b}, KV head {g}: lse off by {err.max()}"


@pytest.mark.parametrize("name", CASES)
def test_against_64_bits(lib, name):
    w = Work(*CASES[name])
    out, lse, status = w.run()
    assert status == 0
    w.check(out, lse, name)


@pytest.mark.parametrize("seed", [1, 2])
@pytest.mark.parametrize("name", CASES)
def test_every_token_counts_once(lib, name, seed):
    w = Work(*CASES[name], seed=seed)
    w.count_tokens()
    out, lse, status = w.run()
    assert status == 0
    w.check_counts(out, lse, name)


@pytest.mark.parametrize("bad", [math.inf, math.nan])
@pytest.mark.parametrize("name", ["draft_ragged", "question", "by_cta_paired"])
def test_hidden_infinities_in_paired_streams(lib, name, bad):
    """V of a drafted token in the middle holds infinities or NaN: they reach
    the rows that see it, in both streams and in units that are cut."""
    w = Work(*CASES[name], seed=5)
    H, Hkv, d, B, T = w.shape
    at = T // 2
    clean = w.vp.clone()
    out, lse, _ = w.run()
    for b in range(B):
        pos = w.nv[b] + w.nt[b] + at
        w.vp[w.bt[b, pos // 16].long(), :, pos % 16, 3::9] = bad
    odd, odd_lse, status = w.run()
    assert status == 0
    w.vp.copy_(clean)
    dims = torch.zeros(d, dtype=torch.bool, device=DEV)
    dims[3::9] = True
    for b in range(B):
        n = w.tn[b]
        hit = w.sees(b)[:, at] if at < n else torch.zeros(n, dtype=torch.bool, device=DEV)
        x = odd[b, :n][hit][..., dims]
        assert (x.isnan() if math.isnan(bad) else x == bad).all()
        assert torch.equal(odd_lse[b, :n], lse[b, :n])
        assert odd[b, :n][~hit].isfinite().all() and odd[b, :n][hit][..., ~dims].isfinite().all()
        # the other dims as without them
        assert torch.equal(odd[b, :n][..., ~dims], out[b, :n][..., ~dims])
        if at >= n:
            assert torch.equal(odd[b, :n], out[b, :n])


@pytest.mark.parametrize("name", ["draft_ragged", "draft_d64", "question_d64", "by_cta_ragged", "by_cta_paired"])
def test_tokens_that_are_not_there_in_every_tile(lib, name):
    """Each 128 entries of the lists have their own indices outside the
    visual tokens, tile after tile: none counts, every other one does."""
    from visual_token_sparsity_gb300 import binding as sv
    w = Work(*CASES[name], seed=9)
    g = np.random.default_rng(4)
    w.vis[g.random(w.vis.shape) < 0.03] = -1
    for g in range(5):
        w.vis[:, :, g::1024] = -1
    w.count_tokens()
    out, lse, status = w.run()
    assert status == sv.SV_DEV_BAD_INDEX
    w.check_counts(out, lse, name)
