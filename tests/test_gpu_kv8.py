"""GPU: the cache in 8 bits (appending, retrieval, attention) against the fp64
oracle, and the calls together as a conversation makes them."""

import math

import numpy as np
import pytest
import torch

import oracle
from kv8_util import (DEV, KV8_WEIGHTS, PROMPT_WEIGHTS, Cache8, assert_close, f64, i32, oracle_decode, oracle_select,
                      select)
from visual_token_sparsity_gb300 import synth

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------------ append

def rotation(rot, axes, N, n_pos, seed, weights=None, interleaved=False, sections=None, pos=None):
    from visual_token_sparsity_gb300 import binding as sv
    g = torch.Generator().manual_seed(seed)
    cs = None
    if rot:
        a = torch.arange(n_pos).double()[:, None] * 10000.0 ** (-torch.arange(rot // 2).double() * 2 / rot)
        cs = torch.stack([a.cos(), a.sin()], -1).float().to(DEV)
    if pos is None:
        pos = torch.randint(0, n_pos, (axes, 1, N) if axes > 1 else (1, N), generator=g, dtype=torch.int32).to(DEV)
    qw, kw = (None, None) if weights is None else weights
    r = sv.Rotation(cs, pos, sections=sections, interleaved=interleaved, q_weight=qw, k_weight=kw, eps=1e-5)
    ref = lambda x, w: oracle.norm_rope(f64(x)[None], None if w is None else f64(w), 1e-5,
                                        None if cs is None else f64(cs), pos.cpu().numpy(), sections, interleaved)[0]
    return r, ref


def weights(d, seed):
    return tuple((1 + 0.2 * synth.normal_bf16((d,), seed + i).float()).to(torch.bfloat16).to(DEV) for i in range(2))


def assert_rows_close(got, ref, what):
    got = f64(got)
    top = np.abs(ref).max(-1, keepdims=True)
    err = np.abs(got - ref) - 2.0 ** -8 * np.abs(ref) - 2.0 ** -20 * top
    assert got.size == 0 or (err <= 0).all(), f"{what}: {err.max()} over the bound"


class Append:
    """A cache and new tokens of each sequence, packed."""

    def __init__(self, H, Hkv, d, base, new, seed, lead=0, behind=0, factor=None, **rot):
        self.H, self.Hkv, self.d, self.base, self.new = H, Hkv, d, list(base), list(new)
        B = len(new)
        self.cache = Cache8(B, Hkv, d, max(b + n for b, n in zip(base, new)) + 5, seed, factor=factor)
        self.start = lead + np.concatenate([[0], np.cumsum(new)])
        self.N = int(self.start[-1]) + behind
        self.proj = synth.normal_bf16((self.N, H + 2 * Hkv, d), seed + 7).to(DEV)
        self.w = weights(d, seed) if rot.pop("norm", False) else None
        rot_dim = rot.pop("rot", d)
        self.rot, self.ref = rotation(rot_dim, rot.pop("axes", 1), self.N, 400, seed, self.w, **rot)

    def seqs(self):
        from visual_token_sparsity_gb300 import binding as sv
        nv = [b // 3 for b in self.base]
        return sv.SeqBatch(self.cache.bt.to(DEV), max(nv), max(b - v for b, v in zip(self.base, nv)), i32(nv),
                           i32([b - v for b, v in zip(self.base, nv)]))

    def run(self, layer, k_out=True, start=True, seqs=None):
        from visual_token_sparsity_gb300 import binding as sv
        ws = sv.workspace(sv.sv_evict_workspace_bytes())
        qo = torch.full((self.N, self.H, self.d), 9.0, dtype=torch.bfloat16, device=DEV)
        ko = torch.full((self.N, self.Hkv, self.d), 9.0, dtype=torch.bfloat16, device=DEV)
        q, k, v = self.parts()
        sv.sv_kv8_append(q, k, v, self.rot, layer, seqs or self.seqs(), qo, ws,
                         seq_start=i32(self.start) if start else None, k_out=ko if k_out else None)
        return qo, ko, sv.sv_read_device_status(ws)

    def parts(self):
        return self.proj[:, :self.H], self.proj[:, self.H: self.H + self.Hkv], self.proj[:, self.H + self.Hkv:]

    def expect(self, keys, skip=()):
        """(codes, scales) after the call, from the keys' bf16 rows."""
        c = self.cache
        codes, scales = [x.copy() for x in c.codes], c.scales.copy()
        v = f64(self.parts()[2])
        for b, n in enumerate(self.new):
            if b in skip:
                continue
            a, e = self.start[b], self.start[b + 1]
            for which, x in ((0, keys), (1, v)):
                s = scales[b, ..., which].copy()
                oracle.kv8_append(codes[which][b], s, self.base[b], x[a:e])
                scales[b, ..., which] = s
        return codes, scales

    def check(self, layer, qo, ko, skip=()):
        a, e = self.start[0], self.start[-1]
        q, k, v = self.parts()
        assert_rows_close(qo[a:e], self.ref(q, self.w and self.w[0])[a:e], "q")
        assert_rows_close(ko[a:e], self.ref(k, self.w and self.w[1])[a:e], "k")
        for x in (qo[:a], qo[e:], ko[:a], ko[e:]):
            assert (x == 9).all(), "rows of no sequence"
        # the 8-bit rows follow from the bf16 ones, bit by bit
        want, want_s = self.expect(f64(ko), skip)
        got, got_s = self.cache.read_back(layer)
        assert np.array_equal(got_s.astype(np.float64), want_s), "scales"
        for name, x, y in zip("kv", got, want):
            diff = (x != y) & ~((x & 127 == 127) & (y & 127 == 127))
            assert not diff.any(), f"{name}: {diff.sum()} codes differ, first at {np.argwhere(diff)[0]}"


APPENDS = [
    # H, Hkv, d, tokens before, new tokens, rotation
    (4, 2, 64, [0], [1], {}), (4, 2, 64, [7], [1], {}), (4, 2, 64, [15, 16, 17], [1, 1, 1], {}),
    (28, 4, 128, [0, 0, 5], [100, 0, 33], dict(norm=True, axes=3, sections=[16, 24, 24])),
    (2, 2, 128, [31, 0, 48, 9], [17, 16, 1, 40], dict(interleaved=True)),
    (16, 1, 64, [3, 250], [200, 6], dict(rot=32, norm=True)),
    (1, 1, 128, [14], [2], dict(rot=0)), (3, 3, 64, [1, 2], [31, 14], dict(rot=0, norm=True)),
    (32, 32, 128, [3008 - 2879] * 4, [1] * 4, {}), (5, 1, 128, [12], [64], dict(rot=64, interleaved=True, norm=True)),
    (2, 1, 64, [0] * 70, [3, 0, 17, 1, 16] * 14, dict(axes=2, sections=[8, 24])),
]


@pytest.mark.parametrize("H,Hkv,d,base,new,rot", APPENDS)
def test_append(lib, H, Hkv, d, base, new, rot):
    a = Append(H, Hkv, d, base, new, seed=3 + H, lead=2, behind=3, **rot)
    layer = a.cache.layer()
    qo, ko, status = a.run(layer)
    assert status == 0
    a.check(layer, qo, ko)


def test_append_again_changes_nothing(lib):
    """The same rows at the same positions: the page keeps its factor."""
    a = Append(4, 2, 64, [5, 40], [30, 9], seed=40)
    layer = a.cache.layer()
    a.run(layer)
    one = a.cache.read_back(layer)
    qo, ko, _ = a.run(layer)
    two = a.cache.read_back(layer)
    assert all(np.array_equal(x, y) for x, y in zip(one[0], two[0])) and np.array_equal(one[1], two[1])


def test_even_shares_need_no_starts(lib):
    a = Append(6, 2, 64, [10, 10, 10], [21, 21, 21], seed=41)
    la, lb = a.cache.layer(), a.cache.layer()
    qa, ka, _ = a.run(la)
    qb, kb, status = a.run(lb, start=False)
    assert status == 0 and torch.equal(qa, qb) and torch.equal(ka, kb)
    a.check(lb, qb, kb)


@pytest.mark.parametrize("grow", [2.0 ** 9, 2.0 ** 40, 2.0 ** -30])
def test_pages_that_grow_and_pages_that_do_not(lib, grow):
    """New rows that are far larger (the old ones are rounded again, into e4m3's
    smallest values or to 0) or far smaller than the page's."""
    a = Append(2, 1, 64, [9, 6], [3, 30], seed=42, rot=0)
    a.proj[:, 2:] *= grow
    layer = a.cache.layer()
    qo, ko, status = a.run(layer)
    assert status == 0
    a.check(layer, qo, ko)


def test_zero_tiny_and_huge_rows(lib):
    a = Append(2, 2, 64, [0, 0, 0, 0], [16, 16, 16, 5], seed=43, rot=0)
    a.proj[0:16] = 0
    a.proj[16:32] *= 2.0 ** -126
    a.proj[32:48] *= 2.0 ** 125
    a.proj[48:53] = 1e-40
    layer = a.cache.layer()
    qo, ko, status = a.run(layer)
    assert status == 0
    a.check(layer, qo, ko)
    got, s = a.cache.read_back(layer)
    assert (got[0][0, :, :16] == 0).all() and (s[0, :, 0] == 2.0 ** -126).all()


def test_infinities_and_nan(lib):
    """They do not count for the factor: infinities become 448 times it, NaN stays."""
    a = Append(2, 1, 128, [0, 4], [20, 12], seed=44, rot=0)
    a.proj[3, 2, 5], a.proj[18, 3, 7], a.proj[25, 2, 0] = float("inf"), float("-inf"), float("nan")
    a.proj[26, 3] = float("nan")
    layer = a.cache.layer()
    q, k, v = a.parts()
    qo, ko, status = a.run(layer)
    assert status == 0 and torch.equal(ko.view(torch.int16), k.view(torch.int16))
    want, want_s = a.expect(f64(k))
    got, got_s = a.cache.read_back(layer)
    assert np.array_equal(got_s.astype(np.float64), want_s)
    for x, y in zip(got, want):
        assert ((x == y) | ((x & 127 == 127) & (y & 127 == 127))).all()
    assert got[0][0, 0, 3, 5] == 0x7E and got[1][0, 0, 18, 7] == 0xFE and (got[1][1, 0, 10] & 127 == 127).all()


def test_an_old_factor_that_is_none(lib):
    """A page's factor that is 0, NaN or negative counts as the smallest one."""
    for bad in (0.0, float("nan"), -3.0, 1e-42):
        a = Append(2, 1, 64, [4], [3], seed=45, rot=0)
        layer = a.cache.layer()
        page = int(a.cache.bt[0, 0])
        layer.scales[page] = bad
        a.cache.scales[0, :, 0] = 2.0 ** -126
        qo, ko, status = a.run(layer)
        assert status == 0
        a.check(layer, qo, ko)


def test_in_place_outputs(lib):
    from visual_token_sparsity_gb300 import binding as sv
    a = Append(4, 2, 128, [3, 20], [18, 40], seed=46, norm=True)
    la, lb = a.cache.layer(), a.cache.layer()
    qo, ko, _ = a.run(la)
    q, k, v = (x.contiguous() for x in a.parts())
    sv.sv_kv8_append(q, k, v, a.rot, lb, a.seqs(), q, sv.workspace(256), seq_start=i32(a.start), k_out=k)
    assert torch.equal(q, qo) and torch.equal(k, ko)
    assert torch.equal(la.k_pool.view(torch.uint8), lb.k_pool.view(torch.uint8))
    assert torch.equal(la.v_pool.view(torch.uint8), lb.v_pool.view(torch.uint8))


def test_skipped_sequences_pages_and_positions(lib):
    from visual_token_sparsity_gb300 import binding as sv
    # a length out of range: that sequence alone
    a = Append(2, 1, 64, [9, 9, 9], [5, 5, 5], seed=47)
    layer, seqs = a.cache.layer(), a.seqs()
    bad = sv.SeqBatch(seqs.block_table, 3, 6, i32([3, 4, 3]), i32([6, 6, 6]))
    qo, ko, status = a.run(layer, seqs=bad)
    assert status == sv.SV_DEV_BAD_LENGTH
    a.check(layer, qo, ko, skip=[1])
    # tokens that overflow the block table
    a = Append(2, 1, 64, [9, 9, 9], [5, 30, 5], seed=48)
    short = a.cache.bt[:, :2].contiguous()
    layer = a.cache.layer()
    qo, ko, status = a.run(layer, seqs=sv.SeqBatch(short.to(DEV), 3, 6))
    assert status == sv.SV_DEV_BAD_LENGTH
    a.check(layer, qo, ko, skip=[1])
    # a page outside the pool
    a = Append(2, 1, 64, [9, 9], [20, 20], seed=49)
    layer = a.cache.layer()
    bt = a.cache.bt.clone()
    bt[1] = torch.tensor([a.cache.blocks, -5, 2 ** 30])[: bt.shape[1]]
    qo, ko, status = a.run(layer, seqs=sv.SeqBatch(bt.to(DEV), 3, 6))
    assert status == sv.SV_DEV_BAD_BLOCK
    a.check(layer, qo, ko, skip=[1])
    # a position outside the table: that token stays as it was, in the cache too
    a = Append(2, 1, 64, [0], [20], seed=50)
    for at, p in ((3, 400), (17, -1)):
        a.rot.pos[0, at] = p
    layer = a.cache.layer()
    qo, ko, status = a.run(layer)
    assert status == sv.SV_DEV_BAD_POSITION
    assert (qo[[3, 17]] == 9).all() and (ko[[3, 17]] == 9).all()
    got, _ = a.cache.read_back(layer)
    for which in range(2):
        assert np.array_equal(got[which][0, :, [3, 17]], a.cache.codes[which][0, :, [3, 17]])
    keep = [i for i in range(20) if i not in (3, 17)]
    want, s = np.zeros((1, 32, 64), np.uint8), np.ones((1, 2))
    keys = f64(ko)
    keys[[3, 17]] = 0
    oracle.kv8_append(want, s, 0, keys)
    assert np.array_equal(got[0][0][:, keep], want[:, keep])


@pytest.mark.parametrize("start", [[0, 7, 3, 12], [-2, 4, 8, 12], [0, 4, 8, 13]])
def test_starts_that_do_not_ascend_are_reported(lib, start):
    from visual_token_sparsity_gb300 import binding as sv
    a = Append(2, 1, 64, [9, 9, 9], [4, 4, 4], seed=51)
    layer = a.cache.layer()
    before = a.cache.read_back(layer)
    a.start = np.array(start)
    _, _, status = a.run(layer)
    assert status == sv.SV_DEV_BAD_LENGTH
    after = a.cache.read_back(layer)
    for which in range(2):                                 # earlier rows of every sequence but for rounding again
        same = before[1][..., which] == after[1][..., which]
        rows = np.repeat(same, 16, 2)[..., :9]
        x, y = before[0][which][:, :, :9], after[0][which][:, :, :9]
        assert (x == y)[rows].all()


# ------------------------------------------------------------------ retrieval

def retrieve(c, q, seqs, k, scores=True):
    from visual_token_sparsity_gb300 import binding as sv
    B, R, H, d = q.shape
    vis = torch.full((B, c.Hkv, k), -7, dtype=torch.int32, device=DEV)
    sc = torch.full((B, c.Hkv, seqs.n_vis), 7.0, device=DEV) if scores else None
    ws = sv.workspace(sv.sv_kv8_retrieve_workspace_bytes(B, H, c.Hkv, d, seqs.n_vis, k))
    sv.sv_kv8_retrieve_topk(q, c.layer(), seqs, k, vis, sc, ws)
    return vis.cpu().numpy(), sc, sv.sv_read_device_status(ws)


@pytest.mark.parametrize("H,Hkv,d,B,R,n_vis,k", [
    (1, 1, 64, 1, 1, 1, 1), (4, 2, 64, 1, 1, 17, 5), (4, 2, 64, 2, 32, 576, 144), (28, 4, 128, 2, 3, 1000, 999),
    (32, 32, 128, 1, 1, 2880, 1440), (7, 1, 128, 1, 193, 300, 300), (16, 1, 64, 3, 2, 5000, 1),
    (8, 4, 128, 1, 1, 20011, 5002), (2, 2, 64, 1, 1, 60001, 15000), (5, 1, 64, 2, 40, 9000, 4500),
    (1, 1, 64, 1, 2, 420007, 100003), (2, 1, 128, 2, 1, 16384, 16383), (3, 1, 64, 1, 1, 16385, 2),
])
def test_retrieval(lib, H, Hkv, d, B, R, n_vis, k):
    from visual_token_sparsity_gb300 import binding as sv
    c = Cache8(B, Hkv, d, n_vis, seed=H + n_vis)
    q = synth.normal_bf16((B, R, H, d), 5).to(DEV)
    vis, sc, status = retrieve(c, q, sv.SeqBatch(c.bt.to(DEV), n_vis, 0), k)
    assert status == 0
    want, scores = oracle_select(q, c.rows(0), [n_vis] * B, [k] * B)
    assert np.array_equal(vis, want)
    for (b, g), s in scores.items():
        assert np.abs(f64(sc[b, g]) - s).max() <= 1e-5 * np.abs(s).max() + 1e-30
    again, _, _ = retrieve(c, q, sv.SeqBatch(c.bt.to(DEV), n_vis, 0), k, scores=False)
    assert np.array_equal(again, want)


@pytest.mark.parametrize("Hkv,d,n_vis,k", [(2, 64, 700, 200), (1, 128, 17000, 6000)])
def test_retrieval_of_different_lengths(lib, Hkv, d, n_vis, k):
    from visual_token_sparsity_gb300 import binding as sv
    nv = [n_vis, n_vis // 2, 1, 0, n_vis // 3, n_vis + 1, 40]
    ks = [k, 0, 1, 0, min(k, n_vis // 3), 1, 41]
    good = [0, 1, 2, 3, 4]
    c = Cache8(7, Hkv, d, n_vis, seed=60)
    q = synth.normal_bf16((7, 1, 2 * Hkv, d), 6).to(DEV)
    seqs = sv.SeqBatch(c.bt.to(DEV), n_vis, 0, i32(nv), None, i32(ks))
    vis, _, status = retrieve(c, q, seqs, k)
    assert status == sv.SV_DEV_BAD_LENGTH
    want, _ = oracle_select(q[:5], c.rows(0)[:5], nv[:5], ks[:5])
    assert np.array_equal(vis[good], want[good])
    assert (vis[5:] == -1).all()


@pytest.mark.parametrize("n_vis,k", [(2000, 700), (20000, 9000), (410000, 70000)])
def test_scores_that_fp32_cannot_tell_apart(lib, n_vis, k):
    """The scores differ beyond fp32's last bit: 2^20 from one element, less than 2^-8
    from another; the selection is the exact one."""
    from visual_token_sparsity_gb300 import binding as sv
    c = Cache8(1, 1, 64, n_vis, seed=61)
    g = np.random.default_rng(3)
    c.codes[0][:] = 0
    c.scales[:] = 1.0
    cap = c.codes[0].shape[2]
    c.codes[0][0, 0, :, 0] = oracle.to_e4m3(256.0)
    c.codes[0][0, 0, :, 1] = g.integers(0, 126, cap)
    c.codes[0][0, 0, :, 2] = g.integers(0, 2, cap) * 0x38
    q = torch.zeros(1, 1, 1, 64, dtype=torch.bfloat16, device=DEV)
    q[..., 0], q[..., 1], q[..., 2] = 4096.0, 2.0 ** -18, 2.0 ** -9
    vis, _, status = retrieve(c, q, sv.SeqBatch(c.bt.to(DEV), n_vis, 0), k)
    want, scores = oracle_select(q, c.rows(0), [n_vis], [k])
    assert len(set(np.float32(scores[0, 0]).tolist())) == 1 and len(set(scores[0, 0].tolist())) > 20
    assert status == 0 and np.array_equal(vis, want)


@pytest.mark.parametrize("n_vis,k,kinds", [(600, 100, 3), (5000, 2500, 2), (30000, 11111, 7), (40, 39, 1), (411000, 200000, 2)])
def test_tied_tokens_go_to_the_lower_index(lib, n_vis, k, kinds):
    """A few different rows, each many times over."""
    from visual_token_sparsity_gb300 import binding as sv
    c = Cache8(2, 2, 64, n_vis, seed=62)
    g = np.random.default_rng(4)
    pick = g.integers(0, kinds, c.codes[0].shape[2])
    c.codes[0] = c.codes[0][:, :, pick]
    c.scales[...] = 0.25
    q = synth.normal_bf16((2, 1, 2, 64), 8).to(DEV)
    vis, _, status = retrieve(c, q, sv.SeqBatch(c.bt.to(DEV), n_vis, 0), k)
    assert status == 0 and np.array_equal(vis, oracle_select(q, c.rows(0), [n_vis] * 2, [k] * 2)[0])
    vis, _, _ = retrieve(c, torch.zeros_like(q), sv.SeqBatch(c.bt.to(DEV), n_vis, 0), k)
    assert (vis == np.arange(k)).all()


def test_rows_that_cancel(lib):
    """Query rows whose sum is small beside them: qbar is taken exactly."""
    from visual_token_sparsity_gb300 import binding as sv
    c = Cache8(1, 1, 64, 3000, seed=63)
    q = synth.normal_bf16((1, 3, 1, 64), 9)
    q[0, 0] *= 2.0 ** 12
    q[0, 2] = -q[0, 0]
    q = q.to(DEV)
    vis, _, status = retrieve(c, q, sv.SeqBatch(c.bt.to(DEV), 3000, 0), 1000)
    assert status == 0 and np.array_equal(vis, oracle_select(q, c.rows(0), [3000], [1000])[0])


def test_retrieval_skips_pages_outside_the_pool(lib):
    from visual_token_sparsity_gb300 import binding as sv
    c = Cache8(1, 2, 64, 500, seed=64)
    bt = c.bt.clone()
    bt[0, 3], bt[0, 9] = -1, c.blocks
    q = synth.normal_bf16((1, 1, 4, 64), 10).to(DEV)
    vis, sc, status = retrieve(c, q, sv.SeqBatch(bt.to(DEV), 500, 0), 100)
    assert status == sv.SV_DEV_BAD_BLOCK
    K = c.rows(0)
    K[:, :, 48:64] = K[:, :, 144:160] = 0                 # their scores are 0
    assert np.array_equal(vis, oracle_select(q, K, [500], [100])[0])
    assert (sc[:, :, 48:64] == 0).all() and (sc[:, :, 144:160] == 0).all()


def test_scores_that_are_not_finite_give_a_valid_choice(lib):
    from visual_token_sparsity_gb300 import binding as sv
    c = Cache8(1, 1, 64, 800, seed=65)
    c.codes[0][0, 0, 100:130, 3] = 0x7F
    q = synth.normal_bf16((1, 1, 1, 64), 11).to(DEV)
    for k in (10, 40, 700, 790):
        vis, _, status = retrieve(c, q, sv.SeqBatch(c.bt.to(DEV), 800, 0), k)
        assert status == 0 and (np.diff(vis[0, 0]) > 0).all() and vis.min() >= 0 and vis.max() < 800
    q[..., 0] = float("inf")
    vis, _, _ = retrieve(c, q, sv.SeqBatch(c.bt.to(DEV), 800, 0), 40)
    assert (np.diff(vis[0, 0]) > 0).all() and vis.min() >= 0 and vis.max() < 800


# ------------------------------------------------------------------ attention

def attend(c, q, seqs, vis, k, scale, lse=True):
    from visual_token_sparsity_gb300 import binding as sv
    B, H, d = q.shape
    out = torch.full_like(q, 7.0)
    norm = torch.full((B, H), 7.0, device=DEV) if lse else None
    n = (k if vis is not None else seqs.n_vis) + seqs.n_text
    ws = sv.workspace(sv.sv_kv8_attn_workspace_bytes(B, H, c.Hkv, d, n))
    for _ in range(2):                                     # (the counters are left at zero)
        sv.sv_kv8_decode_attn(q, scale, c.layer(), seqs, None if vis is None else i32(vis), k, out, norm, ws)
    return out, norm, sv.sv_read_device_status(ws)


@pytest.mark.parametrize("H,Hkv,d,B,n_vis,n_text,k", [
    (1, 1, 64, 1, 1, 0, 1), (1, 1, 128, 1, 0, 1, None), (4, 2, 64, 1, 576, 57, 144), (4, 2, 64, 3, 100, 31, 0),
    (32, 32, 128, 2, 700, 40, 350), (28, 4, 128, 2, 3136, 256, 784), (28, 4, 128, 1, 300, 17, None),
    (16, 1, 128, 2, 999, 1, 500), (16, 1, 64, 1, 33, 0, 33), (9, 1, 128, 1, 2000, 5, 1000), (8, 1, 64, 2, 257, 16, 255),
    (5, 1, 128, 1, 40, 3, 20), (6, 2, 64, 1, 15, 2, 7), (6, 3, 128, 4, 200, 15, None), (12, 4, 64, 1, 5000, 100, 2501),
    (2, 1, 128, 33, 64, 9, 16), (7, 7, 64, 1, 12000, 33, 6000),
])
def test_attention(lib, H, Hkv, d, B, n_vis, n_text, k):
    from visual_token_sparsity_gb300 import binding as sv
    c = Cache8(B, Hkv, d, n_vis + n_text, seed=H + n_vis)
    q = synth.normal_bf16((B, H, d), 5).to(DEV)
    vis = None if k is None else select(B, Hkv, [n_vis] * B, [k] * B, k, 3)
    scale = 1 / math.sqrt(d)
    out, lse, status = attend(c, q, sv.SeqBatch(c.bt.to(DEV), n_vis, n_text), vis, k or 0, scale)
    assert status == 0
    ref = oracle_decode(q, c.rows(0), c.rows(1), vis, [n_vis] * B, [n_text] * B, [k] * B, scale)
    assert_close(out, lse, *ref, KV8_WEIGHTS)
    again, _, _ = attend(c, q, sv.SeqBatch(c.bt.to(DEV), n_vis, n_text), vis, k or 0, scale, lse=False)
    assert torch.equal(out.view(torch.int16), again.view(torch.int16))


@pytest.mark.parametrize("indexed", [True, False])
@pytest.mark.parametrize("H,Hkv,d", [(4, 2, 64), (28, 4, 128), (3, 3, 128)])
def test_attention_of_different_lengths(lib, H, Hkv, d, indexed):
    from visual_token_sparsity_gb300 import binding as sv
    n_vis, n_text, k = 900, 70, 400
    nv = [900, 450, 0, 1, 33, 901, 500]
    nt = [70, 0, 5, 1, 0, 10, 71]
    ks = [400, 0, 0, 1, 33, 5, 100]
    B = len(nv)
    c = Cache8(B, Hkv, d, n_vis + n_text + 2, seed=70)
    q = synth.normal_bf16((B, H, d), 7).to(DEV)
    vis = select(B, Hkv, [min(n, n_vis) for n in nv], ks, k, 8) if indexed else None
    seqs = sv.SeqBatch(c.bt.to(DEV), n_vis, n_text, i32(nv), i32(nt), i32(ks))
    out, lse, status = attend(c, q, seqs, vis, k if indexed else 0, 0.11)
    assert status == sv.SV_DEV_BAD_LENGTH
    nv[5:], nt[5:], ks[5:] = [0, 0], [0, 0], [0, 0]        # skipped: out 0, lse -inf
    ref = oracle_decode(q, c.rows(0), c.rows(1), vis, nv, nt, ks, 0.11)
    assert_close(out, lse, *ref, KV8_WEIGHTS)
    assert (out[5:] == 0).all() and torch.isneginf(lse[5:]).all()
    if indexed:
        assert torch.isneginf(lse[1]).sum() == H and (out[1] == 0).all()   # no text, nothing selected


@pytest.mark.parametrize("H,Hkv,d", [(2, 2, 64), (8, 1, 128), (16, 1, 64)])
def test_pages_of_very_different_factors(lib, H, Hkv, d):
    """Values that are 2^20 apart from page to page, and keys whose products are 2^12
    apart: a weight keeps its bits whatever its page's factor."""
    from visual_token_sparsity_gb300 import binding as sv
    g = np.random.default_rng(5)
    n = 500
    per = synth.blocks_for(n)
    factor = np.exp2(np.stack([g.integers(-9, 3, (1, Hkv, per)), g.integers(-10, 10, (1, Hkv, per))], -1))
    c = Cache8(1, Hkv, d, n, seed=71, factor=factor)
    q = synth.normal_bf16((1, H, d), 9).to(DEV)
    seqs = sv.SeqBatch(c.bt.to(DEV), n - 20, 20)
    out, lse, status = attend(c, q, seqs, None, 0, 1 / math.sqrt(d))
    ref = oracle_decode(q, c.rows(0), c.rows(1), None, [n - 20], [20], None, 1 / math.sqrt(d))
    assert status == 0
    assert_close(out, lse, *ref, KV8_WEIGHTS)


@pytest.mark.parametrize("kf,vf", [(0.0, 1.0), (1.0, 0.0), (2.0 ** -126, 2.0 ** -126), (2.0 ** -120, 2.0 ** 100)])
def test_extreme_factors(lib, kf, vf):
    from visual_token_sparsity_gb300 import binding as sv
    c = Cache8(1, 1, 64, 200, seed=72)
    c.scales[..., 0], c.scales[..., 1] = kf, vf
    q = synth.normal_bf16((1, 2, 64), 10).to(DEV)
    out, lse, status = attend(c, q, sv.SeqBatch(c.bt.to(DEV), 150, 50), None, 0, 0.125)
    ref = oracle_decode(q, c.rows(0), c.rows(1), None, [150], [50], None, 0.125)
    assert status == 0
    if vf >= 2.0 ** -100:
        assert_close(out, lse, *ref, KV8_WEIGHTS)
    else:                                                   # below the smallest numbers of the output's type
        assert (out.abs() <= 2.0 ** -110).all()
        assert np.abs(f64(lse) - ref[1]).max() < 1e-3


def test_queries_of_very_different_magnitudes(lib):
    """Heads 2^40 apart, and elements that reach 2^100 or vanish beside others."""
    from visual_token_sparsity_gb300 import binding as sv
    c = Cache8(1, 1, 128, 300, seed=73)
    q = synth.normal_bf16((1, 8, 128), 11)
    q[0, 1] *= 2.0 ** -40
    q[0, 2] = 0
    q[0, 3] *= 2.0 ** 4
    q[0, 4, ::3] *= 2.0 ** -30
    q[0, 5, 0] = 100.0
    c.codes[0][0, 0, :, 5] = 0
    q[0, 6, 5] = 2.0 ** 100                                 # meets zeros only
    q = q.to(DEV)
    out, lse, status = attend(c, q, sv.SeqBatch(c.bt.to(DEV), 250, 50), None, 0, 0.09)
    ref = oracle_decode(q, c.rows(0), c.rows(1), None, [250], [50], None, 0.09)
    assert status == 0
    keep = [0, 1, 2, 3, 4, 5, 7]
    assert_close(out[:, keep], lse[:, keep], *(r[:, keep] for r in ref), KV8_WEIGHTS)
    # 2^100 beside elements of order 1: fp32's products keep what 24 bits below it keep, nothing
    assert torch.isfinite(out[:, 6]).all()


def test_scale_zero_and_negative(lib):
    from visual_token_sparsity_gb300 import binding as sv
    c = Cache8(1, 2, 64, 90, seed=74)
    q = synth.normal_bf16((1, 4, 64), 12).to(DEV)
    for scale in (0.0, -0.125):
        out, lse, _ = attend(c, q, sv.SeqBatch(c.bt.to(DEV), 60, 30), None, 0, scale)
        assert_close(out, lse, *oracle_decode(q, c.rows(0), c.rows(1), None, [60], [30], None, scale), KV8_WEIGHTS)


def test_rows_behind_the_end_and_skipped_tokens(lib):
    """NaN rows behind the last token (and pages that nobody holds are NaN) have no
    part; indices and pages that are out of range are reported and skipped."""
    from visual_token_sparsity_gb300 import binding as sv
    for H, Hkv, d in ((2, 2, 64), (7, 1, 128)):
        c = Cache8(1, Hkv, d, 100, seed=75)
        c.codes[0][:, :, 91:], c.codes[1][:, :, 91:] = 0x7F, 0x7F
        q = synth.normal_bf16((1, H, d), 13).to(DEV)
        vis = select(1, Hkv, [80], [30], 30, 4)
        out, lse, status = attend(c, q, sv.SeqBatch(c.bt.to(DEV), 80, 11), vis, 30, 0.1)
        assert status == 0
        assert_close(out, lse, *oracle_decode(q, c.rows(0), c.rows(1), vis, [80], [11], [30], 0.1), KV8_WEIGHTS)
        bad = vis.copy()
        bad[:, :, [0, 7, 29]] = [-1, 80, 2 ** 31 - 1]
        out, lse, status = attend(c, q, sv.SeqBatch(c.bt.to(DEV), 80, 11), bad, 30, 0.1)
        assert status == sv.SV_DEV_BAD_INDEX
        good = [i for i in range(30) if i not in (0, 7, 29)]
        ref = oracle_decode(q, c.rows(0), c.rows(1), vis[:, :, good], [80], [11], [27], 0.1)
        assert_close(out, lse, *ref, KV8_WEIGHTS)
        bt = c.bt.clone()
        bt[0, 5] = -1                                       # positions 80 to 95: all the text
        out, lse, status = attend(c, q, sv.SeqBatch(bt.to(DEV), 80, 11), vis, 30, 0.1)
        assert status == sv.SV_DEV_BAD_BLOCK
        assert_close(out, lse, *oracle_decode(q, c.rows(0), c.rows(1), vis, [80], [0], [30], 0.1), KV8_WEIGHTS)
        out, lse, status = attend(c, q, sv.SeqBatch(torch.full_like(bt, -1).to(DEV), 80, 11), vis, 30, 0.1)
        assert (out == 0).all() and torch.isneginf(lse).all()


def test_values_that_are_not_finite(lib):
    """A NaN among the values that are attended makes that dim NaN, one among the
    keys the whole row."""
    from visual_token_sparsity_gb300 import binding as sv
    for H, d in ((1, 64), (8, 128)):
        c = Cache8(1, 1, d, 64, seed=76)
        q = synth.normal_bf16((1, H, d), 14).to(DEV)
        c.codes[1][0, 0, 20, 3] = 0x7F
        out, lse, _ = attend(c, q, sv.SeqBatch(c.bt.to(DEV), 64, 0), None, 0, 0.1)
        assert out[..., 3].isnan().all() and torch.isfinite(out[..., :3]).all() and torch.isfinite(lse).all()
        c.codes[0][0, 0, 33, 3] = 0x7F
        out, lse, _ = attend(c, q, sv.SeqBatch(c.bt.to(DEV), 64, 0), None, 0, 0.1)
        assert out.isnan().all() and lse.isnan().all()


# ------------------------------------------------------------------ together

@pytest.mark.parametrize("graph", [False, True])
@pytest.mark.parametrize("H,Hkv,d,lens,kept", [(4, 2, 64, [90, 33, 140], 0.4), (14, 2, 128, [200, 65], 0.25)])
def test_a_conversation(lib, H, Hkv, d, lens, kept, graph):
    """Prompts enter the cache while they attend to one another, then decode steps
    append, retrieve and attend: each call on what the others left."""
    from visual_token_sparsity_gb300 import binding as sv
    B, steps, scale = len(lens), 4, 1 / math.sqrt(d)
    nv = [int(n * 0.8) for n in lens]
    nt = [n - v for n, v in zip(lens, nv)]
    k = max(1, int(max(nv) * kept))
    ks = [min(k, max(1, int(n * kept))) for n in nv]
    c = Cache8(B, Hkv, d, max(lens) + steps, seed=80)
    layer = c.layer()
    N = sum(lens)
    ws = sv.workspace(max(sv.sv_prompt_attn_workspace_bytes(N, B, H, Hkv, d),
                          sv.sv_kv8_retrieve_workspace_bytes(B, H, Hkv, d, max(nv), k),
                          sv.sv_kv8_attn_workspace_bytes(B, H, Hkv, d, k + max(nt) + steps)))
    start = i32(np.concatenate([[0], np.cumsum(lens)]))
    pos = torch.cat([torch.arange(n, dtype=torch.int32) for n in lens])[None].to(DEV)
    rot, _ = rotation(d, 1, N, 400, 1, weights(d, 2), pos=pos)
    proj = synth.normal_bf16((N, H + 2 * Hkv, d), 81).to(DEV)
    q, ko = torch.empty(N, H, d, dtype=torch.bfloat16, device=DEV), torch.empty(N, Hkv, d, dtype=torch.bfloat16, device=DEV)
    out, lse = torch.empty_like(q), torch.empty(N, H, device=DEV)
    empty = sv.SeqBatch(c.bt.to(DEV), 0, 0)

    def prompt():
        sv.sv_kv8_append(proj[:, :H], proj[:, H: H + Hkv], proj[:, H + Hkv:], rot, layer, empty, q, ws, seq_start=start,
                         k_out=ko)
        sv.sv_prompt_attn(q, ko, proj[:, H + Hkv:], start, scale, out, lse, ws)

    # decode: the text lengths live on the device and grow there
    text_n, vis_n, sel_n = i32(nt), i32(nv), i32(ks)
    seqs = sv.SeqBatch(c.bt.to(DEV), max(nv), max(nt) + steps - 1, vis_n, text_n, sel_n)
    after = sv.SeqBatch(c.bt.to(DEV), max(nv), max(nt) + steps, vis_n, text_n, sel_n)
    dproj = synth.normal_bf16((steps, B, H + 2 * Hkv, d), 82).to(DEV)
    dpos = [i32([[n + s for n in lens]]) for s in range(steps)]
    drots = [rotation(d, 1, B, 400, 1, weights(d, 2), pos=p)[0] for p in dpos]
    dq, dk, dout = (torch.empty(steps, B, h, d, dtype=torch.bfloat16, device=DEV) for h in (H, Hkv, H))
    dlse = torch.empty(steps, B, H, device=DEV)
    dvis = torch.empty(steps, B, Hkv, k, dtype=torch.int32, device=DEV)

    def step(s):
        p = dproj[s]
        sv.sv_kv8_append(p[:, :H], p[:, H: H + Hkv], p[:, H + Hkv:], drots[s], layer, seqs, dq[s], ws, k_out=dk[s])
        text_n.add_(1)
        sv.sv_kv8_retrieve_topk(dq[s].unsqueeze(1), layer, after, k, dvis[s], None, ws)
        sv.sv_kv8_decode_attn(dq[s], scale, layer, after, dvis[s], k, dout[s], dlse[s], ws)

    def everything():
        prompt()
        for s in range(steps):
            step(s)
    if graph:
        g = torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(g):
            everything()
        for _ in range(2):
            text_n.copy_(i32(nt))
            g.replay()
    else:
        everything()
    torch.cuda.synchronize()
    assert sv.sv_read_device_status(ws) == 0

    # the prompt, from the rows that the append wrote
    ref = oracle.prompt_attention(f64(q), f64(ko), f64(proj[:, H + Hkv:]), start.tolist(), scale)
    assert_close(out, lse, *ref, PROMPT_WEIGHTS, "prompt")
    # the cache as the oracle fills it, and each decode step over its own state
    codes, scales = [x.copy() for x in c.codes], c.scales.copy()

    def fill(b, base, rows):
        for which in range(2):
            s = scales[b, ..., which].copy()
            oracle.kv8_append(codes[which][b], s, base, rows[which])
            scales[b, ..., which] = s
    st = start.tolist()
    for b in range(B):
        fill(b, 0, (f64(ko)[st[b]: st[b + 1]], f64(proj[st[b]: st[b + 1], H + Hkv:])))
    for s in range(steps):
        for b in range(B):
            fill(b, lens[b] + s, (f64(dk[s, b: b + 1]), f64(dproj[s, b: b + 1, H + Hkv:])))
        K, V = (np.stack([oracle.kv8_rows(codes[w][b], scales[b, ..., w]) for b in range(B)]) for w in range(2))
        want, _ = oracle_select(dq[s].unsqueeze(1), K, nv, ks)
        got = dvis[s].cpu().numpy()
        assert np.array_equal(got[..., : want.shape[2]], want) and (got[..., want.shape[2]:] == -1).all()
        ref = oracle_decode(dq[s], K, V, got, nv, [n + s + 1 for n in nt], ks, scale)
        assert_close(dout[s], dlse[s], *ref, KV8_WEIGHTS, f"step {s}")
    got, got_s = c.read_back(layer)
    assert np.array_equal(got_s.astype(np.float64), scales)
    assert np.array_equal(got[0], codes[0]) and np.array_equal(got[1], codes[1])


def test_programmatic_launch_on_another_stream(lib):
    """The calls one behind the other on a stream of their own, and twice over."""
    from visual_token_sparsity_gb300 import binding as sv
    c = Cache8(2, 2, 64, 400, seed=90)
    q = synth.normal_bf16((2, 1, 4, 64), 15).to(DEV)
    seqs = sv.SeqBatch(c.bt.to(DEV), 350, 50)
    layer = c.layer()
    ws = sv.workspace(max(sv.sv_kv8_retrieve_workspace_bytes(2, 4, 2, 64, 350, 90),
                          sv.sv_kv8_attn_workspace_bytes(2, 4, 2, 64, 140)))
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    runs = []
    for _ in range(20):
        vis = torch.empty(2, 2, 90, dtype=torch.int32, device=DEV)
        out, lse = torch.empty(2, 4, 64, dtype=torch.bfloat16, device=DEV), torch.empty(2, 4, device=DEV)
        torch.cuda.synchronize()
        sv.sv_kv8_retrieve_topk(q, layer, seqs, 90, vis, None, ws, stream=s)
        sv.sv_kv8_decode_attn(q[:, 0].contiguous(), 0.125, layer, seqs, vis, 90, out, lse, ws, stream=s)
        torch.cuda.synchronize()
        runs.append((vis, out, lse))
    for r in runs[1:]:
        assert all(torch.equal(x, y) for x, y in zip(r, runs[0]))
    assert np.array_equal(runs[0][0].cpu().numpy(), oracle_select(q, c.rows(0), [350] * 2, [90] * 2)[0])
