"""GPU: norm and rotation of new tokens, attention of a draft tree over the
paged cache, compaction of its accepted path, and a whole speculative step,
against the fp64 oracle."""

import math

import numpy as np
import pytest
import torch

import oracle
from draft_util import (DEV, Cache, assert_tree_close, f64, i32, mask64, oracle_tree, random_tree, select)
from visual_token_sparsity_gb300 import synth

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------------ norm and rotation

def rotation(rot, axes, B, T, n_pos, seed, weights=None, interleaved=False, sections=None):
    from visual_token_sparsity_gb300 import binding as sv
    g = torch.Generator().manual_seed(seed)
    cs = None
    if rot:
        a = torch.arange(n_pos).double()[:, None] * 10000.0 ** (-torch.arange(rot // 2).double() * 2 / rot)
        cs = torch.stack([a.cos(), a.sin()], -1).float().to(DEV)
    shape = (axes, B, T) if axes > 1 else (B, T)
    pos = torch.randint(0, n_pos, shape, generator=g, dtype=torch.int32).to(DEV)
    qw, kw = (None, None) if weights is None else weights
    r = sv.Rotation(cs, pos, sections=sections, interleaved=interleaved, q_weight=qw, k_weight=kw, eps=1e-5)
    ref = lambda x, w: oracle.norm_rope(f64(x), None if w is None else f64(w), 1e-5,
                                        None if cs is None else f64(cs), pos.cpu().numpy(), sections, interleaved)
    return r, ref


def assert_rows_close(got, ref, what):
    got = f64(got)
    if got.size == 0:
        return
    top = np.abs(ref).max(-1, keepdims=True)
    err = np.abs(got - ref) - 2.0 ** -8 * np.abs(ref) - 2.0 ** -20 * top
    assert (err <= 0).all(), f"{what}: {err.max()} over the bound"


def weights(d, seed):
    return tuple((1 + 0.2 * synth.normal_bf16((d,), seed + i).float()).to(torch.bfloat16).to(DEV) for i in range(2))


@pytest.mark.parametrize("d,rot_dim", [(128, 64), (80, 40), (72, 0)])
@pytest.mark.parametrize("inter", [False, True])
def test_elements_behind_the_rotation_stay(lib, d, rot_dim, inter):
    """Infinities and NaN behind rot_dim are passed on, each to its own place only."""
    from visual_token_sparsity_gb300 import binding as sv
    rot, ref = rotation(rot_dim, 1, 1, 9, 50, 4, None, inter)
    x = synth.normal_bf16((1, 9, 3, d), 5)
    x[0, :, :, rot_dim + 1::5] = float("inf")
    x[0, ::2, :, rot_dim + 3::7] = float("nan")
    x = x.to(DEV)
    qo, ko = (torch.empty(1, h, 9, d, dtype=torch.bfloat16, device=DEV) for h in (2, 1))
    sv.sv_qk_norm_rope(x[:, :, :2], x[:, :, 2:], rot, qo, ko, sv.workspace(256))
    torch.cuda.synchronize()
    got = torch.cat([qo, ko], 1).transpose(1, 2)
    assert torch.equal(got[..., rot_dim:].view(torch.int16), x[..., rot_dim:].view(torch.int16))
    clean = torch.where(torch.isfinite(x), x, torch.zeros_like(x))
    assert_rows_close(got[..., :rot_dim], ref(clean, None)[..., :rot_dim], "turned part")


@pytest.mark.parametrize("d,rot_dim,inter", [(128, 64, False), (72, 32, True), (80, 0, False)])
def test_an_infinity_behind_the_rotation_of_normed_rows(lib, d, rot_dim, inter):
    """It becomes NaN and the rest of its row 0, as in the formula."""
    from visual_token_sparsity_gb300 import binding as sv
    rot, ref = rotation(rot_dim, 1, 1, 6, 50, 4, weights(d, 2), inter)
    x = synth.normal_bf16((1, 6, 2, d), 8)
    x[0, :3, :, rot_dim + 6] = float("-inf")
    x = x.to(DEV)
    qo, ko = (torch.empty(1, 1, 6, d, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    sv.sv_qk_norm_rope(x[:, :, :1], x[:, :, 1:], rot, qo, ko, sv.workspace(256))
    torch.cuda.synchronize()
    for got in (qo[0, 0], ko[0, 0]):
        assert got[:3, rot_dim + 6].isnan().all()
        rest = torch.cat([got[:3, :rot_dim + 6], got[:3, rot_dim + 7:]], 1)
        assert (rest == 0).all()
        assert got[3:].isfinite().all()


@pytest.mark.parametrize("d,H,Hk,B,N,axes,sections,inter,norm", [
    (80, 16, 16, 1, 37, 2, [20, 20], False, False),
    (72, 5, 5, 2, 19, 1, None, True, True),
    (72, 3, 1, 1, 1, 1, None, False, True),
    (64, 4, 2, 3, 33, 3, [8, 0, 24], False, True),
    (128, 7, 2, 2, 65, 3, [16, 24, 24], True, True),
    (128, 1, 1, 1, 5, 1, None, False, False),
])
def test_encoder_operands(lib, d, H, Hk, B, N, axes, sections, inter, norm):
    from visual_token_sparsity_gb300 import binding as sv
    w = weights(d, 3) if norm else None
    rot, ref = rotation(d, axes, B, N, 200, 5, w, inter, sections)
    proj = synth.normal_bf16((B, N, H + Hk, d), 7).to(DEV)
    q, k = proj[:, :, :H], proj[:, :, H:]
    qo = torch.full((B, H, N, d), 9.0, dtype=torch.bfloat16, device=DEV)
    ko = torch.full((B, Hk, N, d), 9.0, dtype=torch.bfloat16, device=DEV)
    ws = sv.workspace(256)
    sv.sv_qk_norm_rope(q, k, rot, qo, ko, ws)
    assert sv.sv_read_device_status(ws) == 0
    assert_rows_close(qo.transpose(1, 2), ref(q, w and w[0]), "q")
    assert_rows_close(ko.transpose(1, 2), ref(k, w and w[1]), "k")


def test_encoder_feeds_the_salience(lib):
    """The operands go straight into sv_salience_prefill."""
    from visual_token_sparsity_gb300 import binding as sv
    from parity_util import assert_salience_close
    B, N, H, d = 2, 300, 4, 80
    rot, _ = rotation(d, 2, B, N, 64, 11, weights(d, 1), sections=[20, 20])
    proj = synth.normal_bf16((B, N, 2 * H, d), 12).to(DEV)
    qo, ko = (torch.empty(B, H, N, d, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    sv.sv_qk_norm_rope(proj[:, :, :H], proj[:, :, H:], rot, qo, ko, sv.workspace(256))
    sal = torch.empty(B, N, device=DEV)
    sv.sv_salience_prefill(qo, ko, 1 / math.sqrt(d), sal, sv.workspace(sv.sv_salience_workspace_bytes(B, H, N, d)))
    assert_salience_close(f64(sal), oracle.salience(f64(qo), f64(ko)))


def test_rotation_outside_the_table_skips_the_token(lib):
    from visual_token_sparsity_gb300 import binding as sv
    rot, ref = rotation(64, 1, 1, 4, 10, 1)
    rot.pos[0, 1], rot.pos[0, 3] = 10, -1
    q = synth.normal_bf16((1, 4, 2, 64), 1).to(DEV)
    qo, ko = (torch.full((1, 2, 4, 64), 5.0, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    ws = sv.workspace(256)
    sv.sv_qk_norm_rope(q, q.clone(), rot, qo, ko, ws)
    assert sv.sv_read_device_status(ws) == sv.SV_DEV_BAD_POSITION
    assert (qo[:, :, [1, 3]] == 5).all() and (ko[:, :, [1, 3]] == 5).all()
    assert not (qo[:, :, [0, 2]] == 5).all()


@pytest.mark.parametrize("H,Hkv,d,rot,B,T,axes,sections,inter,norm,ragged", [
    (28, 4, 128, 128, 3, 1, 3, [16, 24, 24], False, True, False),
    (28, 4, 128, 128, 2, 21, 3, [16, 24, 24], False, True, True),
    (4, 2, 64, 32, 1, 33, 1, None, False, False, False),
    (8, 8, 64, 64, 2, 7, 1, None, True, True, True),
    (1, 1, 128, 0, 2, 17, 1, None, False, True, False),
])
def test_append(lib, H, Hkv, d, rot, B, T, axes, sections, inter, norm, ragged):
    from visual_token_sparsity_gb300 import binding as sv
    nv, nt = [30 - 7 * b for b in range(B)], [9 + 4 * b for b in range(B)]
    tn = [max(0, T - 3 * b) if ragged else T for b in range(B)]
    if not ragged:
        nv, nt = [30] * B, [9] * B
    c = Cache(B, Hkv, d, 30 + max(nt) + T, seed=H + T)
    kp, vp = c.pools()
    w = weights(d, 3) if norm else None
    r, ref = rotation(rot, axes, B, T, 100, 5, w, inter, sections)
    proj = synth.normal_bf16((B, T, H + 2 * Hkv, d), 7).to(DEV)
    q, k, v = proj[:, :, :H], proj[:, :, H:H + Hkv], proj[:, :, H + Hkv:]
    out = torch.full((B, T, H, d), 9.0, dtype=torch.bfloat16, device=DEV)
    seqs = sv.SeqBatch(c.bt.to(DEV), 30, max(nt), *((i32(nv), i32(nt)) if ragged else ()))
    ws = sv.workspace(256)
    before_k, before_v = kp.clone(), vp.clone()
    sv.sv_qk_norm_rope_append(q, k, v, r, sv.KvLayer(kp, vp), seqs, out, ws, n_new=i32(tn) if ragged else None)
    assert sv.sv_read_device_status(ws) == 0
    q_ref, k_ref = ref(q, w and w[0]), ref(k, w and w[1])
    touched = torch.zeros(kp.shape[0], 16, dtype=torch.bool)
    for b in range(B):
        assert_rows_close(out[b, :tn[b]], q_ref[b, :tn[b]], "q")
        assert (out[b, tn[b]:] == 9).all()
        for t in range(tn[b]):
            page, slot = int(c.bt[b, (nv[b] + nt[b] + t) // 16]), (nv[b] + nt[b] + t) % 16
            touched[page, slot] = True
            assert_rows_close(kp[page, :, slot], k_ref[b, t], "k")
            assert torch.equal(vp[page, :, slot], v[b, t])
    rest = ~touched.to(DEV)
    assert torch.equal(kp.transpose(1, 2)[rest], before_k.transpose(1, 2)[rest])
    assert torch.equal(vp.transpose(1, 2)[rest], before_v.transpose(1, 2)[rest])


@pytest.mark.parametrize("d,inter,norm", [(128, False, True), (64, True, True), (128, True, False)])
def test_appended_rows_are_rounded_as_from_64_bits(lib, d, inter, norm):
    """fp32 is off by 0.6 to 1.6 (rms) of the last bit of a pair's larger member,
    which leaves one in 80 000 on the other side of a bf16 rounding boundary, five
    of this test's.  Results within four last bits are looked at twice: beyond
    2.5 to 6 times the error, of which less than one in 100 is left, none of five.  A
    pair's smaller member has larger errors for its size; of all, fp32 alone
    leaves one in 40 000."""
    from visual_token_sparsity_gb300 import binding as sv
    B, T, H, Hkv = 2, 120, 28, 4
    w = weights(d, 6) if norm else None
    rot, ref = rotation(d, 1, B, T, 3000, 5, w, inter)
    x = [synth.normal_bf16((B, T, h, d), 40 + i).to(DEV) for i, h in enumerate((H, Hkv, Hkv))]
    cache = Cache(B, Hkv, d, T, seed=2)
    q = torch.empty(B, T, H, d, dtype=torch.bfloat16, device=DEV)
    sv.sv_qk_norm_rope_append(*x, rot, cache.layer(), sv.SeqBatch(cache.bt.to(DEV), 0, 0), q, sv.workspace(256))
    torch.cuda.synchronize()
    exact = torch.from_numpy(ref(x[0], w and w[0]))
    pair = exact.view(B, T, H, d // 2, 2) if inter else exact.view(B, T, H, 2, d // 2).transpose(-1, -2)
    large = pair.abs() == pair.abs().amax(-1, keepdim=True)
    got = q.cpu().view(B, T, H, d // 2, 2) if inter else q.cpu().view(B, T, H, 2, d // 2).transpose(-1, -2)
    differ = got != pair.float().to(torch.bfloat16)
    assert int((differ & large).sum()) == 0
    assert int(differ.sum()) <= 5e-5 * differ.numel()


def test_append_without_norm_or_rotation_is_the_plain_append(lib):
    from visual_token_sparsity_gb300 import binding as sv
    c = Cache(2, 4, 128, 70, seed=4)
    pools = [c.pools() for _ in range(2)]
    q, k, v = (synth.normal_bf16((2, 5, h, 128), 6 + i).to(DEV) for i, h in enumerate((8, 4, 4)))
    seqs = sv.SeqBatch(c.bt.to(DEV), 40, 20)
    out = torch.empty_like(q)
    sv.sv_qk_norm_rope_append(q, k, v, sv.Rotation(None, None), sv.KvLayer(*pools[0]), seqs, out, sv.workspace(256))
    sv.sv_kv_append(sv.KvLayer(*pools[1]), seqs, k, v, sv.workspace(256))
    assert torch.equal(out, q)
    assert torch.equal(pools[0][0], pools[1][0]) and torch.equal(pools[0][1], pools[1][1])
    # in place
    keep = q.clone()
    sv.sv_qk_norm_rope_append(q, k, v, sv.Rotation(None, None), sv.KvLayer(*pools[0]), seqs, q, sv.workspace(256))
    assert torch.equal(q, keep)


def test_append_reports_bad_pages_and_lengths(lib):
    from visual_token_sparsity_gb300 import binding as sv
    c = Cache(3, 2, 64, 40, seed=8)
    kp, vp = c.pools()
    keep = kp.clone()
    bt = c.bt.clone()
    bt[0, 1] = c.blocks                               # the page of sequence 0's new tokens
    rot, ref = rotation(64, 1, 3, 4, 50, 2)
    q, k, v = (synth.normal_bf16((3, 4, 2, 64), 6 + i).to(DEV) for i in range(3))
    out = torch.full_like(q, 9.0)
    ws = sv.workspace(256)
    sv.sv_qk_norm_rope_append(q, k, v, rot, sv.KvLayer(kp, vp), sv.SeqBatch(bt.to(DEV), 12, 6), out, ws,
                              n_new=i32([4, 5, -1]))
    assert sv.sv_read_device_status(ws) == sv.SV_DEV_BAD_BLOCK | sv.SV_DEV_BAD_LENGTH
    assert torch.equal(kp, keep)
    assert_rows_close(out[0], ref(q, None)[0], "q")   # the queries do not need the page
    assert (out[1:] == 9).all()


# ------------------------------------------------------------------ tree attention

def run_tree(cache, q, vis, k, nv, nt, ks, tn, mask, scale, layer=None, want_lse=True, bt=None, cap=None, out=None,
             stream=None):
    """One call; per-sequence arrays whenever the sequences differ."""
    from visual_token_sparsity_gb300 import binding as sv
    B, T, H, d = q.shape
    Hkv = cache.K.shape[1]
    cap_v, cap_t = cap or (max(nv), max(nt))
    ragged = cap is not None or len(set(zip(nv, nt, ks))) > 1
    lens = (i32(nv), i32(nt), i32(ks) if vis is not None else None) if ragged else ()
    seqs = sv.SeqBatch((cache.bt if bt is None else bt).to(DEV), cap_v, cap_t, *lens)
    n_new = None if all(t == T for t in tn) else i32(tn)
    out = torch.full((B, T, H, d), 7.0, dtype=torch.bfloat16, device=DEV) if out is None else out
    lse = torch.full((B, T, H), 7.0, device=DEV) if want_lse else None
    ws = sv.workspace(sv.sv_tree_attn_workspace_bytes(B, T, H, Hkv, d, (k if vis is not None else cap_v) + cap_t + T))
    sv.sv_tree_attn(q.to(DEV), scale, layer or cache.layer(), seqs, None if vis is None else i32(vis), k,
                    None if mask is None else mask64(mask), out, lse, ws, n_new=n_new, stream=stream)
    torch.cuda.synchronize()
    return out, lse, sv.sv_read_device_status(ws)


def check_tree(H, Hkv, d, B, T, n_vis, k, n_text, kind, seed=0, std=1.0, scale=None, ragged=False):
    g = np.random.default_rng(seed + H + T + n_vis)
    nv, nt, ks, tn = [n_vis] * B, [n_text] * B, [k or 0] * B, [T] * B
    if ragged:
        nv = [int(g.integers(0, n_vis + 1)) for _ in range(B)]
        nt = [int(g.integers(0, n_text + 1)) for _ in range(B)]
        ks = [int(g.integers(0, min(k or 0, v) + 1)) for v in nv]
        tn = [int(g.integers(0, T + 1)) for _ in range(B)]
        nv[0], nt[0], tn[-1] = n_vis, n_text, T
    cache = Cache(B, Hkv, d, n_vis + n_text + T, seed=seed + T, std=std)
    q = synth.normal_bf16((B, T, H, d), seed + 9)
    vis = None if k is None else select(B, Hkv, nv, ks, k, seed)
    mask = {"chain": None, "tree": [random_tree(T, g) for _ in range(B)],
            "any": [[int(x) for x in g.integers(0, 1 << 63, T, dtype=np.uint64) * np.uint64(2)] for _ in range(B)]}[kind]
    scale = 1 / math.sqrt(d) if scale is None else scale
    out, lse, status = run_tree(cache, q, vis, k or 0, nv, nt, ks, tn, mask, scale,
                                cap=(n_vis, n_text) if ragged else None)
    assert status == 0
    ref = oracle_tree(q, cache, vis, nv, nt, ks, tn, mask, scale)
    for b in range(B):
        n = tn[b]
        assert_tree_close(out[b, :n], lse[b, :n], *(r[b, :n] for r in ref), what=f"sequence {b}")
        assert (out[b, n:] == 7).all() and (lse[b, n:] == 7).all()


@pytest.mark.parametrize("H,Hkv,d,B,T,n_vis,k,n_text,kind", [
    (4, 2, 64, 1, 5, 576, 144, 57, "tree"),        # the round-loop shape
    (4, 2, 64, 2, 1, 100, 30, 3, "tree"),          # one drafted token
    (8, 8, 128, 2, 16, 300, 150, 20, "tree"),      # equal heads
    (28, 4, 128, 2, 27, 400, 100, 31, "tree"),     # 189 rows per KV head
    (28, 4, 128, 1, 64, 700, 175, 0, "tree"),      # the widest mask, no text
    (16, 1, 64, 1, 64, 300, 100, 11, "any"),       # 1024 rows per KV head, arbitrary masks
    (14, 2, 64, 2, 18, 0, None, 110, "tree"),      # text only: 126 rows, 128 tokens
    (14, 2, 128, 1, 19, 0, None, 108, "any"),      # 133 rows, 127 tokens
    (2, 2, 128, 3, 9, 120, None, 0, "tree"),       # 129 tokens
    (2, 1, 64, 1, 3, 0, None, 0, "any"),           # rows that may see nothing
    (7, 1, 128, 1, 37, 250, 1, 0, "chain"),        # two row tiles by a few rows
    (6, 3, 64, 2, 193, 90, None, 17, "chain"),     # a question's rows
    (7, 1, 128, 1, 300, 40, 20, 5, "chain"),       # many row tiles, more drafted than cached
    (1, 1, 64, 1, 1, 1, 1, 0, "chain"),
])
def test_tree_attention(lib, H, Hkv, d, B, T, n_vis, k, n_text, kind):
    check_tree(H, Hkv, d, B, T, n_vis, k, n_text, kind)


@pytest.mark.parametrize("H,Hkv,d,T,kind", [(8, 4, 64, 12, "tree"), (28, 4, 128, 33, "any"), (7, 1, 64, 70, "chain")])
@pytest.mark.parametrize("k", [60, None])
def test_tree_attention_with_per_sequence_lengths(lib, H, Hkv, d, T, kind, k):
    check_tree(H, Hkv, d, 5, T, 150, k, 40, kind, seed=3, ragged=True)


def test_tree_attention_of_many_short_sequences(lib):
    """More sequences than a warp's lanes, some without a token."""
    check_tree(2, 1, 64, 75, 4, 40, 10, 9, "tree", seed=8, ragged=True)


@pytest.mark.parametrize("H,Hkv,d,B,T,n_text", [(14, 2, 128, 80, 18, 108), (28, 4, 128, 40, 9, 50), (32, 32, 64, 12, 20, 90)])
def test_tree_attention_of_units_of_one_tile(lib, H, Hkv, d, B, T, n_text):
    """Several (sequence, KV head) units per CTA, each with a tile for one of
    its two streams only."""
    for seed in range(3):
        check_tree(H, Hkv, d, B, T, 0, None, n_text, "tree", seed=seed)


def test_more_row_tiles_than_a_gpu_has_places(lib):
    check_tree(16, 1, 64, 1, 2450, 30, 20, 3, "chain")


def test_a_batch_of_70000_sequences(lib):
    """Reserve, append, attend and accept with one token of context each."""
    from visual_token_sparsity_gb300 import binding as sv
    B, T, d = 70000, 2, 64
    kp, vp = (torch.zeros(B, 1, 16, d, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    layer = sv.KvLayer(kp, vp)
    table = torch.full((B, 1), -1, dtype=torch.int32, device=DEV)
    pool = sv.PagePool(torch.zeros(B, dtype=torch.int32, device=DEV), torch.zeros(B, dtype=torch.int32, device=DEV))
    seqs = sv.SeqBatch(table, 0, 0)
    ws = sv.workspace(max(sv.sv_pages_workspace_bytes(B, 1, B), sv.sv_tree_attn_workspace_bytes(B, T, 1, 1, d, T)))
    sv.sv_pages_reserve(pool, [layer], seqs, T, ws)
    x = synth.normal_bf16((3, B, T, 1, d), 4).to(DEV)
    q, out = torch.empty_like(x[0]), torch.empty_like(x[0])
    sv.sv_qk_norm_rope_append(x[0], x[1], x[2], sv.Rotation(None, None), layer, seqs, q, ws)
    # token 0 sees itself, token 1 only itself
    mask = torch.tensor([1, 2], dtype=torch.int64, device=DEV).repeat(B, 1)
    sv.sv_tree_attn(q, 0.125, layer, seqs, None, 0, mask, out, None, ws)
    path = torch.ones(B, 1, dtype=torch.int32, device=DEV)
    sv.sv_kv_accept([layer], seqs, T, path, ws)
    torch.cuda.synchronize()
    assert sv.sv_read_device_status(ws) == 0
    assert torch.equal(table[:, 0], torch.arange(B, dtype=torch.int32, device=DEV))
    assert torch.equal(q, x[0]) and torch.equal(out, x[2])
    assert torch.equal(kp[:, 0, 0], x[1][:, 1, 0]) and torch.equal(vp[:, 0, 0], x[2][:, 1, 0])


@pytest.mark.parametrize("std,scale", [(4.0, 0.5), (16.0, 0.7), (1.0, 0.0)])
def test_tree_attention_with_peaked_and_flat_weights(lib, std, scale):
    check_tree(8, 2, 128, 1, 20, 500, 250, 30, "tree", seed=5, std=std, scale=scale)


def test_tree_attention_with_growing_logits(lib):
    """Every tile's maximum is far above the last one's."""
    c = Cache(1, 2, 64, 1200, seed=21, std=0.1)
    ramp = torch.arange(c.K.shape[2]).float()[None, None, :, None] / 40
    for sign in (1, -1):
        c.K = (c.K.float() * 0.1 + sign * ramp / 8).to(torch.bfloat16)
        q = (1 + 0.05 * synth.normal_bf16((1, 20, 4, 64), 3).float()).to(torch.bfloat16)
        out, lse, status = run_tree(c, q, None, 0, [1100], [40], [0], [20], None, 0.5)
        ref = oracle_tree(q, c, None, [1100], [40], [0], [20], None, 0.5)
        assert status == 0
        assert_tree_close(out, lse, *ref)


def test_tree_rows_without_any_token(lib):
    c = Cache(2, 2, 64, 40, seed=2)
    q = synth.normal_bf16((2, 6, 4, 64), 3)
    mask = [[0, 2, 0, 8, 0, 63], [0] * 6]
    out, lse, status = run_tree(c, q, None, 0, [0, 0], [0, 0], [0, 0], [6, 6], mask, 0.125)
    assert status == 0
    assert (out[1] == 0).all() and torch.isneginf(lse[1]).all()
    assert (out[0, [0, 2, 4]] == 0).all() and torch.isneginf(lse[0, [0, 2, 4]]).all()
    assert_tree_close(out, lse, *oracle_tree(q, c, None, [0, 0], [0, 0], [0, 0], [6, 6], mask, 0.125))


@pytest.mark.parametrize("bad", [math.inf, -math.inf, math.nan])
@pytest.mark.parametrize("H,Hkv,T", [(4, 2, 7), (28, 4, 40)])
def test_hidden_tokens_have_no_part_whatever_they_hold(lib, bad, H, Hkv, T):
    """A drafted token's infinities and NaN reach the rows that see it and no
    others; what lies behind the last token reaches none."""
    d, n_vis, n_text = 64, 130, 10
    c = Cache(1, Hkv, d, n_vis + n_text + T, seed=31)
    q = synth.normal_bf16((1, T, H, d), 4)
    mask = [[(1 << t) | (1 if t % 3 == 0 else 0) for t in range(T)]]     # token 0: seen by every third
    clean = oracle_tree(q, c, None, [n_vis], [n_text], [0], [T], mask, 0.125)
    n = n_vis + n_text
    for which in (c.K, c.V):
        keep = which.clone()
        which[0, :, n, 5] = bad
        which[0, :, n + T:] = bad                       # behind the last token
        out, lse, status = run_tree(c, q, None, 0, [n_vis], [n_text], [0], [T], mask, 0.125)
        which.copy_(keep)
        assert status == 0
        blind = [t for t in range(T) if not mask[0][t] & 1]
        assert_tree_close(out[:, blind], lse[:, blind], *(x[:, blind] for x in clean))
        if which is c.V:
            seeing = [t for t in range(T) if mask[0][t] & 1]
            hit = f64(out[:, seeing][..., 5])
            assert np.isnan(hit).all() if math.isnan(bad) else (hit == bad).all()
            other = [e for e in range(d) if e != 5]
            assert_tree_close(out[..., other], None, clean[0][..., other], None, clean[2][..., other])


def test_tree_attention_reports_and_skips_bad_pages_and_indices(lib):
    from visual_token_sparsity_gb300 import binding as sv
    B, H, Hkv, d, T, n_vis, k, n_text = 2, 8, 4, 64, 9, 200, 60, 30
    c = Cache(B, Hkv, d, n_vis + n_text + T, seed=41)
    q = synth.normal_bf16((B, T, H, d), 5)
    vis = select(B, Hkv, [n_vis] * B, [k] * B, k, 6)
    mask = [random_tree(T, np.random.default_rng(b)) for b in range(B)]
    args = (k, [n_vis] * B, [n_text] * B, [k] * B, [T] * B, mask, 0.125)
    # indices outside the visual tokens: as if the list were shorter
    bad = vis.copy()
    bad[0, 1, 5], bad[0, 1, 6] = n_vis, -1
    out, lse, status = run_tree(c, q, bad, *args)
    assert status == sv.SV_DEV_BAD_INDEX
    ref = oracle_tree(q, c, vis, *args[1:])
    short = oracle.tree_attention(f64(q[0]), f64(c.K[0]), f64(c.V[0]), [np.delete(v, [5, 6]) for v in vis[0]],
                                  n_vis, n_text, mask[0], 0.125)
    G = H // Hkv
    for x, y in zip(ref, short):
        x[0][:, G:2 * G] = y[:, G:2 * G]
    assert_tree_close(out, lse, *ref)
    # a page outside the pool
    bt = c.bt.clone()
    bt[1, 2] = -5
    out, lse, status = run_tree(c, q, vis, *args, bt=bt)
    assert status == sv.SV_DEV_BAD_BLOCK
    gone = oracle.tree_attention(f64(q[1]), f64(c.K[1]), f64(c.V[1]), [v[(v < 32) | (v >= 48)] for v in vis[1]],
                                 n_vis, n_text, mask[1], 0.125)
    assert_tree_close(out[1], lse[1], *gone)
    # lengths out of range: the sequence reads as empty
    out, lse, status = run_tree(c, q, vis, k, [n_vis, n_vis + 1], [n_text] * 2, [k] * 2, [T] * B, mask, 0.125,
                                cap=(n_vis, n_text))
    assert status == sv.SV_DEV_BAD_LENGTH
    assert (out[1] == 0).all() and torch.isneginf(lse[1]).all() and (out[0] != 0).any()
    out, lse, status = run_tree(c, q, vis, k, [n_vis] * 2, [n_text] * 2, [k] * 2, [T + 1, T], mask, 0.125)
    assert status == sv.SV_DEV_BAD_LENGTH
    assert (out[0] == 0).all() and torch.isneginf(lse[0]).all() and (out[1] != 0).any()


def test_tree_attention_in_place_and_without_lse(lib):
    c = Cache(1, 2, 64, 300, seed=51)
    q = synth.normal_bf16((1, 11, 4, 64), 5)
    args = (None, 0, [250], [20], [0], [11], None, 0.125)
    a, _, _ = run_tree(c, q, *args)
    buf = q.to(DEV)
    b, _, _ = run_tree(c, buf, *args, want_lse=False, out=buf)
    assert torch.equal(a, b)


def test_tree_attention_with_an_empty_list(lib):
    """k = 0 with a list is text alone, not every visual token."""
    c = Cache(1, 2, 64, 200, seed=91)
    q = synth.normal_bf16((1, 5, 4, 64), 5)
    args = (0, [150], [30], [0], [5], None, 0.125)
    out, lse, status = run_tree(c, q, np.zeros((1, 2, 0), np.int32), *args)
    assert status == 0
    assert_tree_close(out, lse, *oracle_tree(q, c, np.zeros((1, 2, 0), int), *args[1:]))


def test_calls_share_a_workspace_with_the_decode_attention(lib):
    """In one workspace, between tree attention and page calls, the decode
    attention finds its counters as it left them."""
    from visual_token_sparsity_gb300 import binding as sv
    B, H, Hkv, d, T, n_vis, n_text = 3, 8, 8, 64, 30, 700, 40
    c = Cache(B, Hkv, d, n_vis + n_text + T, seed=95)
    layer, bt = c.layer(), c.bt.to(DEV)
    seqs, after = sv.SeqBatch(bt, n_vis, n_text), sv.SeqBatch(bt, n_vis, n_text + T)
    pool = sv.PagePool(torch.ones(c.blocks, dtype=torch.int32, device=DEV), i32([c.per] * B))
    n = n_vis + n_text + T
    ws = sv.workspace(max(sv.sv_tree_attn_workspace_bytes(B, T, H, Hkv, d, n),
                          sv.sv_attn_workspace_bytes(B, H, Hkv, d, n),
                          sv.sv_pages_workspace_bytes(B, c.per, c.blocks)))
    q = synth.normal_bf16((B, T, H, d), 5).to(DEV)
    q1 = q[:, -1].contiguous()
    outs = []
    for _ in range(3):
        out, one = torch.empty_like(q), torch.empty_like(q1)
        sv.sv_tree_attn(q, 0.125, layer, seqs, None, 0, None, out, None, ws)
        sv.sv_pages_reserve(pool, [layer], seqs, T, ws)
        sv.sv_sparse_decode_attn(q1, 0.125, layer, after, None, 0, one, None, ws)
        outs.append((out, one))
    assert sv.sv_read_device_status(ws) == 0
    for out, one in outs:
        assert torch.equal(out, outs[0][0]) and torch.equal(one, outs[0][1])
        # the last drafted token of a chain attends to what the decode token does
        assert (out[:, -1].float() - one.float()).abs().max() <= 0.02


def test_binding_refuses_what_the_kernels_could_not_read(lib):
    from visual_token_sparsity_gb300 import binding as sv
    c = Cache(2, 2, 64, 60, seed=3)
    layer, seqs = c.layer(), sv.SeqBatch(c.bt.to(DEV), 20, 10)
    q = synth.normal_bf16((2, 4, 4, 64), 5).to(DEV)
    out, ws = torch.empty_like(q), sv.workspace(sv.sv_tree_attn_workspace_bytes(2, 4, 4, 2, 64, 34))
    good = dict(q=q, scale=0.1, layer=layer, seqs=seqs, vis_idx=None, k=0, tree_mask=None, out=out, lse=None, ws=ws)
    sv.sv_tree_attn(**good)
    for change in (dict(q=q.float()), dict(q=q.cpu()), dict(q=q[:1]), dict(out=out[:, :3]), dict(ws=ws.cpu()),
                   dict(q=q.transpose(1, 2).contiguous().transpose(1, 2)), dict(lse=out),
                   dict(tree_mask=torch.zeros(2, 4, dtype=torch.int32, device=DEV)),
                   dict(tree_mask=torch.zeros(2, 3, dtype=torch.int64, device=DEV)),
                   dict(vis_idx=i32(np.zeros((2, 2, 5))), k=4), dict(n_new=i32([1, 2, 3]))):
        with pytest.raises(ValueError):
            sv.sv_tree_attn(**{**good, **change})
    rot = sv.Rotation(None, None)
    k = synth.normal_bf16((2, 4, 2, 64), 6).to(DEV)
    with pytest.raises(ValueError, match="evenly"):
        sv.sv_qk_norm_rope_append(q, k.transpose(0, 1).contiguous().transpose(0, 1), k, rot, layer, seqs, out, ws)
    with pytest.raises(ValueError, match="tokens"):
        cs = torch.zeros(9, 32, 2, device=DEV)
        sv.sv_qk_norm_rope_append(q, k, k, sv.Rotation(cs, i32(np.zeros((2, 3)))), layer, seqs, out, ws)
    with pytest.raises(sv.SvError, match="overflow"):
        sv.sv_tree_attn(**{**good, "seqs": sv.SeqBatch(c.bt.to(DEV), 20, 41)})
    with pytest.raises(sv.SvError) as e:
        sv.sv_tree_attn(**{**good, "ws": ws[:128]})
    assert e.value.status == 4


def test_tree_attention_is_deterministic_on_streams_and_in_graphs(lib):
    """The same bits eager, on another stream, and captured; two graphs over
    one workspace replay in turn."""
    from visual_token_sparsity_gb300 import binding as sv
    B, H, Hkv, d, T, n_vis, n_text = 2, 28, 4, 128, 20, 1500, 60
    c = Cache(B, Hkv, d, n_vis + n_text + T, seed=61)
    layer = c.layer()
    seqs = sv.SeqBatch(c.bt.to(DEV), n_vis, n_text)
    qs = [synth.normal_bf16((B, T, H, d), s).to(DEV) for s in (1, 2)]
    mask = mask64([random_tree(T, np.random.default_rng(b)) for b in range(B)])
    ws = sv.workspace(sv.sv_tree_attn_workspace_bytes(B, T, H, Hkv, d, n_vis + n_text + T))
    outs = [torch.empty_like(q) for q in qs]
    lses = [torch.empty(B, T, H, device=DEV) for _ in qs]
    call = lambda i: sv.sv_tree_attn(qs[i], 0.1, layer, seqs, None, 0, mask, outs[i], lses[i], ws)
    eager = []
    for i in range(2):
        call(i)
        torch.cuda.synchronize()
        eager.append((outs[i].clone(), lses[i].clone()))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graphs = []
    for i in range(2):
        outs[i].zero_()
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            call(i)
        side.synchronize()
        assert torch.equal(outs[i], eager[i][0]) and torch.equal(lses[i], eager[i][1])
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            call(i)
        graphs.append(g)
    for _ in range(3):
        for i in range(2):
            outs[i].zero_()
            graphs[i].replay()
        torch.cuda.synchronize()
        for i in range(2):
            assert torch.equal(outs[i], eager[i][0]) and torch.equal(lses[i], eager[i][1])
    assert sv.sv_read_device_status(ws) == 0


def test_offsets_beyond_32_bits(lib):
    """A pool of more than 2^32 bytes and elements, read and written near its
    end."""
    from visual_token_sparsity_gb300 import binding as sv
    Hkv, d, T, n = 32, 128, 6, 90
    blocks = 70000                                        # 4.6e9 elements per pool
    c = Cache(1, Hkv, d, n + T, seed=71)
    kp, vp = (torch.empty(blocks, Hkv, 16, d, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    small_k, small_v = c.pools()
    ids = torch.randperm(500)[: c.per] + blocks - 500
    kp[ids.to(DEV)] = small_k[c.bt[0].long().to(DEV)]
    vp[ids.to(DEV)] = small_v[c.bt[0].long().to(DEV)]
    layer = sv.KvLayer(kp, vp)
    q = synth.normal_bf16((1, T, Hkv, d), 6)
    out, lse, status = run_tree(c, q, None, 0, [60], [30], [0], [T], None, 0.1, layer=layer, bt=ids.int()[None])
    assert status == 0
    assert_tree_close(out, lse, *oracle_tree(q, c, None, [60], [30], [0], [T], None, 0.1))
    seqs = sv.SeqBatch(ids.int()[None].contiguous().to(DEV), 60, 30)
    ws = sv.workspace(256)
    new = synth.normal_bf16((1, T, Hkv, d), 8).to(DEV)
    sv.sv_qk_norm_rope_append(new, new, new, sv.Rotation(None, None), layer, seqs, torch.empty_like(new), ws)
    sv.sv_kv_accept([layer], seqs, T, i32([[1, 4]]), ws)
    for i, t in ((0, 1), (1, 4)):
        page, slot = int(ids[(n + i) // 16]), (n + i) % 16
        assert torch.equal(kp[page, :, slot], new[0, t]) and torch.equal(vp[page, :, slot], new[0, t])
    assert sv.sv_read_device_status(ws) == 0
    # a private copy of a page at the far end
    ref = torch.ones(blocks, dtype=torch.int32, device=DEV)
    ref[int(ids[5])], ref[blocks - 501] = 2, 0
    pool = sv.PagePool(ref, i32([c.per]))
    wp = sv.workspace(sv.sv_pages_workspace_bytes(1, c.per, blocks))
    last = int(ids[5])
    sv.sv_pages_reserve(pool, [layer], seqs, T, wp)
    assert sv.sv_read_device_status(wp) == 0 and int(seqs.block_table[0, 5]) == blocks - 501
    assert torch.equal(kp[blocks - 501], kp[last]) and torch.equal(vp[blocks - 501], vp[last])


def test_tree_lse_serves_the_softmax_retrieval(lib):
    """A question's chain attention gives the lse that the softmax-normalised
    retrieval takes: scores as the oracle's with that normaliser."""
    from visual_token_sparsity_gb300 import binding as sv
    from parity_util import assert_softmax_scores_close
    B, H, Hkv, d, R, n_vis, n_text, k = 1, 8, 4, 64, 12, 300, 20, 50
    c = Cache(B, Hkv, d, n_vis + n_text + R, seed=81)
    q = synth.normal_bf16((B, R, H, d), 7)
    scale = 1 / math.sqrt(d)
    _, lse, _ = run_tree(c, q, None, 0, [n_vis], [n_text], [0], [R], None, scale)
    vis = torch.empty(B, Hkv, k, dtype=torch.int32, device=DEV)
    sc = torch.empty(B, Hkv, n_vis, device=DEV)
    ws = sv.workspace(sv.sv_retrieve_softmax_workspace_bytes(B, R, H, Hkv, d, n_vis, n_text))
    sv.sv_retrieve_topk_softmax(q.to(DEV), scale, c.layer(), sv.SeqBatch(c.bt.to(DEV), n_vis, n_text), k, vis, sc, ws,
                                lse=lse)
    ref = oracle.retrieval_scores_softmax(f64(q), f64(c.K), n_vis, n_text, scale=scale, lse=f64(lse))
    assert_softmax_scores_close(sc, ref)


# ------------------------------------------------------------------ accept

@pytest.mark.parametrize("Hkv,d,T", [(4, 128, 64), (2, 64, 7), (1, 128, 200)])
def test_accept_moves_the_path(lib, Hkv, d, T):
    from visual_token_sparsity_gb300 import binding as sv
    g = np.random.default_rng(T)
    B, nv, nt = 4, [20, 3, 0, 11], [7, 0, 16, 5]
    P = min(T, 64)
    n_path = [P, 0, min(3, P), P - 1]
    path = np.full((B, P), -7)
    for b in range(B):
        path[b, :n_path[b]] = np.sort(g.permutation(T)[:n_path[b]])
    caches = [Cache(B, Hkv, d, 36 + T, seed=l) for l in range(3)]
    for c in caches[1:]:
        c.bt = caches[0].bt
    layers = [c.layer() for c in caches]
    seqs = sv.SeqBatch(caches[0].bt.to(DEV), 20, 16, i32(nv), i32(nt))
    ws = sv.workspace(256)
    sv.sv_kv_accept(layers, seqs, T, i32(path), ws, n_path=i32(n_path))
    assert sv.sv_read_device_status(ws) == 0
    for c, layer in zip(caches, layers):
        for b in range(B):
            base = nv[b] + nt[b]
            for X, pool in ((c.K, layer.k_pool), (c.V, layer.v_pool)):
                ref = oracle.accept_path(X[b].view(torch.int16).numpy(), base, path[b, :n_path[b]])
                got = pool.cpu()[c.bt[b].long()].permute(1, 0, 2, 3).reshape(Hkv, -1, d).view(torch.int16).numpy()
                assert np.array_equal(got, ref)


def test_accept_skips_a_path_that_does_not_ascend(lib):
    from visual_token_sparsity_gb300 import binding as sv
    c = Cache(4, 2, 64, 40, seed=5)
    layer = c.layer()
    keep = layer.k_pool.clone()
    ws = sv.workspace(256)
    seqs = sv.SeqBatch(c.bt.to(DEV), 8, 8)
    sv.sv_kv_accept([layer], seqs, 9, i32([[2, 2], [3, 1], [0, 9], [-1, 4]]), ws)
    assert sv.sv_read_device_status(ws, clear=True) == sv.SV_DEV_BAD_INDEX
    sv.sv_kv_accept([layer], seqs, 9, i32([[2, 3]] * 4), ws, n_path=i32([3, -1, 0, 0]))
    assert sv.sv_read_device_status(ws) == sv.SV_DEV_BAD_LENGTH
    assert torch.equal(layer.k_pool, keep)


# ------------------------------------------------------------------ together

def test_speculative_step(lib):
    """Branch a conversation, reserve, append and rotate a draft, verify it
    under its tree, accept a path, and decode the next token over the result:
    as the oracle says at every stage, in the branch and not in the parent."""
    from visual_token_sparsity_gb300 import binding as sv
    H, Hkv, d, n_vis, n_text, T, k, L = 8, 4, 64, 70, 21, 9, 30, 2
    n = n_vis + n_text
    per, blocks = 9, 30
    g = np.random.default_rng(0)
    K = [synth.normal_bf16((1, Hkv, per * 16, d), 10 + l) for l in range(L)]
    V = [synth.normal_bf16((1, Hkv, per * 16, d), 20 + l) for l in range(L)]
    held = synth.blocks_for(n)
    ids = torch.randperm(blocks, generator=synth.generator(1))[:held]
    table = torch.full((2, per), -1, dtype=torch.int32)
    table[0, :held] = ids.int()
    pools = []
    for l in range(L):
        kp, vp = (torch.zeros(blocks, Hkv, 16, d, dtype=torch.bfloat16) for _ in range(2))
        for x, pool in ((K[l], kp), (V[l], vp)):
            pool[ids] = x[0, :, : held * 16].reshape(Hkv, held, 16, d).transpose(0, 1)
        pools.append((kp.to(DEV), vp.to(DEV)))
    layers = [sv.KvLayer(*p) for p in pools]
    ref = torch.zeros(blocks, dtype=torch.int32)
    ref[ids] = 1
    pool = sv.PagePool(ref.to(DEV), i32([held, 0]))
    table = table.to(DEV)
    both = sv.SeqBatch(table, n_vis, n_text)
    ws = sv.workspace(sv.sv_pages_workspace_bytes(2, per, blocks))
    parent_before = [p[0][ids.to(DEV)].clone() for p in pools]
    sv.sv_pages_fork(pool, both, i32([0]), i32([1]), ws)
    sv.sv_pages_reserve(pool, layers, both, T, ws, n_new=i32([0, T]))
    child = sv.SeqBatch(table[1:], n_vis, n_text)
    rot, rot_ref = rotation(d, 1, 1, T, 300, 3, weights(d, 4))
    mask = [random_tree(T, g)]
    vis = select(1, Hkv, [n_vis], [k], k, 2)
    path = [0, 3, 8]
    wa = sv.workspace(sv.sv_tree_attn_workspace_bytes(1, T, H, Hkv, d, k + n_text + T))
    for l in range(L):
        proj = synth.normal_bf16((1, T, H + 2 * Hkv, d), 30 + l).to(DEV)
        q = torch.empty(1, T, H, d, dtype=torch.bfloat16, device=DEV)
        sv.sv_qk_norm_rope_append(proj[:, :, :H], proj[:, :, H:H + Hkv], proj[:, :, H + Hkv:], rot, layers[l], child,
                                  q, ws)
        out, lse = torch.empty_like(q), torch.empty(1, T, H, device=DEV)
        sv.sv_tree_attn(q, 0.125, layers[l], child, i32(vis), k, mask64(mask), out, lse, wa)
        # the logical cache with the rows as the call stored them
        pages = table[1].long()[n // 16: (n + T - 1) // 16 + 1]
        got = pools[l][0][pages].transpose(0, 1).reshape(Hkv, -1, d)[:, n % 16: n % 16 + T]
        assert_rows_close(got.transpose(0, 1)[None], rot_ref(proj[:, :, H:H + Hkv], rot.k_weight), "k")
        K[l][0, :, n:n + T] = got.cpu()
        V[l][0, :, n:n + T] = proj[0, :, H + Hkv:].transpose(0, 1).cpu()
        assert_tree_close(out, lse, *(x[None] for x in oracle.tree_attention(
            f64(q[0]), f64(K[l][0]), f64(V[l][0]), vis[0], n_vis, n_text, mask[0], 0.125)))
    sv.sv_kv_accept(layers, child, T, i32([path]), ws)
    after = sv.SeqBatch(table[1:], n_vis, n_text + len(path))
    q1 = synth.normal_bf16((1, H, d), 50)
    for l in range(L):
        Kl, Vl = (oracle.accept_path(f64(X[l][0]), n, path)[None] for X in (K, V))
        out = torch.empty(1, H, d, dtype=torch.bfloat16, device=DEV)
        wd = sv.workspace(sv.sv_attn_workspace_bytes(1, H, Hkv, d, k + n_text + len(path)))
        sv.sv_sparse_decode_attn(q1.to(DEV), 0.125, layers[l], after, i32(vis), k, out, None, wd)
        o_ref, _ = oracle.sparse_decode_attention(f64(q1), Kl, Vl, vis, n_vis, n_text + len(path), scale=0.125)
        assert np.abs(f64(out) - o_ref).max() <= 0.02
        assert torch.equal(pools[l][0][ids.to(DEV)], parent_before[l])
    assert sv.sv_read_device_status(ws) == 0 and sv.sv_read_device_status(wa) == 0
    sv.sv_pages_release(pool, both, i32([-1, 0]), ws)
    assert torch.equal(pool.ref.cpu(), ref) and pool.n_pages.tolist() == [held, 0]


def test_a_step_without_drafted_tokens(lib):
    """T = 0 through the whole step: nothing is launched, nothing is refused."""
    from visual_token_sparsity_gb300 import binding as sv
    c = Cache(2, 2, 64, 60, seed=3)
    layer, seqs, ws = c.layer(), sv.SeqBatch(c.bt.to(DEV), 20, 10), sv.workspace(1 << 20)
    keep = layer.k_pool.clone()
    none = lambda *s, t=torch.bfloat16: torch.empty(*s, dtype=t, device=DEV)
    cs = torch.zeros(9, 32, 2, device=DEV)
    rot = sv.Rotation(cs, none(2, 0, t=torch.int32))
    q, kv = none(2, 0, 4, 64), none(2, 0, 2, 64)
    sv.sv_qk_norm_rope(q, kv, rot, none(2, 4, 0, 64), none(2, 2, 0, 64), ws)
    sv.sv_pages_reserve(sv.PagePool(torch.ones(c.blocks, dtype=torch.int32, device=DEV), i32([c.per] * 2)), [layer], seqs,
                        0, sv.workspace(sv.sv_pages_workspace_bytes(2, c.per, c.blocks)))
    sv.sv_qk_norm_rope_append(q, kv, kv, rot, layer, seqs, none(2, 0, 4, 64), ws)
    sv.sv_tree_attn(q, 0.1, layer, seqs, None, 0, none(2, 0, t=torch.int64), none(2, 0, 4, 64), none(2, 0, 4, t=torch.float32),
                    ws)
    sv.sv_kv_accept([layer], seqs, 0, none(2, 0, t=torch.int32), ws)
    assert sv.sv_read_device_status(ws) == 0
    assert torch.equal(layer.k_pool, keep)


@pytest.mark.parametrize("d,H,T", [(64, 4, 9), (128, 14, 30)])
def test_scale_zero_whatever_the_products(lib, d, H, T):
    """Every token weighs the same: products near fp32's largest value count
    0, hidden tokens stay hidden, and 0 times an infinity is NaN."""
    n_vis, n_text, std = 140, 9, 1.2e18 / math.sqrt(d / 64)
    c = Cache(1, 2, d, n_vis + n_text + T, seed=61, std=std)
    q = synth.normal_bf16((1, T, H, d), 4, std=std)
    mask = [random_tree(T, np.random.default_rng(3))]
    args = ([n_vis], [n_text], [0], [T], mask, 0.0)
    out, lse, status = run_tree(c, q, None, 0, *args)
    assert status == 0
    ref = oracle_tree(q, c, None, *args)
    assert_tree_close(out, lse, *ref)
    q[0, 2, 1, 7], q[0, 4, 0, d - 1] = math.inf, math.nan
    out, lse, _ = run_tree(c, q, None, 0, *args)
    for t, h in ((2, 1), (4, 0)):
        assert out[0, t, h].isnan().all() and lse[0, t, h].isnan()
        out[0, t, h], lse[0, t, h] = torch.from_numpy(ref[0][0, t, h]), float(ref[1][0, t, h])
    assert_tree_close(out, lse, *ref)


@pytest.mark.parametrize("H,Hkv,d,B,T", [(32, 32, 128, 2, 150), (28, 4, 128, 2, 150), (28, 4, 128, 4, 1), (8, 2, 64, 2, 150),
                                         (8, 8, 64, 3, 2)])
@pytest.mark.parametrize("ragged", [False, True])
def test_append_of_plain_rotate_half_heads(lib, H, Hkv, d, B, T, ragged):
    """The whole head rotated by halves, one position, no norm: a prefill and
    single tokens as most decoders have them."""
    test_append(lib, H, Hkv, d, d, B, T, 1, None, False, False, ragged)


@pytest.mark.parametrize("d", [64, 128])
def test_plain_rotate_half_rows_are_rounded_as_from_64_bits(lib, d):
    test_appended_rows_are_rounded_as_from_64_bits(lib, d, False, False)
