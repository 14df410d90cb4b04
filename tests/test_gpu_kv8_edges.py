"""GPU: calls of the 8-bit cache at the edges of what the header allows: sequences
that are skipped for any of their counts, rows that are taken whole."""

import numpy as np
import pytest
import torch

from kv8_util import DEV, KV8_WEIGHTS, Cache8, assert_close, i32, oracle_decode, oracle_select
from test_gpu_kv8 import attend
from visual_token_sparsity_gb300 import synth

pytestmark = pytest.mark.gpu

GUARD = 4096          # elements behind the indices, left as they were


def retrieve(c, q, seqs, k):
    """(indices, fp32 scores, status); nothing is written behind the indices."""
    from visual_token_sparsity_gb300 import binding as sv
    B, R, H, d = q.shape
    n = B * c.Hkv * k
    buf = torch.full((n + GUARD,), -7, dtype=torch.int32, device=DEV)
    sc = torch.full((B, c.Hkv, seqs.n_vis), 7.0, device=DEV)
    ws = sv.workspace(sv.sv_kv8_retrieve_workspace_bytes(B, H, c.Hkv, d, seqs.n_vis, k))
    sv.sv_kv8_retrieve_topk(q, c.layer(), seqs, k, buf[:n].view(B, c.Hkv, k), sc, ws)
    status = sv.sv_read_device_status(ws)
    assert (buf[n:] == -7).all()
    return buf[:n].view(B, c.Hkv, k).cpu().numpy(), sc, status


def long_cache(B, Hkv, d, tokens, seed):
    """A cache whose pages come again behind 8192 tokens: (cache, block table, keys of `tokens`)."""
    c = Cache8(B, Hkv, d, min(tokens, 8192), seed)
    bt = c.bt.repeat(1, -(-tokens // (c.per * 16)))[:, : synth.blocks_for(tokens)].contiguous()
    return c, bt.to(DEV), c.rows(0)[:, :, np.arange(tokens) % (c.per * 16)]


@pytest.mark.parametrize("Hkv,d,n_vis,k", [(2, 64, 700, 200), (4, 64, 5000, 5000), (4, 64, 20011, 6000),
                                           (1, 64, 402000, 90000)])
@pytest.mark.parametrize("which", ["some", "all"])
def test_retrieval_skips_sequences_whose_text_count_is_out_of_range(lib, Hkv, d, n_vis, k, which):
    """They are not scored, so their rows have no selection either: all -1.  The valid
    ones, a short one first, are as they would be without them."""
    from visual_token_sparsity_gb300 import binding as sv
    n_text = 9
    nv = [16, n_vis, n_vis // 2, n_vis]
    nt = [0, n_text + 1, n_text, -1] if which == "some" else [n_text + 1, -1, 2 ** 31 - 1, -2 ** 31]
    ks = [min(3, k), k, k // 3, k]
    good = [b for b in range(4) if 0 <= nt[b] <= n_text]
    c, bt, K = long_cache(4, Hkv, d, n_vis + n_text, seed=91)
    q = synth.normal_bf16((4, 1, 2 * Hkv, d), 6).to(DEV)
    vis, sc, status = retrieve(c, q, sv.SeqBatch(bt, n_vis, n_text, i32(nv), i32(nt), i32(ks)), k)
    assert status == sv.SV_DEV_BAD_LENGTH
    for b in range(4):
        if b not in good:
            assert (vis[b] == -1).all() and (sc[b] == 7.0).all()
    if good:
        want, _ = oracle_select(q[good], K[good], [nv[b] for b in good], [ks[b] for b in good])
        assert np.array_equal(vis[good][..., :want.shape[2]], want) and (vis[good][..., want.shape[2]:] == -1).all()
    # the text counts alone, the others uniform
    vis, _, status = retrieve(c, q, sv.SeqBatch(bt, n_vis, n_text, None, i32(nt), None), k)
    assert status == sv.SV_DEV_BAD_LENGTH
    for b in range(4):
        if b not in good:
            assert (vis[b] == -1).all()
        else:
            assert np.array_equal(vis[b: b + 1], oracle_select(q[b: b + 1], K[b: b + 1], [n_vis], [k])[0])


LONG = [5000, 20011, 402000]       # a CTA per row, a cluster, a cluster whose keys lie in global memory


def kinds_of_rows(n, kinds, seed):
    """A cache of one head whose keys are `kinds` different rows, row i's kind pick[i]; d 64."""
    c, bt, _ = long_cache(1, 1, 64, n, seed)
    cap = c.codes[0].shape[2]
    pick = np.random.default_rng(seed).integers(0, kinds, cap)
    c.codes[0] = np.ascontiguousarray(c.codes[0][:, :, pick])
    c.scales[...] = 0.25
    return c, bt, pick[np.arange(n) % cap]


@pytest.mark.parametrize("n", LONG)
def test_rows_taken_whole_without_a_difference(lib, n):
    """k == n_vis and all scores equal: every token lies next to the border and is needed."""
    from visual_token_sparsity_gb300 import binding as sv
    c, bt, _ = long_cache(2, 2, 64, n, seed=92)
    q = torch.zeros(2, 1, 4, 64, dtype=torch.bfloat16, device=DEV)
    vis, sc, status = retrieve(c, q, sv.SeqBatch(bt, n, 0), n)
    assert status == 0 and (sc == 0).all() and (vis == np.arange(n)).all()


@pytest.mark.parametrize("kinds,better", [(2, 1), (3, 2), (2, 2)])
@pytest.mark.parametrize("n", LONG)
def test_ties_that_the_selection_uses_up(lib, n, kinds, better):
    """k is the number of tokens of the better kinds: the last of them is needed."""
    from visual_token_sparsity_gb300 import binding as sv
    c, bt, pick = kinds_of_rows(n, kinds, seed=93)
    q = synth.normal_bf16((1, 1, 1, 64), 16).to(DEV)
    qn = q.double().cpu().numpy()[0, 0, 0]
    K = c.rows(0)[0, 0]
    cap = K.shape[0]
    value = {p: (K[np.flatnonzero(pick[:cap] == p)[0]] @ qn) for p in range(kinds)}
    best = sorted(value, key=value.get)[-better:]
    want = np.flatnonzero(np.isin(pick, best))
    assert len(set(value.values())) == kinds and want.size > 600
    vis, _, status = retrieve(c, q, sv.SeqBatch(bt, n, 0), want.size)
    assert status == 0 and np.array_equal(vis[0, 0], want)


@pytest.mark.parametrize("less", [0, 1, 1000])
@pytest.mark.parametrize("n", LONG)
def test_one_key_that_is_not_finite_in_a_long_row(lib, n, less):
    """The choice is open, but ascending, distinct and in range."""
    from visual_token_sparsity_gb300 import binding as sv
    c, bt, _ = long_cache(1, 1, 64, n, seed=94)
    c.codes[0][0, 0, 4321, 3] = 0x7F
    q = synth.normal_bf16((1, 1, 1, 64), 17).to(DEV)
    vis, _, status = retrieve(c, q, sv.SeqBatch(bt, n, 0), n - less)
    assert status == 0
    assert (np.diff(vis[0, 0]) > 0).all() and vis.min() >= 0 and vis.max() < n


@pytest.mark.parametrize("n", LONG)
def test_a_short_sequence_taken_whole_beside_long_ones(lib, n):
    """The kernel is chosen by the capacity; equal scores, k_seq == n_vis_seq or one less."""
    from visual_token_sparsity_gb300 import binding as sv
    nv, ks = [n, 3000, 4001, 513, 512], [n // 3, 3000, 4000, 513, 512]
    c, bt, _ = long_cache(5, 1, 64, n, seed=95)
    q = torch.zeros(5, 1, 1, 64, dtype=torch.bfloat16, device=DEV)
    vis, _, status = retrieve(c, q, sv.SeqBatch(bt, n, 0, i32(nv), None, i32(ks)), max(ks))
    assert status == 0
    for b in range(5):
        assert np.array_equal(vis[b, 0, : ks[b]], np.arange(ks[b])) and (vis[b, 0, ks[b]:] == -1).all()


@pytest.mark.parametrize("arrays", [True, False])
@pytest.mark.parametrize("B,H,Hkv,d", [(700, 8, 1, 128), (2100, 4, 2, 64), (1100, 20, 4, 128), (460, 16, 1, 64)])
def test_attention_of_more_rows_than_pieces(lib, B, H, Hkv, d, arrays):
    """The cut of the line leaves most rows whole and some in two pieces or, where a long
    sequence stands among short ones, in many; each is joined once.  Sequences share the
    pages of a small pool; a few are compared with the oracle, the others with their like."""
    from visual_token_sparsity_gb300 import binding as sv
    n_vis, n_text, kinds = (1500, 20, 9) if arrays else (130, 20, 9)
    g = np.random.default_rng(96)
    c = Cache8(kinds, Hkv, d, n_vis + n_text, seed=97)
    kind = g.integers(0, kinds, B)
    if arrays:
        long = g.random(kinds) < 0.3
        long[:2] = True, False
        kv = np.where(long, g.integers(600, n_vis + 1, kinds), g.integers(0, 40, kinds))
        kt = g.integers(0, n_text + 1, kinds)
        kv[2] = kt[2] = 0
        kind[[b for b in range(B) if long[kind[b]] and b % 37]] = 1            # (few long ones)
        kind[[5, B - 1]] = 0
    else:
        kv, kt = np.full(kinds, n_vis), np.full(kinds, n_text)
    q9 = synth.normal_bf16((kinds, H, d), 20)
    q, bt = q9[torch.from_numpy(kind)].to(DEV), c.bt[torch.from_numpy(kind)].contiguous().to(DEV)
    seqs = sv.SeqBatch(bt, n_vis, n_text, *((i32(kv[kind]), i32(kt[kind])) if arrays else (None, None)))
    out, lse, status = attend(c, q, seqs, None, 0, 0.11)
    assert status == 0
    first = [int(np.flatnonzero(kind == i)[0]) for i in range(kinds) if (kind == i).any()]
    used = [int(kind[f]) for f in first]
    ref = oracle_decode(q9[used], c.rows(0)[used], c.rows(1)[used], None, kv[used].tolist(), kt[used].tolist(), None, 0.11)
    for nth, i in enumerate(used):
        for b in np.flatnonzero(kind == i):
            assert_close(out[b], lse[b], *(r[nth] for r in ref), KV8_WEIGHTS, f"sequence {b} of kind {i}")


@pytest.mark.parametrize("B,Hkv,n_vis,k", [(33, 2, 400, 90), (300, 1, 150, 40), (1000, 3, 70, 20), (65, 1, 17000, 60)])
@pytest.mark.parametrize("bad", [False, True])
def test_retrieval_of_many_sequences_of_their_own_lengths(lib, B, Hkv, n_vis, k, bad):
    """Empty ones and, bad, some that are skipped among them; sequences share the pages of a
    small pool, so that each can be compared with its like."""
    from visual_token_sparsity_gb300 import binding as sv
    g = np.random.default_rng(98)
    kinds = 7
    c = Cache8(kinds, Hkv, 64, min(n_vis, 800), seed=99)
    kind = g.integers(0, kinds, B)
    nv = g.integers(0, min(n_vis, 800) + 1, B)
    nv[[3, B - 1]] = 0, min(n_vis, 800)
    ks = np.minimum(nv, g.integers(0, k + 1, B))
    ks[B - 1] = min(k, nv[B - 1])
    nt = g.integers(0, 6, B)
    if bad:
        nt[[0, 5, B // 2]] = 6, -1, 99
        nv[7], ks[9] = n_vis + 1, nv[9] + 1
    good = (nt >= 0) & (nt <= 5) & (nv <= n_vis) & (ks <= nv) & (ks <= k)
    bt = torch.zeros(B, synth.blocks_for(n_vis + 5), dtype=torch.int32)
    bt[:, : c.per] = c.bt[torch.from_numpy(kind)][:, : bt.shape[1]]
    q = synth.normal_bf16((B, 1, Hkv, 64), 21).to(DEV)
    vis, _, status = retrieve(c, q, sv.SeqBatch(bt.to(DEV), n_vis, 5, i32(nv), i32(nt), i32(ks)), k)
    assert status == (sv.SV_DEV_BAD_LENGTH if bad else 0)
    assert bad != good.all() and (vis[~good] == -1).all()
    at = np.flatnonzero(good)
    want, _ = oracle_select(q[at], c.rows(0)[kind[at]], nv[at].tolist(), ks[at].tolist())
    assert np.array_equal(vis[at][..., : want.shape[2]], want) and (vis[at][..., want.shape[2]:] == -1).all()
