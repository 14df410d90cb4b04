"""The prompt and 8-bit cache calls beside the others: one workspace for all of
them, two streams at once, programmatic launch on and off, pages behind the 4 GiB
that 32-bit offsets reach, and batches of many short sequences."""

import math
import os
import subprocess
import sys
import textwrap

import numpy as np
import pytest
import torch

import oracle
from kv8_util import DEV, KV8_WEIGHTS, Cache8, assert_close, f64, i32, oracle_decode, oracle_select
from visual_token_sparsity_gb300 import synth

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_one_workspace_serves_old_and_new_calls(lib):
    """A 16-bit and an 8-bit layer in turn, on one workspace: both leave it as the
    others need it, eager and replayed."""
    from visual_token_sparsity_gb300 import binding as sv
    B, H, Hkv, d, n_vis, n_text, k, N = 3, 8, 2, 128, 900, 30, 300, 200
    c = Cache8(B, Hkv, d, n_vis + n_text, seed=5)
    layer8, seqs = c.layer(), sv.SeqBatch(c.bt.to(DEV), n_vis, n_text)
    pools = [synth.normal_bf16((c.blocks, Hkv, 16, d), 30 + i).to(DEV) for i in range(2)]
    layer = sv.KvLayer(*pools)
    q = synth.normal_bf16((B, 1, H, d), 7).to(DEV)
    x = synth.normal_bf16((N, H + 2 * Hkv, d), 8).to(DEV)
    start = i32([0, 77, 77, N])
    n = k + n_text
    need = max(sv.sv_prompt_attn_workspace_bytes(N, B, H, Hkv, d),
               sv.sv_kv8_retrieve_workspace_bytes(B, H, Hkv, d, n_vis, k), sv.sv_kv8_attn_workspace_bytes(B, H, Hkv, d, n),
               sv.sv_retrieve_workspace_bytes(B, H, Hkv, d, n_vis, k), sv.sv_attn_workspace_bytes(B, H, Hkv, d, n))

    def new(ws, o):
        sv.sv_prompt_attn(x[:, :H], x[:, H: H + Hkv], x[:, H + Hkv:], start, 0.1, o["po"], o["pl"], ws)
        sv.sv_kv8_retrieve_topk(q, layer8, seqs, k, o["vis8"], None, ws)
        sv.sv_kv8_decode_attn(q[:, 0], 0.1, layer8, seqs, o["vis8"], k, o["out8"], o["lse8"], ws)

    def old(ws, o):
        sv.sv_retrieve_topk(q, layer, seqs, k, o["vis"], o["sc"], ws)
        sv.sv_sparse_decode_attn(q[:, 0], 0.1, layer, seqs, o["vis"], k, o["out"], o["lse"], ws)

    def outputs():
        bf = dict(dtype=torch.bfloat16, device=DEV)
        return dict(po=torch.zeros(N, H, d, **bf), pl=torch.zeros(N, H, device=DEV),
                    vis8=torch.zeros(B, Hkv, k, dtype=torch.int32, device=DEV), out8=torch.zeros(B, H, d, **bf),
                    lse8=torch.zeros(B, H, device=DEV), vis=torch.zeros(B, Hkv, k, dtype=torch.int32, device=DEV),
                    sc=torch.zeros(B, Hkv, n_vis, device=DEV), out=torch.zeros(B, H, d, **bf),
                    lse=torch.zeros(B, H, device=DEV))
    alone = outputs()
    new(sv.workspace(need), alone)
    old(sv.workspace(need), alone)
    ws, mixed = sv.workspace(need), outputs()
    for f in (new, old, old, new, new, old):
        f(ws, mixed)
    torch.cuda.synchronize()
    graphs, replayed = [], outputs()
    for f in (new, old):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            f(ws, replayed)
        graphs.append(g)
    for i in (0, 1, 1, 0, 0, 1):
        graphs[i].replay()
    assert sv.sv_read_device_status(ws) == 0
    for name, t in alone.items():
        assert torch.equal(t, mixed[name]) and torch.equal(t, replayed[name]), name
        assert t.abs().max() > 0, name


def test_two_streams_at_once(lib):
    from visual_token_sparsity_gb300 import binding as sv
    B, H, Hkv, d, n_vis, k, N = 4, 28, 4, 128, 20000, 5000, 2000
    c = Cache8(B, Hkv, d, n_vis, seed=6)
    layer, seqs = c.layer(), sv.SeqBatch(c.bt.to(DEV), n_vis, 0)
    q = synth.normal_bf16((B, 1, H, d), 7).to(DEV)
    x = synth.normal_bf16((N, H + 2 * Hkv, d), 8).to(DEV)
    start = i32([0, 500, N])

    def run(ws, stream=None):
        vis = torch.empty(B, Hkv, k, dtype=torch.int32, device=DEV)
        out, po = torch.empty(B, H, d, dtype=torch.bfloat16, device=DEV), torch.empty(N, H, d, dtype=torch.bfloat16, device=DEV)
        torch.cuda.synchronize()
        return (vis, out, po), lambda: (
            sv.sv_kv8_retrieve_topk(q, layer, seqs, k, vis, None, ws, stream=stream),
            sv.sv_prompt_attn(x[:, :H], x[:, H: H + Hkv], x[:, H + Hkv:], start, 0.1, po, None, ws, stream=stream),
            sv.sv_kv8_decode_attn(q[:, 0], 0.1, layer, seqs, vis, k, out, None, ws, stream=stream))
    size = max(sv.sv_kv8_retrieve_workspace_bytes(B, H, Hkv, d, n_vis, k),
               sv.sv_kv8_attn_workspace_bytes(B, H, Hkv, d, k), sv.sv_prompt_attn_workspace_bytes(N, 2, H, Hkv, d))
    want, go = run(sv.workspace(size))
    go()
    torch.cuda.synchronize()
    streams, spaces = [torch.cuda.Stream() for _ in range(2)], [sv.workspace(size) for _ in range(2)]
    for _ in range(5):
        both = [run(w, s) for w, s in zip(spaces, streams)]
        for _, go in both:
            go()
        torch.cuda.synchronize()
        for got, _ in both:
            assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert [sv.sv_read_device_status(w) for w in spaces] == [0, 0]


@pytest.mark.parametrize("d", [64, 128])
def test_pages_behind_four_gib(lib, d):
    """The last pages of pools of more than 2^32 bytes: appended, retrieved, attended."""
    from visual_token_sparsity_gb300 import binding as sv
    H, n_vis, new = 2, 100, 40
    blocks = 2 ** 32 // (16 * d) + 50
    pools = [torch.zeros(blocks, 1, 16, d, dtype=torch.uint8, device=DEV) for _ in range(2)]
    layer = sv.Kv8Layer(*pools, torch.zeros(blocks, 1, 2, device=DEV))
    bt = (blocks - 1 - torch.randperm(40, generator=torch.Generator().manual_seed(1))[:9]).int()[None].to(DEV)
    x = synth.normal_bf16((n_vis + new, H + 2, d), 9).to(DEV)
    rot = sv.Rotation(None, None)
    q = torch.empty(n_vis + new, H, d, dtype=torch.bfloat16, device=DEV)
    ws = sv.workspace(max(sv.sv_kv8_retrieve_workspace_bytes(1, H, 1, d, n_vis, 30),
                          sv.sv_kv8_attn_workspace_bytes(1, H, 1, d, 30 + new)))
    sv.sv_kv8_append(x[:, :H], x[:, H: H + 1], x[:, H + 1:], rot, layer, sv.SeqBatch(bt, 0, 0), q, ws)
    seqs = sv.SeqBatch(bt, n_vis, new)
    vis = torch.empty(1, 1, 30, dtype=torch.int32, device=DEV)
    out, lse = torch.empty(1, H, d, dtype=torch.bfloat16, device=DEV), torch.empty(1, H, device=DEV)
    sv.sv_kv8_retrieve_topk(q[-1:].unsqueeze(0), layer, seqs, 30, vis, None, ws)
    sv.sv_kv8_decode_attn(q[-1:], 0.1, layer, seqs, vis, 30, out, lse, ws)
    assert sv.sv_read_device_status(ws) == 0
    assert torch.equal(q, x[:, :H])
    K, V = [], []
    for to, at in ((K, H), (V, H + 1)):
        codes, scales = np.zeros((1, 144, d), np.uint8), np.full((1, 9), np.nan)
        oracle.kv8_append(codes, scales, 0, f64(x[:, at: at + 1]))
        to.append(oracle.kv8_rows(codes, scales))
    K, V = np.stack(K), np.stack(V)
    want, _ = oracle_select(q[-1:].unsqueeze(0), K, [n_vis], [30])
    assert np.array_equal(vis.cpu().numpy(), want)
    assert_close(out, lse, *oracle_decode(q[-1:], K, V, want, [n_vis], [new], [30], 0.1), KV8_WEIGHTS)
    assert not any(p[: 2 ** 32 // (16 * d)].any() for p in pools)
    del pools, layer
    torch.cuda.empty_cache()


def test_many_short_sequences(lib):
    """70001 sequences of one token each: appended, then attended by itself."""
    from visual_token_sparsity_gb300 import binding as sv
    B, d = 70001, 64
    pools = [torch.full((B, 1, 16, d), 0x7F, dtype=torch.uint8, device=DEV) for _ in range(2)]
    layer = sv.Kv8Layer(*pools, torch.full((B, 1, 2), math.nan, device=DEV))
    bt = torch.randperm(B, generator=torch.Generator().manual_seed(2)).int()[:, None].to(DEV)
    x = synth.normal_bf16((B, 3, d), 10).to(DEV)
    rot = sv.Rotation(None, None)
    q, ko = (torch.empty(B, 1, d, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    ws = sv.workspace(max(sv.sv_kv8_attn_workspace_bytes(B, 1, 1, d, 1), sv.sv_prompt_attn_workspace_bytes(B, B, 1, 1, d)))
    sv.sv_kv8_append(x[:, :1], x[:, 1:2], x[:, 2:], rot, layer, sv.SeqBatch(bt, 0, 0), q, ws, k_out=ko)
    out, lse = torch.empty_like(q), torch.empty(B, 1, device=DEV)
    sv.sv_kv8_decode_attn(q, 0.125, layer, sv.SeqBatch(bt, 0, 1), None, 0, out, lse, ws)
    # one token: its row, as the cache holds it (a power of two times e4m3 is bf16)
    top = x[:, 2].float().abs().amax(-1, keepdim=True)
    s = torch.exp2(torch.ceil(torch.log2(top.double() / 448))).float()
    want = ((x[:, 2].float() / s).to(torch.float8_e4m3fn).float() * s).bfloat16()
    assert torch.equal(out[:, 0], want)
    po = torch.empty_like(q)
    sv.sv_prompt_attn(q, ko, x[:, 2:], torch.arange(B + 1, dtype=torch.int32, device=DEV), 0.125, po, None, ws)
    assert torch.equal(po[:, 0], x[:, 2])
    assert sv.sv_read_device_status(ws) == 0


@pytest.mark.parametrize("d,interleaved,norm", [(128, False, True), (64, True, True), (128, True, False), (64, False, False)])
def test_keys_are_rounded_from_more_than_fp32(lib, d, interleaved, norm):
    """Keys whose turned pairs cancel among ten million elements: bf16 results on the
    right side of every border, where fp32 alone would fall on the other now and then."""
    from visual_token_sparsity_gb300 import binding as sv
    N, H, Hkv, n_pos = 80000 * 64 // d, 2, 2, 500
    g = torch.Generator().manual_seed(4)
    angle = torch.rand(n_pos, d // 2, generator=g, dtype=torch.float64) * 2 * math.pi
    turns = torch.stack([angle.cos(), angle.sin()], -1).float().to(DEV)
    pos = torch.randint(n_pos, (1, N), generator=g, dtype=torch.int32).to(DEV)
    w = (1 + 0.1 * synth.normal_bf16((d,), 12).float()).bfloat16().to(DEV) if norm else None
    x = synth.normal_bf16((N, H + 2 * Hkv, d), 13).to(DEV)
    k = x[:, H: H + Hkv]
    bt = torch.arange((N + 15) // 16, dtype=torch.int32)[None].to(DEV)
    pools = [torch.zeros(bt.numel(), Hkv, 16, d, dtype=torch.uint8, device=DEV) for _ in range(2)]
    layer = sv.Kv8Layer(*pools, torch.zeros(bt.numel(), Hkv, 2, device=DEV))
    q = torch.empty(N, H, d, dtype=torch.bfloat16, device=DEV)
    ko = torch.empty(N, Hkv, d, dtype=torch.bfloat16, device=DEV)
    ws = sv.workspace(sv.sv_evict_workspace_bytes())
    sv.sv_kv8_append(x[:, :H], k, x[:, H + Hkv:], sv.Rotation(turns, pos, interleaved=interleaved, q_weight=w, k_weight=w),
                     layer, sv.SeqBatch(bt, 0, 0), q, ws, k_out=ko)
    assert sv.sv_read_device_status(ws) == 0
    y = k.double()
    if norm:
        y = y / torch.sqrt((y * y).mean(-1, keepdim=True) + 1e-6) * w.double()
    c, s = turns.double()[pos[0].long()][:, None].unbind(-1)
    a, b = (y[..., 0::2], y[..., 1::2]) if interleaved else (y[..., : d // 2], y[..., d // 2:])
    re, im = a * c - b * s, a * s + b * c
    want = (torch.stack([re, im], -1).flatten(-2) if interleaved else torch.cat([re, im], -1)).bfloat16()
    assert int((want.view(torch.int16) != ko.view(torch.int16)).sum()) == 0


@pytest.mark.parametrize("times", [40.0, 3e4, 2.0 ** 70])
@pytest.mark.parametrize("n_vis,k", [(3000, 700), (20000, 9000)])
def test_retrieval_beside_keys_of_another_magnitude(lib, n_vis, k, times):
    """One page's keys are many times larger: its scores stretch the range that the
    others lie in a small part of, and its factor the error that fp32 may have made."""
    from visual_token_sparsity_gb300 import binding as sv
    H, Hkv, d, per = 4, 2, 64, -(-n_vis // 16)
    factor = np.ones((1, Hkv, per, 2))
    factor[:, 0, 5], factor[:, 1, per - 1] = times, times
    c = Cache8(1, Hkv, d, n_vis, seed=44, factor=factor)
    q = synth.normal_bf16((1, 2, H, d), 16).to(DEV)
    vis = torch.full((1, Hkv, k), -7, dtype=torch.int32, device=DEV)
    ws = sv.workspace(sv.sv_kv8_retrieve_workspace_bytes(1, H, Hkv, d, n_vis, k))
    sv.sv_kv8_retrieve_topk(q, c.layer(), sv.SeqBatch(c.bt.to(DEV), n_vis, 0), k, vis, None, ws)
    assert sv.sv_read_device_status(ws) == 0
    want, _ = oracle_select(q, c.rows(0), [n_vis], [k])
    assert np.array_equal(vis.cpu().numpy(), want)


RUN = textwrap.dedent("""
    import sys, torch
    sys.path.insert(0, {root!r})
    from visual_token_sparsity_gb300 import binding as sv, synth
    dev, out = "cuda", {{}}
    for name, H, Hkv, d, n, k, R in (("small", 4, 2, 64, 300, 90, 1), ("mha", 8, 8, 128, 2000, 500, 3),
                                     ("gqa", 28, 4, 128, 17000, 4000, 1)):
        per = -(-(n + 6) // 16)
        bt = torch.randperm(2 * per, generator=torch.Generator().manual_seed(1)).int().view(2, per).to(dev)
        layer = sv.Kv8Layer(*(torch.zeros(2 * per, Hkv, 16, d, dtype=torch.uint8, device=dev) for _ in range(2)),
                            torch.zeros(2 * per, Hkv, 2, device=dev))
        x = synth.normal_bf16((2 * (n + 6), H + 2 * Hkv, d), 5).to(dev)
        cs = torch.randn(n + 6, d // 2, 2, generator=torch.Generator().manual_seed(3)).to(dev)
        pos = torch.arange(n + 6, dtype=torch.int32, device=dev)
        ws = sv.workspace(max(sv.sv_prompt_attn_workspace_bytes(2 * n, 2, H, Hkv, d),
                              sv.sv_kv8_retrieve_workspace_bytes(2, H, Hkv, d, n, k),
                              sv.sv_kv8_attn_workspace_bytes(2, H, Hkv, d, k + 6)))
        bf = dict(dtype=torch.bfloat16, device=dev)
        start = torch.tensor([0, n, 2 * n], dtype=torch.int32, device=dev)
        first, q, ko = x[: 2 * n], torch.zeros(2 * n, H, d, **bf), torch.zeros(2 * n, Hkv, d, **bf)
        po, pl = torch.zeros(2 * n, H, d, **bf), torch.zeros(2 * n, H, device=dev)
        rot = sv.Rotation(cs, pos[:n].repeat(2)[None])
        rots = [sv.Rotation(cs, pos[n + s: n + s + 1].repeat(2)[None]) for s in range(6)]
        o = torch.zeros(6, 2, H, d, **bf)
        dq = torch.zeros(6, 2, H, d, **bf)
        vis = torch.zeros(6, 2, Hkv, k, dtype=torch.int32, device=dev)
        qq = torch.zeros(2, R, H, d, **bf)
        torch.cuda.synchronize()
        sv.sv_kv8_append(first[:, :H], first[:, H:H + Hkv], first[:, H + Hkv:], rot, layer, sv.SeqBatch(bt, 0, 0), q, ws,
                         seq_start=start, k_out=ko)
        sv.sv_prompt_attn(q, ko, first[:, H + Hkv:], start, 0.1, po, pl, ws)
        for s in range(6):
            p = x[2 * (n + s): 2 * (n + s) + 2]
            sv.sv_kv8_append(p[:, :H], p[:, H:H + Hkv], p[:, H + Hkv:], rots[s], layer, sv.SeqBatch(bt, n, s), dq[s], ws)
            qq.copy_(dq[s][:, None].expand(2, R, H, d))
            seqs = sv.SeqBatch(bt, n, s + 1)
            sv.sv_kv8_retrieve_topk(qq, layer, seqs, k, vis[s], None, ws)
            sv.sv_kv8_decode_attn(dq[s], 0.1, layer, seqs, vis[s], k, o[s], None, ws)
        assert sv.sv_read_device_status(ws) == 0
        out.update({{f"{{name}}_{{w}}": t.cpu() for w, t in (("q", q), ("ko", ko), ("po", po), ("pl", pl), ("dq", dq),
                   ("vis", vis), ("o", o), ("k", layer.k_pool.view(torch.uint8)), ("v", layer.v_pool.view(torch.uint8)),
                   ("s", layer.scales))}})
    torch.save(out, sys.argv[1])
""")


def test_programmatic_launch_does_not_change_a_run(lib, tmp_path):
    runs = []
    for pdl in ("1", "0"):
        env, path = dict(os.environ, SV_PDL=pdl), str(tmp_path / f"{pdl}.pt")
        r = subprocess.run([sys.executable, "-c", RUN.format(root=ROOT), path], env=env, capture_output=True, text=True,
                           timeout=600)
        assert r.returncode == 0, r.stderr[-2000:]
        runs.append(torch.load(path))
    assert runs[0].keys() == runs[1].keys()
    for key, t in runs[0].items():
        assert torch.equal(t, runs[1][key]), key
        assert t.float().abs().max() > 0, key


def test_many_ragged_sequences(lib):
    """3001 sequences of 0 to 40 tokens: each row's own selection and attention."""
    from visual_token_sparsity_gb300 import binding as sv
    B, H, Hkv, d, n_vis, n_text, k = 3001, 4, 1, 64, 33, 7, 9
    g = np.random.default_rng(5)
    nv, nt = g.integers(0, n_vis + 1, B), g.integers(0, n_text + 1, B)
    ks = np.minimum(nv, g.integers(0, k + 1, B))
    c = Cache8(B, Hkv, d, n_vis + n_text, seed=91)
    layer, seqs = c.layer(), sv.SeqBatch(c.bt.to(DEV), n_vis, n_text, i32(nv), i32(nt), i32(ks))
    q = synth.normal_bf16((B, 1, H, d), 17).to(DEV)
    vis = torch.full((B, Hkv, k), -7, dtype=torch.int32, device=DEV)
    out, lse = torch.full((B, H, d), 7.0, dtype=torch.bfloat16, device=DEV), torch.full((B, H), 7.0, device=DEV)
    ws = sv.workspace(max(sv.sv_kv8_retrieve_workspace_bytes(B, H, Hkv, d, n_vis, k),
                          sv.sv_kv8_attn_workspace_bytes(B, H, Hkv, d, k + n_text)))
    sv.sv_kv8_retrieve_topk(q, layer, seqs, k, vis, None, ws)
    sv.sv_kv8_decode_attn(q[:, 0], 0.125, layer, seqs, vis, k, out, lse, ws)
    assert sv.sv_read_device_status(ws) == 0
    K, V, got = c.rows(0), c.rows(1), vis.cpu().numpy()
    want, _ = oracle_select(q, K, nv.tolist(), ks.tolist())
    assert np.array_equal(got[..., : want.shape[2]], want) and (got[..., want.shape[2]:] == -1).all()
    assert_close(out, lse, *oracle_decode(q[:, 0], K, V, got, nv.tolist(), nt.tolist(), ks.tolist(), 0.125), KV8_WEIGHTS)
