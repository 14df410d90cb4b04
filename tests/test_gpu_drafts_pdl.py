"""Draft, branch and rotation calls launched one behind the other give the
same bits with programmatic dependent launch (the default) and without it
(SV_PDL=0, in a child process, since the library reads the switch once)."""

import os
import subprocess
import sys
import textwrap

import pytest
import torch

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

RUN = textwrap.dedent("""
    import sys, torch
    sys.path.insert(0, {root!r})
    from visual_token_sparsity_gb300 import binding as sv, synth
    dev, out = "cuda", {{}}
    bf = dict(dtype=torch.bfloat16, device=dev)
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device=dev)
    # a prefix of n tokens, forked into three branches that draft T tokens each, in every layer
    for name, H, Hkv, d, n_vis, n_text, T, L in (("small", 4, 2, 64, 300, 21, 7, 3), ("mha", 8, 8, 128, 2000, 50, 16, 3),
                                                 ("gqa", 28, 4, 128, 12000, 40, 27, 2)):
        n = n_vis + n_text
        held, per = -(-n // 16), -(-(n + 3 * T) // 16)
        blocks = held + 3 * (per - held + 1) + 2
        g = torch.Generator().manual_seed(3)
        table = torch.full((4, per), -1, dtype=torch.int32)
        table[0, :held] = torch.randperm(blocks, generator=g)[:held].int()
        ref = torch.zeros(blocks, dtype=torch.int32)
        ref[table[0, :held].long()] = 1
        table, ref, n_pages = table.to(dev), ref.to(dev), i32(held, 0, 0, 0)
        layers = [sv.KvLayer(*(synth.normal_bf16((blocks, Hkv, 16, d), 10 * l + i).to(dev) for i in range(2)))
                  for l in range(L)]
        pool, seqs = sv.PagePool(ref, n_pages), sv.SeqBatch(table, n_vis, n_text)
        kids = sv.SeqBatch(table[1:], n_vis, n_text)
        cs = torch.randn(n + T, d // 2, 2, generator=g).to(dev)
        rot = sv.Rotation(cs, (n + torch.arange(T, dtype=torch.int32, device=dev)).repeat(3, 1))
        proj = synth.normal_bf16((L, 3, T, H + 2 * Hkv, d), 5).to(dev)
        mask = torch.tensor([[(2 << t) - 1 if b == 0 else (1 << t) | 1 for t in range(T)] for b in range(3)], device=dev)
        k = n_vis // 2
        vis = torch.stack([torch.sort(torch.randperm(n_vis, generator=g)[:k]).values for _ in range(3 * Hkv)])
        vis = vis.int().view(3, Hkv, k).to(dev)
        ws = sv.workspace(max(sv.sv_pages_workspace_bytes(4, per, blocks),
                              sv.sv_tree_attn_workspace_bytes(3, T, H, Hkv, d, k + n_text + T)))
        q, o = (torch.zeros(L, 3, T, H, d, **bf) for _ in range(2))
        lse = torch.zeros(L, 3, T, H, device=dev)
        path = i32(0, T - 1).repeat(3, 1)
        torch.cuda.synchronize()
        for step in range(3):
            sv.sv_pages_fork(pool, seqs, i32(0, 0, 0), i32(1, 2, 3), ws)
            sv.sv_pages_reserve(pool, layers, seqs, T, ws, n_new=i32(0, T, T, T))
            for l in range(L):
                p = proj[l]
                sv.sv_qk_norm_rope_append(p[:, :, :H], p[:, :, H:H + Hkv], p[:, :, H + Hkv:], rot, layers[l], kids, q[l], ws)
                sv.sv_tree_attn(q[l], 0.125, layers[l], kids, vis, k, mask, o[l], lse[l], ws)
            sv.sv_kv_accept(layers, kids, T, path, ws)
            out.update({{f"{{name}}_{{what}}{{step}}": t.clone() for what, t in (("q", q), ("o", o), ("lse", lse),
                                                                              ("table", table), ("ref", ref))}})
            out.update({{f"{{name}}_pool{{step}}_{{l}}": x.k_pool.clone() for l, x in enumerate(layers)}})
            sv.sv_pages_release(pool, seqs, i32(-1, 0, 0, 0), ws)
        qo = torch.zeros(3, H, T, d, **bf)
        ko = torch.zeros(3, Hkv, T, d, **bf)
        sv.sv_qk_norm_rope(proj[0][:, :, :H], proj[0][:, :, H:H + Hkv], rot, qo, ko, ws)
        out[name + "_qo"], out[name + "_ko"] = qo, ko
        assert sv.sv_read_device_status(ws) == 0
    torch.cuda.synchronize()
    torch.save({{k: v.cpu() for k, v in out.items()}}, sys.argv[1])
""")


def run(path, pdl):
    env = dict(os.environ)
    env["SV_PDL"] = "1" if pdl else "0"
    r = subprocess.run([sys.executable, "-c", RUN.format(root=ROOT), path], env=env, capture_output=True, text=True,
                       timeout=600)
    assert r.returncode == 0, r.stderr[-2000:]
    return torch.load(path)


def test_programmatic_launch_does_not_change_a_draft_step(lib, tmp_path):
    on, off = run(str(tmp_path / "on.pt"), True), run(str(tmp_path / "off.pt"), False)
    assert on.keys() == off.keys()
    for key in on:
        assert torch.equal(on[key], off[key]), key
    for name in ("small", "mha", "gqa"):
        assert on[name + "_o0"].float().abs().max() > 0
        for step in (1, 2):              # every step from the same prefix
            assert torch.equal(on[f"{name}_o{step}"], on[f"{name}_o0"])
