"""GPU: prompt attention's outputs where they lie in other places than a fresh
allocation, rows that are formed twice, and its lse in the retrieval that takes one."""

import numpy as np
import pytest
import torch

import oracle
from kv8_util import DEV, i32, f64
from parity_util import SOFTMAX_SCORE_REL, assert_selection, assert_softmax_scores_close
from test_gpu_prompt import Prompt
from visual_token_sparsity_gb300 import synth

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("odd", [False, True])
@pytest.mark.parametrize("H,Hkv,d,lens", [(4, 2, 64, [176]), (7, 1, 128, [33, 0, 200]), (28, 4, 128, [97, 18, 150])])
def test_an_output_on_a_16_byte_boundary(lib, H, Hkv, d, lens, odd):
    """Addresses that are no multiple of 32 get the same bits, nothing beside them changes.
    odd: with a value that is not finite, so that rows are formed again."""
    from visual_token_sparsity_gb300 import binding as sv
    p = Prompt(H, Hkv, d, lens, seed=40)
    if odd:
        p.v[20, 0, 5] = float("nan")
    want, want_lse = p.run()
    n = p.N * H * d
    ws = sv.workspace(sv.sv_prompt_attn_workspace_bytes(p.N, len(lens), H, Hkv, d))
    for off in (8, 24):
        buf = torch.full((n + 64,), 7.0, dtype=torch.bfloat16, device=DEV)
        norm = torch.full((p.N * H + 8,), 7.0, device=DEV)
        out, lse = buf[off: off + n].view(p.N, H, d), norm[1: 1 + p.N * H].view(p.N, H)
        assert out.data_ptr() % 32 == 16
        sv.sv_prompt_attn(p.q, p.k, p.v, i32(p.start), p.scale, out, lse, ws)
        assert sv.sv_read_device_status(ws) == 0
        assert torch.equal(out.view(torch.int16), want.view(torch.int16))
        assert torch.equal(lse.view(torch.int32), want_lse.view(torch.int32))
        assert (buf[:off] == 7).all() and (buf[off + n:] == 7).all() and norm[0] == 7 and (norm[1 + p.N * H:] == 7).all()


@pytest.mark.parametrize("H,Hkv,d,n,R", [(4, 2, 64, 200, 8), (28, 4, 128, 400, 3)])
def test_lse_normalises_the_softmax_retrieval(lib, H, Hkv, d, n, R):
    """The last R rows of a prompt retrieve from its own visual tokens, with the prompt's
    lse as their normaliser.  The lse is off by 1e-3 at most, so a score is by as much of
    itself beside the retrieval's own tolerance."""
    from visual_token_sparsity_gb300 import binding as sv
    p = Prompt(H, Hkv, d, [n], seed=41)
    _, lse = p.run()
    n_vis, k = n - 50, 40
    per = synth.blocks_for(n)
    bt = synth.random_block_table(1, per, per + 2, seed=42)
    pool = torch.zeros(per + 2, Hkv, 16, d, dtype=torch.bfloat16, device=DEV)
    rows = torch.zeros(per * 16, Hkv, d, dtype=torch.bfloat16, device=DEV)
    rows[:n] = p.k
    pool[bt[0].long().to(DEV)] = rows.view(per, 16, Hkv, d).transpose(1, 2)
    q = p.q[n - R:].contiguous().unsqueeze(0)
    vis = torch.empty(1, Hkv, k, dtype=torch.int32, device=DEV)
    sc = torch.empty(1, Hkv, n_vis, device=DEV)
    ws = sv.workspace(sv.sv_retrieve_softmax_workspace_bytes(1, R, H, Hkv, d, n_vis, 50))
    sv.sv_retrieve_topk_softmax(q, p.scale, sv.KvLayer(pool, torch.zeros_like(pool)), sv.SeqBatch(bt.to(DEV), n_vis, 50),
                                k, vis, sc, ws, lse=lse[n - R:].contiguous().unsqueeze(0))
    assert sv.sv_read_device_status(ws) == 0
    K = f64(p.k).transpose(1, 0, 2)[None]
    given = oracle.retrieval_scores_softmax(f64(q), K, n_vis, 50, p.scale, lse=f64(lse[n - R:])[None])
    assert_softmax_scores_close(sc, given)
    assert_selection(vis.cpu().numpy(), given, k)
    _, ref_lse, _ = p.ref()
    exact = oracle.retrieval_scores_softmax(f64(q), K, n_vis, 50, p.scale, lse=ref_lse[n - R:][None])
    assert (np.abs(f64(sc) - exact) <= (SOFTMAX_SCORE_REL + 1.001e-3) * exact + 1e-7 * exact.max()).all()
    # what the rows' weights add up to over all that each sees is 1, so over the visual tokens it is less
    assert (f64(sc).sum(-1) < R * (H // Hkv)).all()
