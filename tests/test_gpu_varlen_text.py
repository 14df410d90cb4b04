"""GPU: retrieval of a batch in which a sequence's text count is out of range.  The
sequence is skipped: not scored, and its indices read -1, whichever of the selections
(fused, a CTA per row, a cluster) a row gets."""

import numpy as np
import pytest
import torch

from test_gpu_varlen import DEV, check_retrieval, retrieve, varlen_batch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("Hkv,batch,n_cap", [(2, 4, 200), (20, 4, 200), (2, 4, 14000), (2, 4, 20000)])
@pytest.mark.parametrize("noalloc", [False, True])
def test_text_counts_out_of_range(lib, Hkv, batch, n_cap, noalloc):
    from visual_token_sparsity_gb300 import binding as sv
    nv, nt = [n_cap, n_cap - 3, n_cap // 2, n_cap], [7, 16, 0, 16]
    kseq = [n_cap // 4, n_cap - 3, 0, n_cap // 3]
    shape, lay, layer, seqs, kseq = varlen_batch(2 * Hkv, Hkv, 64, nv, nt, seed=n_cap + Hkv, kseq=kseq)
    bad = torch.tensor([7, 17, 0, -1], dtype=torch.int32, device=DEV)
    seqs = sv.SeqBatch(seqs.block_table, shape.n_vis, shape.n_text, seqs.n_vis_seq, bad, seqs.k_seq)
    vis, sc, st = retrieve(shape, layer, seqs, torch.ones(4, 1, 2 * Hkv, 64, dtype=torch.bfloat16, device=DEV),
                           max(kseq), noalloc=noalloc)
    if not noalloc:
        assert st == sv.SV_DEV_BAD_LENGTH
    q = torch.ones(4, 1, 2 * Hkv, 64, dtype=torch.bfloat16)
    check_retrieval(shape, lay, q, vis, sc, nv, kseq, max(kseq), valid=[True, False, True, False])
    assert (sc[[1, 3]] == 7.0).all()
    assert np.array_equal(np.unique(vis[[1, 3]].cpu().numpy()), [-1])
