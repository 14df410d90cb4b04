"""Shared by the prompt and 8-bit cache GPU tests: caches with known logical
rows, and the tolerances.

Prompt attention (bf16 in and out, fp32 logits, softmax and accumulation; the
weights enter the value product as bf16): as for tree attention, the output's own
rounding is at most 2^-8 |ref|; a weight's is at most 2^-8 of it, so the average
moves by at most 2^-8 sum p |v|; the fp32 logits (d <= 128 products of bf16
values, |z| < 2^7, relative error below 2^-18) move each weight by at most
2^-11, and the weights' sum by as much.  lse: the same logit error, and sums of
up to 2^16 terms.

Attention over the 8-bit cache: the rows' values are exact in fp16 and the
query's are taken with more bits than it has, so the logits carry fp32's error
alone, as above; the weights enter the value product with fp16's eleven bits,
2^-11 of each, and the sum once more the logits' error: 2^-11 + 2 * 2^-11 of
sum p |v|, below 2^-9.
"""

import math

import numpy as np
import torch

import oracle
from visual_token_sparsity_gb300 import synth

DEV = "cuda"


def i32(x):
    return torch.as_tensor(np.asarray(x, dtype=np.int32)).to(DEV)


def f64(t):
    return t.detach().double().cpu().numpy()


def assert_close(out, lse, ref, ref_lse, mag, weights, what=""):
    """weights: the share of sum p |v| that the product's weights may be off by."""
    out = f64(out)
    if out.size:
        bad = np.abs(out - ref) - (2.0 ** -8 * np.abs(ref) + weights * mag + 1e-30)
        i = np.unravel_index(np.argmax(np.where(np.isnan(bad), np.inf, bad)), bad.shape)
        assert (bad <= 0).all(), f"{what} at {i}: {out[i]} against {ref[i]}, sum p|v| {mag[i]}"
    if lse is not None:
        lse = f64(lse)
        none = np.isneginf(ref_lse)
        assert (np.isneginf(lse) == none).all(), f"{what}: lse of rows that see nothing"
        err = np.abs(lse[~none] - ref_lse[~none])
        assert err.size == 0 or err.max() <= 1e-3, f"{what}: lse off by {err.max()}"


PROMPT_WEIGHTS = 2.0 ** -8 + 2.0 ** -10
KV8_WEIGHTS = 2.0 ** -9


class Cache8:
    """One layer: logical codes and scales of both pools, and the paged ones."""

    def __init__(self, B, Hkv, d, tokens, seed, spare=2, factor=None):
        self.B, self.Hkv, self.d = B, Hkv, d
        self.per = synth.blocks_for(tokens) or 1
        self.blocks = B * self.per + spare
        self.bt = synth.random_block_table(B, self.per, self.blocks, seed=seed + 1)
        x = [synth.normal_bf16((B, Hkv, self.per, 16, d), seed + 2 + i).double().numpy() for i in range(2)]
        if factor is not None:                     # [B][Hkv][per][2], a factor of each page's rows
            x = [y * factor[..., i, None, None] for i, y in enumerate(x)]
        top = [np.abs(y).max((3, 4)) for y in x]
        self.scales = np.stack([np.exp2(np.maximum(np.ceil(np.log2(t / 448)), -126)) for t in top], -1)
        self.codes = [oracle.to_e4m3(y / self.scales[..., i, None, None]).reshape(B, Hkv, -1, d)
                      for i, y in enumerate(x)]

    def rows(self, which):
        """Logical values [B][Hkv][capacity][d]."""
        return np.stack([oracle.kv8_rows(self.codes[which][b], self.scales[b, ..., which]) for b in range(self.B)])

    def pools(self):
        """k_pool, v_pool (float8), scales on the device; pages that nobody holds are NaN."""
        out = []
        bt = self.bt.numpy()
        for which in range(2):
            pool = np.full((self.blocks, self.Hkv, 16, self.d), 0x7F, np.uint8)
            c = self.codes[which].reshape(self.B, self.Hkv, self.per, 16, self.d)
            for b in range(self.B):
                pool[bt[b]] = c[b].transpose(1, 0, 2, 3)
            out.append(torch.from_numpy(pool).to(DEV).view(torch.float8_e4m3fn))
        sc = np.full((self.blocks, self.Hkv, 2), np.nan, np.float32)
        for b in range(self.B):
            sc[bt[b]] = self.scales[b].transpose(1, 0, 2)
        return out[0], out[1], torch.from_numpy(sc).to(DEV)

    def layer(self):
        from visual_token_sparsity_gb300 import binding as sv
        return sv.Kv8Layer(*self.pools())

    def read_back(self, layer):
        """(codes, scales) in logical order, from the device's pools."""
        bt = self.bt.numpy()
        pools = [p.view(torch.uint8).cpu().numpy() for p in (layer.k_pool, layer.v_pool)]
        codes = [np.stack([p[bt[b]].transpose(1, 0, 2, 3).reshape(self.Hkv, -1, self.d) for b in range(self.B)])
                 for p in pools]
        sc = layer.scales.cpu().numpy()
        return codes, np.stack([sc[bt[b]].transpose(1, 0, 2) for b in range(self.B)])


def select(B, Hkv, nv, ks, k, seed):
    """[B][Hkv][k] ascending distinct indices below nv[b], -1 behind ks[b]."""
    g = np.random.default_rng(seed)
    out = np.full((B, Hkv, k), -1, dtype=np.int32)
    for b in range(B):
        for h in range(Hkv):
            out[b, h, :ks[b]] = np.sort(g.permutation(nv[b])[:ks[b]])
    return out


def oracle_decode(q, K, V, vis, nv, nt, ks, scale):
    """(out, lse, mag) [B][H].. of every sequence's own counts; vis None: all visual tokens."""
    B, H, d = q.shape
    G = H // K.shape[1]
    out, lse, mag = np.zeros((B, H, d)), np.full((B, H), -math.inf), np.zeros((B, H, d))
    for b in range(B):
        for h in range(H):
            g = h // G
            tok = list(range(nv[b])) if vis is None else vis[b, g, :ks[b]].tolist()
            tok = np.array(tok + list(range(nv[b], nv[b] + nt[b])), dtype=np.int64)
            out[b, h], lse[b, h], mag[b, h] = oracle.attend(f64(q[b, h]), K[b, g, tok], V[b, g, tok], scale)
    return out, lse, mag


def oracle_select(q, K, nv, ks):
    """([B][Hkv][max ks] ascending indices of the exact scores, -1 behind ks[b]; scores per (b, g))."""
    B, R, H, d = q.shape
    Hkv = K.shape[1]
    vis, scores = np.full((B, Hkv, max(ks)), -1, np.int32), {}
    for b in range(B):
        for g in range(Hkv):
            qbar = f64(q[b]).reshape(R, Hkv, H // Hkv, d)[:, g].sum((0, 1))
            s = K[b, g, :nv[b]] @ qbar
            scores[b, g] = s
            vis[b, g, :ks[b]] = np.sort(np.argsort(-s, kind="stable")[:ks[b]])
    return vis, scores
