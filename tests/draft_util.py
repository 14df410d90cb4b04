"""Shared by the draft and branch GPU tests: caches with known logical rows,
random trees, and the tolerances.

Tree attention (bf16 in and out, fp32 logits, softmax and accumulation; the
weights enter the value product as bf16): the output's own rounding is at most
2^-8 |ref|; a weight's is at most 2^-8 of it, so the average moves by at most
2^-8 sum p |v|; the fp32 logits (d <= 128 products of bf16 values, |z| < 2^7,
relative error below 2^-18) move each weight by at most 2^-11, and the weights'
sum by as much.  lse: the same logit error, and sums of up to 2^16 terms.

Norm and rotation: the output's rounding, 2^-8 |ref|, and a handful of fp32
roundings of terms no larger than the row's largest, below 2^-20 of it.
"""

import numpy as np
import torch

import oracle
from visual_token_sparsity_gb300 import synth

DEV = "cuda"


def i32(x):
    return torch.as_tensor(np.asarray(x, dtype=np.int32)).to(DEV)


def mask64(rows):
    """[B][T] Python ints (unsigned 64 bit) -> int64 device tensor."""
    return torch.as_tensor(np.array(rows, dtype=np.uint64).view(np.int64)).to(DEV)


def random_tree(T, g):
    m = []
    for t in range(T):
        p = int(g.integers(-1, t)) if t else -1
        m.append((m[p] if p >= 0 else 0) | 1 << t)
    return m


class Cache:
    """One layer: logical rows K, V [B][Hkv][capacity][d] and their pools."""

    def __init__(self, B, Hkv, d, tokens, seed, spare=2, std=1.0):
        self.per = synth.blocks_for(tokens) or 1
        self.blocks = B * self.per + spare
        self.bt = synth.random_block_table(B, self.per, self.blocks, seed=seed + 1)
        self.K = synth.normal_bf16((B, Hkv, self.per * 16, d), seed + 2, std=std)
        self.V = synth.normal_bf16((B, Hkv, self.per * 16, d), seed + 3)

    def pools(self):
        kp = synth.scatter_to_pool(self.K, self.bt, self.blocks)
        vp = synth.scatter_to_pool(self.V, self.bt, self.blocks)
        return kp.to(DEV), vp.to(DEV)

    def layer(self):
        from visual_token_sparsity_gb300 import binding as sv
        return sv.KvLayer(*self.pools())


def select(B, Hkv, nv, ks, k, seed):
    """[B][Hkv][k] ascending distinct indices below nv[b], -1 behind ks[b]."""
    g = np.random.default_rng(seed)
    out = np.full((B, Hkv, k), -1, dtype=np.int32)
    for b in range(B):
        for h in range(Hkv):
            out[b, h, :ks[b]] = np.sort(g.permutation(nv[b])[:ks[b]])
    return out


def f64(t):
    return t.detach().double().cpu().numpy()


def assert_tree_close(out, lse, ref, ref_lse, mag, what=""):
    out = f64(out)
    if out.size == 0:
        return
    bad = np.abs(out - ref) - (2.0 ** -8 * np.abs(ref) + (2.0 ** -8 + 2.0 ** -10) * mag + 1e-30)
    i = np.unravel_index(np.argmax(bad), bad.shape)
    assert (bad <= 0).all(), f"{what} at {i}: {out[i]} against {ref[i]}, sum p|v| {mag[i]}"
    if lse is not None:
        lse = f64(lse)
        none = np.isneginf(ref_lse)
        assert (np.isneginf(lse) == none).all(), f"{what}: lse of rows that see nothing"
        err = np.abs(lse[~none] - ref_lse[~none])
        assert err.size == 0 or err.max() <= 1e-3, f"{what}: lse off by {err.max()}"


def oracle_tree(q, cache, vis, nv, nt, ks, tn, mask, scale):
    """[B][T]... references over every sequence's own counts."""
    B, T, H, d = q.shape
    out, lse, mag = np.zeros((B, T, H, d)), np.full((B, T, H), -np.inf), np.zeros((B, T, H, d))
    for b in range(B):
        n = tn[b]
        v = None if vis is None else vis[b, :, :ks[b]]
        m = None if mask is None else mask[b][:n]
        out[b, :n], lse[b, :n], mag[b, :n] = oracle.tree_attention(
            f64(q[b, :n]), f64(cache.K[b]), f64(cache.V[b]), v, nv[b], nt[b], m, scale)
    return out, lse, mag
