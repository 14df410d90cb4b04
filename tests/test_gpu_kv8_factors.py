"""GPU: attention over 8-bit pages whose factors lie far apart.

What the kernel promises: a token's weight in the value product is its softmax weight
times its page's factor, rounded to fp16's eleven bits, or to 2^-30 of the largest such
product of the row where that is coarser.  So with p the softmax weights, f the factors
and v8 the e4m3 values

  |error| <= 2^-8 |out| + 2^-9 sum p f |v8| + 2^-31 max(p f) sum |v8|

(the output's own rounding; the weights' bits and twice the logits' error, 2^-11 each;
the products' step)."""

import math

import numpy as np
import pytest
import torch

import oracle
from kv8_util import DEV, KV8_WEIGHTS, Cache8, f64
from test_gpu_kv8 import attend
from visual_token_sparsity_gb300 import synth

pytestmark = pytest.mark.gpu


def check(out, lse, q, c, n, scale):
    """Every head over tokens [0, n) of sequence 0."""
    H, Hkv = q.shape[1], c.Hkv
    K, V = c.rows(0), c.rows(1)
    page = np.arange(n) // 16
    got, norm = f64(out), f64(lse)
    for h in range(H):
        g = h // (H // Hkv)
        ref, ref_lse, mag = oracle.attend(f64(q[0, h]), K[0, g, :n], V[0, g, :n], scale)
        p = np.exp(scale * (K[0, g, :n] @ f64(q[0, h])) - ref_lse)
        f = c.scales[0, g, page, 1]
        v8 = np.abs(oracle.E4M3[c.codes[1][0, g, :n]])
        bound = 2.0 ** -8 * np.abs(ref) + KV8_WEIGHTS * mag + 2.0 ** -31 * (p * f).max() * v8.sum(0) + 1e-30
        err = np.abs(got[0, h] - ref) / bound
        assert err.max() <= 1, f"head {h}: {err.max()} of the bound"
        assert abs(norm[0, h] - ref_lse) <= 1e-3


@pytest.mark.parametrize("H,Hkv,d", [(2, 2, 64), (8, 1, 128), (16, 1, 128), (16, 1, 64), (7, 1, 128)])
@pytest.mark.parametrize("exponent,gap", [(16, 20), (29, 30), (30, 60), (60, 100), (90, 100), (110, 100)])
def test_large_values_of_tokens_without_weight(lib, H, Hkv, d, exponent, gap):
    """Some pages' values are 2^exponent larger, their softmax weights 2^gap smaller: they
    take no bit from the others.  Odd heads weigh the same tokens 2^gap more."""
    from visual_token_sparsity_gb300 import binding as sv
    n, scale = 700, 0.125
    c = Cache8(1, Hkv, d, n, seed=100)
    g = np.random.default_rng(7)
    big = g.random(c.per) < 0.3
    big[[0, 20]] = True, False
    tok = np.repeat(big, 16)
    c.scales[..., 0] = 2.0 ** -6
    c.codes[0][..., 0] = np.where(tok, oracle.to_e4m3(-448.0), 0)          # -7
    c.scales[0, :, big, 1] *= 2.0 ** exponent
    q = synth.normal_bf16((1, H, d), 18)
    q[..., 0] = gap * math.log(2) / (7 * scale)
    q[:, 1::2, 0] *= -1
    q = q.to(DEV)
    out, lse, status = attend(c, q, sv.SeqBatch(c.bt.to(DEV), n - 30, 30), None, 0, scale)
    assert status == 0
    check(out, lse, q, c, n, scale)


@pytest.mark.parametrize("exponent", [0, 10, 19, 20, 21, 25, 28, 30, 33, 60])
def test_bits_of_values_beside_larger_ones(lib, exponent):
    """Tokens of equal weight, give or take, whose pages' factors are 2^exponent apart, in
    dims of their own: eleven bits down to 2^-20, fewer below."""
    from visual_token_sparsity_gb300 import binding as sv
    n, d = 320, 64
    c = Cache8(1, 1, d, n, seed=101)
    tok = np.arange(c.codes[0].shape[2]) // 16 % 2 == 1
    c.codes[1][0, 0, tok, : d // 2] = 0
    c.codes[1][0, 0, ~tok, d // 2:] = 0
    c.scales[..., 1] = np.where(np.arange(c.per) % 2 == 1, 2.0 ** (exponent // 2), 2.0 ** (exponent // 2 - exponent))
    q = synth.normal_bf16((1, 3, d), 19).to(DEV)
    out, lse, status = attend(c, q, sv.SeqBatch(c.bt.to(DEV), n, 0), None, 0, 0.06)
    assert status == 0
    check(out, lse, q, c, n, 0.06)
