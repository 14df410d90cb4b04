"""CPU pins of the prompt and 8-bit cache oracle: closed forms, library routines
and brute force."""

import math

import numpy as np
import pytest
import torch

import oracle


def test_e4m3_values_and_rounding_are_torchs():
    codes = torch.arange(256, dtype=torch.uint8)
    want = codes.view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(np.isnan(want), np.isnan(oracle.E4M3))
    assert np.array_equal(want[~np.isnan(want)], oracle.E4M3[~np.isnan(want)])
    g = torch.Generator().manual_seed(1)
    x = torch.cat([torch.randn(20000, generator=g) * 2.0 ** torch.randint(-12, 9, (20000,), generator=g),
                   torch.tensor(oracle.E4M3[:127]), torch.tensor((oracle.E4M3[:126] + oracle.E4M3[1:127]) / 2),
                   torch.tensor([0.0, -0.0, 2.0 ** -10, -2.0 ** -10, 3 * 2.0 ** -10])]).double().clamp(-448, 448)
    want = x.float().to(torch.float8_e4m3fn).view(torch.uint8).numpy()     # (every x is an fp32 number)
    assert (x.float().double() == x).all()
    assert np.array_equal(oracle.to_e4m3(x.numpy()), want)


def test_e4m3_beyond_the_range():
    got = oracle.to_e4m3(np.array([449.0, 1e9, -1e9, math.inf, -math.inf, math.nan]))
    assert got.tolist() == [0x7E, 0x7E, 0xFE, 0x7E, 0xFE, 0x7F]


@pytest.mark.parametrize("top,scale", [(448.0, 1.0), (450.0, 2.0), (224.0, 0.5), (226.0, 1.0), (0.0, 2.0 ** -126),
                                       (1e-40, 2.0 ** -126), (3.0 * 2.0 ** 126, 2.0 ** 119), (1.75, 2.0 ** -8)])
def test_page_scale(top, scale):
    assert oracle.page_scale(np.array([0.0, -top, top / 3, math.inf, math.nan])) == scale


def test_append_in_pieces_equals_append_at_once_when_the_scale_is_the_first_ones():
    g = np.random.default_rng(2)
    rows = g.normal(size=(37, 3, 64)).astype(np.float32)
    rows = torch.tensor(rows).to(torch.bfloat16).double().numpy()
    rows[::16] *= 64                                       # the first row of each page is its largest
    whole = [np.zeros((3, 48, 64), np.uint8), np.full((3, 3), 7.0)]
    parts = [np.zeros((3, 48, 64), np.uint8), np.full((3, 3), 7.0)]
    oracle.kv8_append(*whole, 0, rows)
    for a, b in ((0, 1), (1, 9), (9, 20), (20, 37)):
        oracle.kv8_append(*parts, a, rows[a:b])
    assert np.array_equal(whole[0], parts[0]) and np.array_equal(whole[1], parts[1])
    # within half a step of e4m3, or of its smallest values
    back = oracle.kv8_rows(*whole)[:, :37]
    step = np.maximum(np.abs(rows.transpose(1, 0, 2)) / 16, 2.0 ** -10 * np.repeat(whole[1], 16, 1)[:, :37, None])
    assert (np.abs(back - rows.transpose(1, 0, 2)) <= step).all()


def test_growing_page_rounds_its_rows_again():
    codes, scales = np.zeros((1, 16, 64), np.uint8), np.zeros((1, 1))
    oracle.kv8_append(codes, scales, 0, np.full((2, 1, 64), 3.0))
    assert scales[0, 0] == 2.0 ** -7
    oracle.kv8_append(codes, scales, 2, np.full((1, 1, 64), 6000.0))
    assert scales[0, 0] == 16.0
    got = oracle.kv8_rows(codes, scales)[0, :3, 0]
    assert got.tolist() == [3.0, 3.0, 6144.0]              # 3/16 is a value; 6000/16 = 375 lies nearest to 384


def test_prompt_attention_is_torchs():
    g = torch.Generator().manual_seed(3)
    start = [2, 2, 7, 20]
    q, k, v = (torch.randn(21, h, 64, generator=g, dtype=torch.float64) for h in (6, 2, 2))
    out, lse, mag = oracle.prompt_attention(q.numpy(), k.numpy(), v.numpy(), start, 0.3)
    for a, b in ((2, 7), (7, 20)):
        x = [t[a:b].transpose(0, 1) for t in (q, k.repeat_interleave(3, 1), v.repeat_interleave(3, 1))]
        want = torch.nn.functional.scaled_dot_product_attention(*x, is_causal=True, scale=0.3).transpose(0, 1)
        assert np.allclose(out[a:b], want.numpy(), rtol=1e-12, atol=1e-13)
    assert np.isnan(out[:2]).all() and np.isnan(out[20:]).all()
    assert np.allclose(lse[2], 0.3 * (q[2].numpy() * k[2].repeat_interleave(3, 0).numpy()).sum(-1))
    assert (mag[2:20] >= np.abs(out[2:20]) - 1e-15).all()


def test_attend_is_the_sparse_decode_oracle():
    g = np.random.default_rng(4)
    q, K, V = g.normal(size=(1, 2, 64)), g.normal(size=(1, 1, 30, 64)), g.normal(size=(1, 1, 30, 64))
    vis = np.array([[[1, 5, 17]]])
    out, lse = oracle.sparse_decode_attention(q, K, V, vis, 20, 10, 0.2)
    tok = [1, 5, 17] + list(range(20, 30))
    for h in range(2):
        o, l, mag = oracle.attend(q[0, h], K[0, 0, tok], V[0, 0, tok], 0.2)
        assert np.allclose(o, out[0, h]) and np.allclose(l, lse[0, h]) and (mag >= np.abs(o) - 1e-15).all()
    o, l, _ = oracle.attend(q[0, 0], K[0, 0, :0], V[0, 0, :0], 0.2)
    assert (o == 0).all() and l == -math.inf
