"""GPU: causal attention of packed prompts against the fp64 oracle."""

import math

import numpy as np
import pytest
import torch

import oracle
from kv8_util import DEV, PROMPT_WEIGHTS, assert_close, f64, i32
from visual_token_sparsity_gb300 import synth

pytestmark = pytest.mark.gpu


class Prompt:
    """Packed sequences of a fused projection; `lead` tokens before the first
    and `behind` tokens after the last one belong to none."""

    def __init__(self, H, Hkv, d, lens, seed, lead=0, behind=0, std=1.0):
        self.H, self.Hkv, self.d = H, Hkv, d
        self.start = lead + np.concatenate([[0], np.cumsum(lens)])
        self.N = int(self.start[-1]) + behind
        proj = synth.normal_bf16((self.N, H + 2 * Hkv, d), seed, std=std)
        self.proj = proj.to(DEV)
        self.q, self.k, self.v = self.proj[:, :H], self.proj[:, H: H + Hkv], self.proj[:, H + Hkv:]
        self.scale = 1 / math.sqrt(d)

    def ref(self):
        return oracle.prompt_attention(f64(self.q), f64(self.k), f64(self.v), self.start, self.scale)

    def run(self, lse=True, ws=None, stream=None):
        from visual_token_sparsity_gb300 import binding as sv
        out = torch.full((self.N, self.H, self.d), 7.0, dtype=torch.bfloat16, device=DEV)
        norm = torch.full((self.N, self.H), 7.0, device=DEV) if lse else None
        own = ws is None
        if own:
            ws = sv.workspace(sv.sv_prompt_attn_workspace_bytes(self.N, len(self.start) - 1, self.H, self.Hkv, self.d))
        sv.sv_prompt_attn(self.q, self.k, self.v, i32(self.start), self.scale, out, norm, ws, stream=stream)
        if own:
            assert sv.sv_read_device_status(ws) == 0
        return out, norm

    def check(self, out, lse, what=""):
        a, b = self.start[0], self.start[-1]
        ref, ref_lse, mag = self.ref()
        assert_close(out[a:b], lse[a:b], ref[a:b], ref_lse[a:b], mag[a:b], PROMPT_WEIGHTS, what)
        for x in (out[:a], out[b:], lse[:a], lse[b:]):
            assert (x == 7).all(), f"{what}: rows of no sequence"


CASES = [
    # H, Hkv, d, lengths
    (1, 1, 64, [1]), (2, 1, 128, [0, 0]), (4, 2, 64, [1, 0, 2, 17, 1]), (4, 4, 128, [127, 128, 129]),
    (28, 4, 128, [18, 1, 36, 37, 0, 97]), (6, 2, 64, [42, 43, 85, 300]), (5, 1, 128, [25, 26, 51, 230]),
    (16, 1, 64, [8, 7, 9, 16, 17, 140]), (16, 1, 128, [3, 257]), (8, 4, 128, [64, 128, 65, 383]),
    (4, 1, 64, [513, 31]), (2, 2, 64, [255, 256, 257, 1]), (2, 2, 128, [1000, 3, 512]), (14, 2, 128, [700]),
    (32, 32, 128, [130]), (13, 1, 128, [9, 10, 200]), (3, 1, 64, [1] * 70 + [33] * 9),
]


@pytest.mark.parametrize("H,Hkv,d,lens", CASES)
def test_lengths_and_heads(lib, H, Hkv, d, lens):
    p = Prompt(H, Hkv, d, lens, seed=11 + H, lead=3, behind=5)
    p.check(*p.run())


@pytest.mark.parametrize("H,Hkv,d,n,std", [(4, 2, 64, 400, 3.0), (7, 1, 128, 333, 2.0), (2, 2, 128, 260, 0.05)])
def test_sharp_and_flat_weights(lib, H, Hkv, d, n, std):
    p = Prompt(H, Hkv, d, [n], seed=5, std=std)
    p.check(*p.run())


def test_growing_logits_move_the_maximum(lib):
    """Each later key outweighs the earlier ones by far, tile after tile, and back."""
    for order in (1, -1):
        p = Prompt(2, 1, 64, [700], seed=6)
        grow = torch.linspace(0, 60, 700, device=DEV).to(torch.bfloat16)
        p.q[:] = 0
        p.q[:, :, 0] = 8.0
        p.k[:] = 0
        p.k[:, :, 0] = (grow if order > 0 else grow.flip(0))[:, None]
        p.check(*p.run(), what=str(order))


def test_equal_keys_average_the_values(lib):
    p = Prompt(2, 1, 128, [300], seed=7)
    p.k[:] = 0
    out, lse = p.run()
    p.check(out, lse)
    n = torch.arange(1, 301, device=DEV)
    assert (lse - n.log()[:, None]).abs().max() < 1e-5


def test_contiguous_operands_and_no_lse(lib):
    p = Prompt(4, 2, 64, [50, 77], seed=8)
    with_lse = p.run()[0]
    p.q, p.k, p.v = (x.contiguous() for x in (p.q, p.k, p.v))
    assert torch.equal(p.run(lse=False)[0].view(torch.int16), with_lse.view(torch.int16))


def test_the_same_bits_every_time_and_wherever_a_sequence_lies(lib):
    p = Prompt(28, 4, 128, [210, 333, 5, 64], seed=9)
    a, la = p.run()
    for _ in range(3):
        b, lb = p.run()
        assert torch.equal(a.view(torch.int16), b.view(torch.int16)) and torch.equal(la, lb)
    one = Prompt(28, 4, 128, [333], seed=9)
    one.q, one.k, one.v = (x[210:543] for x in (p.q, p.k, p.v))
    b, lb = one.run()
    assert torch.equal(a[210:543].view(torch.int16), b.view(torch.int16)) and torch.equal(la[210:543], lb)


@pytest.mark.parametrize("H,Hkv,d", [(4, 2, 64), (7, 1, 128), (2, 2, 128)])
@pytest.mark.parametrize("at", [0, 40, 130, 299])
def test_what_a_row_does_not_see_has_no_part(lib, H, Hkv, d, at):
    """Infinities and NaN in K and V of a token reach the rows from it on, and no
    other sequence's."""
    from visual_token_sparsity_gb300 import binding as sv
    clean = Prompt(H, Hkv, d, [100, 300, 60], seed=12)
    ref, ref_lse, mag = clean.ref()
    t = 100 + at
    for what in ("v", "k"):
        p = Prompt(H, Hkv, d, [100, 300, 60], seed=12)
        if what == "v":
            p.v[t, 0, 3] = float("inf")
            p.v[t, 0, d - 1] = float("nan")
        else:
            p.k[t, 0, 5] = float("nan")
        out, lse = p.run()
        G = H // Hkv
        heads = [h for h in range(H) if h // G == 0]
        other = [h for h in range(H) if h // G != 0]
        seen = np.zeros((p.N, H), bool)
        seen[t:400, heads] = True
        got, want = f64(out), ref.copy()
        if what == "v":
            assert np.isposinf(got[..., 3][seen]).all() and np.isnan(got[..., d - 1][seen]).all()
            cols = [c for c in range(d) if c not in (3, d - 1)]
            assert_close(out[..., cols], lse, ref[..., cols], ref_lse, mag[..., cols], PROMPT_WEIGHTS, what)
        else:
            assert np.isnan(got[seen]).all() and np.isnan(f64(lse)[seen]).all()
        rest = ~seen
        assert_close(out[torch.from_numpy(rest).to(DEV)], lse[torch.from_numpy(rest).to(DEV)], want[rest], ref_lse[rest],
                     mag[rest], PROMPT_WEIGHTS, what)


def test_infinite_values_of_both_signs(lib):
    p = Prompt(2, 1, 64, [200], seed=13)
    p.v[10, 0, 0], p.v[20, 0, 0], p.v[150, 0, 1] = float("inf"), float("-inf"), float("-inf")
    out, _ = p.run()
    got = f64(out)
    assert np.isfinite(got[:10]).all()
    assert np.isposinf(got[10:20, :, 0]).all() and np.isnan(got[20:, :, 0]).all()
    assert np.isfinite(got[:150, :, 1]).all() and np.isneginf(got[150:, :, 1]).all()
    assert np.isfinite(got[..., 2:]).all()


@pytest.mark.parametrize("start", [[0, 10, 5, 40], [0, 50], [-1, 20, 40], [3, 2], [0, 20, 41]])
def test_starts_that_do_not_ascend_compute_nothing(lib, start):
    from visual_token_sparsity_gb300 import binding as sv
    p = Prompt(4, 2, 64, [40], seed=14)
    ws = sv.workspace(sv.sv_prompt_attn_workspace_bytes(40, 3, 4, 2, 64))
    out, lse = torch.full((40, 4, 64), 7.0, dtype=torch.bfloat16, device=DEV), torch.full((40, 4), 7.0, device=DEV)
    sv.sv_prompt_attn(p.q, p.k, p.v, i32(start), 0.1, out, lse, ws)
    assert sv.sv_read_device_status(ws, clear=True) == sv.SV_DEV_BAD_LENGTH
    assert (out == 7).all() and (lse == 7).all()
    p.check(*p.run(ws=ws))                    # the workspace serves the next call
    assert sv.sv_read_device_status(ws) == 0


def test_graph_replay_another_stream_and_a_shared_workspace(lib):
    from visual_token_sparsity_gb300 import binding as sv
    ps = [Prompt(28, 4, 128, [150, 9, 300], seed=20), Prompt(4, 2, 64, [33] * 8, seed=21), Prompt(2, 2, 128, [1], seed=22)]
    want = [p.run() for p in ps]
    ws = sv.workspace(max(sv.sv_prompt_attn_workspace_bytes(p.N, len(p.start) - 1, p.H, p.Hkv, p.d) for p in ps))
    s = torch.cuda.Stream()
    starts = [i32(p.start) for p in ps]
    outs = [torch.zeros_like(w[0]) for w in want]
    lses = [torch.zeros_like(w[1]) for w in want]
    torch.cuda.synchronize()

    def all_calls(stream=None):
        for p, st, o, l in zip(ps, starts, outs, lses):
            sv.sv_prompt_attn(p.q, p.k, p.v, st, p.scale, o, l, ws, stream=stream)

    def check():
        torch.cuda.synchronize()
        for w, o, l in zip(want, outs, lses):
            assert torch.equal(w[0].view(torch.int16), o.view(torch.int16)) and torch.equal(w[1], l)
            o.zero_()
            l.zero_()
        torch.cuda.synchronize()
    all_calls(stream=s)
    check()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        all_calls()
    for _ in range(3):
        graph.replay()
        check()
    # other inputs through the same graph
    ps[0].proj.copy_(synth.normal_bf16(tuple(ps[0].proj.shape), 77).to(DEV))
    graph.replay()
    torch.cuda.synchronize()
    ps[0].check(outs[0], lses[0])
    assert sv.sv_read_device_status(ws) == 0


def test_a_long_prompt(lib):
    """Rows of a sequence whose keys span many tiles, against sampled references."""
    H, Hkv, d, n = 14, 2, 128, 5000
    p = Prompt(H, Hkv, d, [n], seed=30)
    out, lse = p.run()
    K, V, Q = f64(p.k), f64(p.v), f64(p.q)
    rows = [0, 1, 127, 128, 2047, 2500, 4095, 4096, n - 2, n - 1]
    for h in (0, 6, 7, 13):
        ref = [oracle.attend(Q[i, h], K[: i + 1, h // 7], V[: i + 1, h // 7], p.scale) for i in rows]
        assert_close(out[rows, h], lse[rows, h], *(np.stack([r[j] for r in ref]) for j in (0, 1, 2)), PROMPT_WEIGHTS)


def test_lse_feeds_the_softmax_retrieval(lib):
    """The prompt's lse of its last rows is the normaliser of their attention."""
    p = Prompt(4, 2, 64, [200], seed=31)
    _, lse = p.run()
    _, ref, _ = p.ref()
    assert np.abs(f64(lse) - ref).max() < 1e-4
