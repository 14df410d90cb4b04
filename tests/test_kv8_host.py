"""CPU: the prompt and 8-bit cache calls refuse bad arguments before anything is
launched, report their sizes, and the binding's struct matches the header."""

import ctypes
import os
import shutil
import subprocess

import pytest
import torch

from test_drafts_host import BAD_ROTATIONS, INVALID, UNSUPPORTED, WORKSPACE, P, rot, seqs

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEAD = 256 + 4 * 4096


@pytest.fixture(scope="module")
def lib():
    if not shutil.which("nvcc") and not os.path.exists("/usr/local/cuda/bin/nvcc"):
        pytest.skip("nvcc not available")
    from visual_token_sparsity_gb300 import binding, build
    return binding.load(build.build())


def layer8(Hkv=2, d=64, blocks=100, k=0x10000, scales=0x20000):
    from visual_token_sparsity_gb300 import binding as sv
    return sv.sv_kv8_layer(P(k), P(), P(scales), blocks, Hkv, d)


def test_prompt_arguments(lib):
    def call(q=P(0x1000000), qs=256, k=P(0x2000000), ks=128, v=P(0x3000000), vs=128, N=8, H=4, Hkv=2, d=64, scale=0.1,
             start=P(), B=2, out=P(0x4000000), ws=P(0x5000000), nb=HEAD - 1):
        return lib.sv_prompt_attn(q, qs, k, ks, v, vs, N, H, Hkv, d, scale, start, B, out, None, ws, nb, None)
    assert call() == WORKSPACE                           # (nothing before it is wrong)
    assert call(q=None) == call(k=None) == call(v=None) == call(out=None) == call(start=None) == INVALID
    assert call(ws=None) == call(N=-1) == call(B=-1) == call(H=3) == call(H=0) == call(Hkv=0) == INVALID
    assert call(H=34, qs=34 * 64) == call(d=80) == call(N=1 << 29, H=4) == UNSUPPORTED
    assert call(qs=255) == call(qs=248) == call(ks=120) == call(vs=132) == INVALID
    assert call(q=P(0x1000008)) == call(k=P(0x2000008)) == call(v=P(0x3000002)) == call(start=P(0x10002)) == INVALID
    for bad in (0.0, -0.1, float("inf"), float("nan"), 2.4e38):
        assert call(scale=bad) == INVALID
    assert call(scale=2.3e38) == call(scale=1e-45) == WORKSPACE
    # the output on an input, or misaligned
    full = dict(nb=HEAD)
    assert call(out=P(0x4000008), **full) == INVALID
    last = 7 * 256 * 2 + 4 * 64 * 2
    assert call(out=P(0x1000000), **full) == call(out=P(0x1000000 + last - 16), **full) == INVALID
    assert call(out=P(0x2000000 - 16), **full) == call(out=P(0x3000000), **full) == INVALID
    # nothing to do
    assert call(N=0, **full) == call(B=0, **full) == 0
    assert call(q=None, k=None, v=None, out=None, start=None, N=0, **full) == 0


def test_append_arguments(lib):
    r = rot()
    def call(q=P(0x1000000), qs=256, k=P(0x2000000), ks=128, v=P(0x3000000), vs=128, N=8, H=4, R=r, L=None, S=None,
             start=P(), qo=P(0x4000000), ko=None, ws=P(), nb=256):
        return lib.sv_kv8_append(q, qs, k, ks, v, vs, N, H, ctypes.byref(R), ctypes.byref(L or layer8()),
                                 ctypes.byref(S or seqs()), start, qo, ko, ws, nb, None)
    assert call(q=None) == call(v=None) == call(qo=None) == call(N=-1) == call(H=3) == call(ws=None) == INVALID
    assert call(nb=255) == WORKSPACE
    assert call(vs=120) == call(ks=132) == call(start=P(0x10001)) == call(ko=P(0x5000008)) == INVALID
    assert call(L=layer8(d=72)) == UNSUPPORTED
    assert call(L=layer8(scales=0)) == call(L=layer8(scales=0x20004)) == call(L=layer8(k=0x10008)) == INVALID
    # even shares: a multiple of the batch that the block table has room for
    assert call(start=None, N=9) == INVALID and b"multiple" in lib.sv_last_error()
    assert call(start=None, N=102) == INVALID and b"overflow" in lib.sv_last_error()
    assert call(S=seqs(n_vis=150, n_text=11)) == INVALID
    assert call(S=seqs(2 ** 30, 1, per=2 ** 27)) == UNSUPPORTED
    assert call(N=1 << 30, qs=256) == UNSUPPORTED
    # in place only with the same layout, and outputs apart
    assert call(qo=P(0x1000000), qs=512) == call(qo=P(0x2000000)) == call(qo=P(0x1000010)) == INVALID
    assert call(ko=P(0x2000000), ks=256) == call(ko=P(0x3000000)) == call(ko=P(0x4000000)) == INVALID
    assert call(ko=P(0x1000000 + 8 * 256 * 2 - 16)) == INVALID
    assert call(N=0) == call(N=0, q=None, k=None, v=None, qo=None, R=rot(pos=None)) == call(S=seqs(batch=0)) == 0
    for change, status in BAD_ROTATIONS:
        assert call(R=rot(**change)) == status


def test_retrieve_arguments(lib):
    def call(q=P(), R=1, H=4, L=None, S=None, k=10, idx=P(), ws=P(), nb=1 << 20):
        return lib.sv_kv8_retrieve_topk(q, R, H, ctypes.byref(L or layer8()), ctypes.byref(S or seqs()), k, idx, None,
                                        ws, nb, None)
    assert call(q=None) == call(idx=None) == call(R=0) == call(H=3) == call(k=0) == call(k=101) == INVALID
    assert call(q=P(0x10008)) == call(S=seqs(n_vis=0, n_text=10)) == call(L=layer8(scales=0)) == INVALID
    assert call(L=layer8(d=96)) == UNSUPPORTED
    assert call(nb=300) == WORKSPACE
    assert call(S=seqs(batch=2 ** 23)) == WORKSPACE and call(S=seqs(batch=2 ** 23 + 1)) == UNSUPPORTED
    assert call(S=seqs(batch=0)) == 0


def test_attention_arguments(lib):
    def call(q=P(0x1000000), H=4, scale=0.1, L=None, S=None, vis=None, k=0, out=P(0x2000000), ws=P(0x3000000), nb=255):
        return lib.sv_kv8_decode_attn(q, H, scale, ctypes.byref(L or layer8()), ctypes.byref(S or seqs()), vis, k, out,
                                      None, ws, nb, None)
    assert call() == WORKSPACE
    assert call(q=None) == call(out=None) == call(q=P(0x1000008)) == call(out=P(0x2000008)) == INVALID
    assert call(H=3) == call(H=0) == call(scale=float("nan")) == call(scale=2.4e38) == INVALID
    assert call(scale=0.0) == call(scale=-1.0) == WORKSPACE
    assert call(H=34) == call(L=layer8(d=80)) == UNSUPPORTED
    assert call(vis=P(), k=101) == call(vis=P(), k=-1) == call(S=seqs(0, 0)) == INVALID
    assert call(L=layer8(scales=0x20002)) == INVALID
    assert call(out=P(0x1000000)) == call(out=P(0x1000000 + 2 * 4 * 64 * 2 - 16)) == INVALID
    assert call(out=P(0x1000000 + 2 * 4 * 64 * 2)) == WORKSPACE
    assert call(S=seqs(2 ** 30, 5, per=2 ** 27)) == UNSUPPORTED
    assert call(S=seqs(batch=0), nb=1 << 20) == 0


@pytest.mark.parametrize("H,Hkv,d", [(28, 4, 128), (4, 2, 64), (32, 32, 128), (16, 1, 64), (1, 1, 64)])
def test_workspaces_serve_every_smaller_call(lib, H, Hkv, d):
    for B in (1, 2, 8, 16, 33):
        sizes = [lib.sv_kv8_attn_workspace_bytes(B, H, Hkv, d, n) for n in range(1, 60000, 61)]
        assert sizes == sorted(sizes) and sizes[0] >= HEAD
        sizes = [lib.sv_kv8_retrieve_workspace_bytes(B, H, Hkv, d, n, 1) for n in range(1, 60000, 61)]
        assert sizes == sorted(sizes)
    for n in (1, 33, 200, 1568, 12800, 50432):
        sizes = [lib.sv_kv8_attn_workspace_bytes(B, H, Hkv, d, n) for B in range(1, 300)]
        assert sizes == sorted(sizes), n
    assert lib.sv_kv8_attn_workspace_bytes(1, 5, 2, 64, 9) == lib.sv_kv8_attn_workspace_bytes(-1, 4, 2, 64, 9) == 256
    assert lib.sv_kv8_retrieve_workspace_bytes(-1, 4, 2, 64, 9, 1) == 256
    assert lib.sv_prompt_attn_workspace_bytes(100, 4, H, Hkv, d) >= HEAD


def test_struct_layout(lib, tmp_path):
    if not shutil.which("gcc"):
        pytest.skip("gcc not available")
    from visual_token_sparsity_gb300 import binding as sv
    fields = [f for f, _ in sv.sv_kv8_layer._fields_]
    lines = ["#include <stddef.h>", "#include <stdio.h>", '#include "sv.h"', "int main(void) {",
             'printf("%zu\\n", sizeof(sv_kv8_layer));']
    lines += [f'printf("%zu\\n", offsetof(sv_kv8_layer, {f}));' for f in fields]
    (tmp_path / "a.c").write_text("\n".join(lines + ["return 0;", "}"]) + "\n")
    subprocess.run(["gcc", "-I", os.path.join(ROOT, "include"), str(tmp_path / "a.c"), "-o", str(tmp_path / "a")],
                   check=True)
    got = subprocess.run([str(tmp_path / "a")], capture_output=True, text=True, check=True).stdout.split()
    assert [int(x) for x in got] == [ctypes.sizeof(sv.sv_kv8_layer)] + [getattr(sv.sv_kv8_layer, f).offset for f in fields]


def test_binding_refuses_before_the_library(lib):
    from visual_token_sparsity_gb300 import binding as sv
    pool = lambda t=torch.uint8, n=16: torch.zeros(3, 2, n, 64, dtype=t)
    with pytest.raises(ValueError, match="pools"):
        sv.Kv8Layer(pool(n=8), pool(n=8), torch.zeros(3, 2, 2))
    with pytest.raises(ValueError, match="float8"):
        sv.Kv8Layer(pool(torch.int8), pool(), torch.zeros(3, 2, 2))
    with pytest.raises(ValueError, match="scales"):
        sv.Kv8Layer(pool(), pool(), torch.zeros(3, 2))
    with pytest.raises(ValueError, match="CUDA"):
        sv.Kv8Layer(pool(), pool(), torch.zeros(3, 2, 2))
