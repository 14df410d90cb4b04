"""CPU: the draft and branch calls refuse bad arguments before anything is
launched, report their sizes, and the binding's structs match the header."""

import ctypes
import os
import shutil
import subprocess

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
INVALID, UNSUPPORTED, WORKSPACE = 1, 2, 4


@pytest.fixture(scope="module")
def lib():
    if not shutil.which("nvcc") and not os.path.exists("/usr/local/cuda/bin/nvcc"):
        pytest.skip("nvcc not available")
    from visual_token_sparsity_gb300 import binding, build
    return binding.load(build.build())


def P(addr=0x10000):
    return ctypes.c_void_p(addr)


def layer(Hkv=2, d=64, blocks=100, k=0x10000):
    from visual_token_sparsity_gb300 import binding as sv
    return sv.sv_kv_layer(P(k), P(), blocks, Hkv, d)


def seqs(n_vis=100, n_text=10, batch=2, per=10):
    from visual_token_sparsity_gb300 import binding as sv
    return sv.sv_seq_batch(P(), batch, per, n_vis, n_text)


def rot(**kw):
    from visual_token_sparsity_gb300 import binding as sv
    v = dict(cos_sin=P(), n_pos=50, rot_dim=64, interleaved=0, pos=P(), n_axes=1, section=(ctypes.c_int32 * 3)(),
             q_weight=None, k_weight=None, eps=1e-6)
    v.update(kw)
    return sv.sv_rotation(*v.values())


BAD_ROTATIONS = [
    (dict(rot_dim=12), INVALID), (dict(rot_dim=72), INVALID), (dict(rot_dim=-8), INVALID),
    (dict(eps=-1.0), INVALID), (dict(eps=float("nan")), INVALID), (dict(q_weight=P(0x10008)), INVALID),
    (dict(cos_sin=None), INVALID), (dict(cos_sin=P(0x10008)), INVALID), (dict(pos=None), INVALID),
    (dict(n_pos=0), INVALID), (dict(n_axes=0), UNSUPPORTED), (dict(n_axes=4), UNSUPPORTED),
    (dict(n_axes=2, section=(ctypes.c_int32 * 3)(16, 15, 1)), INVALID),
    (dict(n_axes=2, section=(ctypes.c_int32 * 3)(33, -1, 0)), INVALID),
]


@pytest.mark.parametrize("change,status", BAD_ROTATIONS)
def test_rotation_descriptor(lib, change, status):
    r = rot(**change)
    out = lambda i: P(0x1000000 * (i + 1))
    assert lib.sv_qk_norm_rope(P(), 256, P(0x400000), 256, 1, 8, 4, 4, 64, ctypes.byref(r), out(1), out(2), P(), 256,
                               None) == status
    assert lib.sv_qk_norm_rope_append(P(), 256, P(0x400000), 128, P(0x500000), 128, 3, 4, ctypes.byref(r),
                                      ctypes.byref(layer()), ctypes.byref(seqs()), None, out(1), P(), 256,
                                      None) == status


def test_encoder_arguments(lib):
    r = rot()
    def call(q=P(0x1000000), qs=256, k=P(0x2000000), ks=256, B=1, N=8, H=4, Hk=4, d=64, R=r, qo=P(0x3000000),
             ko=P(0x4000000), ws=P(), nb=256):
        return lib.sv_qk_norm_rope(q, qs, k, ks, B, N, H, Hk, d, None if R is None else ctypes.byref(R), qo, ko, ws,
                                   nb, None)
    assert call(q=None) == call(ko=None) == call(R=None) == call(ws=None) == INVALID
    assert call(nb=255) == WORKSPACE
    assert call(d=96) == UNSUPPORTED
    assert call(H=0) == call(B=-1) == call(N=-1) == INVALID
    assert call(qs=255) == call(qs=260) == call(ks=248) == INVALID
    assert call(q=P(0x1000008)) == call(qo=P(0x3000008)) == INVALID
    # outputs on the inputs or on one another
    assert call(qo=P(0x1000000)) == call(qo=P(0x1000000 - 16)) == call(ko=P(0x3000000 + 4 * 8 * 64 * 2 - 16)) == INVALID
    assert call(N=0) == 0                       # nothing to do, nothing launched


def test_append_arguments(lib):
    r = rot()
    def call(q=P(0x1000000), qs=256, k=P(0x2000000), ks=128, v=P(0x3000000), vs=128, T=4, H=4, L=None, S=None,
             qo=P(0x4000000), ws=P(), nb=256):
        return lib.sv_qk_norm_rope_append(q, qs, k, ks, v, vs, T, H, ctypes.byref(r), ctypes.byref(L or layer()),
                                          ctypes.byref(S or seqs()), None, qo, ws, nb, None)
    assert call(v=None) == call(qo=None) == call(T=-1) == call(H=3) == INVALID
    assert call(S=seqs(n_vis=150, n_text=7)) == INVALID                # 161 tokens, 160 positions
    assert b"overflow" in lib.sv_last_error()
    assert call(vs=120) == call(ks=132) == INVALID
    assert call(L=layer(d=72)) == UNSUPPORTED
    assert call(nb=0) == WORKSPACE
    # in place only with the same layout
    assert call(qo=P(0x1000000), qs=512) == INVALID
    assert call(qo=P(0x2000000)) == INVALID
    assert call(T=0) == 0


def test_tree_arguments(lib):
    def call(q=P(0x1000000), T=5, H=4, scale=0.1, L=None, S=None, vis=None, k=0, mask=None, out=P(0x2000000),
             ws=P(0x3000000), nb=1 << 26):
        return lib.sv_tree_attn(q, T, H, scale, ctypes.byref(L or layer()), ctypes.byref(S or seqs()), vis, k, mask,
                                None, out, None, ws, nb, None)
    assert call(q=None) == call(out=None) == call(q=P(0x1000008)) == call(out=P(0x2000008)) == INVALID
    assert call(H=3) == call(H=0) == call(T=-1) == call(T=65537) == INVALID
    assert call(H=34) == UNSUPPORTED                                    # 17 query heads per KV head
    assert call(scale=-0.1) == call(scale=float("inf")) == call(scale=float("nan")) == INVALID
    assert call(T=65, mask=P(), S=seqs(0, 10)) == UNSUPPORTED
    assert call(vis=P(), k=101) == call(vis=P(), k=-1) == INVALID
    assert call(T=51) == INVALID and b"overflow" in lib.sv_last_error()
    assert call(nb=255) == WORKSPACE
    assert call(L=layer(d=80)) == UNSUPPORTED
    assert call(T=0) == call(S=seqs(batch=0)) == 0


def test_tree_mask_and_output_addresses(lib):
    def call(mask=None, out=P(0x2000000), T=5):
        return lib.sv_tree_attn(P(0x1000000), T, 4, 0.1, ctypes.byref(layer()), ctypes.byref(seqs(0, 10)), None, 0,
                                mask, None, out, None, P(0x3000000), 255, None)
    assert call() == call(mask=P(0x10008)) == WORKSPACE                  # (nothing before it is wrong)
    assert call(mask=P(0x10004)) == INVALID
    rows = 2 * 5 * 4 * 64 * 2                                           # bytes of q
    assert call(out=P(0x1000000 + rows - 16)) == call(out=P(0x1000000 - rows + 16)) == INVALID
    assert call(out=P(0x1000000 + rows)) == call(out=P(0x1000000 - rows)) == call(out=P(0x1000000)) == WORKSPACE


def test_accept_arguments(lib):
    from visual_token_sparsity_gb300 import binding as sv
    def call(layers=(layer(),), S=None, T=9, path=P(), n=4, ws=P(), nb=256):
        arr = (sv.sv_kv_layer * max(1, len(layers)))(*layers)
        return lib.sv_kv_accept(arr, len(layers), ctypes.byref(S or seqs()), T, path, n, None, ws, nb, None)
    assert call(path=None) == call(n=10) == call(n=-1) == call(T=-1) == INVALID
    assert call(T=51) == INVALID
    assert call(S=seqs(0, 10), T=70, n=65) == UNSUPPORTED
    assert call(layers=(layer(), layer(d=128))) == call(layers=(layer(), layer(blocks=101))) == INVALID
    assert call(nb=100) == WORKSPACE
    assert call(layers=()) == call(n=0) == 0


def test_page_arguments(lib):
    from visual_token_sparsity_gb300 import binding as sv
    pool = lambda ref=P(), n=P(), pages=100: sv.sv_page_pool(ref, n, pages)
    need = lib.sv_pages_workspace_bytes(2, 10, 100)
    def release(p=pool(), S=None, nb=need):
        return lib.sv_pages_release(ctypes.byref(p), ctypes.byref(S or seqs(batch=0)), None, P(), nb, None)
    assert release(pool(ref=None)) == release(pool(n=None)) == release(pool(pages=0)) == INVALID
    assert release(pool(ref=P(0x10004))) == INVALID
    assert release(pool(pages=(1 << 30) + 1)) == UNSUPPORTED
    assert release(S=seqs(), nb=need - 1) == WORKSPACE
    assert release(S=seqs(batch=-1)) == release(S=seqs(per=0)) == INVALID
    assert release() == 0                       # an empty batch
    def fork(parent=P(), child=P(), n=2):
        return lib.sv_pages_fork(ctypes.byref(pool()), ctypes.byref(seqs()), parent, child, n, None, P(), need, None)
    assert fork(n=-1) == fork(parent=None) == fork(child=None) == INVALID
    assert fork(n=0) == 0
    def reserve(p=pool(), layers=(), S=None, T=4):
        arr = (sv.sv_kv_layer * max(1, len(layers)))(*layers)
        return lib.sv_pages_reserve(ctypes.byref(p), arr, len(layers), ctypes.byref(S or seqs()), T, None, P(), need,
                                    None)
    assert reserve(T=-1) == reserve(T=51) == reserve(S=seqs(n_text=-1)) == INVALID
    assert reserve(layers=(layer(blocks=99),)) == INVALID
    assert reserve(layers=(layer(), layer(Hkv=3))) == INVALID
    assert reserve(layers=tuple(layer() for _ in range(1025))) == UNSUPPORTED
    assert reserve(T=0) == 0


def test_workspace_sizes(lib):
    assert lib.sv_pages_workspace_bytes(0, 0, 0) >= 256
    assert lib.sv_pages_workspace_bytes(-1, 4, 4) == 256
    assert lib.sv_pages_workspace_bytes(16, 3152, 60000) >= 256 + 16 * 3152 * 20
    for bad in ((-1, 4, 4, 4, 64, 9), (1, 4, 5, 2, 64, 9), (1, 4, 4, 4, 64, -1)):
        assert lib.sv_tree_attn_workspace_bytes(*bad) == 256
    # a shorter call of the same shape fits the workspace of a longer one
    for B, H, Hkv, d in ((1, 4, 2, 64), (16, 32, 32, 128), (8, 28, 4, 128), (1, 16, 1, 64)):
        for T in (1, 7, 64, 500):
            last = 256
            for n in range(T, 60000, 487):
                w = lib.sv_tree_attn_workspace_bytes(B, T, H, Hkv, d, n)
                assert w >= last
                last = w


def test_struct_layouts(lib, tmp_path):
    if not shutil.which("gcc"):
        pytest.skip("gcc not available")
    from visual_token_sparsity_gb300 import binding as sv
    lines = ["#include <stddef.h>", "#include <stdio.h>", '#include "sv.h"', "int main(void) {"]
    want = []
    for st in ("sv_rotation", "sv_page_pool"):
        cls = getattr(sv, st)
        want.append(ctypes.sizeof(cls))
        lines.append(f'printf("%zu\\n", sizeof({st}));')
        for f, _ in cls._fields_:
            want.append(getattr(cls, f).offset)
            lines.append(f'printf("%zu\\n", offsetof({st}, {f}));')
    (tmp_path / "a.c").write_text("\n".join(lines + ["return 0;", "}"]) + "\n")
    subprocess.run(["gcc", "-I", os.path.join(ROOT, "include"), str(tmp_path / "a.c"), "-o", str(tmp_path / "a")],
                   check=True)
    got = subprocess.run([str(tmp_path / "a")], capture_output=True, text=True, check=True).stdout.split()
    assert [int(x) for x in got] == want


def test_binding_refuses_before_the_library(lib):
    from visual_token_sparsity_gb300 import binding as sv
    with pytest.raises(ValueError, match="CUDA"):
        sv.PagePool(torch.zeros(4, dtype=torch.int32), torch.zeros(1, dtype=torch.int32))
    with pytest.raises(ValueError, match="cos_sin"):
        sv.Rotation(torch.zeros(4, 8), torch.zeros(1, 2, dtype=torch.int32))
    with pytest.raises(ValueError, match="pos"):
        sv.Rotation(torch.zeros(4, 8, 2), torch.zeros(2, dtype=torch.int32))
    with pytest.raises(ValueError, match="pos"):
        sv.Rotation(torch.zeros(4, 8, 2), torch.zeros(1, 2, dtype=torch.int32), sections=[4, 4])
    with pytest.raises(ValueError, match="add up"):
        sv.Rotation(torch.zeros(4, 8, 2), torch.zeros(1, 2, dtype=torch.int32), sections=[4])
    with pytest.raises(ValueError, match="weight"):
        sv.Rotation(None, None, q_weight=torch.zeros(2, 8))


def test_calls_without_tokens_take_null_tensors(lib):
    """An empty tensor has no address: a step that drafted nothing is no error."""
    r = rot(pos=None)
    L, S = ctypes.byref(layer()), ctypes.byref(seqs())
    for B, N in ((1, 0), (0, 8)):
        assert lib.sv_qk_norm_rope(None, 256, None, 256, B, N, 4, 4, 64, ctypes.byref(r), None, None, P(), 256, None) == 0
    assert lib.sv_qk_norm_rope_append(None, 256, None, 128, None, 128, 0, 4, ctypes.byref(r), L, S, None, None, P(), 256,
                                      None) == 0
    assert lib.sv_tree_attn(None, 0, 4, 0.1, L, S, None, 0, None, None, None, None, P(), 1 << 26, None) == 0
    assert lib.sv_kv_accept(L, 1, S, 0, None, 0, None, P(), 256, None) == 0
    # with tokens they are still refused
    assert lib.sv_qk_norm_rope(None, 256, None, 256, 1, 8, 4, 4, 64, ctypes.byref(rot()), None, None, P(), 256, None) == INVALID
    assert lib.sv_qk_norm_rope(P(0x1000000), 256, P(0x2000000), 256, 1, 8, 4, 4, 64, ctypes.byref(r), P(0x3000000),
                               P(0x4000000), P(), 256, None) == INVALID
    assert lib.sv_qk_norm_rope_append(None, 256, None, 128, None, 128, 1, 4, ctypes.byref(rot()), L, S, None, None, P(),
                                      256, None) == INVALID
    assert lib.sv_tree_attn(None, 1, 4, 0.1, L, S, None, 0, None, None, None, None, P(), 1 << 26, None) == INVALID


@pytest.mark.parametrize("H,Hkv,d", [(28, 4, 128), (4, 2, 64), (32, 32, 128), (16, 1, 64), (1, 1, 64)])
def test_tree_workspace_serves_every_smaller_call(lib, H, Hkv, d):
    """Never larger for fewer sequences, drafted tokens or context tokens,
    whatever tiles and pieces the sizes are cut into."""
    size = lambda B, T, ctx: lib.sv_tree_attn_workspace_bytes(B, T, H, Hkv, d, ctx + T)
    Ts = list(range(1, 301)) + list(range(301, 4000, 37)) + [5600, 9728, 20000, 65535, 65536]
    for B in (1, 2, 8, 33):
        for ctx in (0, 100, 500, 1000, 3392, 12800, 50199):
            sizes = [size(B, T, ctx) for T in Ts]
            drop = [(T, a, b) for T, a, b in zip(Ts[1:], sizes, sizes[1:]) if b < a]
            assert not drop, (B, ctx, drop[0])
    for T in (1, 9, 33, 73, 74, 193, 2000):
        for ctx in (0, 300, 3000, 50000):
            by_batch = [size(B, T, ctx) for B in range(1, 160)]
            assert by_batch == sorted(by_batch), (T, ctx)
    # counters, and partial results for a GPU of CTAs: no more
    assert size(8, 65536, 50000) <= 256 + 4 * 4096 + 4 * 256 + 152 * 2 * 256 * (4 * d + 8) + 152 * 16


def test_the_plan_cases_take_the_plans_they_name(lib):
    """The GPU cases of test_gpu_tree_plans.py name the row tile and pieces that
    they were made for.  The rule, written again, has to give both those and the
    library's workspace size, which tells the row tile: (m, l) and O of two
    units' rows per CTA."""
    from test_gpu_tree_plans import CASES
    up = lambda a, b: -(-a // b)
    for name, (H, Hkv, d, B, T, n_vis, k, n_text, _, _, tile, row_tiles, pieces, by_unit) in CASES.items():
        rows, n = T * (H // Hkv), (n_vis if k is None else k) + n_text + T
        tiles = B * Hkv * up(n, 128)
        qt = 256 if rows > 128 and tiles >= up(8 * 152, up(rows, 256)) else 128
        rt = up(rows, qt)
        cols = max(1, min(152 // rt, tiles // 2))
        assert (qt, rt, cols, B * Hkv * rt <= cols * rt) == (tile, row_tiles, pieces, by_unit), name
        ctas = min(152, rt * (tiles // 2))
        size = up(ctas * 16, 256) * 256 + up(ctas * 2 * qt * 8, 256) * 256 + ctas * 2 * qt * d * 4
        assert lib.sv_tree_attn_workspace_bytes(B, T, H, Hkv, d, n) == 256 + 4 * 4096 + up(size, 256) * 256, name


def test_positions_stay_within_32_bits(lib):
    """A block table may have room for more positions than int32 counts; the
    calls whose kernels count them in 32 bits refuse such lengths."""
    from visual_token_sparsity_gb300 import binding as sv
    L = ctypes.byref(layer())
    for n_vis, n_text in ((2 ** 31 - 9, 4), (2 ** 30 - 4, 0), (2 ** 30, 2 ** 30)):
        S = seqs(n_vis, n_text, batch=1, per=2 ** 29)
        s = ctypes.byref(S)
        tree = lambda T: lib.sv_tree_attn(P(0x1000000), T, 4, 0.1, L, s, None, 0, None, None, P(0x2000000), None,
                                          P(0x3000000), 1 << 40, None)
        append = lambda T: lib.sv_qk_norm_rope_append(P(0x1000000), 256, P(0x2000000), 128, P(0x3000000), 128, T, 4,
                                                      ctypes.byref(rot()), L, s, None, P(0x4000000), P(), 256, None)
        accept = lambda T: lib.sv_kv_accept(L, 1, s, T, P(), 1, None, P(), 256, None)
        pool = sv.sv_page_pool(P(), P(), 100)
        reserve = lambda T: lib.sv_pages_reserve(ctypes.byref(pool), None, 0, s, T, None, P(), 1 << 40, None)
        assert tree(5) == append(5) == accept(5) == reserve(5) == UNSUPPORTED, (n_vis, n_text)
        assert b"2^30" in lib.sv_last_error()


def test_tree_scale_stays_finite_in_base_two(lib):
    """The kernel works with scale * log2(e): where that is infinite, products
    of 0 would be NaN."""
    call = lambda scale: lib.sv_tree_attn(P(0x1000000), 5, 4, scale, ctypes.byref(layer()), ctypes.byref(seqs()), None, 0,
                                          None, None, P(0x2000000), None, P(0x3000000), 255, None)
    assert call(2.3e38) == call(0.0) == call(1e-45) == WORKSPACE          # (nothing before it is wrong)
    assert call(2.4e38) == call(3.4e38) == call(float("inf")) == INVALID
