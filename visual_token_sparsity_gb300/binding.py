"""ctypes binding of libsv (include/sv.h): argument marshalling only.

Every function here has the name of the C entry point it calls, checks that
tensors have the dtype / layout the C ABI documents, passes raw device
pointers and raises :class:`SvError` on a non-OK status.  All arithmetic runs
in the library's CUDA kernels; there is no other implementation behind these
calls, and loading fails loudly when the library is missing.
"""

import ctypes
import os

import torch

from . import build as _build

_lib = None

SV_OK = 0
SV_DEV_BAD_BLOCK = 0x1
SV_DEV_BAD_INDEX = 0x2
SV_DEV_BAD_LENGTH = 0x4
SV_DEV_BAD_POSITION = 0x8
SV_DEV_TIMEOUT = 0x10
SV_DEV_NO_PAGES = 0x20
BLOCK_TOKENS = 16


class SvError(RuntimeError):
    def __init__(self, status, msg):
        super().__init__(f"sv status {status}: {msg}")
        self.status = status


class sv_kv_layer(ctypes.Structure):
    _fields_ = [("k_pool", ctypes.c_void_p), ("v_pool", ctypes.c_void_p),
                ("num_blocks", ctypes.c_int32), ("n_kv_heads", ctypes.c_int32),
                ("head_dim", ctypes.c_int32)]


class sv_seq_batch(ctypes.Structure):
    _fields_ = [("block_table", ctypes.c_void_p), ("batch", ctypes.c_int32),
                ("max_blocks", ctypes.c_int32), ("n_vis", ctypes.c_int32),
                ("n_text", ctypes.c_int32), ("n_vis_seq", ctypes.c_void_p),
                ("n_text_seq", ctypes.c_void_p), ("k_seq", ctypes.c_void_p)]


class sv_rotation(ctypes.Structure):
    _fields_ = [("cos_sin", ctypes.c_void_p), ("n_pos", ctypes.c_int32), ("rot_dim", ctypes.c_int32),
                ("interleaved", ctypes.c_int32), ("pos", ctypes.c_void_p), ("n_axes", ctypes.c_int32),
                ("section", ctypes.c_int32 * 3), ("q_weight", ctypes.c_void_p), ("k_weight", ctypes.c_void_p),
                ("eps", ctypes.c_float)]


class sv_page_pool(ctypes.Structure):
    _fields_ = [("ref", ctypes.c_void_p), ("n_pages", ctypes.c_void_p), ("num_blocks", ctypes.c_int32)]


# (module constants and fields of their own: the calls of a decode step look them
# up a dozen times each)
_BF16, _F32, _I32, _U8 = torch.bfloat16, torch.float32, torch.int32, torch.uint8
_VP, _SZ, _I, _F, _I64 = ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int, ctypes.c_float, ctypes.c_int64
_SIGS = {
    "sv_status_string": (ctypes.c_char_p, [_I]),
    "sv_last_error": (ctypes.c_char_p, []),
    "sv_version": (ctypes.c_char_p, []),
    "sv_salience_workspace_bytes": (_SZ, [_I, _I, _I, _I]),
    "sv_retrieve_kernel_count": (_I, [_I, _I, _I]),
    "sv_salience_kernel_count": (_I, [_I, _I]),
    "sv_attn_kernel_count": (_I, [_I, _I, _I, _I]),
    "sv_topk_workspace_bytes": (_SZ, [_I, _I, _I]),
    "sv_prune_workspace_bytes": (_SZ, [_I, _I, _I]),
    "sv_retrieve_workspace_bytes": (_SZ, [_I, _I, _I, _I, _I, _I]),
    "sv_attn_workspace_bytes": (_SZ, [_I, _I, _I, _I, _I]),
    "sv_evict_workspace_bytes": (_SZ, []),
    "sv_salience_prefill": (_I, [_VP, _VP, _I, _I, _I, _I, _F, _VP, _VP, _SZ, _VP]),
    "sv_topk_rows": (_I, [_VP, _I, _I, _I, _VP, _VP, _SZ, _VP]),
    "sv_prune_compact": (_I, [_VP, _I, _I, _I, _VP, _I64, _VP, _VP, _VP, _SZ, _VP]),
    "sv_retrieve_topk": (_I, [_VP, _I, _I, ctypes.POINTER(sv_kv_layer),
                              ctypes.POINTER(sv_seq_batch), _I, _VP, _VP, _VP, _SZ, _VP]),
    "sv_retrieve_topk_noalloc": (_I, [_VP, _I, _I, ctypes.POINTER(sv_kv_layer),
                                      ctypes.POINTER(sv_seq_batch), _I, _VP, _VP, _VP]),
    "sv_sparse_decode_attn": (_I, [_VP, _I, _F, ctypes.POINTER(sv_kv_layer),
                                   ctypes.POINTER(sv_seq_batch), _VP, _I, _VP, _VP, _VP, _SZ, _VP]),
    "sv_decode_append_attn": (_I, [_VP, _I, _F, ctypes.POINTER(sv_kv_layer), ctypes.POINTER(sv_seq_batch),
                                   _VP, _VP, _VP, _I, _VP, _VP, _VP, _SZ, _VP]),
    "sv_evict_qa_tokens": (_I, [ctypes.POINTER(sv_kv_layer), _I, ctypes.POINTER(sv_seq_batch),
                                ctypes.c_int32, ctypes.c_int32, _VP, _VP, _SZ, _VP]),
    "sv_kv_append": (_I, [ctypes.POINTER(sv_kv_layer), ctypes.POINTER(sv_seq_batch), _VP, _VP, _I,
                          _VP, _SZ, _VP]),
    "sv_pack_kv": (_I, [ctypes.POINTER(sv_kv_layer), ctypes.POINTER(sv_seq_batch), _VP, _I,
                        ctypes.POINTER(sv_kv_layer), ctypes.POINTER(sv_seq_batch), _VP, _SZ, _VP]),
    "sv_salience_summary_workspace_bytes": (_SZ, [_I, _I, _I, _I, _I]),
    "sv_salience_summary": (_I, [_VP, _VP, _I, _I, _I, _I, _I, ctypes.c_float, _VP, _VP, _SZ, _VP]),
    "sv_prune_threshold": (_I, [_VP, _I, _I, ctypes.c_float, _VP, ctypes.c_int64, _VP, _VP, _VP, _VP, _SZ, _VP]),
    "sv_retrieve_softmax_workspace_bytes": (_SZ, [_I, _I, _I, _I, _I, _I, _I]),
    "sv_retrieve_topk_softmax": (_I, [_VP, _I, _I, ctypes.c_float, ctypes.POINTER(sv_kv_layer),
                                      ctypes.POINTER(sv_seq_batch), _VP, _I, _VP, _VP, _VP, _SZ, _VP]),
    "sv_qk_norm_rope": (_I, [_VP, _I64, _VP, _I64, _I, _I, _I, _I, _I, ctypes.POINTER(sv_rotation), _VP, _VP, _VP,
                             _SZ, _VP]),
    "sv_qk_norm_rope_append": (_I, [_VP, _I64, _VP, _I64, _VP, _I64, _I, _I, ctypes.POINTER(sv_rotation),
                                    ctypes.POINTER(sv_kv_layer), ctypes.POINTER(sv_seq_batch), _VP, _VP, _VP, _SZ,
                                    _VP]),
    "sv_tree_attn_workspace_bytes": (_SZ, [_I, _I, _I, _I, _I, _I]),
    "sv_tree_attn": (_I, [_VP, _I, _I, _F, ctypes.POINTER(sv_kv_layer), ctypes.POINTER(sv_seq_batch), _VP, _I, _VP,
                          _VP, _VP, _VP, _VP, _SZ, _VP]),
    "sv_kv_accept": (_I, [ctypes.POINTER(sv_kv_layer), _I, ctypes.POINTER(sv_seq_batch), _I, _VP, _I, _VP, _VP, _SZ,
                          _VP]),
    "sv_pages_workspace_bytes": (_SZ, [_I, _I, _I]),
    "sv_pages_release": (_I, [ctypes.POINTER(sv_page_pool), ctypes.POINTER(sv_seq_batch), _VP, _VP, _SZ, _VP]),
    "sv_pages_fork": (_I, [ctypes.POINTER(sv_page_pool), ctypes.POINTER(sv_seq_batch), _VP, _VP, _I, _VP, _VP, _SZ,
                           _VP]),
    "sv_pages_reserve": (_I, [ctypes.POINTER(sv_page_pool), ctypes.POINTER(sv_kv_layer), _I,
                              ctypes.POINTER(sv_seq_batch), _I, _VP, _VP, _SZ, _VP]),
    "sv_read_device_status": (_I, [_VP, _I, ctypes.POINTER(ctypes.c_int32), _VP]),
}
EXPORTED = tuple(_SIGS)


def library_path():
    return _build.LIB


def load(path=None):
    """Load libsv.so (built by ``build.build()``); raises if it is missing."""
    global _lib
    if _lib is not None:
        return _lib
    path = path or library_path()
    if not os.path.exists(path):
        raise RuntimeError(f"libsv.so is not built ({path}); run visual_token_sparsity_gb300.build")
    lib = ctypes.CDLL(path)
    for name, (res, args) in _SIGS.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    _lib = lib
    return lib


def _check(status):
    if status != SV_OK:
        raise SvError(status, _lib.sv_last_error().decode())


def _stream(stream):
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream))


def _ptr(t, dtype=None, name="tensor"):
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    return ctypes.c_void_p(t.data_ptr())


def _ws(ws):
    return _ptr(ws, torch.uint8, "ws"), ctypes.c_size_t(ws.numel())


def workspace(nbytes, device="cuda"):
    """Zero-filled device workspace of ``nbytes`` bytes (status word cleared)."""
    return torch.zeros(int(nbytes), dtype=torch.uint8, device=device)


def _one_device(*tensors):
    """Index of the device that all these tensors are on (None: no tensor)."""
    devs = {t.get_device() for t in tensors if t is not None}
    if len(devs) > 1:
        raise ValueError(f"tensors on different devices: {sorted(devs)}")
    return devs.pop() if devs else None


# ------------------------------------------------------------------ descriptors

class KvLayer:
    """One layer's paged cache: bf16 pools [num_blocks][Hkv][16][d], both on one
    device (ValueError otherwise, as for the descriptors below)."""

    def __init__(self, k_pool, v_pool):
        assert k_pool.shape == v_pool.shape and k_pool.shape[2] == BLOCK_TOKENS
        self.k_pool, self.v_pool = k_pool, v_pool
        self.c = sv_kv_layer(_ptr(k_pool, torch.bfloat16, "k_pool"), _ptr(v_pool, torch.bfloat16, "v_pool"),
                             k_pool.shape[0], k_pool.shape[1], k_pool.shape[3])
        self.by_ref, self.n_kv_heads, self.head_dim = ctypes.byref(self.c), k_pool.shape[1], k_pool.shape[3]
        self.device = _one_device(k_pool, v_pool)


class SeqBatch:
    """Block table (int32 [batch][max_blocks]) plus lengths: uniform n_vis /
    n_text, or -- with the optional int32 [batch] device tensors n_vis_seq,
    n_text_seq, k_seq -- per-sequence counts, n_vis / n_text then being the
    capacities."""

    def __init__(self, block_table, n_vis, n_text, n_vis_seq=None, n_text_seq=None, k_seq=None):
        self.block_table = block_table
        self.n_vis_seq, self.n_text_seq, self.k_seq = n_vis_seq, n_text_seq, k_seq
        B = block_table.shape[0]

        def opt(t, name):
            if t is None:
                return None
            if t.shape != (B,):
                raise ValueError(f"{name} must have shape ({B},), got {tuple(t.shape)}")
            return _ptr(t, torch.int32, name)
        self.c = sv_seq_batch(_ptr(block_table, torch.int32, "block_table"), B,
                              block_table.shape[1], int(n_vis), int(n_text), opt(n_vis_seq, "n_vis_seq"),
                              opt(n_text_seq, "n_text_seq"), opt(k_seq, "k_seq"))
        self.by_ref, self.batch = ctypes.byref(self.c), B
        self.device = _one_device(block_table, n_vis_seq, n_text_seq, k_seq)

    @property
    def n_vis(self):
        return self.c.n_vis

    @property
    def n_text(self):
        return self.c.n_text

    @n_text.setter
    def n_text(self, v):
        self.c.n_text = int(v)


class Rotation:
    """Norm and rotation of queries and keys: cos_sin fp32 [n_pos][rot / 2][2]
    (or None: no rotation), pos int32 [B][T] or, with ``sections`` (pairs of
    each axis, adding up to rot / 2), [axes][B][T]; optional bf16 [d] weights of
    the per-head RMS norm (None: not normalised)."""

    def __init__(self, cos_sin, pos, sections=None, interleaved=False, q_weight=None, k_weight=None, eps=1e-6):
        self.cos_sin, self.pos, self.q_weight, self.k_weight = cos_sin, pos, q_weight, k_weight
        n_pos = rot = 0
        n_axes, sec = 1, [0, 0, 0]
        self.tokens = None
        if cos_sin is not None:
            if cos_sin.dim() != 3 or cos_sin.shape[2] != 2:
                raise ValueError(f"cos_sin must be [n_pos][rot / 2][2], got {tuple(cos_sin.shape)}")
            n_pos, rot = cos_sin.shape[0], 2 * cos_sin.shape[1]
            if sections is not None:
                n_axes = len(sections)
                if not 1 <= n_axes <= 3:
                    raise ValueError(f"1 to 3 sections, got {n_axes}")
                sec[:n_axes] = [int(x) for x in sections]
                if n_axes == 1 and sec[0] != rot // 2:
                    raise ValueError(f"sections add up to {sec[0]}, not to {rot // 2}")
            lead = (n_axes,) if pos is not None and pos.dim() == 3 else ()
            if pos is None or pos.dim() != 2 + len(lead) or (n_axes > 1 and not lead) or pos.shape[:-2] != lead:
                raise ValueError(f"pos must be [B][T] or [{n_axes}][B][T]")
            self.tokens = tuple(pos.shape[-2:])
        for w, name in ((q_weight, "q_weight"), (k_weight, "k_weight")):
            if w is not None and w.dim() != 1:
                raise ValueError(f"{name} must be [head_dim]")
        self.c = sv_rotation(_ptr(cos_sin, torch.float32, "cos_sin"), n_pos, rot, 1 if interleaved else 0,
                             _ptr(pos if cos_sin is not None else None, torch.int32, "pos"), n_axes,
                             (ctypes.c_int32 * 3)(*sec), _ptr(q_weight, torch.bfloat16, "q_weight"),
                             _ptr(k_weight, torch.bfloat16, "k_weight"), float(eps))
        self.by_ref = ctypes.byref(self.c)
        self.device = _one_device(cos_sin, pos if cos_sin is not None else None, q_weight, k_weight)

    def check(self, B, T, d):
        """The call's tokens and head dim are the descriptor's."""
        if self.tokens is not None and self.tokens != (B, T):
            raise ValueError(f"pos is for {self.tokens} tokens, the call has {(B, T)}")
        for w, name in ((self.q_weight, "q_weight"), (self.k_weight, "k_weight")):
            if w is not None and w.shape[0] != d:
                raise ValueError(f"{name} has {w.shape[0]} elements, head_dim is {d}")


class PagePool:
    """Reference counts of a cache's pages (ref int32 [num_blocks], 0: free)
    and the block-table entries each sequence holds (n_pages int32 [batch])."""

    def __init__(self, ref, n_pages):
        if ref.dim() != 1 or n_pages.dim() != 1:
            raise ValueError("ref must be [num_blocks], n_pages [batch]")
        self.ref, self.n_pages = ref, n_pages
        self.c = sv_page_pool(_ptr(ref, torch.int32, "ref"), _ptr(n_pages, torch.int32, "n_pages"), ref.shape[0])
        self.by_ref = ctypes.byref(self.c)
        self.device = _one_device(ref, n_pages)


class _Call:
    """Pointers of one call's tensors, checked: on the current device (the
    launch goes there), of the given type and shape, contiguous.  These calls
    are made many times per decoded token, so the checks are lean."""

    def __init__(self, ws, stream, *descriptors):
        self.dev = dev = torch._C._cuda_getDevice()
        for d in descriptors:
            if d.device not in (dev, None):
                raise ValueError(f"descriptor on cuda:{d.device}, current device is cuda:{dev}")
        if ws.dtype != _U8:
            raise ValueError(f"ws must be {_U8}, got {ws.dtype}")
        self.ws = self.device_ptr(ws, "ws"), ws.numel()
        if stream is None:
            self.stream = torch._C._cuda_getCurrentRawStream(dev)
        else:
            self.stream = stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)

    def device_ptr(self, t, name):
        if t.get_device() != self.dev:
            raise ValueError(f"{name} must be a CUDA tensor on the current device cuda:{self.dev}, is on {t.device}")
        if not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous")
        return t.data_ptr()

    def ptr(self, t, dtype, shape, name):
        if t is None:
            return None
        if t.dtype != dtype:
            raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
        if t.shape != shape:
            raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
        return self.device_ptr(t, name)

    def rows(self, t, shape, name):
        """Pointer and token stride of a bf16 [B][T][heads][d] tensor whose
        tokens lie evenly apart (a slice of a fused projection, for instance)."""
        if t.dtype != _BF16:
            raise ValueError(f"{name} must be {_BF16}, got {t.dtype}")
        if t.shape != shape:
            raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
        if t.get_device() != self.dev:
            raise ValueError(f"{name} must be a CUDA tensor on the current device cuda:{self.dev}, is on {t.device}")
        B, T, h, d = shape
        if B * T * h * d == 0:
            return t.data_ptr(), h * d
        sb, st, sh, sd = t.stride()
        if (sd != 1 and d > 1) or (sh != d and h > 1) or (B > 1 and T > 1 and sb != T * st):
            raise ValueError(f"{name}: heads must be contiguous and tokens evenly spaced, strides {t.stride()}")
        return t.data_ptr(), st if T > 1 else sb if B > 1 else h * d


# ------------------------------------------------------------------ sizes

def sv_salience_workspace_bytes(B, H, N, d):
    return load().sv_salience_workspace_bytes(B, H, N, d)


def sv_topk_workspace_bytes(rows, n, k):
    return load().sv_topk_workspace_bytes(rows, n, k)


def sv_prune_workspace_bytes(B, N, k):
    return load().sv_prune_workspace_bytes(B, N, k)


def sv_retrieve_workspace_bytes(B, H, n_kv_heads, head_dim, n_vis, k):
    return load().sv_retrieve_workspace_bytes(B, H, n_kv_heads, head_dim, n_vis, k)


def sv_attn_workspace_bytes(B, H, n_kv_heads, head_dim, n_tokens):
    return load().sv_attn_workspace_bytes(B, H, n_kv_heads, head_dim, n_tokens)


def sv_evict_workspace_bytes():
    return load().sv_evict_workspace_bytes()


def sv_salience_kernel_count(N, d):
    """Kernels one sv_salience_prefill call launches (3, or 4 for long sequences)."""
    return load().sv_salience_kernel_count(int(N), int(d))


def sv_retrieve_kernel_count(batch, n_kv_heads, n_vis):
    """Kernels one sv_retrieve_topk call launches (1: fused top-k, 2: separate top-k)."""
    return load().sv_retrieve_kernel_count(int(batch), int(n_kv_heads), int(n_vis))


def sv_attn_kernel_count(B, H, n_kv_heads, n_tokens):
    """Kernels one sv_sparse_decode_attn call launches (1: fused split merge, 2: merge kernel)."""
    return load().sv_attn_kernel_count(int(B), int(H), int(n_kv_heads), int(n_tokens))


# ------------------------------------------------------------------ calls

def sv_salience_prefill(q, k, scale, salience, ws, stream=None):
    """q, k: bf16 [B][H][N][d]; salience: fp32 [B][N] (written)."""
    lib = load()
    B, H, N, d = q.shape
    assert k.shape == q.shape and salience.shape == (B, N)
    _check(lib.sv_salience_prefill(_ptr(q, torch.bfloat16, "q"), _ptr(k, torch.bfloat16, "k"), B, H, N, d,
                                   float(scale), _ptr(salience, torch.float32, "salience"), *_ws(ws),
                                   _stream(stream)))


def sv_salience_summary_workspace_bytes(B, H, N, d, R):
    return load().sv_salience_summary_workspace_bytes(B, H, N, d, R)


def sv_salience_summary(q, k, R, scale, salience, ws, stream=None):
    """q, k: bf16 [B][H][N][d] (summary tokens first); salience: fp32 [B][N] (written)."""
    lib = load()
    B, H, N, d = q.shape
    assert k.shape == q.shape and salience.shape == (B, N)
    _check(lib.sv_salience_summary(_ptr(q, torch.bfloat16, "q"), _ptr(k, torch.bfloat16, "k"), B, H, N, d, int(R),
                                   float(scale), _ptr(salience, torch.float32, "salience"), *_ws(ws),
                                   _stream(stream)))


def sv_prune_threshold(salience, threshold, feat, feat_out, kept_idx, kept_count, ws, stream=None):
    """salience fp32 [B][N]; feat / feat_out [B][N][...] rows (or None); kept_idx int32 [B][N];
    kept_count int32 [B] (device)."""
    lib = load()
    B, N = salience.shape
    row_bytes = 0 if feat is None else feat.shape[2] * feat.element_size()
    _check(lib.sv_prune_threshold(_ptr(salience, torch.float32, "salience"), B, N, float(threshold),
                                  _ptr(feat, None, "feat"), row_bytes, _ptr(feat_out, None, "feat_out"),
                                  _ptr(kept_idx, torch.int32, "kept_idx"), _ptr(kept_count, torch.int32, "kept_count"),
                                  *_ws(ws), _stream(stream)))


def sv_topk_rows(scores, k, idx, ws, stream=None):
    """scores: fp32 [rows][n]; idx: int32 [rows][k] (written, ascending)."""
    lib = load()
    rows, n = scores.shape
    assert idx.shape == (rows, k)
    _check(lib.sv_topk_rows(_ptr(scores, torch.float32, "scores"), rows, n, k,
                            _ptr(idx, torch.int32, "idx"), *_ws(ws), _stream(stream)))


def sv_prune_compact(salience, k, feat, feat_out, kept_idx, ws, stream=None):
    """salience fp32 [B][N]; feat [B][N][C] (any dtype); feat_out [B][k][C]; kept_idx int32 [B][k]."""
    lib = load()
    B, N = salience.shape
    row_bytes = 0 if feat is None else feat.shape[2] * feat.element_size()
    _check(lib.sv_prune_compact(_ptr(salience, torch.float32, "salience"), B, N, k,
                                _ptr(feat, None, "feat"), row_bytes, _ptr(feat_out, None, "feat_out"),
                                _ptr(kept_idx, torch.int32, "kept_idx"), *_ws(ws), _stream(stream)))


def sv_retrieve_topk(q, layer, seqs, k, vis_idx, scores, ws, stream=None):
    """q bf16 [B][R][H][d]; vis_idx int32 [B][Hkv][k]; scores fp32 [B][Hkv][n_vis] or None."""
    lib = load()
    B, R, H, d = q.shape
    _check(lib.sv_retrieve_topk(_ptr(q, torch.bfloat16, "q"), R, H, ctypes.byref(layer.c),
                                ctypes.byref(seqs.c), k, _ptr(vis_idx, torch.int32, "vis_idx"),
                                _ptr(scores, torch.float32, "scores"), *_ws(ws), _stream(stream)))


def sv_retrieve_softmax_workspace_bytes(B, R, H, n_kv_heads, head_dim, n_vis, n_text):
    return load().sv_retrieve_softmax_workspace_bytes(B, R, H, n_kv_heads, head_dim, n_vis, n_text)


def sv_retrieve_topk_softmax(q, scale, layer, seqs, k, vis_idx, scores, ws, lse=None, stream=None):
    """q bf16 [B][R][H][d]; lse fp32 [B][R][H] (natural log) or None; vis_idx int32 [B][Hkv][k]."""
    lib = load()
    B, R, H, d = q.shape
    _check(lib.sv_retrieve_topk_softmax(_ptr(q, torch.bfloat16, "q"), R, H, float(scale), ctypes.byref(layer.c),
                                        ctypes.byref(seqs.c), _ptr(lse, torch.float32, "lse"), int(k),
                                        _ptr(vis_idx, torch.int32, "vis_idx"), _ptr(scores, torch.float32, "scores"),
                                        *_ws(ws), _stream(stream)))


def sv_retrieve_topk_noalloc(q, layer, seqs, k, vis_idx, scores=None, stream=None):
    """As sv_retrieve_topk, for callers that cannot allocate: no workspace; the
    library's fixed device scratch holds the scores (limit B * Hkv * n_vis <= 2^21)."""
    lib = load()
    B, R, H, d = q.shape
    _check(lib.sv_retrieve_topk_noalloc(_ptr(q, torch.bfloat16, "q"), R, H, ctypes.byref(layer.c),
                                        ctypes.byref(seqs.c), k, _ptr(vis_idx, torch.int32, "vis_idx"),
                                        _ptr(scores, torch.float32, "scores"), _stream(stream)))


def sv_sparse_decode_attn(q, scale, layer, seqs, vis_idx, k, out, lse, ws, stream=None):
    """q bf16 [B][H][d]; vis_idx int32 [B][Hkv][k] or None; out bf16 [B][H][d]; lse fp32 [B][H] or None."""
    lib = load()
    B, H, d = q.shape
    _check(lib.sv_sparse_decode_attn(_ptr(q, torch.bfloat16, "q"), H, float(scale), ctypes.byref(layer.c),
                                     ctypes.byref(seqs.c), _ptr(vis_idx, torch.int32, "vis_idx"), k,
                                     _ptr(out, torch.bfloat16, "out"), _ptr(lse, torch.float32, "lse"),
                                     *_ws(ws), _stream(stream)))


def sv_decode_append_attn(q, scale, layer, seqs, k_new, v_new, vis_idx, k, out, lse, ws, stream=None):
    """sv_kv_append of one token (k_new, v_new bf16 [B][Hkv][d]) then sparse attention over it and the
    cache, in one launch; n_text unchanged (the caller adds 1)."""
    lib = load()
    B, H, d = q.shape
    _check(lib.sv_decode_append_attn(_ptr(q, torch.bfloat16, "q"), H, float(scale), ctypes.byref(layer.c),
                                     ctypes.byref(seqs.c), _ptr(k_new, torch.bfloat16, "k_new"),
                                     _ptr(v_new, torch.bfloat16, "v_new"), _ptr(vis_idx, torch.int32, "vis_idx"),
                                     k, _ptr(out, torch.bfloat16, "out"), _ptr(lse, torch.float32, "lse"),
                                     *_ws(ws), _stream(stream)))


def sv_evict_qa_tokens(layers, seqs, text_begin, text_end, ws, stream=None):
    """Evicts text span [text_begin, text_end) in every layer; returns pages in use per sequence."""
    lib = load()
    arr = (sv_kv_layer * len(layers))(*[l.c for l in layers])
    used = (ctypes.c_int32 * max(1, seqs.c.batch))()
    _check(lib.sv_evict_qa_tokens(arr, len(layers), ctypes.byref(seqs.c), int(text_begin), int(text_end),
                                  ctypes.cast(used, ctypes.c_void_p), *_ws(ws), _stream(stream)))
    return list(used)[: seqs.c.batch]


def sv_kv_append(layer, seqs, k_new, v_new, ws, stream=None):
    """k_new, v_new bf16 [B][T][Hkv][d] written at positions n_vis + n_text ...; n_text unchanged."""
    lib = load()
    T = k_new.shape[1]
    _check(lib.sv_kv_append(ctypes.byref(layer.c), ctypes.byref(seqs.c), _ptr(k_new, torch.bfloat16, "k_new"),
                            _ptr(v_new, torch.bfloat16, "v_new"), T, *_ws(ws), _stream(stream)))


def sv_pack_kv(src, seqs, vis_idx, k, dst, dst_seqs, ws, stream=None):
    """Copy the selected visual (vis_idx int32 [B][Hkv][k], or None = all) and all
    text K/V rows of src to positions [0, k + n_text) of dst (see include/sv.h)."""
    lib = load()
    _check(lib.sv_pack_kv(ctypes.byref(src.c), ctypes.byref(seqs.c), _ptr(vis_idx, torch.int32, "vis_idx"), int(k),
                          ctypes.byref(dst.c), ctypes.byref(dst_seqs.c), *_ws(ws), _stream(stream)))


def sv_qk_norm_rope(q, k, rot, q_out, k_out, ws, stream=None):
    """q bf16 [B][N][H][d], k bf16 [B][N][Hk][d] (tokens may be strided: slices of a fused projection),
    normalised and rotated as ``rot`` says -> q_out [B][H][N][d], k_out [B][Hk][N][d] (written)."""
    lib = load()
    B, N, H, d = q.shape
    Hk = k.shape[2]
    c = _Call(ws, stream, rot)
    rot.check(B, N, d)
    _check(lib.sv_qk_norm_rope(*c.rows(q, (B, N, H, d), "q"), *c.rows(k, (B, N, Hk, d), "k"), B, N, H, Hk, d,
                               rot.by_ref, c.ptr(q_out, _BF16, (B, H, N, d), "q_out"),
                               c.ptr(k_out, _BF16, (B, Hk, N, d), "k_out"), *c.ws, c.stream))


def sv_qk_norm_rope_append(q, k, v, rot, layer, seqs, q_out, ws, n_new=None, stream=None):
    """T new tokens per sequence: q bf16 [B][T][H][d], k, v bf16 [B][T][Hkv][d] (tokens may be strided);
    q normalised and rotated -> q_out [B][T][H][d]; k likewise, and v, -> the cache at n_vis + n_text + t;
    n_text unchanged (the caller adds T or n_new).  n_new int32 [B]: new tokens of each sequence, or None."""
    lib = load()
    B, T, H, d = q.shape
    kv = (B, T, layer.n_kv_heads, d)
    c = _Call(ws, stream, rot, layer, seqs)
    rot.check(B, T, d)
    _check(lib.sv_qk_norm_rope_append(*c.rows(q, (seqs.batch, T, H, layer.head_dim), "q"), *c.rows(k, kv, "k"),
                                      *c.rows(v, kv, "v"), T, H, rot.by_ref, layer.by_ref,
                                      seqs.by_ref, c.ptr(n_new, _I32, (B,), "n_new"),
                                      c.ptr(q_out, _BF16, q.shape, "q_out"), *c.ws, c.stream))


def sv_tree_attn_workspace_bytes(B, T, H, n_kv_heads, head_dim, n_tokens):
    return load().sv_tree_attn_workspace_bytes(B, T, H, n_kv_heads, head_dim, n_tokens)


def sv_tree_attn(q, scale, layer, seqs, vis_idx, k, tree_mask, out, lse, ws, n_new=None, stream=None):
    """T drafted tokens per sequence, already appended behind n_text, over the cache: q, out bf16
    [B][T][H][d]; vis_idx int32 [B][Hkv][k] or None; tree_mask int64 (or uint64) [B][T], bit s of row t: t sees
    s, or None: causal; lse fp32 [B][T][H] or None; n_new int32 [B]: drafted tokens of each sequence, or None."""
    lib = load()
    B, T, H, d = q.shape
    c = _Call(ws, stream, layer, seqs)
    vis = c.ptr(vis_idx, _I32, (B, layer.n_kv_heads, k), "vis_idx")
    if vis_idx is not None and k == 0:
        vis = c.ws[0]            # an empty list, not "all visual tokens": any address, nothing is read
    mask = None
    if tree_mask is not None:
        if tree_mask.dtype not in (torch.int64, torch.uint64):
            raise ValueError(f"tree_mask must be 64-bit integers, got {tree_mask.dtype}")
        mask = c.ptr(tree_mask, tree_mask.dtype, (B, T), "tree_mask")
    _check(lib.sv_tree_attn(c.ptr(q, _BF16, (seqs.batch, T, H, layer.head_dim), "q"), T, H, scale,
                            layer.by_ref, seqs.by_ref, vis, k, mask,
                            c.ptr(n_new, _I32, (B,), "n_new"), c.ptr(out, _BF16, q.shape, "out"),
                            c.ptr(lse, _F32, (B, T, H), "lse"), *c.ws, c.stream))


def _layer_array(layers):
    return (sv_kv_layer * max(1, len(layers)))(*[l.c for l in layers])


def sv_kv_accept(layers, seqs, T, path, ws, n_path=None, stream=None):
    """Compacts the accepted path of a draft of T tokens in every layer: path int32 [B][P] ascending drafted
    indices (the first n_path[b] of a row, or all); n_text unchanged (the caller adds the accepted count)."""
    lib = load()
    B, P = path.shape
    c = _Call(ws, stream, seqs, *layers)
    _check(lib.sv_kv_accept(_layer_array(layers), len(layers), seqs.by_ref, T,
                            c.ptr(path, _I32, (seqs.batch, P), "path"), P,
                            c.ptr(n_path, _I32, (B,), "n_path"), *c.ws, c.stream))


def sv_pages_workspace_bytes(batch, max_blocks, num_blocks):
    return load().sv_pages_workspace_bytes(batch, max_blocks, num_blocks)


def _pages(pool, seqs, ws, stream, *layers):
    if pool.n_pages.shape != (seqs.batch,):
        raise ValueError(f"n_pages must have shape ({seqs.batch},), got {tuple(pool.n_pages.shape)}")
    return _Call(ws, stream, pool, seqs, *layers)


def sv_pages_release(pool, seqs, keep, ws, stream=None):
    """Drops every sequence's pages behind its first keep[b] tokens (int32 [B]; -1: leave it; None: drop all)."""
    lib = load()
    c = _pages(pool, seqs, ws, stream)
    _check(lib.sv_pages_release(pool.by_ref, seqs.by_ref,
                                c.ptr(keep, _I32, (seqs.batch,), "keep"), *c.ws, c.stream))


def sv_pages_fork(pool, seqs, parent, child, ws, n_tok=None, stream=None):
    """Rows child[i] (holding no pages) share the pages of rows parent[i] (int32 [n]), or of their first
    n_tok[i] tokens."""
    lib = load()
    n, = parent.shape
    c = _pages(pool, seqs, ws, stream)
    _check(lib.sv_pages_fork(pool.by_ref, seqs.by_ref,
                             c.ptr(parent, _I32, (n,), "parent"), c.ptr(child, _I32, (n,), "child"), n,
                             c.ptr(n_tok, _I32, (n,), "n_tok"), *c.ws, c.stream))


def sv_pages_reserve(pool, layers, seqs, T, ws, n_new=None, stream=None):
    """Makes the T (or n_new[b], int32 [B]) positions behind each sequence's tokens writable: fresh pages, and
    private copies, in every layer, of the shared pages among them."""
    lib = load()
    c = _pages(pool, seqs, ws, stream, *layers)
    _check(lib.sv_pages_reserve(pool.by_ref, _layer_array(layers), len(layers), seqs.by_ref, T,
                                c.ptr(n_new, _I32, (seqs.batch,), "n_new"), *c.ws, c.stream))


def sv_read_device_status(ws, clear=False, stream=None):
    lib = load()
    out = ctypes.c_int32(0)
    _check(lib.sv_read_device_status(_ptr(ws, torch.uint8, "ws"), 1 if clear else 0, ctypes.byref(out),
                                     _stream(stream)))
    return out.value
