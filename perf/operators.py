"""Workloads of the speculative-decoding operators over the paged cache.

A draft step takes T drafted tokens per sequence through a layer: their
queries and keys are normalised per head and rotated while they enter the
paged cache, they attend over the selected visual tokens, the text and their
own ancestors in the draft tree, and after verification the accepted path is
compacted to the end of the text.  Conversations that branch from one visual
cache share its pages until they write to them.  Five kinds of case:

  encode  per-head RMS norm and position rotation of an encoder's queries and
          keys, token-major projections to the head-major salience operands
  append  the same for a decoder's new tokens, keys and values written into
          the paged cache
  tree    attention of drafted (or question) tokens over the paged cache
  pages   release of old branches, fork of new ones from their prefix, and
          private copies of the shared pages that they will write to
  step    append and tree attention in every layer, then the compaction of
          the accepted path in all layers
"""

import math

import numpy as np
import torch

own = False

PAGE = 16          # tokens of a cache page
DEV = "cuda"


# ------------------------------------------------------------------ cases

def listed():
    return [
        # Qwen2-VL vision tower (16 heads, d 80, rows and columns rotated
        # apart) over one long clip: the operands of the long salience
        dict(name="encode_vision_16384", kind="encode", B=1, N=16384, H=16, Hk=16, d=80, axes=2, norm=False,
             interleaved=False),
        # a SigLIP-sized encoder (729 tokens, 16 heads, d 72) with normalised
        # queries and keys, a batch of frames, one plain position axis
        dict(name="encode_frames_b16", kind="encode", B=16, N=729, H=16, Hk=16, d=72, axes=1, norm=True,
             interleaved=True),
        # one decode token per sequence of the LongVILA-7B attention (28 query,
        # 4 KV heads): the smallest call, bound by its launch
        dict(name="append_decode_b8", kind="append", B=8, T=1, H=28, Hkv=4, d=128, n_vis=3136, n_text=256, axes=3,
             rot=128, norm=True, interleaved=False, ragged=False),
        # a prefill of the same model's pruned visual prefix, odd length, the
        # sequences of different lengths
        dict(name="append_prefill_b4", kind="append", B=4, T=2885, H=28, Hkv=4, d=128, n_vis=0, n_text=0, axes=3,
             rot=128, norm=True, interleaved=False, ragged=True),
        # the round-loop shape (4 query, 2 KV heads, d 64) with a draft of five
        dict(name="tree_tiny", kind="tree", B=1, T=5, H=4, Hkv=2, d=64, n_vis=576, k=144, n_text=57, mask="tree",
             ragged=False),
        # LLaVA-NeXT-7B, 16 sequences, half of the visual tokens, 16 drafted
        dict(name="tree_llava_next_b16", kind="tree", B=16, T=16, H=32, Hkv=32, d=128, n_vis=2880, k=1440,
             n_text=128, mask="tree", ragged=False),
        # LongVILA-7B, 8 sequences of different lengths, 27 drafted tokens
        dict(name="tree_longvila_b8", kind="tree", B=8, T=27, H=28, Hkv=4, d=128, n_vis=50176, k=12544, n_text=256,
             mask="tree", ragged=True),
        # a long question of the same model read against its whole visual
        # cache: many rows per KV head, bound by the matrix products
        dict(name="tree_question_193", kind="tree", B=1, T=193, H=28, Hkv=4, d=128, n_vis=50176, k=0, n_text=23,
             mask="chain", ragged=False),
        # two branches of one small conversation
        dict(name="pages_small", kind="pages", parents=1, forks=2, layers=2, Hkv=2, d=64, n_tok=611, T=5),
        # 32 branches over four cached clips of the LongVILA-7B at 16 frames
        dict(name="pages_branches", kind="pages", parents=4, forks=8, layers=8, Hkv=4, d=128, n_tok=3370, T=24),
        # one speculative step, small shapes
        dict(name="step_tiny", kind="step", layers=2, B=2, T=7, H=4, Hkv=2, d=64, n_vis=576, k=144, n_text=41,
             axes=1, rot=64, norm=False, interleaved=False, mask="tree", ragged=True),
        # one speculative step of four LongVILA-7B layers at 16 frames
        dict(name="step_longvila_16f", kind="step", layers=4, B=8, T=32, H=28, Hkv=4, d=128, n_vis=3136, k=784,
             n_text=256, axes=3, rot=128, norm=True, interleaved=False, mask="tree", ragged=True),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _heads(rng):
    """(H, Hkv): equal heads, or groups of up to 16."""
    Hkv = rng.choice([1, 2, 3, 4, 8, 32])
    G = rng.choice([1, 1, 2, 4, 7, 8, 16]) if Hkv <= 8 else 1
    return Hkv * G, Hkv


def draw(rng):
    kind = rng.choice(["encode", "append", "tree", "tree", "pages", "step"])
    if kind == "encode":
        d = rng.choice([64, 72, 80, 128])
        H = rng.choice([2, 5, 12, 16])
        N = _log_int(rng, 1, 16384)
        B = max(1, min(_log_int(rng, 1, 64), 16384 * 16 // (N * H) or 1))
        return dict(kind=kind, B=B, N=N, H=H, Hk=rng.choice([H, 1]), d=d, axes=rng.choice([1, 2]),
                    norm=rng.random() < 0.5, interleaved=rng.random() < 0.5)
    if kind == "append":
        H, Hkv = _heads(rng)
        T = _log_int(rng, 1, 2885)
        B = max(1, min(_log_int(rng, 1, 32), 4 * 2885 * 36 // (T * (H + 2 * Hkv)) or 1))
        d = rng.choice([64, 128])
        return dict(kind=kind, B=B, T=T, H=H, Hkv=Hkv, d=d, n_vis=_log_int(rng, 1, 3136), n_text=_log_int(rng, 1, 300),
                    axes=rng.choice([1, 3]), rot=rng.choice([d, d, d // 2]), norm=rng.random() < 0.5,
                    interleaved=rng.random() < 0.5, ragged=rng.random() < 0.5)
    if kind == "tree":
        H, Hkv = _heads(rng)
        d = rng.choice([64, 128])
        mask = rng.choice(["tree", "tree", "chain"])
        T = _log_int(rng, 1, 64 if mask == "tree" else 193)
        n_vis = _log_int(rng, 16, 50176)
        # at most the cost of the largest listed cases, in cache rows and in products
        B = _log_int(rng, 1, 16)
        B = max(1, min(B, int(3.0e5 // (n_vis * Hkv)), int(1.2e11 // (4.0 * n_vis * T * H * d))))
        if n_vis * Hkv > 4.0e5:
            n_vis = int(4.0e5 // Hkv)
        k = 0 if rng.random() < 0.3 else max(1, int(n_vis * rng.choice([0.25, 0.5, 0.9])))
        return dict(kind=kind, B=B, T=T, H=H, Hkv=Hkv, d=d, n_vis=n_vis, k=k, n_text=_log_int(rng, 1, 300), mask=mask,
                    ragged=rng.random() < 0.5)
    if kind == "pages":
        parents = rng.choice([1, 2, 3, 4])
        return dict(kind=kind, parents=parents, forks=rng.choice([1, 2, 3, 5, 8]), layers=rng.choice([1, 2, 5, 8]),
                    Hkv=rng.choice([1, 2, 4]), d=rng.choice([64, 128]), n_tok=_log_int(rng, 1, 3370),
                    T=_log_int(rng, 1, 64))
    H, Hkv = rng.choice([(4, 2), (8, 8), (28, 4), (16, 1)])
    d = rng.choice([64, 128])
    n_vis = _log_int(rng, 32, 3136)
    return dict(kind="step", layers=rng.choice([1, 2, 4]), B=_log_int(rng, 1, 8), T=_log_int(rng, 1, 32), H=H, Hkv=Hkv,
                d=d, n_vis=n_vis, k=max(1, n_vis // 4), n_text=_log_int(rng, 1, 256), axes=rng.choice([1, 3]), rot=d,
                norm=rng.random() < 0.5, interleaved=rng.random() < 0.5, mask="tree", ragged=rng.random() < 0.5)


def _lengths(c):
    """Visual, text, selected and new tokens of every sequence."""
    B, T, k = c["B"], c["T"], c.get("k", 0)
    if not c["ragged"]:
        return [c["n_vis"]] * B, [c["n_text"]] * B, [k] * B, [T] * B
    nv, nt, ks, tn = [], [], [], []
    for b in range(B):
        part = 1.0 - 0.6 * ((b * 5) % B) / B
        nv.append(int(c["n_vis"] * part))
        nt.append(int(c["n_text"] * (1.0 - 0.5 * ((b * 3) % B) / B)))
        ks.append(min(int(k * part), nv[-1]))
        tn.append(max(1, int(T * (1.0 - 0.4 * ((b * 7) % B) / B))))
    return nv, nt, ks, tn


def _accepted(c, b):
    """How many drafted tokens of sequence b were accepted."""
    return min(_lengths(c)[3][b], 1 + (b * 3) % 5)


def _sections(c, rot):
    """Rotation pairs of each position axis."""
    half = rot // 2
    if c["axes"] == 1:
        return None
    if c["axes"] == 2:
        return [half // 2, half - half // 2]
    a = half // 4
    b = (half - a) // 2
    return [a, b, half - a - b]


def work(case):
    c = case
    if c["kind"] == "encode":
        n = c["B"] * c["N"] * (c["H"] + c["Hk"]) * c["d"]
        return {"bytes": 4 * n + 4 * c["B"] * c["N"] * c["axes"], "flops": (7 if c["norm"] else 3) * n}
    if c["kind"] == "pages":
        page = c["Hkv"] * PAGE * c["d"] * 2
        kids = c["parents"] * c["forks"]
        held = -(-c["n_tok"] // PAGE)
        copied = kids * (1 if c["n_tok"] % PAGE else 0)
        return {"bytes": 2 * copied * page * 2 * c["layers"] + kids * held * 4 * 5, "flops": kids * held * 4}
    nv, nt, ks, tn = _lengths(c)
    new = sum(tn)
    append_b = 4 * new * (c["H"] + 2 * c["Hkv"]) * c["d"]
    append_f = 7 * new * (c["H"] + c["Hkv"]) * c["d"]
    if c["kind"] == "append":
        return {"bytes": append_b + 4 * new * c["axes"], "flops": append_f}
    rows = [(ks[b] if c["k"] else nv[b]) + nt[b] + tn[b] for b in range(c["B"])]
    attn_b = sum(r * c["Hkv"] * c["d"] * 4 for r in rows) + 4 * new * c["H"] * c["d"] + 4 * new * c["H"]
    if c["k"]:
        attn_b += 4 * sum(ks) * c["Hkv"]
    attn_f = sum(4 * tn[b] * c["H"] * c["d"] * rows[b] for b in range(c["B"]))
    if c["kind"] == "tree":
        return {"bytes": attn_b, "flops": attn_f}
    moved = sum(_accepted(c, b) for b in range(c["B"])) * c["Hkv"] * c["d"] * 8
    return {"bytes": c["layers"] * (append_b + attn_b + moved), "flops": c["layers"] * (append_f + attn_f)}


# ------------------------------------------------------------------ inputs

class _Rand:
    """Seeded draws on the device."""

    def __init__(self, seed):
        self.g = torch.Generator(device=DEV)
        self.g.manual_seed(int(seed) * 7919 + 13)

    def normal(self, *shape, std=1.0):
        return torch.randn(*shape, generator=self.g, device=DEV).mul_(std).to(torch.bfloat16)

    def perm(self, n):
        return torch.randperm(n, generator=self.g, device=DEV)

    def ints(self, lo, hi, *shape):
        return torch.randint(lo, hi, shape, generator=self.g, device=DEV, dtype=torch.int32)


def _i32(x):
    return torch.as_tensor(np.asarray(x, dtype=np.int32)).to(DEV)


def _table(n_pos, rot):
    """(cos, sin) of every position and pair, angles in 64 bits."""
    freq = 10000.0 ** (-torch.arange(rot // 2, dtype=torch.float64, device=DEV) * 2 / rot)
    a = torch.arange(n_pos, dtype=torch.float64, device=DEV)[:, None] * freq
    return torch.stack([a.cos(), a.sin()], dim=-1).float().contiguous()


def _rotation(c, r, rot, pos, n_pos):
    s = dict(rot=rot, sections=_sections(c, rot), interleaved=c["interleaved"], eps=1e-6, pos=pos,
             table=_table(n_pos, rot), qw=None, kw=None)
    if c["norm"]:
        s["qw"] = (1 + 0.1 * r.normal(c["d"]).float()).to(torch.bfloat16)
        s["kw"] = (1 + 0.1 * r.normal(c["d"]).float()).to(torch.bfloat16)
    return s


def _tree(c, r, lens):
    """Random draft trees: every token's parent is an earlier one or the text."""
    B, T = c["B"], c["T"]
    u = np.random.default_rng(int(r.ints(0, 1 << 30, 1).item())).random((B, T))
    m = np.zeros((B, T), dtype=np.uint64)
    for b in range(B):
        for t in range(lens[b]):
            parent = int(u[b, t] * (t + 1)) - 1
            m[b, t] = (m[b, parent] if parent >= 0 else 0) | np.uint64(1 << t)
    return torch.as_tensor(m.view(np.int64)).to(DEV)


def _cache(c, r, layers, blocks, outliers):
    """`layers` pools of K and V; some rows are the outliers that real keys have."""
    ks, vs = [], []
    for _ in range(layers):
        k = r.normal(blocks, c["Hkv"], PAGE, c["d"])
        v = r.normal(blocks, c["Hkv"], PAGE, c["d"])
        if outliers:
            hit = r.ints(0, 50, blocks, 1, PAGE, 1) == 0
            k = torch.where(hit, k * 4, k)
        ks.append(k)
        vs.append(v)
    return ks, vs


def _select(r, B, Hkv, nv, ks, k):
    """Ascending distinct visual indices per sequence and KV head, -1 behind them."""
    out = torch.full((B, Hkv, k), -1, dtype=torch.int32, device=DEV)
    for b in range(B):
        for g in range(Hkv):
            out[b, g, : ks[b]] = torch.sort(r.perm(max(nv[b], 1))[: ks[b]]).values.to(torch.int32)
    return out


def _pairs(counts):
    """(b, i) of every i < counts[b]."""
    n = torch.tensor(counts)
    b = torch.repeat_interleave(torch.arange(len(counts)), n)
    i = torch.arange(int(n.sum())) - torch.repeat_interleave(torch.cumsum(n, 0) - n, n)
    return b.to(DEV), i.to(DEV)


def _prepare_lengths(c, s):
    nv, nt, ks, tn = _lengths(c)
    s.update(nv=nv, nt=nt, ks=ks, tn=tn)
    # the same on the device, and the (sequence, token) pairs that are computed
    s.update(vis_n=_i32(nv), text_n=_i32(nt), new_n=_i32(tn), sel_n=_i32(ks if c.get("k") else nv))
    s["base"] = s["vis_n"] + s["text_n"]
    s["live"] = _pairs(tn)
    if c["ragged"]:
        s["lens"] = tuple(_i32(x) for x in (nv, nt, ks))
        s["n_new"] = _i32(tn)
    else:
        s["lens"], s["n_new"] = (None, None, None), None


def prepare(case, seed):
    c, r = case, _Rand(seed)
    s = {"c": c}
    if c["kind"] == "encode":
        B, N, H, Hk, d = c["B"], c["N"], c["H"], c["Hk"], c["d"]
        # one fused projection: the queries and keys are slices of its rows
        s["proj"] = r.normal(B, N, H + Hk, d)
        side = max(1, int(math.isqrt(N)))
        t = torch.arange(N, device=DEV)
        pos = [t] if c["axes"] == 1 else [t // side, t % side]
        n_pos = N + 1
        pos = torch.stack([p.to(torch.int32).expand(B, N) for p in pos]).contiguous()
        s["rot"] = _rotation(c, r, d, pos, n_pos)
        s["q_out"] = torch.zeros(B, H, N, d, dtype=torch.bfloat16, device=DEV)
        s["k_out"] = torch.zeros(B, Hk, N, d, dtype=torch.bfloat16, device=DEV)
        return _own_prepare(c, s) if own else s
    if c["kind"] == "pages":
        return _prepare_pages(c, r, s)
    B, T, H, Hkv, d = c["B"], c["T"], c["H"], c["Hkv"], c["d"]
    _prepare_lengths(c, s)
    per = -(-(c["n_vis"] + c["n_text"] + T) // PAGE)
    blocks = B * per + 3
    L = c.get("layers", 1)
    s["table"] = r.perm(blocks)[: B * per].to(torch.int32).view(B, per).contiguous()
    if c["kind"] == "append":
        s["kp"] = [torch.zeros(blocks, Hkv, PAGE, d, dtype=torch.bfloat16, device=DEV)]
        s["vp"] = [torch.zeros(blocks, Hkv, PAGE, d, dtype=torch.bfloat16, device=DEV)]
    else:
        s["kp"], s["vp"] = _cache(c, r, L, blocks, True)
    if c["kind"] != "tree":
        s["proj"] = [r.normal(B, T, H + 2 * Hkv, d) for _ in range(L)]
        n_pos = c["n_vis"] + c["n_text"] + T + 1
        at = torch.tensor([a + b for a, b in zip(s["nv"], s["nt"])], device=DEV)[:, None] + torch.arange(T, device=DEV)
        axes = [at] + [(at * (3 + a)) % n_pos for a in range(c["axes"] - 1)]
        s["rot"] = _rotation(c, r, c["rot"], torch.stack(axes).to(torch.int32).contiguous(), n_pos)
        s["q_out"] = [torch.zeros(B, T, H, d, dtype=torch.bfloat16, device=DEV) for _ in range(L)]
    if c["kind"] != "append":
        s["mask"] = _tree(c, r, s["tn"]) if c["mask"] == "tree" else None
        s["vis"] = _select(r, B, Hkv, s["nv"], s["ks"], c["k"]) if c["k"] else None
        s["out"] = [torch.zeros(B, T, H, d, dtype=torch.bfloat16, device=DEV) for _ in range(L)]
        s["lse"] = [torch.zeros(B, T, H, device=DEV) for _ in range(L)]
    if c["kind"] == "tree":
        s["q"] = r.normal(B, T, H, d)
    if c["kind"] == "step":
        acc = [_accepted(c, b) for b in range(B)]
        width = max(acc)
        path = torch.full((B, width), -1, dtype=torch.int32, device=DEV)
        for b in range(B):
            path[b, : acc[b]] = torch.sort(r.perm(s["tn"][b])[: acc[b]]).values.to(torch.int32)
        s["acc"], s["path"], s["n_path"], s["took"] = acc, path, _i32(acc), _pairs(acc)
    return _own_prepare(c, s) if own else s


def _prepare_pages(c, r, s):
    """`parents` cached prefixes, each with `forks` older branches that hold
    one page of their own behind the shared ones."""
    P, F, n, T = c["parents"], c["forks"], c["n_tok"], c["T"]
    held = -(-n // PAGE)
    grow = -(-(n + T) // PAGE) - held + 1
    rows, per = P + P * F, held + grow
    blocks = P * held + P * F * (grow + 1) + 7
    order = r.perm(blocks).cpu().numpy().astype(np.int32)
    table = np.full((rows, per), -1, dtype=np.int32)
    ref = np.zeros(blocks, dtype=np.int32)
    pages = np.full(rows, held, dtype=np.int32)
    at = 0
    for p in range(P):
        table[p, :held] = order[at: at + held]
        at += held
    for f in range(P * F):
        table[P + f, : held - 1] = table[f // F, : held - 1]
        table[P + f, held - 1] = order[at]
        at += 1
    for row in range(rows):
        for e in table[row, :held]:
            ref[e] += 1
    s["table"], s["ref"], s["n_pages"] = _i32(table), _i32(ref), _i32(pages)
    s["kp"], s["vp"] = _cache(c, r, c["layers"], blocks, False)
    s["child"] = _i32(np.arange(P, rows))
    s["parent"] = _i32(np.arange(P * F) // F)
    s["keep"] = _i32([-1] * P + [0] * (P * F))        # -1: the prefixes keep what they hold
    s["n_new"] = _i32([0] * P + [T] * (P * F))
    return _own_prepare(c, s) if own else s


# ------------------------------------------------------------------ one pass

def run(state):
    c = state["c"]
    return (_own_run if own else _plain_run)(c, state)


def _own_prepare(c, s):
    """The descriptors and workspaces that a program keeps."""
    from visual_token_sparsity_gb300 import binding as sv
    if "rot" in s:
        R = s["rot"]
        s["sv_rot"] = sv.Rotation(R["table"], R["pos"], sections=R["sections"], interleaved=R["interleaved"],
                                  q_weight=R["qw"], k_weight=R["kw"], eps=R["eps"])
    s["ws"] = sv.workspace(256)
    if c["kind"] == "encode":
        return s
    s["sv_layers"] = [sv.KvLayer(k, v) for k, v in zip(s["kp"], s["vp"])]
    if c["kind"] == "pages":
        s["sv_pool"] = sv.PagePool(s["ref"], s["n_pages"])
        s["sv_seqs"] = sv.SeqBatch(s["table"], 0, c["n_tok"])
        s["ws"] = sv.workspace(sv.sv_pages_workspace_bytes(s["table"].shape[0], s["table"].shape[1], s["ref"].numel()))
        return s
    nv, nt, ks = s["lens"]
    s["sv_seqs"] = sv.SeqBatch(s["table"], c["n_vis"], c["n_text"], nv, nt, ks if c.get("k") else None)
    if c["kind"] != "append":
        n_tok = (c["k"] or c["n_vis"]) + c["n_text"] + c["T"]
        s["ws"] = sv.workspace(sv.sv_tree_attn_workspace_bytes(c["B"], c["T"], c["H"], c["Hkv"], c["d"], n_tok))
    return s


def _own_run(c, s):
    from visual_token_sparsity_gb300 import binding as sv
    H = c.get("H")
    if c["kind"] == "encode":
        q, k = s["proj"][:, :, :H], s["proj"][:, :, H:]
        sv.sv_qk_norm_rope(q, k, s["sv_rot"], s["q_out"], s["k_out"], s["ws"])
        return {"q": s["q_out"], "k": s["k_out"]}
    if c["kind"] == "pages":
        sv.sv_pages_release(s["sv_pool"], s["sv_seqs"], s["keep"], s["ws"])
        sv.sv_pages_fork(s["sv_pool"], s["sv_seqs"], s["parent"], s["child"], s["ws"])
        sv.sv_pages_reserve(s["sv_pool"], s["sv_layers"], s["sv_seqs"], c["T"], s["ws"], n_new=s["n_new"])
        return {"table": s["table"], "n_pages": s["n_pages"], "ref": s["ref"], "k": s["kp"], "v": s["vp"]}
    scale = 1.0 / math.sqrt(c["d"])
    L = c.get("layers", 1)
    for l in range(L):
        layer = s["sv_layers"][l]
        q = s.get("q")
        if c["kind"] != "tree":
            p, Hkv = s["proj"][l], c["Hkv"]
            q = s["q_out"][l]
            sv.sv_qk_norm_rope_append(p[:, :, :H], p[:, :, H: H + Hkv], p[:, :, H + Hkv:], s["sv_rot"], layer,
                                      s["sv_seqs"], q, s["ws"], n_new=s["n_new"])
        if c["kind"] != "append":
            sv.sv_tree_attn(q, scale, layer, s["sv_seqs"], s["vis"], c["k"], s["mask"], s["out"][l], s["lse"][l],
                            s["ws"], n_new=s["n_new"])
    if c["kind"] == "append":
        return {"q": s["q_out"][0], "k": s["kp"][0], "v": s["vp"][0]}
    if c["kind"] == "tree":
        return {"out": s["out"][0], "lse": s["lse"][0]}
    sv.sv_kv_accept(s["sv_layers"], s["sv_seqs"], c["T"], s["path"], s["ws"], n_path=s["n_path"])
    return {"q": s["q_out"], "out": s["out"], "lse": s["lse"], "k": s["kp"], "v": s["vp"]}


# ---- plain form: elementary operations in 32 bits, rounded once

def _plain_norm_rope(x, w, R):
    """x [B][T][h][d] -> normalised and rotated, fp32."""
    x = x.float()
    if w is not None:
        x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + R["eps"]) * w.float()
    rot, half = R["rot"], R["rot"] // 2
    pos = R["pos"].long()                                     # [axes][B][T]
    cs = R["table"][pos]                                      # [axes][B][T][half][2]
    if R["sections"] is None:
        cs = cs[0]
    else:
        parts, at = [], 0
        for a, n in enumerate(R["sections"]):
            parts.append(cs[a, :, :, at: at + n])
            at += n
        cs = torch.cat(parts, dim=2)
    cos, sin = cs[..., 0].unsqueeze(2), cs[..., 1].unsqueeze(2)
    if R["interleaved"]:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        y = torch.stack([a * cos - b * sin, a * sin + b * cos], dim=-1).flatten(-2)
    else:
        a, b = x[..., :half], x[..., half:rot]
        y = torch.cat([a * cos - b * sin, a * sin + b * cos], dim=-1)
    return torch.cat([y, x[..., rot:]], dim=-1)


def _plain_append(c, s, l):
    H, Hkv = c["H"], c["Hkv"]
    p, (b, t) = s["proj"][l], s["live"]
    q = _plain_norm_rope(p[:, :, :H], s["rot"]["qw"], s["rot"]).to(torch.bfloat16)
    k = _plain_norm_rope(p[:, :, H: H + Hkv], s["rot"]["kw"], s["rot"]).to(torch.bfloat16)
    s["q_out"][l][b, t] = q[b, t]
    at = s["base"][b] + t
    page = s["table"][b, at // PAGE].long()
    s["kp"][l][page, :, at % PAGE] = k[b, t]
    s["vp"][l][page, :, at % PAGE] = p[b, t, H + Hkv:]


def _plain_tree(c, s, l, q):
    B, T, Hkv, d, G = c["B"], c["T"], c["Hkv"], c["d"], c["H"] // c["Hkv"]
    scale = 1.0 / math.sqrt(d)
    per_seq = lambda x: x.view(B, 1, 1)
    # the tokens of every sequence and KV head: selected (or all) visual ones, text, drafted ones
    n_sel = c["k"] or c["n_vis"]
    sel = torch.arange(n_sel, device=DEV).expand(B, Hkv, n_sel) if s["vis"] is None else s["vis"].long()
    tail = torch.arange(c["n_text"] + T, device=DEV).expand(B, Hkv, c["n_text"] + T)
    have = torch.cat([torch.arange(n_sel, device=DEV) < per_seq(s["sel_n"]),
                      torch.arange(c["n_text"] + T, device=DEV) < per_seq(s["text_n"] + s["new_n"])], dim=2)
    at = torch.cat([sel, tail + per_seq(s["vis_n"])], dim=2)
    at = torch.where(have, at, 0)
    page = torch.gather(s["table"].long().unsqueeze(1).expand(B, Hkv, -1), 2, at // PAGE)
    head = torch.arange(Hkv, device=DEV).view(1, Hkv, 1)
    K = s["kp"][l][page, head, at % PAGE].float()              # [B][Hkv][tokens][d]
    V = s["vp"][l][page, head, at % PAGE].float()
    x = q.float().view(B, T, Hkv, G, d).transpose(1, 2).reshape(B, Hkv, T * G, d)
    z = torch.matmul(x, K.transpose(2, 3)) * scale
    # the drafted token of each column (negative: context), and whether a row sees it
    j = torch.cat([torch.full((B, n_sel), -1, device=DEV),
                   torch.arange(c["n_text"] + T, device=DEV) - s["text_n"].view(B, 1)], dim=1).view(B, 1, -1)
    if s["mask"] is None:
        seen = j <= torch.arange(T, device=DEV).view(1, T, 1)
    else:
        seen = (j < 0) | (((s["mask"].unsqueeze(2) >> j.clamp(0, 63)) & 1) != 0)
    seen = seen.repeat_interleave(G, 1).unsqueeze(1) & have.unsqueeze(2)
    z = torch.where(seen, z, -math.inf)
    m = z.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, 0.0, m)
    w = torch.exp(z - m)
    total = w.sum(-1, keepdim=True)
    o = torch.matmul(w, V) / torch.where(total == 0, 1.0, total)
    o = o.view(B, Hkv, T, G, d).transpose(1, 2).reshape(B, T, Hkv * G, d)
    lse = (m + torch.log(total)).view(B, Hkv, T, G).transpose(1, 2).reshape(B, T, Hkv * G)
    b, t = s["live"]
    s["out"][l][b, t] = o[b, t].to(torch.bfloat16)
    s["lse"][l][b, t] = lse[b, t]


def _plain_accept(c, s):
    b, i = s["took"]
    src, dst = s["base"][b] + s["path"][b, i], s["base"][b] + i
    src_page, dst_page = s["table"][b, src // PAGE].long(), s["table"][b, dst // PAGE].long()
    for pool in s["kp"] + s["vp"]:
        pool[dst_page, :, dst % PAGE] = pool[src_page, :, src % PAGE]


def _plain_pages(c, s):
    table, ref, n_pages = s["table"], s["ref"], s["n_pages"]
    rows, per = table.shape
    col = torch.arange(per, device=DEV)
    # release: the rows' entries behind what they keep
    keep = torch.where(s["keep"] < 0, n_pages, torch.minimum(n_pages, (s["keep"] + PAGE - 1) // PAGE))
    drop = (col >= keep[:, None]) & (col < n_pages[:, None])
    ref.index_put_((torch.where(drop, table, 0).long(),), -drop.to(torch.int32), accumulate=True)
    table.copy_(torch.where(drop, -1, table))
    n_pages.copy_(keep)
    # fork: the children share their parents' pages
    par, kid = s["parent"].long(), s["child"].long()
    took = col < n_pages[par][:, None]
    ref.index_put_((torch.where(took, table[par], 0).long(),), took.to(torch.int32), accumulate=True)
    table[kid] = torch.where(took, table[par], table[kid])
    n_pages[kid] = n_pages[par]
    # reserve: missing pages, and private copies of shared ones
    n, T, new = c["n_tok"], c["T"], s["n_new"][:, None]
    first, last = n // PAGE, (n + new - 1) // PAGE
    held = n_pages[:, None]
    wanted = (new > 0) & (col >= first) & (col <= last)
    shared = wanted & (col < held) & (ref[table.clamp(min=0).long()] > 1)
    fresh = (new > 0) & (col >= held) & (col <= last)
    need = shared | fresh
    free = torch.argsort((ref != 0).to(torch.int8), stable=True).to(torch.int32)
    nth = (torch.cumsum(need.view(-1).to(torch.int32), 0) - 1).clamp(min=0).view(rows, per)
    page = torch.where(need, free[nth], table)
    width = (T - 1) // PAGE + 2
    cols = (first + torch.arange(width, device=DEV)).clamp(max=per - 1)
    # a column without a copy moves a page onto itself: its own, or one in use
    src = torch.where(table < 0, table[0, 0], table)[:, cols]
    dst = torch.where(shared[:, cols], page[:, cols], src).long().view(-1)
    src = src.long().view(-1)
    for pool in s["kp"] + s["vp"]:
        pool[dst] = pool[src]
    ref.index_put_((torch.where(shared, table, 0).long(),), -shared.to(torch.int32), accumulate=True)
    ref.index_put_((torch.where(need, page, 0).long(),), need.to(torch.int32), accumulate=True)
    n_pages.copy_(torch.maximum(n_pages, torch.where(new > 0, last + 1, 0).view(-1)))
    table.copy_(page)


def _plain_run(c, s):
    if c["kind"] == "encode":
        H = c["H"]
        q = _plain_norm_rope(s["proj"][:, :, :H], s["rot"]["qw"], s["rot"])
        k = _plain_norm_rope(s["proj"][:, :, H:], s["rot"]["kw"], s["rot"])
        return {"q": q.transpose(1, 2).to(torch.bfloat16).contiguous(),
                "k": k.transpose(1, 2).to(torch.bfloat16).contiguous()}
    if c["kind"] == "pages":
        _plain_pages(c, s)
        return {"table": s["table"], "n_pages": s["n_pages"], "ref": s["ref"], "k": s["kp"], "v": s["vp"]}
    for l in range(c.get("layers", 1)):
        if c["kind"] != "tree":
            _plain_append(c, s, l)
        if c["kind"] != "append":
            _plain_tree(c, s, l, s["q"] if c["kind"] == "tree" else s["q_out"][l])
    if c["kind"] == "append":
        return {"q": s["q_out"][0], "k": s["kp"][0], "v": s["vp"][0]}
    if c["kind"] == "tree":
        return {"out": s["out"][0], "lse": s["lse"][0]}
    _plain_accept(c, s)
    return {"q": s["q_out"], "out": s["out"], "lse": s["lse"], "k": s["kp"], "v": s["vp"]}


# ------------------------------------------------------------------ 64 bits

def _exact_rotate(x, w, R):
    """One token-major tensor from the definition: complex products per pair."""
    x = x.double()
    B, T, h, d = x.shape
    if w is not None:
        x = x / torch.sqrt((x ** 2).sum(-1, keepdim=True) / d + R["eps"]) * w.double()
    y = x.clone()
    axis = []
    for a, n in enumerate(R["sections"] or [R["rot"] // 2]):
        axis += [a] * n
    turn = torch.view_as_complex(R["table"].double())
    for p, a in enumerate(axis):
        i, j = (2 * p, 2 * p + 1) if R["interleaved"] else (p, p + R["rot"] // 2)
        z = torch.complex(x[..., i], x[..., j]) * turn[R["pos"][a].long(), p][:, :, None]
        y[..., i], y[..., j] = z.real, z.imag
    return y


def _exact_attend(q, K, V, seen, scale):
    """q [rows][d], K and V [tokens][d], seen [rows][tokens], 64 bits."""
    z = (q @ K.T * scale).masked_fill(~seen, -math.inf)
    lse = torch.logsumexp(z, -1)
    p = torch.exp(z - torch.where(lse == -math.inf, 0.0, lse)[:, None])
    return p @ V, lse


def _exact_tree(c, s, l, q, out, lse):
    G = c["H"] // c["Hkv"]
    for b in range(c["B"]):
        n, ctx = s["tn"][b], s["nv"][b] + s["nt"][b]
        row = s["table"][b].long()
        tree = torch.zeros(n, n, dtype=torch.bool)
        bits = None if s["mask"] is None else s["mask"][b].cpu().numpy().view(np.uint64)
        for t in range(n):
            for j in range(n):
                tree[t, j] = j <= t if bits is None else bool((int(bits[t]) >> j) & 1)
        tree = tree.to(DEV)
        for g in range(c["Hkv"]):
            where = list(range(s["nv"][b])) if s["vis"] is None else s["vis"][b, g, : s["ks"][b]].tolist()
            where = torch.tensor(where + list(range(s["nv"][b], ctx + n)), device=DEV)
            K = s["kp"][l][row[where // PAGE], g, where % PAGE].double()
            V = s["vp"][l][row[where // PAGE], g, where % PAGE].double()
            seen = torch.cat([torch.ones(n, len(where) - n, dtype=torch.bool, device=DEV), tree], dim=1)
            for h in range(g * G, (g + 1) * G):
                out[b, :n, h], lse[b, :n, h] = _exact_attend(q[b, :n, h].double(), K, V, seen, 1.0 / math.sqrt(c["d"]))


def _exact_append(c, s, l):
    """Queries in 64 bits; the pools as 64-bit tensors with the new rows."""
    H, Hkv = c["H"], c["Hkv"]
    p = s["proj"][l]
    q = _exact_rotate(p[:, :, :H], s["rot"]["qw"], s["rot"])
    k = _exact_rotate(p[:, :, H: H + Hkv], s["rot"]["kw"], s["rot"])
    kp, vp = s["kp"][l].double(), s["vp"][l].double()
    for b in range(c["B"]):
        q[b, s["tn"][b]:] = 0
        for t in range(s["tn"][b]):
            at = s["nv"][b] + s["nt"][b] + t
            page = s["table_host"][b][at // PAGE]
            kp[page, :, at % PAGE] = k[b, t]
            vp[page, :, at % PAGE] = p[b, t, H + Hkv:].double()
    return q, kp, vp


def _exact_pages(c, s):
    """The three calls, page by page."""
    table, ref, held = s["table"].tolist(), s["ref"].tolist(), s["n_pages"].tolist()
    keep, new = s["keep"].tolist(), s["n_new"].tolist()
    for row in range(len(table)):
        if keep[row] >= 0:
            for i in range(-(-keep[row] // PAGE), held[row]):
                ref[table[row][i]] -= 1
                table[row][i] = -1
            held[row] = min(held[row], -(-keep[row] // PAGE))
    for par, kid in zip(s["parent"].tolist(), s["child"].tolist()):
        for i in range(held[par]):
            table[kid][i] = table[par][i]
            ref[table[par][i]] += 1
        held[kid] = held[par]
    free = iter([p for p, n in enumerate(ref) if n == 0])
    before, copies = list(ref), []
    for row, T in enumerate(new):
        if T == 0:
            continue
        for i in range(c["n_tok"] // PAGE, (c["n_tok"] + T - 1) // PAGE + 1):
            if i < held[row]:
                if before[table[row][i]] <= 1:
                    continue
                to = next(free)
                copies.append((table[row][i], to))
                ref[table[row][i]] -= 1
            else:
                to = next(free)
            table[row][i] = to
            ref[to] += 1
        held[row] = max(held[row], (c["n_tok"] + T - 1) // PAGE + 1)
    pools = []
    for group in (s["kp"], s["vp"]):
        pools.append([])
        for x in group:
            y = x.clone()
            for a, b in copies:
                y[b] = x[a]
            pools[-1].append(y)
    as32 = lambda x: torch.tensor(x, dtype=torch.int32)
    return {"table": as32(table), "n_pages": as32(held), "ref": as32(ref), "k": pools[0], "v": pools[1]}


def exact(case, seed):
    global own
    c = case
    was, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = was
    if c["kind"] == "pages":
        return _exact_pages(c, s)
    if c["kind"] == "encode":
        H = c["H"]
        q = _exact_rotate(s["proj"][:, :, :H], s["rot"]["qw"], s["rot"])
        k = _exact_rotate(s["proj"][:, :, H:], s["rot"]["kw"], s["rot"])
        return {"q": q.transpose(1, 2).contiguous(), "k": k.transpose(1, 2).contiguous()}
    s["table_host"] = s["table"].tolist()
    if c["kind"] == "append":
        q, kp, vp = _exact_append(c, s, 0)
        return {"q": q, "k": kp, "v": vp}
    outs = {"q": [], "out": [], "lse": [], "k": [], "v": []}
    for l in range(c.get("layers", 1)):
        q = s.get("q")
        if c["kind"] == "step":
            q, kp, vp = _exact_append(c, s, l)
            outs["q"].append(q)
            # attention reads the rows as the cache and the query tensor hold them
            q = q.to(torch.bfloat16)
            s["kp"][l].copy_(kp)
            s["vp"][l].copy_(vp)
        out = torch.zeros(c["B"], c["T"], c["H"], c["d"], dtype=torch.float64, device=DEV)
        lse = torch.zeros(c["B"], c["T"], c["H"], dtype=torch.float64, device=DEV)
        _exact_tree(c, s, l, q, out, lse)
        if c["kind"] == "tree":
            return {"out": out, "lse": lse}
        for pool in (kp, vp):
            old = pool.clone()
            for b in range(c["B"]):
                base = s["nv"][b] + s["nt"][b]
                for i, j in enumerate(s["path"][b, : s["acc"][b]].tolist()):
                    to, at = base + i, base + j
                    pool[s["table_host"][b][to // PAGE], :, to % PAGE] = \
                        old[s["table_host"][b][at // PAGE], :, at % PAGE]
        outs["out"].append(out)
        outs["lse"].append(lse)
        outs["k"].append(kp)
        outs["v"].append(vp)
    return outs
