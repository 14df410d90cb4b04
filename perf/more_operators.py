"""Workloads of the prompt and of the cache in 8 bits.

A prompt's packed tokens enter the layer: queries and keys are normalised and
rotated, attend to one another within their sequences, and keys and values go
into a paged cache of 8-bit values (e4m3) with one power of two per page of 16
tokens and KV head.  Decode steps then append to that cache, retrieve from its
visual keys and attend over what they selected.  Four kinds of case:

  prompt    causal attention of packed sequences of different lengths, grouped
            heads, read from the slices of a fused projection
  append    norm, rotation and rounding of new tokens into the 8-bit pages
  retrieve  scores of the cached visual keys and the selection of the largest
  attend    one query per head over the selected visual tokens and the text
"""

import math

import numpy as np
import torch

own = False

PAGE = 16          # tokens of a cache page
DEV = "cuda"
E4M3 = torch.float8_e4m3fn
TOP = 448.0        # the largest e4m3 value
LEAST = 2.0 ** -126  # the smallest scale


# ------------------------------------------------------------------ cases

def listed():
    return [
        # the round-loop shape (4 query, 2 KV heads, d 64): the visual tokens
        # that a prune kept, and a short text; latency
        dict(name="prompt_tiny", kind="prompt", B=1, T=176, H=4, Hkv=2, d=64, ragged=False),
        # short questions of many users, packed: lengths from 0 to 97
        dict(name="prompt_questions_b48", kind="prompt", B=48, T=97, H=28, Hkv=4, d=128, ragged=True),
        # LLaVA-NeXT-7B prefill of four requests: 2880 visual and 128 text tokens
        dict(name="prompt_llava_next_b4", kind="prompt", B=4, T=3008, H=32, Hkv=32, d=128, ragged=False),
        # LongVILA-7B prefill of one long video, a quarter of its visual tokens
        # kept: bound by the matrix products
        dict(name="prompt_longvila_12800", kind="prompt", B=1, T=12800, H=28, Hkv=4, d=128, ragged=False),
        # one decode token per sequence of LLaVA-NeXT-7B, batch 16: latency
        dict(name="append_decode_b16", kind="append", B=16, T=1, H=32, Hkv=32, d=128, n_vis=2880, n_text=128, axes=1,
             rot=128, norm=False, interleaved=False, ragged=False, k_out=False),
        # a second question of 193 tokens, behind a text that ends inside a page
        dict(name="append_question_193", kind="append", B=2, T=193, H=4, Hkv=2, d=64, n_vis=576, n_text=41, axes=1,
             rot=64, norm=False, interleaved=False, ragged=False, k_out=False),
        # prefill of eight LongVILA-7B clips at 16 frames, the sequences of
        # different lengths, with the norms and axes that other decoders bring;
        # the rotated keys also go to the prompt's attention
        dict(name="append_prompt_b8", kind="append", B=8, T=3392, H=28, Hkv=4, d=128, n_vis=0, n_text=0, axes=3,
             rot=128, norm=True, interleaved=False, ragged=True, k_out=True),
        # LLaVA-NeXT-7B, 16 sequences, half of the visual tokens selected by
        # the decode token's own queries
        dict(name="retrieve_llava_next_b16", kind="retrieve", B=16, R=1, H=32, Hkv=32, d=128, n_vis=2880, k=1440,
             n_text=128, ragged=False),
        # LongVILA-7B, 8 sequences of up to 50176 visual tokens, a quarter of them
        dict(name="retrieve_longvila_b8", kind="retrieve", B=8, R=1, H=28, Hkv=4, d=128, n_vis=50176, k=12544,
             n_text=256, ragged=True),
        # the round-loop shape: latency
        dict(name="attend_tiny", kind="attend", B=1, H=4, Hkv=2, d=64, n_vis=576, k=144, n_text=57, ragged=False),
        # LLaVA-NeXT-7B, 16 sequences, half of the visual tokens: bound by the cache
        dict(name="attend_llava_next_b16", kind="attend", B=16, H=32, Hkv=32, d=128, n_vis=2880, k=1440, n_text=128,
             ragged=False),
        # LongVILA-7B, 8 sequences of different lengths
        dict(name="attend_longvila_b8", kind="attend", B=8, H=28, Hkv=4, d=128, n_vis=50176, k=12544, n_text=256,
             ragged=True),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _heads(rng):
    """(H, Hkv): equal heads, or groups of up to 16."""
    Hkv = rng.choice([1, 2, 3, 4, 8, 32])
    G = rng.choice([1, 1, 2, 4, 5, 7, 8, 16]) if Hkv <= 8 else 1
    return Hkv * G, Hkv


def draw(rng):
    kind = rng.choice(["prompt", "append", "retrieve", "attend"])
    H, Hkv = _heads(rng)
    d = rng.choice([64, 128])
    ragged = rng.random() < 0.5
    if kind == "prompt":
        # at most the logits and the rows of the largest listed cases
        T = _log_int(rng, 1, 12800)
        T = min(T, int(math.isqrt(int(4.5e9) // H)))
        B = max(1, min(_log_int(rng, 1, 64), int(4.5e9 / (T * T * H)), int(1.15e6 / (T * (H + 2 * Hkv)))))
        return dict(kind=kind, B=B, T=T, H=H, Hkv=Hkv, d=d, ragged=ragged)
    if kind == "append":
        T = _log_int(rng, 1, 3392)
        B = max(1, min(_log_int(rng, 1, 32), 8 * 3392 * 36 // (T * (H + 2 * Hkv)) or 1))
        return dict(kind=kind, B=B, T=T, H=H, Hkv=Hkv, d=d, n_vis=_log_int(rng, 1, 3136), n_text=_log_int(rng, 1, 300),
                    axes=rng.choice([1, 3]), rot=rng.choice([d, d, d // 2]), norm=rng.random() < 0.5,
                    interleaved=rng.random() < 0.5, ragged=ragged, k_out=rng.random() < 0.5)
    n_vis = _log_int(rng, 16, 50176)
    # at most the cache rows of the largest listed cases
    B = max(1, min(_log_int(rng, 1, 16), int((1.45e6 if kind == "retrieve" else 0.8e6) / (n_vis * Hkv))))
    k = max(1, int(n_vis * rng.choice([0.1, 0.25, 0.5, 0.9])))
    c = dict(kind=kind, B=B, H=H, Hkv=Hkv, d=d, n_vis=n_vis, k=k, n_text=_log_int(rng, 1, 300), ragged=ragged)
    if kind == "retrieve":
        c["R"] = rng.choice([1, 1, 2, 9, 32])
    elif rng.random() < 0.25:
        c["k"] = 0               # no index list: every visual token
    return c


def _new_tokens(c):
    """New tokens of every sequence; ragged batches have short and empty ones."""
    B, T = c["B"], c["T"]
    if not c["ragged"]:
        return [T] * B
    return [0 if b % 9 == 8 else max(1, int(T * (1.0 - 0.95 * ((b * 5) % B) / B))) for b in range(B)]


def _lengths(c):
    """Visual, text and selected tokens of every sequence."""
    B, k = c["B"], c.get("k", 0)
    if not c["ragged"]:
        return [c["n_vis"]] * B, [c["n_text"]] * B, [k] * B
    nv, nt, ks = [], [], []
    for b in range(B):
        part = 1.0 - 0.6 * ((b * 5) % B) / B
        nv.append(int(c["n_vis"] * part))
        nt.append(int(c["n_text"] * (1.0 - 0.5 * ((b * 3) % B) / B)))
        ks.append(min(int(k * part), nv[-1]))
    return nv, nt, ks


def _sections(c):
    """Rotation pairs of each position axis."""
    if c["axes"] == 1:
        return None
    half = c["rot"] // 2
    a = half // 4
    b = (half - a) // 2
    return [a, b, half - a - b]


def work(case):
    c = case
    H, Hkv, d = c["H"], c["Hkv"], c["d"]
    if c["kind"] == "prompt":
        n = _new_tokens(c)
        return {"bytes": 4 * sum(n) * (H + Hkv) * d + 4 * sum(n) * H,
                "flops": sum(2 * t * (t + 1) for t in n) * H * d}
    if c["kind"] == "append":
        n = sum(_new_tokens(c))
        return {"bytes": n * d * (4 * H + (8 if c["k_out"] else 6) * Hkv) + 4 * n * c["axes"],
                "flops": (7 if c["norm"] else 3) * n * (H + Hkv) * d + 4 * n * Hkv * d}
    nv, nt, ks = _lengths(c)
    if c["kind"] == "retrieve":
        keys = sum(nv) * Hkv
        return {"bytes": keys * (d + 4) + sum(-(-n // PAGE) for n in nv) * Hkv * 4 + 4 * sum(ks) * Hkv
                + 2 * c["B"] * c["R"] * H * d, "flops": 2 * keys * d + c["B"] * c["R"] * H * d}
    rows = sum((ks[b] if c["k"] else nv[b]) + nt[b] for b in range(c["B"])) * Hkv
    return {"bytes": rows * 2 * d + rows * 8 // PAGE + 4 * (sum(ks) if c["k"] else 0) * Hkv + 4 * c["B"] * H * d
            + 4 * c["B"] * H, "flops": 4 * rows * (H // Hkv) * d}


# ------------------------------------------------------------------ inputs

class _Rand:
    """Seeded draws on the device."""

    def __init__(self, seed):
        self.g = torch.Generator(device=DEV)
        self.g.manual_seed(int(seed) * 6007 + 29)

    def normal(self, *shape):
        return torch.randn(*shape, generator=self.g, device=DEV).to(torch.bfloat16)

    def perm(self, n):
        return torch.randperm(n, generator=self.g, device=DEV)

    def ints(self, lo, hi, *shape):
        return torch.randint(lo, hi, shape, generator=self.g, device=DEV, dtype=torch.int32)


def _i32(x):
    return torch.as_tensor(np.asarray(x, dtype=np.int32)).to(DEV)


def _outliers(r, x, dim):
    """Some tokens' rows are the outliers that real keys have."""
    shape = [1] * x.dim()
    shape[dim] = x.shape[dim]
    return torch.where(r.ints(0, 50, *shape) == 0, x * 4, x)


def _scale_of(top):
    """The smallest power of two, at least 2^-126, that brings `top` (fp32) into e4m3's range."""
    m, e = torch.frexp(top)                               # top = m 2^e, m in [0.5, 1); 448 = 0.875 2^9
    e = torch.where(top == 0, -126, (e - 9 + (m > 0.875)).clamp(min=-126))
    return torch.ldexp(torch.ones_like(top), e)


def _as_e4m3(x):
    return x.clamp(-TOP, TOP).to(E4M3)


def _cache(r, blocks, Hkv, d, outliers):
    """Pools of 8-bit rows and their scales, from normally distributed rows."""
    pools, scales = [], []
    for which in range(2):
        x = r.normal(blocks, Hkv, PAGE, d)
        if outliers:
            x = torch.where(r.ints(0, 50, blocks, 1, PAGE, 1) == 0, x * 4, x)
        x = x.float()
        s = _scale_of(x.abs().amax((2, 3)))
        pools.append(_as_e4m3(x / s[:, :, None, None]))
        scales.append(s)
    return pools[0], pools[1], torch.stack(scales, dim=-1).contiguous()


def _rows_of(counts):
    """(sequence, index) of every i < counts[b]."""
    n = torch.tensor(counts)
    b = torch.repeat_interleave(torch.arange(len(counts)), n)
    i = torch.arange(int(n.sum())) - torch.repeat_interleave(torch.cumsum(n, 0) - n, n)
    return b.to(DEV), i.to(DEV)


def prepare(case, seed):
    c, r = case, _Rand(seed)
    s = {"c": c}
    B, H, Hkv, d = c["B"], c["H"], c["Hkv"], c["d"]
    if c["kind"] in ("prompt", "append"):
        s["n"] = _new_tokens(c)
        N = sum(s["n"])
        # one fused projection: queries, keys and values are slices of its rows
        s["proj"] = r.normal(N, H + 2 * Hkv, d)
        s["start"] = _i32(np.concatenate([[0], np.cumsum(s["n"])]))
        s["row"] = _rows_of(s["n"])
    if c["kind"] == "prompt":
        s["proj"][:, H: H + Hkv] = _outliers(r, s["proj"][:, H: H + Hkv], 0)
        s["out"] = torch.zeros(N, H, d, dtype=torch.bfloat16, device=DEV)
        s["lse"] = torch.zeros(N, H, device=DEV)
        return _plan(c, s) if own else s
    nv, nt, ks = _lengths(c)
    s.update(nv=nv, nt=nt, ks=ks, vis_n=_i32(nv), text_n=_i32(nt), sel_n=_i32(ks if c.get("k") else nv))
    s["lens"] = tuple(_i32(x) for x in (nv, nt, ks)) if c["ragged"] else (None, None, None)
    per = -(-(c["n_vis"] + c["n_text"] + c.get("T", 0)) // PAGE)
    blocks = B * per + 3
    s["table"] = r.perm(blocks)[: B * per].to(torch.int32).view(B, per).contiguous()
    s["k8"], s["v8"], s["scales"] = _cache(r, blocks, Hkv, d, True)
    if c["kind"] == "append":
        n_pos = c["n_vis"] + c["n_text"] + c["T"] + 1
        half = c["rot"] // 2
        freq = 10000.0 ** (-torch.arange(half, dtype=torch.float64, device=DEV) / half)
        a = torch.arange(n_pos, dtype=torch.float64, device=DEV)[:, None] * freq
        s["turns"] = torch.stack([a.cos(), a.sin()], dim=-1).float().contiguous()
        b, i = s["row"]
        at = (s["vis_n"] + s["text_n"])[b] + i
        s["at"] = at
        s["pos"] = torch.stack([at] + [(at * (3 + x)) % n_pos for x in range(c["axes"] - 1)]).to(torch.int32)
        s["pos"] = s["pos"].unsqueeze(1).contiguous()         # [axes][1][N]
        s["qw"] = s["kw"] = None
        if c["norm"]:
            s["qw"] = (1 + 0.1 * r.normal(d).float()).to(torch.bfloat16)
            s["kw"] = (1 + 0.1 * r.normal(d).float()).to(torch.bfloat16)
        s["q_out"] = torch.zeros(N, H, d, dtype=torch.bfloat16, device=DEV)
        s["k_out"] = torch.zeros(N, Hkv, d, dtype=torch.bfloat16, device=DEV) if c["k_out"] else None
    elif c["kind"] == "retrieve":
        s["q"] = r.normal(B, c["R"], H, d)
        s["vis"] = torch.zeros(B, Hkv, c["k"], dtype=torch.int32, device=DEV)
        s["scores"] = torch.zeros(B, Hkv, c["n_vis"], device=DEV)
    else:
        s["q"] = r.normal(B, H, d)
        s["vis"] = None
        if c["k"]:
            s["vis"] = torch.full((B, Hkv, c["k"]), -1, dtype=torch.int32, device=DEV)
            for b in range(B):
                pick = torch.rand(Hkv, max(nv[b], 1), generator=r.g, device=DEV).topk(ks[b], dim=1).indices
                s["vis"][b, :, : ks[b]] = pick.sort(dim=1).values.to(torch.int32)
        s["out"] = torch.zeros(B, H, d, dtype=torch.bfloat16, device=DEV)
        s["lse"] = torch.zeros(B, H, device=DEV)
    return _plan(c, s) if own else s


# ------------------------------------------------------------------ one pass

def run(state):
    c = state["c"]
    return (_own_run if own else _plain_run)(c, state)


def _plan(c, s):
    """The descriptors and workspaces that a program keeps."""
    from visual_token_sparsity_gb300 import binding as sv
    B, H, Hkv, d = c["B"], c["H"], c["Hkv"], c["d"]
    if c["kind"] == "prompt":
        s["ws"] = sv.workspace(sv.sv_prompt_attn_workspace_bytes(s["proj"].shape[0], B, H, Hkv, d))
        return s
    s["sv_layer"] = sv.Kv8Layer(s["k8"], s["v8"], s["scales"])
    nv, nt, ks = s["lens"]
    s["sv_seqs"] = sv.SeqBatch(s["table"], c["n_vis"], c["n_text"], nv, nt, ks if c.get("k") else None)
    if c["kind"] == "append":
        s["sv_rot"] = sv.Rotation(s["turns"], s["pos"] if c["axes"] > 1 else s["pos"][0], sections=_sections(c),
                                  interleaved=c["interleaved"], q_weight=s["qw"], k_weight=s["kw"], eps=1e-6)
        s["ws"] = sv.workspace(sv.sv_evict_workspace_bytes())
    elif c["kind"] == "retrieve":
        s["ws"] = sv.workspace(sv.sv_kv8_retrieve_workspace_bytes(B, H, Hkv, d, c["n_vis"], c["k"]))
    else:
        s["ws"] = sv.workspace(sv.sv_kv8_attn_workspace_bytes(B, H, Hkv, d, (c["k"] or c["n_vis"]) + c["n_text"]))
    return s


def _outputs(c, s):
    if c["kind"] == "prompt":
        return {"out": s["out"], "lse": s["lse"]}
    if c["kind"] == "append":
        # the cache as values: e4m3 ones, and what they are multiplied with
        return {"q": s["q_out"], "k": s["k8"], "v": s["v8"], "scales": s["scales"], "k_out": s["k_out"]}
    if c["kind"] == "retrieve":
        return {"vis": s["vis"], "scores": s["scores"]}
    return {"out": s["out"], "lse": s["lse"]}


def _own_run(c, s):
    from visual_token_sparsity_gb300 import binding as sv
    H, Hkv = c["H"], c["Hkv"]
    if c["kind"] in ("prompt", "append"):
        p = s["proj"]
        q, k, v = p[:, :H], p[:, H: H + Hkv], p[:, H + Hkv:]
    if c["kind"] == "prompt":
        sv.sv_prompt_attn(q, k, v, s["start"], 1.0 / math.sqrt(c["d"]), s["out"], s["lse"], s["ws"])
    elif c["kind"] == "append":
        sv.sv_kv8_append(q, k, v, s["sv_rot"], s["sv_layer"], s["sv_seqs"], s["q_out"], s["ws"],
                         seq_start=s["start"], k_out=s["k_out"])
    elif c["kind"] == "retrieve":
        sv.sv_kv8_retrieve_topk(s["q"], s["sv_layer"], s["sv_seqs"], c["k"], s["vis"], s["scores"], s["ws"])
    else:
        sv.sv_kv8_decode_attn(s["q"], 1.0 / math.sqrt(c["d"]), s["sv_layer"], s["sv_seqs"], s["vis"], c["k"],
                              s["out"], s["lse"], s["ws"])
    return _outputs(c, s)


# ---- plain form: elementary operations in 32 bits, rounded once

def _plain_prompt(c, s):
    B, T, H, Hkv, d = c["B"], c["T"], c["H"], c["Hkv"], c["d"]
    G = H // Hkv
    b, i = s["row"]
    # padded to the longest sequence; a row behind its end reads the sequence's first
    at = s["start"][:-1, None] + torch.arange(T, device=DEV)
    at = torch.where(at < s["start"][1:, None], at, s["start"][:-1, None]).clamp(max=s["proj"].shape[0] - 1)
    x = s["proj"][at].float().transpose(1, 2)                  # [B][heads][T][d]
    q = x[:, :H].reshape(B, Hkv, G * T, d)
    k, v = x[:, H: H + Hkv], x[:, H + Hkv:]
    z = torch.matmul(q, k.transpose(2, 3)).mul_(1.0 / math.sqrt(d)).view(B, Hkv, G, T, T)
    later = torch.arange(T, device=DEV)[:, None] < torch.arange(T, device=DEV)
    z.masked_fill_(later, -math.inf)
    m = z.amax(-1, keepdim=True)
    z.sub_(m).exp_()
    total = z.sum(-1, keepdim=True)
    o = torch.matmul(z.view(B, Hkv, G * T, T), v).view(B, Hkv, G, T, d) / total
    lse = (m + total.log()).view(B, H, T)
    s["out"].copy_(o.view(B, H, T, d)[b, :, i])
    s["lse"].copy_(lse[b, :, i])


def _plain_norm_rotate(c, s, x, w):
    """x [N][h][d] -> normalised and rotated, rounded to bf16.  In 64 bits: the 8-bit
    rows follow from the bf16 ones, and a result next to a border must fall on its side."""
    x = x.double()
    if w is not None:
        x = x / torch.sqrt((x * x).mean(-1, keepdim=True) + 1e-6) * w.double()
    rot, half = c["rot"], c["rot"] // 2
    cs = s["turns"].double()[s["pos"][:, 0].long()]            # [axes][N][half][2]
    sec = _sections(c)
    axis = torch.zeros(half, dtype=torch.long) if sec is None else \
        torch.repeat_interleave(torch.arange(3), torch.tensor(sec))
    cs = cs[axis.to(DEV), :, torch.arange(half, device=DEV)].transpose(0, 1)     # [N][half][2]
    cos, sin = cs[:, None, :, 0], cs[:, None, :, 1]
    if c["interleaved"]:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        y = torch.stack([a * cos - b * sin, a * sin + b * cos], dim=-1).flatten(-2)
    else:
        a, b = x[..., :half], x[..., half:rot]
        y = torch.cat([a * cos - b * sin, a * sin + b * cos], dim=-1)
    return torch.cat([y, x[..., rot:]], dim=-1).to(torch.bfloat16)


def _plain_append(c, s):
    H, Hkv = c["H"], c["Hkv"]
    p = s["proj"]
    s["q_out"].copy_(_plain_norm_rotate(c, s, p[:, :H], s["qw"]))
    k = _plain_norm_rotate(c, s, p[:, H: H + Hkv], s["kw"])
    if s["k_out"] is not None:
        s["k_out"].copy_(k)
    b, i = s["row"]
    at = s["at"]
    page, slot = s["table"][b, at // PAGE].long(), at % PAGE
    # per touched page: the first new slot, and the largest new magnitude of each head
    pages, nth = torch.unique(page, return_inverse=True)
    first = torch.full(pages.shape, PAGE, device=DEV).scatter_reduce_(0, nth, slot.long(), "amin")
    earlier = (torch.arange(PAGE, device=DEV) < first[:, None]).view(-1, 1, PAGE, 1)
    for which, x, pool in ((0, k, s["k8"]), (1, p[:, H + Hkv:], s["v8"])):
        x, pool = x.float(), pool.view(torch.uint8)
        top = torch.zeros(pages.shape[0], Hkv, device=DEV)
        top.scatter_reduce_(0, nth[:, None].expand(-1, Hkv), x.abs().amax(-1), "amax")
        old = torch.where((first == 0)[:, None], LEAST, s["scales"][pages, :, which])
        new = torch.maximum(old, _scale_of(top))
        rows = pool[pages]
        grown = _as_e4m3(rows.view(E4M3).float() * (old / new)[:, :, None, None])
        pool[pages] = torch.where(earlier, grown.view(torch.uint8), rows)
        pool[page, :, slot] = _as_e4m3(x / new[nth][:, :, None]).view(torch.uint8)
        s["scales"][pages, :, which] = new


def _read(c, s, which, at, head):
    """Cache rows at logical positions [B][Hkv][n] in fp32."""
    page = torch.gather(s["table"].long().unsqueeze(1).expand(-1, c["Hkv"], -1), 2, at // PAGE)
    pool = (s["k8"], s["v8"])[which].view(torch.uint8)
    return pool[page, head, at % PAGE].view(E4M3).float() * s["scales"][page, head, which].unsqueeze(-1)


def _plain_retrieve(c, s):
    B, Hkv, n, k = c["B"], c["Hkv"], c["n_vis"], c["k"]
    head = torch.arange(Hkv, device=DEV).view(1, Hkv, 1)
    at = torch.arange(n, device=DEV).expand(B, Hkv, n)
    qbar = s["q"].double().sum(1).view(B, Hkv, -1, c["d"]).sum(2)
    # in 64 bits: the selection is made at a border between neighbouring scores
    z = torch.matmul(_read(c, s, 0, at, head).double(), qbar.unsqueeze(-1)).squeeze(-1)
    there = torch.arange(n, device=DEV) < s["vis_n"].view(B, 1, 1)
    z = torch.where(there, z, -math.inf)
    best = torch.sort(z, dim=-1, descending=True, stable=True).indices[..., :k]
    best = torch.where(torch.arange(k, device=DEV) < s["sel_n"].view(B, 1, 1), best, n).sort(-1).values
    s["vis"].copy_(torch.where(best == n, -1, best))
    s["scores"].copy_(torch.where(there, z, s["scores"].double()))


def _plain_attend(c, s):
    B, H, Hkv, d = c["B"], c["H"], c["Hkv"], c["d"]
    per_seq = lambda x: x.view(B, 1, 1)
    head = torch.arange(Hkv, device=DEV).view(1, Hkv, 1)
    n_sel, n_text = c["k"] or c["n_vis"], c["n_text"]
    sel = torch.arange(n_sel, device=DEV).expand(B, Hkv, n_sel) if s["vis"] is None else s["vis"].long()
    text = torch.arange(n_text, device=DEV).expand(B, Hkv, n_text)
    have = torch.cat([torch.arange(n_sel, device=DEV) < per_seq(s["sel_n"]),
                      torch.arange(n_text, device=DEV) < per_seq(s["text_n"])], dim=2)
    at = torch.where(have, torch.cat([sel, text + per_seq(s["vis_n"])], dim=2), 0)
    K, V = _read(c, s, 0, at, head), _read(c, s, 1, at, head)
    z = torch.matmul(s["q"].float().view(B, Hkv, H // Hkv, d), K.transpose(2, 3)) * (1.0 / math.sqrt(d))
    z = torch.where(have.unsqueeze(2), z, -math.inf)
    m = z.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, 0.0, m)
    w = torch.exp(z - m)
    total = w.sum(-1, keepdim=True)
    o = torch.matmul(w, V) / torch.where(total == 0, 1.0, total)
    s["out"].copy_(o.view(B, H, d))
    s["lse"].copy_((m + torch.log(total)).view(B, H))


def _plain_run(c, s):
    {"prompt": _plain_prompt, "append": _plain_append, "retrieve": _plain_retrieve, "attend": _plain_attend}[
        c["kind"]](c, s)
    return _outputs(c, s)


# ------------------------------------------------------------------ 64 bits

def _exact_prompt(c, s):
    H, Hkv, d = c["H"], c["Hkv"], c["d"]
    N = s["proj"].shape[0]
    out = torch.zeros(N, H, d, dtype=torch.float64, device=DEV)
    lse = torch.zeros(N, H, dtype=torch.float64, device=DEV)
    begin = 0
    for n in s["n"]:
        for g in range(Hkv):
            K = s["proj"][begin: begin + n, H + g].double()
            V = s["proj"][begin: begin + n, H + Hkv + g].double()
            for h in range(g * (H // Hkv), (g + 1) * (H // Hkv)):
                for r0 in range(0, n, 2048):                    # rows that see r1 tokens at most
                    r1 = min(n, r0 + 2048)
                    z = s["proj"][begin + r0: begin + r1, h].double() @ K[:r1].T / math.sqrt(d)
                    z = z + torch.full((r1 - r0, r1), -math.inf, dtype=torch.float64, device=DEV).triu(r0 + 1)
                    norm = torch.logsumexp(z, -1)
                    out[begin + r0: begin + r1, h] = torch.exp(z - norm[:, None]) @ V[:r1]
                    lse[begin + r0: begin + r1, h] = norm
        begin += n
    return {"out": out, "lse": lse}


def _exact_rotate(c, s, x, w):
    """Pair by pair, as complex products; the result rounded to bf16, as the cache's rows are."""
    x = x.double()
    if w is not None:
        x = x * torch.rsqrt((x ** 2).sum(-1, keepdim=True) / c["d"] + 1e-6) * w.double()
    y = x.clone()
    turn = torch.view_as_complex(s["turns"].double())
    axis = []
    for a, n in enumerate(_sections(c) or [c["rot"] // 2]):
        axis += [a] * n
    for p, a in enumerate(axis):
        i, j = (2 * p, 2 * p + 1) if c["interleaved"] else (p, p + c["rot"] // 2)
        z = torch.complex(x[..., i], x[..., j]) * turn[s["pos"][a, 0].long(), p][:, None]
        y[..., i], y[..., j] = z.real, z.imag
    return y


def _exact_e4m3(x):
    """Nearest e4m3 value of each 64-bit one, ties to the even one."""
    e = torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -300))).clamp(min=-6)
    step = torch.exp2(e - 3)
    return (torch.round(x / step) * step).clamp(-TOP, TOP)


def _exact_append(c, s):
    H, Hkv = c["H"], c["Hkv"]
    p = s["proj"]
    q, k = _exact_rotate(c, s, p[:, :H], s["qw"]), _exact_rotate(c, s, p[:, H: H + Hkv], s["kw"])
    pools = [s["k8"].double(), s["v8"].double()]
    scales = s["scales"].double()
    table = s["table"].tolist()
    begin = 0
    for b, n in enumerate(s["n"]):
        base = s["nv"][b] + s["nt"][b]
        done = 0
        while done < n:
            at = base + done
            page, r0 = table[b][at // PAGE], at % PAGE
            take = min(PAGE - r0, n - done)
            for which, x in ((0, k), (1, p[:, H + Hkv:])):
                new = x[begin + done: begin + done + take].to(torch.bfloat16).double().transpose(0, 1)
                top = new.abs().amax((1, 2)).clamp(min=1e-300)
                need = torch.exp2(torch.ceil(torch.log2(top / TOP)).clamp(min=-126))
                before = scales[page, :, which] if r0 else torch.full_like(need, LEAST)
                s_new = torch.maximum(need, before)
                if r0:
                    ratio = (before / s_new)[:, None, None]
                    pools[which][page, :, :r0] = _exact_e4m3(pools[which][page, :, :r0] * ratio)
                pools[which][page, :, r0: r0 + take] = _exact_e4m3(new / s_new[:, None, None])
                scales[page, :, which] = s_new
            done += take
        begin += n
    return {"q": q, "k": pools[0], "v": pools[1], "scales": scales, "k_out": k if c["k_out"] else None}


def _exact_rows(s, which, b, g, where):
    page = s["table"][b].long()[where // PAGE]
    rows = (s["k8"], s["v8"])[which].view(torch.uint8)[page, g, where % PAGE].view(E4M3)
    return rows.double() * s["scales"][page, g, which].double()[:, None]


def _exact_retrieve(c, s):
    vis, scores = torch.full_like(s["vis"], -1), s["scores"].double()
    G = c["H"] // c["Hkv"]
    for b in range(c["B"]):
        n = s["nv"][b]
        for g in range(c["Hkv"]):
            K = _exact_rows(s, 0, b, g, torch.arange(n, device=DEV))
            z = (s["q"][b, :, g * G: (g + 1) * G].double().reshape(-1, c["d"]) @ K.T).sum(0)
            scores[b, g, :n] = z
            order = np.argsort(-z.cpu().numpy(), kind="stable")[: s["ks"][b]]
            vis[b, g, : s["ks"][b]] = torch.as_tensor(np.sort(order).astype(np.int32)).to(DEV)
    return {"vis": vis, "scores": scores}


def _exact_attend(c, s):
    G = c["H"] // c["Hkv"]
    out = torch.zeros(c["B"], c["H"], c["d"], dtype=torch.float64, device=DEV)
    lse = torch.zeros(c["B"], c["H"], dtype=torch.float64, device=DEV)
    for b in range(c["B"]):
        nv = s["nv"][b]
        text = torch.arange(nv, nv + s["nt"][b], device=DEV)
        for g in range(c["Hkv"]):
            seen = torch.arange(nv, device=DEV) if s["vis"] is None else s["vis"][b, g, : s["ks"][b]].long()
            where = torch.cat([seen, text])
            K, V = _exact_rows(s, 0, b, g, where), _exact_rows(s, 1, b, g, where)
            z = s["q"][b, g * G: (g + 1) * G].double() @ K.T / math.sqrt(c["d"])
            norm = torch.logsumexp(z, -1)
            out[b, g * G: (g + 1) * G] = torch.softmax(z, -1) @ V
            lse[b, g * G: (g + 1) * G] = norm
    return {"out": out, "lse": lse}


def exact(case, seed):
    global own
    was, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = was
    return {"prompt": _exact_prompt, "append": _exact_append, "retrieve": _exact_retrieve, "attend": _exact_attend}[
        case["kind"]](case, s)
