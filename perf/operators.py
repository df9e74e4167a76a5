"""The cases by which the decoder layer's operators around the MoE layer are measured: moe_block_norm
(norms before and after a block, its gate and residual scale), moe_kv_append (position rotation and
the 8-bit paged cache) and moe_attention (attention over that cache).

Each case is run in one of two forms: elementary torch operations in 32 or 64 bits (`own` false), or
the library's entry points (`own` true).
"""
import math
import random

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16}
MIN_EXP = -60  # the smallest exponent of a cache scale
ROPE_BASE = 1.0e6


# ------------------------------------------------------------------------------- cases --

def _norm(name, **kw):
    return dict({"name": name, "op": "norm", "tokens": 1, "hidden": 2048, "dtype": "bf16", "gate": "none", "sigmoid": False,
                 "post": True, "pre": True, "wide": 0}, **kw)


def _kv(name, op, **kw):
    return dict({"name": name, "op": op, "seqs": 1, "new": 1, "kv": 1024, "ragged": False, "lens": 0, "q_heads": 16, "kv_heads": 2,
                 "head_dim": 128, "rotary": 128, "interleaved": False, "page": 64, "window": 0, "causal": True,
                 "dtype": "bf16"}, **kw)


def listed():
    return [
        # one token between attention and the MoE layer of a decode step: post norm, residual, pre norm
        _norm("norm_token"),
        # a prompt piece of the framework's largest size with a learned sigmoid gate on each element
        _norm("norm_prompt", tokens=8192, gate="element", sigmoid=True),
        # an odd batch of tokens, rows cut out of a wider tensor, a learned scale on each channel
        _norm("norm_odd", tokens=1031, hidden=4096, dtype="f16", gate="channel", wide=4096 + 136),
        # a decode step of 48 conversations: one new token each, far apart in length
        _kv("append_decode", "append", seqs=48, new=1, kv=16384, ragged=True, lens=1),
        # a prompt piece of 8192 tokens behind 1000 tokens that are in the cache (the first page is half full)
        _kv("append_prompt", "append", new=8192, kv=9192),
        # several prompts and single tokens at once; small pages, interleaved pairs, part of the head rotated
        _kv("append_mixed", "append", seqs=11, new=700, kv=5000, ragged=True, lens=2, q_heads=24, kv_heads=8, head_dim=64, rotary=32,
            interleaved=True, page=16, dtype="f16"),
        # one user, one token, a short conversation: latency counts
        _kv("attn_token", "attention", kv=1500),
        # a decode step of 48 conversations of very different length
        _kv("attn_decode", "attention", seqs=48, new=1, kv=32768, ragged=True, lens=3),
        # one token behind a very long document, more key heads
        _kv("attn_long", "attention", kv=131071, q_heads=32, kv_heads=8),
        # wide heads, four tokens that are checked at once (speculative decoding), a sliding window
        _kv("attn_draft", "attention", seqs=8, new=4, kv=9000, ragged=True, lens=4, head_dim=256, rotary=64, window=4096, page=32),
        # a prompt piece of 8192 tokens from an empty cache
        _kv("attn_prompt", "attention", new=8192, kv=8192),
        # pieces of several prompts behind what is already in the cache, odd lengths, narrow heads
        _kv("attn_pieces", "attention", seqs=5, new=1031, kv=6007, ragged=True, lens=5, q_heads=24, kv_heads=8, head_dim=64,
            rotary=64, page=16, dtype="f16"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _seconds(case):
    w = work(case)
    return max(w["bytes"] / 6.7e12, w["flops"] / 1.9e15)


_MOST = {}


def draw(rng):
    op = rng.choice(["norm", "append", "attention", "attention"])
    if not _MOST:
        for c in listed():
            _MOST[c["op"]] = max(_MOST.get(c["op"], 0.0), _seconds(c))
    while True:
        if op == "norm":
            hidden = 128 * _log(rng, 2, 64)
            case = _norm("", tokens=_log(rng, 1, 13337), hidden=hidden, dtype=rng.choice(["bf16", "bf16", "f16"]),
                         gate=rng.choice(["none", "channel", "token", "element"]), sigmoid=rng.random() < 0.5,
                         post=rng.random() < 0.7, pre=rng.random() < 0.8, wide=rng.choice([0, 0, hidden + 8, 3 * hidden]))
        else:
            dim = rng.choice([64, 128, 128, 256])
            kv_heads = rng.choice([1, 2, 4, 8])
            many = op == "attention" and rng.random() < 0.5
            new = _log(rng, 16, 8192) if many else _log(rng, 1, 8192 if op == "append" else 4)
            seqs = _log(rng, 1, 8) if new > 16 else _log(rng, 1, 64)
            case = _kv("", op, seqs=seqs, new=new, kv=new + _log(rng, 1, 131072) - 1, ragged=rng.random() < 0.6,
                       lens=rng.randrange(1 << 20), q_heads=kv_heads * rng.choice([1, 2, 3, 4, 8]), kv_heads=kv_heads, head_dim=dim,
                       rotary=rng.choice([dim, dim, dim // 2]), interleaved=rng.random() < 0.3, page=rng.choice([16, 32, 64, 64, 128]),
                       window=rng.choice([0, 0, _log(rng, 16, 8192)]), causal=rng.random() < 0.85, dtype=rng.choice(["bf16", "bf16", "f16"]))
            if op == "append":
                case.update(window=0, causal=True)
            # the plain form's padded logits, and the caches of three states, have to fit
            if seqs * case["q_heads"] * new * case["kv"] > 1.2e9 or seqs * case["kv"] * kv_heads * dim > 3e8:
                continue
        if _seconds(case) <= _MOST[op]:
            del case["name"]
            return case


def _lens(case):
    """(new tokens, cached tokens after them) of each sequence; the first has the case's own lengths."""
    r = random.Random(case["lens"])
    new, kv = [case["new"]], [case["kv"]]
    for _ in range(case["seqs"] - 1):
        n = _log(r, 1, case["new"]) if case["ragged"] else case["new"]
        new.append(n)
        kv.append(n + _log(r, 1, case["kv"] - case["new"] + 1) - 1 if case["ragged"] else case["kv"])
    return new, kv


def _pairs(case):
    """(query, key) pairs that the masks leave, over all sequences."""
    total = 0
    for n, kv in zip(*_lens(case)):
        pos = np.arange(kv - n, kv, dtype=np.int64)
        hi = pos + 1 if case["causal"] else np.full(n, kv, dtype=np.int64)
        lo = np.maximum(pos + 1 - case["window"], 0) if case["window"] else np.zeros(n, dtype=np.int64)
        total += int(np.maximum(hi - lo, 0).sum())
    return total


def _keys(case):
    """Cached tokens that at least one query sees."""
    total = 0
    for n, kv in zip(*_lens(case)):
        lo = max(kv - n + 1 - case["window"], 0) if case["window"] else 0
        total += kv - lo
    return total


def work(case):
    if case["op"] == "norm":
        rows = 1 + 1 + 1 + (1 if case["pre"] else 0) + (1 if case["gate"] == "element" else 0)
        n = case["tokens"] * case["hidden"]
        return {"bytes": 2 * n * rows + 4 * case["hidden"], "flops": 12 * n}
    new, kv = _lens(case)
    T, D, QH, KH = sum(new), case["head_dim"], case["q_heads"], case["kv_heads"]
    if case["op"] == "append":
        table = 4 * case["rotary"] * T
        return {"bytes": T * D * (4 * QH + 2 * KH * 3) + table + 8 * KH * (T // case["page"] + case["seqs"]),
                "flops": 3 * T * case["rotary"] * (QH + KH)}
    keys = _keys(case)
    return {"bytes": 4 * T * QH * D + keys * KH * (2 * D + 8.0 / case["page"]), "flops": 4 * D * QH * _pairs(case)}


# ------------------------------------------------------------------------------ inputs --

def _rows(gen, shape, dtype, wide, std):
    """[T, H] values, or H columns cut out of rows of `wide` values."""
    t = torch.randn(shape[0], wide or shape[1], device="cuda", generator=gen) * std
    return t.to(dtype)[:, 8 if wide else 0:][:, :shape[1]]


def _pow2(e):
    """2^e, exactly, in 64 bits (the power functions may be a bit off on a GPU)."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def _encode(values):
    """E4M3 values and power-of-two scales of pages [pages, heads, tokens, dim] (fp32)."""
    m, e = torch.frexp(values.abs().amax(dim=(2, 3)))
    scale = _pow2(torch.where(m > 0, e - 9 + (m > 0.875).to(e.dtype), MIN_EXP).clamp(min=MIN_EXP)).float()
    return (values / scale[:, :, None, None]).to(torch.float8_e4m3fn), scale


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    dt = DTYPES[case["dtype"]]
    if case["op"] == "norm":
        T, H, wide = case["tokens"], case["hidden"], case["wide"]
        s = {"case": case, "x": _rows(gen, (T, H), dt, wide, 0.7), "resid": _rows(gen, (T, H), dt, wide, 3.0), "gate": None,
             "w_post": None, "w_pre": None, "eps": 1e-6, "scale": 0.8}
        if case["gate"] != "none":
            shape = {"channel": (1, H), "token": (T, 1), "element": (T, H)}[case["gate"]]
            s["gate"] = _rows(gen, shape, dt, wide if case["gate"] == "element" else 0, 1.0)
        for k in ("post", "pre"):
            if case[k]:
                s["w_" + k] = (1 + 0.1 * torch.randn(H, device="cuda", generator=gen)).to(dt)
        return s
    new, kv = _lens(case)
    B, T, P, D, QH, KH = len(new), sum(new), case["page"], case["head_dim"], case["q_heads"], case["kv_heads"]
    pages = [-(-n // P) for n in kv]
    n_pages = sum(pages) + 3
    order = torch.randperm(n_pages, device="cuda", generator=gen).to(torch.int32)
    at = np.concatenate([[0], np.cumsum(pages)])
    table = torch.full((B, max(pages)), -1, dtype=torch.int32, device="cuda")
    col = torch.arange(max(pages), device="cuda")
    used = torch.tensor(pages, device="cuda")
    index = torch.tensor(at[:-1], device="cuda")[:, None] + col
    table = torch.where(col < used[:, None], order[index.clamp(max=n_pages - 1)], table)
    s = {"case": case, "new": torch.tensor(new, device="cuda"), "kv_len": torch.tensor(kv, dtype=torch.int32, device="cuda"),
         "q_start": torch.tensor(np.concatenate([[0], np.cumsum(new)]), dtype=torch.int32, device="cuda"), "table": table,
         "tokens": T, "most_new": max(new), "most_kv": max(kv)}
    # what the cache holds: the strength of a page's keys and values goes up and down along a text
    for n in ("k", "v"):
        v = torch.randn(n_pages, KH, P, D, device="cuda", generator=gen)
        v *= torch.exp(0.6 * torch.randn(n_pages, KH, 1, 1, device="cuda", generator=gen))
        s[n + "_codes"], s[n + "_scale"] = _encode(v)
    if case["op"] == "append":
        # q, k and v as one product leaves them: columns of one row
        qkv = torch.randn(T, QH + 2 * KH, D, device="cuda", generator=gen)
        qkv *= torch.exp(0.6 * torch.randn(T, 1, 1, device="cuda", generator=gen))
        s["q"], s["k"], s["v"] = qkv.to(dt).split([QH, KH, KH], dim=1)
        half = case["rotary"] // 2
        angle = torch.arange(max(kv), device="cuda", dtype=torch.float64)[:, None]
        angle = angle * ROPE_BASE ** (-torch.arange(half, device="cuda", dtype=torch.float64) / half)
        s["rope"] = torch.cat([angle.cos(), angle.sin()], dim=1).float()
    else:
        s["q"] = (1.2 * torch.randn(T, QH, D, device="cuda", generator=gen)).to(dt)
    return s


# ----------------------------------------------------------------------- the plain form --

def _unit(t, w, eps):
    t = t * torch.rsqrt(t.square().mean(dim=-1, keepdim=True) + eps)
    return t if w is None else t * w.float()


def _plain_norm(s):
    dt = s["x"].dtype
    n = s["x"].float()
    if s["w_post"] is not None:
        n = _unit(n, s["w_post"], s["eps"])
    if s["gate"] is not None:
        g = s["gate"].float()
        n = n * (1 / (1 + torch.exp(-g)) if s["case"]["sigmoid"] else g)
    r = s["resid"].float() + s["scale"] * n
    return [r.to(dt)] + ([_unit(r, s["w_pre"], s["eps"]).to(dt)] if s["w_pre"] is not None else [])


def _places(s):
    """Sequence, position, page and slot of every new token."""
    seq = torch.repeat_interleave(torch.arange(len(s["new"]), device="cuda"), s["new"], output_size=s["tokens"])
    i = torch.arange(s["tokens"], device="cuda")
    pos = i - s["q_start"][seq] + s["kv_len"][seq] - s["new"][seq]
    P = s["case"]["page"]
    return seq, pos, s["table"][seq, pos // P].long(), pos % P


def _rotate(t, pos, s):
    """The rotation in 64 bits: [T, heads, D]."""
    rot, half = s["case"]["rotary"], s["case"]["rotary"] // 2
    t = t.double()
    cos, sin = s["rope"][pos].double()[:, None].split(half, dim=2)
    if s["case"]["interleaved"]:
        a, b = t[..., 0:rot:2], t[..., 1:rot:2]
        both = torch.stack([a * cos - b * sin, b * cos + a * sin], dim=-1).flatten(-2)
    else:
        a, b = t[..., :half], t[..., half:rot]
        both = torch.cat([a * cos - b * sin, b * cos + a * sin], dim=-1)
    return torch.cat([both, t[..., rot:]], dim=-1)


def _fit(amax):
    """The smallest power of two s with amax <= 448 s."""
    m, e = torch.frexp(amax)
    e = torch.where(m > 0, e - 9 + (m > 0.875).to(e.dtype), MIN_EXP).clamp(min=MIN_EXP)
    return _pow2(e).float()


def _nearest(t):
    """The E4M3 values nearest to t, |t| <= 448, ties to even."""
    step = _pow2((torch.frexp(t)[1] - 1).clamp(min=-6) - 3)
    return (torch.round(t / step) * step).float().to(torch.float8_e4m3fn)


def _put(t, codes, scale, s):
    """Rows t [T, heads, D] (64 bits) into the pages; a page that was begun before keeps the larger scale."""
    seq, pos, page, slot = _places(s)
    P = s["case"]["page"]
    start = s["kv_len"] - s["new"]
    begun = start % P != 0
    first = s["table"].gather(1, (start // P)[:, None].long())[:, 0].long()
    most = torch.zeros(scale.shape, dtype=t.dtype, device="cuda")
    most.scatter_reduce_(0, page[:, None].expand(-1, scale.shape[1]), t.abs().amax(dim=2), "amax")
    before = scale[first]
    new = _fit(most)
    new[first] = torch.where(begun[:, None], torch.maximum(before, new[first]), new[first])
    scale[page] = new[page]
    old = codes.view(torch.uint8)[first].view(torch.float8_e4m3fn)
    ratio = torch.where(begun[:, None], before / new[first], torch.ones_like(before))
    codes.view(torch.uint8)[first] = _nearest(old.double() * ratio[:, :, None, None].double()).view(torch.uint8)
    codes.view(torch.uint8)[page, :, slot] = _nearest(t / scale[page][:, :, None].double()).view(torch.uint8)


def _plain_append(s):
    pos = _places(s)[1]
    _put(_rotate(s["k"], pos, s), s["k_codes"], s["k_scale"], s)
    _put(s["v"].double(), s["v_codes"], s["v_scale"], s)
    return [_rotate(s["q"], pos, s).to(s["q"].dtype), s["k_codes"], s["v_codes"], s["k_scale"], s["v_scale"]]


def _gathered(s, name):
    """The cached values of every sequence, padded to the longest: [B, heads, L, D]."""
    page = s["table"].clamp(min=0).long()
    v = s[name + "_codes"].view(torch.uint8)[page].view(torch.float8_e4m3fn).float() * s[name + "_scale"][page][..., None, None]
    return v.transpose(1, 2).flatten(2, 3)[:, :, :s["most_kv"]]


def _plain_attention(s):
    c = s["case"]
    B, N, KH, G, D = len(s["new"]), s["most_new"], c["kv_heads"], c["q_heads"] // c["kv_heads"], c["head_dim"]
    seq = torch.repeat_interleave(torch.arange(B, device="cuda"), s["new"], output_size=s["tokens"])
    row = torch.arange(s["tokens"], device="cuda") - s["q_start"][seq]
    q = torch.zeros(B, N, KH, G, D, device="cuda")
    q[seq, row] = s["q"].float().view(-1, KH, G, D)
    q = q.permute(0, 2, 1, 3, 4).reshape(B, KH, N * G, D)
    z = (q @ _gathered(s, "k").transpose(2, 3)) * (1 / math.sqrt(D))
    pos = (s["kv_len"] - s["new"])[:, None] + torch.arange(N, device="cuda")
    key = torch.arange(s["most_kv"], device="cuda")
    seen = (key < s["kv_len"][:, None])[:, None, :].expand(B, N, -1)
    if c["causal"]:
        seen = seen & (key <= pos[:, :, None])
    if c["window"]:
        seen = seen & (key > pos[:, :, None] - c["window"])
    seen = seen.repeat_interleave(G, dim=1)[:, None]
    z = torch.where(seen, z, -math.inf)
    top = z.amax(dim=-1, keepdim=True)
    p = torch.exp(z - torch.where(top > -math.inf, top, 0.0))
    total = p.sum(dim=-1, keepdim=True)
    o = (p @ _gathered(s, "v")) / torch.where(total > 0, total, 1.0)
    o = o.view(B, KH, N, G, D).permute(0, 2, 1, 3, 4)[seq, row]
    return o.reshape(-1, KH * G, D).to(s["q"].dtype)


# ------------------------------------------------------------------------- the library --

def _handles(s):
    """What a program makes once for a cache, a batch layout or a layer and keeps."""
    from sparse_moe_router_gb300 import abi
    c = s["case"]
    if c["op"] == "norm":
        h = {"cfg": abi.norm_config(c["hidden"], dtype=s["x"].dtype, gate=c["gate"], sigmoid=c["sigmoid"], eps=s["eps"],
                                    residual_scale=s["scale"]),
             "resid_out": torch.empty(s["x"].shape, dtype=s["x"].dtype, device="cuda")}
        h["y"] = torch.empty_like(h["resid_out"]) if s["w_pre"] is not None else None
        return abi, h
    cfg = abi.attn_config(c["q_heads"], c["kv_heads"], c["head_dim"], c["page"], rotary_dim=c["rotary"], interleaved=c["interleaved"],
                          dtype=s["q"].dtype)
    h = {"cfg": cfg, "cache": abi.KVCache(cfg, s["k_codes"].view(torch.uint8), s["v_codes"].view(torch.uint8), s["k_scale"], s["v_scale"]),
         "batch": abi.KVBatch(s["q_start"], s["kv_len"], s["table"], s["tokens"]),
         "ws": abi.alloc_attn_workspace(cfg, len(s["new"]), s["tokens"]),
         "out": torch.empty(s["q"].shape, dtype=s["q"].dtype, device="cuda")}
    return abi, h


def _own(s):
    if "handles" not in s:
        s["handles"] = _handles(s)
    abi, h = s["handles"]
    c = s["case"]
    if c["op"] == "norm":
        abi.moe_block_norm(h["cfg"], s["x"], s["resid"], h["resid_out"], h["y"], gate=s["gate"], w_post=s["w_post"], w_pre=s["w_pre"])
        return [h["resid_out"]] + ([h["y"]] if h["y"] is not None else [])
    if c["op"] == "append":
        abi.moe_kv_append(h["cfg"], h["cache"], h["batch"], s["q"], s["k"], s["v"], s["rope"], h["out"], h["ws"])
        return [h["out"], s["k_codes"], s["v_codes"], s["k_scale"], s["v_scale"]]
    abi.moe_attention(h["cfg"], h["cache"], h["batch"], s["q"], h["out"], h["ws"], causal=c["causal"], window=c["window"])
    return h["out"]


def run(state):
    if own:
        return _own(state)
    return {"norm": _plain_norm, "append": _plain_append, "attention": _plain_attention}[state["case"]["op"]](state)


# --------------------------------------------------------------------------- 64 bits --

def _exact_norm(s):
    v = {k: s[k].double() for k in ("x", "resid", "gate", "w_post", "w_pre") if s[k] is not None}
    n = v["x"]
    if "w_post" in v:
        n = n / (n.pow(2).sum(1, keepdim=True) / n.shape[1] + s["eps"]).sqrt() * v["w_post"]
    g = v.get("gate", torch.ones((), dtype=torch.float64, device="cuda"))
    r = v["resid"] + s["scale"] * (torch.sigmoid(g) if s["case"]["sigmoid"] and "gate" in v else g) * n
    out = [r]
    if "w_pre" in v:
        out.append(r / (r.pow(2).sum(1, keepdim=True) / r.shape[1] + s["eps"]).sqrt() * v["w_pre"])
    return out


#: the non-negative E4M3 values in order, and the borders between neighbours
def _grid():
    g = [m * 2.0 ** -9 for m in range(8)] + [(8 + m) * 2.0 ** (e - 3) for e in range(-6, 9) for m in range(8)][:-1]
    return torch.tensor(g, dtype=torch.float64, device="cuda")


def _on_grid(t, grid):
    """t rounded onto the grid by looking its place up; a border goes to the even neighbour."""
    a = t.abs().contiguous()
    mid = (grid[1:] + grid[:-1]) / 2
    i = torch.bucketize(a, mid)
    tie = (i < len(mid)) & (mid[i.clamp(max=len(mid) - 1)] == a) & (i % 2 == 1)
    return torch.copysign(grid[i + tie.long()], t)


def _exact_append(s):
    c = s["case"]
    P, rot, half = c["page"], c["rotary"], c["rotary"] // 2
    grid = _grid()
    codes = {n: s[n + "_codes"].double() for n in "kv"}
    scale = {n: s[n + "_scale"].double() for n in "kv"}
    turned = []
    for b, (n, kv) in enumerate(zip(*_lens(c))):
        at = int(s["q_start"][b])
        pos = torch.arange(kv - n, kv, device="cuda")
        turn = torch.complex(s["rope"][pos, :half].double(), s["rope"][pos, half:].double())[:, None]
        rows = {}
        for name in "qk":
            t = s[name][at:at + n].double()
            z = torch.complex(t[..., 0:rot:2], t[..., 1:rot:2]) if c["interleaved"] else torch.complex(t[..., :half], t[..., half:rot])
            z = z * turn
            z = torch.view_as_real(z).flatten(-2) if c["interleaved"] else torch.cat([z.real, z.imag], dim=-1)
            rows[name] = torch.cat([z, t[..., rot:]], dim=-1)
        rows["v"] = s["v"][at:at + n].double()
        turned.append(rows["q"])
        table = s["table"][b].tolist()
        for name in "kv":
            # the pages as [pages touched, heads, P, D], with what they held before
            p0, p1 = (kv - n) // P, (kv - 1) // P + 1
            ids = torch.tensor(table[p0:p1], device="cuda")
            old = torch.zeros(p1 - p0, c["kv_heads"], P, c["head_dim"], dtype=torch.float64, device="cuda")
            held = (kv - n) % P
            was = scale[name][ids[0]].clone()
            old[0, :, :held] = codes[name][ids[0], :, :held] * was[:, None, None]
            flat = old.transpose(1, 2).flatten(0, 1)
            flat[held:held + n] = rows[name]
            full = flat.view(p1 - p0, P, c["kv_heads"], -1).transpose(1, 2)
            fresh = full.clone()
            fresh[0, :, :held] = 0
            top = fresh.abs().amax(dim=(2, 3))
            powers = torch.tensor([2.0 ** e for e in range(MIN_EXP, 121)], dtype=torch.float64, device="cuda")
            new = powers[torch.bucketize(top, 448 * powers)]
            if held:
                new[0] = torch.maximum(new[0], was)
            value = _on_grid(full / new[:, :, None, None], grid)
            keep = torch.arange((p1 - p0) * P, device="cuda").view(p1 - p0, 1, P, 1) < held + n
            shrunk = codes[name][ids]
            shrunk[0] = _on_grid(shrunk[0] * (was / new[0])[:, None, None], grid) if held else shrunk[0]
            codes[name][ids] = torch.where(keep, value, shrunk)
            scale[name][ids] = new
    return [torch.cat(turned), codes["k"], codes["v"], scale["k"], scale["v"]]


def _exact_attention(s):
    c = s["case"]
    G, D, P = c["q_heads"] // c["kv_heads"], c["head_dim"], c["page"]
    out = []
    for b, (n, kv) in enumerate(zip(*_lens(c))):
        at, heads = int(s["q_start"][b]), []
        ids = s["table"][b, :-(-kv // P)].long()
        pos, key = torch.arange(kv - n, kv, device="cuda")[:, None], torch.arange(kv, device="cuda")[None]
        hidden = torch.zeros(n, kv, dtype=torch.bool, device="cuda")
        if c["causal"]:
            hidden |= key > pos
        if c["window"]:
            hidden |= pos - key >= c["window"]
        for h in range(c["q_heads"]):
            k, v = ((s[x + "_codes"].view(torch.uint8)[ids, h // G].view(torch.float8_e4m3fn).double()
                     * s[x + "_scale"][ids, h // G].double()[:, None, None]).reshape(-1, D)[:kv] for x in "kv")
            z = torch.einsum("nd,kd->nk", s["q"][at:at + n, h].double(), k) / D ** 0.5
            z.masked_fill_(hidden, -math.inf)
            heads.append(torch.nan_to_num(torch.softmax(z, dim=1)) @ v)
        out.append(torch.stack(heads, dim=1))
    return torch.cat(out)


def exact(case, seed):
    s = prepare(case, seed)
    return {"norm": _exact_norm, "append": _exact_append, "attention": _exact_attention}[case["op"]](s)
