"""Plain 64-bit forms of the decoder layer's norms, cache append and attention, on the CPU, written
from the formulas of include/moe.h, and the bounds their tests use."""
import math

import torch

BF16, F16 = torch.bfloat16, torch.float16
HALF_STEP = {BF16: 2.0 ** -8, F16: 2.0 ** -11}   # a rounding's largest relative error
TINY = {BF16: 0.0, F16: 2.0 ** -25}              # and its absolute one among fp16 subnormals
MIN_EXP = -60

# the non-negative E4M3 values in code order (code 127 is NaN)
GRID = torch.tensor([m * 2.0 ** -9 for m in range(8)] +
                    [(8 + m) * 2.0 ** (e - 3) for e in range(-6, 9) for m in range(8)][:-1], dtype=torch.float64)


def decode(codes):
    """uint8 codes -> the values they stand for (NaN for the code 127)."""
    c = codes.long()
    v = torch.cat([GRID, torch.tensor([math.nan], dtype=torch.float64)])[c & 127]
    return torch.where(c >= 128, -v, v)


def encode(v):
    """Codes of the nearest values, ties to even, saturating; NaN -> 0."""
    v = torch.nan_to_num(v, nan=0.0, posinf=1e30, neginf=-1e30)
    a = v.abs().clamp(max=448.0).contiguous()
    mid = (GRID[1:] + GRID[:-1]) / 2
    i = torch.bucketize(a, mid)
    tie = (i < len(mid)) & (mid[i.clamp(max=len(mid) - 1)] == a) & (i % 2 == 1)
    i = i + tie.long()
    return (i + 128 * torch.signbit(v).long()).to(torch.uint8)


def pow2_scale(amax):
    powers = torch.tensor([2.0 ** e for e in range(MIN_EXP, 121)], dtype=torch.float64)
    amax = amax.clamp(max=3.4028234663852886e38).contiguous()
    return powers[torch.bucketize(amax, 448 * powers).clamp(max=len(powers) - 1)]


def round16(v, dtype):
    """64-bit values rounded ONCE to a 16-bit type's values, still in 64 bits (a cast of a 64-bit tensor
    may pass through 32 bits and round twice)."""
    digits, lowest = {BF16: (8, -126), F16: (11, -14)}[dtype]
    e = (torch.frexp(v)[1].long() - 1).clamp(min=lowest) - (digits - 1)
    step = ((e + 1023) << 52).view(torch.float64)
    return torch.round(v / step) * step


def block_norm(x, resid, gate, w_post, w_pre, eps, alpha, sigmoid=False, unit_offset=False):
    """(r', y, size of the terms of r', size of the terms of y) in 64 bits."""
    d = lambda t: None if t is None else t.detach().cpu().double()  # noqa: E731
    x, resid, gate, w_post, w_pre = d(x), d(resid), d(gate), d(w_post), d(w_pre)
    off = 1.0 if unit_offset else 0.0
    r = torch.zeros_like(x if x is not None else resid)
    size = torch.zeros_like(r)
    if x is not None:
        n = x
        if w_post is not None:
            n = n / (n.square().mean(-1, keepdim=True) + eps).sqrt() * (w_post + off)
        if gate is not None:
            n = n * (1 / (1 + torch.exp(-gate)) if sigmoid else gate)
        r = r + alpha * n
        size = size + (alpha * n).abs()
    if resid is not None:
        r = r + resid
        size = size + resid.abs()
    if w_pre is None:
        return r, None, size, None
    inv = 1 / (r.square().mean(-1, keepdim=True) + eps).sqrt() * (w_pre + off)
    return r, r * inv, size, size * inv.abs()


def rotate(t, angles, rot, interleaved):
    """t [n, heads, D] (64 bits) rotated by angles [n, rot] (cosines, then sines)."""
    half = rot // 2
    cos, sin = angles[:, None, :half].double(), angles[:, None, half:].double()
    out = t.clone()
    if interleaved:
        a, b = t[..., 0:rot:2], t[..., 1:rot:2]
        out[..., 0:rot:2] = a * cos - b * sin
        out[..., 1:rot:2] = b * cos + a * sin
    else:
        a, b = t[..., :half], t[..., half:rot]
        out[..., :half] = a * cos - b * sin
        out[..., half:rot] = b * cos + a * sin
    return out


def kv_append(cfg, cache, q_start, kv_len, table, q, k, v, rope):
    """cache: dict of CPU tensors k_codes, v_codes, k_scale, v_scale, changed in place; returns q_out in
    64 bits.  One token at a time is not the definition: a page's scale is settled over all of a
    call's tokens in it."""
    P, rot = cfg.page_size, cfg.rotary_dim
    q_out = torch.zeros(q.shape, dtype=torch.float64) if q is not None else None
    for b in range(len(kv_len)):
        q0, q1, kv = int(q_start[b]), int(q_start[b + 1]), int(kv_len[b])
        first = kv - (q1 - q0)
        pos = torch.arange(max(first, 0), kv)
        rows = q0 + pos - first
        rows = rows[:max(0, q1 - q0)]
        if len(pos) == 0:
            continue
        turn = (lambda t: rotate(t.double(), rope[pos], rot, bool(cfg.interleaved))) if rot else (lambda t: t.double())
        if q is not None:
            q_out[rows] = turn(q[rows])
        for name, new in (("k", turn(k[rows])), ("v", v[rows].double())):
            codes, scale = cache[name + "_codes"], cache[name + "_scale"]
            for col in range(int(pos[0]) // P, (kv - 1) // P + 1):
                page = int(table[b, col])
                here = (pos >= col * P) & (pos < (col + 1) * P)
                val = new[here]
                slots = pos[here] % P
                s = pow2_scale(torch.nan_to_num(val.abs(), nan=0.0).amax(dim=(0, 2)))
                if col * P < first:
                    old = scale[page].double()
                    s = torch.maximum(s, old)
                    grown = encode(decode(codes[page]) * (old / s)[:, None, None])
                    codes[page] = torch.where((s > old)[:, None, None], grown, codes[page])
                scale[page] = s.float()
                codes[page][:, slots] = encode(val / s[None, :, None]).transpose(0, 1)
    return q_out


def attention(cfg, cache, q_start, kv_len, table, q, scale, causal=True, window=0):
    """(out, lse, bound of out's error before its rounding, bound of lse's) in 64 bits.

    The bound counts: fp16 weights (2^-11 relative, or 2^-25 absolute when subnormal, against a
    largest weight of at least 1 in units of the largest value scale), fp32 sums on the tensor
    cores (2^-22 an addition, D/16 + n/16 of them), the exponential (2^-21)."""
    G, D, P = cfg.q_heads // cfg.kv_heads, cfg.head_dim, cfg.page_size
    T = q.shape[0]
    out = torch.zeros(T, cfg.q_heads, D, dtype=torch.float64)
    tol = torch.zeros(T, cfg.q_heads, D, dtype=torch.float64)
    lse = torch.full((T, cfg.q_heads), -math.inf, dtype=torch.float64)
    lse_tol = torch.zeros(T, cfg.q_heads, dtype=torch.float64)
    for b in range(len(kv_len)):
        q0, q1, kv = int(q_start[b]), int(q_start[b + 1]), int(kv_len[b])
        n = q1 - q0
        if n == 0 or kv == 0:
            continue
        ids = table[b, :-(-kv // P)].long()
        pos = torch.arange(kv - n, kv)[:, None]
        key = torch.arange(kv)[None]
        seen = torch.ones(n, kv, dtype=torch.bool)
        if causal:
            seen &= key <= pos
        if window:
            seen &= key > pos - window
        for h in range(cfg.q_heads):
            kh = h // G
            K, V, S = {}, {}, {}
            for name, into in (("k", K), ("v", V)):
                s = cache[name + "_scale"][ids, kh].double()
                into["x"] = (decode(cache[name + "_codes"][ids, kh]) * s[:, None, None]).reshape(-1, D)[:kv]
                S[name] = s
            qq = q[q0:q1, h].double()
            z = qq @ K["x"].T * scale
            size = (qq.abs() @ K["x"].abs().T * scale).amax(1, keepdim=True)
            z = z.masked_fill(~seen, -math.inf)
            top = z.amax(1, keepdim=True)
            p = torch.exp(z - torch.where(top > -math.inf, top, 0.0)) * seen
            total = p.sum(1, keepdim=True)
            safe = torch.where(total > 0, total, 1.0)
            o = p @ V["x"] / safe
            a = p @ V["x"].abs() / safe
            out[q0:q1, h] = o
            lse[q0:q1, h] = (top + torch.log(total))[:, 0]
            dz = size * (D / 16 + 2) * 2.0 ** -22 + 2.0 ** -21 * 8
            tol[q0:q1, h] = a * (2.0 ** -11 + 2 * dz + (kv / 16 + 8) * 2.0 ** -22) + kv * 2.0 ** -25 * 448 * S["v"].max()
            lse_tol[q0:q1, h] = (dz + 2.0 ** -20)[:, 0] + 2.0 ** -22 * lse[q0:q1, h].abs().nan_to_num(posinf=0.0)
    return out, lse, tol, lse_tol
