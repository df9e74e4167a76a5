"""A bound for moe_attention's rows that counts only what each row sees, and the 64-bit form it goes with.

Per row, relative to a = sum_j p_j |v_j|: the weights' rounding to fp16 (2^-11), the error of the logits twice
(numerator and sum) and the fp32 sums (2^-22 an addition, n/16 on the tensor cores and some for parts).
Beside it an absolute term: fp16 weights below 2^-14 are off by up to 2^-25.  They are taken in units in
which the largest weight that the row sees, its value's scale drawn in, is at least `top`, so a
value v_j = s_j code_j adds at most 2^-25 / top * max_seen(p s) * |code_j|.  Logits: products exact, fp32 sums
(2^-22 an addition, D/16 + 2 of them), 2^-22 for the factor's rounding, and z = logit - reference
rounded in base 2 (2^-23 of both); q in fp16 is off by 2^-25 of its row's power of two at most."""
import math

import torch

import layer_ref as ref


def attention(cfg, cache, q_start, kv_len, table, q, scale, causal=True, window=0, top=1.0):
    """(out, lse, bound of out before its rounding, bound of lse), [T, q_heads, (D)] in 64 bits."""
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
        pos, key = torch.arange(kv - n, kv)[:, None], torch.arange(kv)[None]
        seen = torch.ones(n, kv, dtype=torch.bool)
        if causal:
            seen &= key <= pos
        if window:
            seen &= key > pos - window
        used = torch.nonzero(seen.any(0))[:, 0]  # keys that a row sees; no other page is looked up
        if len(used) == 0:
            continue
        k0, k1 = int(used[0]), int(used[-1]) + 1
        seen = seen[:, k0:k1]
        ids = table[b, k0 // P:-(-k1 // P)].long()
        part = slice(k0 - k0 // P * P, k1 - k0 // P * P)
        for kh in range(cfg.kv_heads):
            x = {}
            for name in "kv":
                code = ref.decode(cache[name + "_codes"][ids, kh]).reshape(-1, D)[part]
                s = cache[name + "_scale"][ids, kh].double().repeat_interleave(P)[part]
                x[name], x[name + "s"], x[name + "c"] = code * s[:, None], s, code
            qq = q[q0:q1, kh * G:(kh + 1) * G].double()  # [n, G, D]
            z = (qq @ x["k"].T * scale).masked_fill(~seen[:, None], -math.inf)
            size = (qq.abs() @ x["k"].abs().T * scale).masked_fill(~seen[:, None], 0.0).amax(2, keepdim=True)
            digits = torch.where(qq.abs().amax(2, keepdim=True) > 0, 2.0 ** (torch.frexp(qq.abs().amax(2, keepdim=True))[1] - 1).double(), 0.0)
            size_k = (x["k"].abs().sum(1) * scale).expand(n, G, -1).masked_fill(~seen[:, None], 0.0).amax(2, keepdim=True)
            high = z.amax(2, keepdim=True)
            p = torch.exp(z - torch.where(high > -math.inf, high, 0.0)).masked_fill(~seen[:, None], 0.0)
            total = p.sum(2, keepdim=True)
            p = p / torch.where(total > 0, total, 1.0)
            rows, heads = slice(q0, q1), slice(kh * G, (kh + 1) * G)
            out[rows, heads] = p @ x["v"]
            a = p @ x["v"].abs()
            lse[rows, heads] = (high + torch.log(total))[..., 0]
            far = torch.where(high > -math.inf, (z.masked_fill(~seen[:, None], 0.0)).abs().amax(2, keepdim=True), 0.0)
            dz = size * (D / 16 + 4) * 2.0 ** -22 + 2.0 ** -25 * digits * size_k + (far + 200) * 2.0 ** -22 + 2.0 ** -21
            unit = 2.0 ** -25 / top * (p * x["vs"]).amax(2, keepdim=True)
            lost = unit * (seen.double() @ x["vc"].abs())[:, None]
            tol[rows, heads] = a * (2.0 ** -11 + 2 * dz + (kv / 16 + 8) * 2.0 ** -22) + lost
            lse_tol[rows, heads] = (dz + (kv / 16 + 8) * 2.0 ** -22)[..., 0] + 2.0 ** -22 * lse[rows, heads].abs().nan_to_num(posinf=0.0)
    return out, lse, tol, lse_tol


def check(cfg, cache, q_start, kv_len, table, q, out, lse, scale=None, causal=True, window=0, rows=None, top=1.0):
    """out and lse (on any device) within the bound, rows that see nothing 0 and -infinity.  rows: only these."""
    scale = cfg.head_dim ** -0.5 if scale is None else scale
    want, wl, tol, ltol = attention(cfg, cache, q_start, kv_len, table, q.cpu(), scale, causal, window, top)
    out, lse = out.cpu(), lse.cpu()
    if rows is not None:
        want, wl, tol, ltol, out, lse = (t[rows] for t in (want, wl, tol, ltol, out, lse))
    half = ref.HALF_STEP[out.dtype]
    far = (out.double() - want).abs() - (half * want.abs() + (1 + half) * tol + ref.TINY[out.dtype])
    assert not bool(far.isnan().any()), int(far.isnan().sum())
    assert float(far.max()) <= 0, (float(far.max()), int((far > 0).sum()), float(want.abs().max()))
    empty = wl == -math.inf
    assert torch.equal(lse == -math.inf, empty) and not out[empty].any()
    if bool((~empty).any()):
        assert float(((lse.double() - wl).abs() - ltol)[~empty].max()) <= 0
