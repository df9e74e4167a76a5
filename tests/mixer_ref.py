"""Plain 64-bit forms of the recurrent token mixer's calls, on the CPU, written from the formulas of
include/moe.h, each with the sum of its terms' sizes (what a rounding's error is relative to)."""
import math

import torch

EPS32 = 2.0 ** -24  # half a step of fp32


def _d(t):
    return None if t is None else t.detach().cpu().double()


def linear_attention(cfg, states, q_start, kv_len, slots, q, k, v, decay, scale):
    """(out, states, size of out's terms, size of the states' terms); out is NaN where the call leaves rows alone."""
    KH, VH, DK, DV = cfg.key_heads, cfg.value_heads, cfg.key_dim, cfg.value_dim
    G = VH // KH
    q, k = (_d(t).reshape(-1, KH, DK).repeat_interleave(G, dim=1) for t in (q, k))
    v = _d(v).reshape(-1, VH, DV)
    T = q.shape[0]
    f = torch.ones(T, VH, dtype=torch.float64)
    if decay is not None:
        f = f * torch.exp(_d(decay))
    states, out = _d(states).clone(), torch.full((T, VH, DV), math.nan, dtype=torch.float64)
    sizes, out_size = states.abs(), torch.zeros_like(out)
    for b in range(len(kv_len)):
        t0, t1 = q_start[b], q_start[b + 1]
        n = t1 - t0
        if n == 0:
            continue
        slot = slots[b]
        fresh = kv_len[b] <= n
        S = torch.zeros(VH, DK, DV, dtype=torch.float64) if fresh else states[slot].clone()
        A = S.abs()
        pad = min(max(n - kv_len[b], 0), n)
        out[t0:t0 + pad] = 0
        for t in range(t0 + pad, t1):
            S = f[t][:, None, None] * S + k[t][:, :, None] * v[t][:, None, :]
            A = f[t][:, None, None] * A + (k[t][:, :, None] * v[t][:, None, :]).abs()
            out[t] = scale * (q[t][:, None, :] @ S)[:, 0]
            out_size[t] = abs(scale) * (q[t].abs()[:, None, :] @ A)[:, 0]
        if pad < n:
            states[slot], sizes[slot] = S, A
    return out, states, out_size, sizes


def steps(n):
    """Roundings one after another that a state of n tokens has been through: token by token up to 64, chunk by chunk of 64
    beyond."""
    return min(n, 64) + n / 64


def head_norm(x, weight, gate, heads, dim, center, kind, eps, unit_offset=False):
    x = _d(x).reshape(-1, heads, dim)
    if center:
        x = x - x.mean(-1, keepdim=True)
    y = x / (x.square().mean(-1, keepdim=True) + eps).sqrt()
    if weight is not None:
        y = y * (_d(weight) + (1.0 if unit_offset else 0.0))
    if gate is not None:
        g = _d(gate).reshape(y.shape)
        y = y * torch.sigmoid(g) * (g if kind == "silu" else 1.0)
    return y.flatten(1)


def activation(z, act):
    F = torch.nn.functional
    return {"none": lambda: z, "relu": lambda: F.relu(z), "gelu": lambda: F.gelu(z), "silu": lambda: F.silu(z),
            "sigmoid": lambda: torch.sigmoid(z), "log_sigmoid": lambda: F.logsigmoid(z)}[act]()


def project(x, w, bias, resid, act, scale):
    """(y, size of z's terms)."""
    x, w, bias, resid = _d(x), _d(w), _d(bias), _d(resid)
    z, size = x @ w.T, x.abs() @ w.abs().T
    if bias is not None:
        z, size = z + bias, size + bias.abs()
    y = scale * activation(z, act)
    return (y if resid is None else resid + y), size
