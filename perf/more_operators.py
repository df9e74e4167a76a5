"""The cases by which the recurrent token mixer of a decoder layer is measured: moe_linear_attention
(linear attention with a decay for each head over a state that each sequence keeps), moe_head_norm
(the norm of each head with its gate) and moe_project (the products around them, with bias, activation
and residual in the epilogue).

Each case is run in one of two forms: elementary torch operations in 32 or 64 bits (`own` false), or
the library's entry points (`own` true).
"""
import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


# ------------------------------------------------------------------------------- cases --

def _mix(name, **kw):
    return dict({"name": name, "op": "mix", "seqs": 1, "new": 1, "past": 1500, "ragged": False, "lens": 0, "key_heads": 16, "value_heads": 32,
                 "key_dim": 128, "value_dim": 128, "decay": "token", "dtype": "bf16"}, **kw)


def _norm(name, **kw):
    return dict({"name": name, "op": "norm", "tokens": 1, "heads": 32, "dim": 128, "gate": "silu", "center": False, "each": False, "wide": 0,
                 "dtype": "bf16"}, **kw)


def _project(name, **kw):
    return dict({"name": name, "op": "project", "tokens": 1, "inputs": 2048, "outputs": 8192, "bias": False, "act": "none", "resid": False,
                 "scale": 1.0, "dtype": "bf16", "out": "same"}, **kw)


def listed():
    return [
        # one user, one token: 16 key heads, each of two value heads; latency counts
        _mix("mix_token"),
        # a decode step of 48 conversations
        _mix("mix_decode", seqs=48),
        # four tokens at once of 8 conversations (checked drafts), narrow heads, a fixed decay for each head
        _mix("mix_draft", seqs=8, new=4, key_heads=8, value_heads=8, key_dim=64, value_dim=64, decay="head", dtype="f16"),
        # a prompt piece of the framework's largest size from an empty state
        _mix("mix_prompt", new=8192, past=0),
        # a prompt piece of one conversation beside pieces and single tokens of others, odd lengths
        _mix("mix_pieces", seqs=12, new=1031, past=3000, ragged=True, lens=2, key_heads=20, value_heads=20, key_dim=64, dtype="f16"),
        # the heads' norm and gate of one token, and of a prompt piece
        _norm("norm_token"),
        _norm("norm_prompt", tokens=8192),
        # queries, keys, values and gates of one token in one product
        _project("project_token", outputs=12288),
        # the product back into the residual stream in a decode step of 48 conversations
        _project("project_decode", tokens=48, inputs=4096, outputs=2048, resid=True),
        # the decays of a prompt piece: few outputs, in 32 bits, with a bias and a log-sigmoid
        _project("project_decays", tokens=8192, outputs=32, bias=True, act="log_sigmoid", scale=0.0625, out="f32"),
        # an odd batch through a projection with bias and activation
        _project("project_odd", tokens=1031, inputs=1032, outputs=4104, bias=True, act="gelu", dtype="f16"),
        # queries, keys, values and gates of a prompt piece
        _project("project_prompt", tokens=8192, outputs=12288),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _seconds(case):
    w = work(case)
    return max(w["bytes"] / 6.7e12, w["flops"] / 1.9e15)


_MOST = {}


def draw(rng):
    op = rng.choice(["mix", "mix", "norm", "project", "project"])
    if not _MOST:
        for c in listed():
            _MOST[c["op"]] = max(_MOST.get(c["op"], 0.0), _seconds(c))
    while True:
        dtype = rng.choice(["bf16", "bf16", "f16"])
        if op == "norm":
            heads, dim = _log(rng, 1, 64), rng.choice([64, 128, 128, 256])
            case = _norm("", tokens=_log(rng, 1, 13337), heads=heads, dim=dim, gate=rng.choice(["none", "silu", "silu", "sigmoid"]),
                         center=rng.random() < 0.3, each=rng.random() < 0.3, wide=rng.choice([0, 0, heads * dim + 72]), dtype=dtype)
        elif op == "project":
            case = _project("", tokens=_log(rng, 1, 13337), inputs=8 * _log(rng, 8, 1024), outputs=8 * _log(rng, 2, 2048),
                            bias=rng.random() < 0.4, act=rng.choice(["none", "none", "silu", "gelu", "relu", "sigmoid", "log_sigmoid"]),
                            resid=rng.random() < 0.4, scale=rng.choice([1.0, 1.0, 0.5]), dtype=dtype, out=rng.choice(["same", "same", "f32"]))
        else:
            many = rng.random() < 0.6
            key_heads = _log(rng, 1, 32)
            case = _mix("", new=_log(rng, 16, 32768) if many else _log(rng, 1, 8), seqs=_log(rng, 1, 16) if many else _log(rng, 1, 64),
                        past=rng.choice([0, _log(rng, 1, 100000)]), ragged=rng.random() < 0.6, lens=rng.randrange(1 << 20),
                        key_heads=key_heads, value_heads=key_heads * rng.choice([1, 1, 2, 4]), key_dim=rng.choice([64, 128, 128]),
                        value_dim=rng.choice([64, 128, 128, 256]), decay=rng.choice(["token", "token", "head", "none"]), dtype=dtype)
            # the plain form's chunk states have to fit
            if case["value_heads"] > 64 or case["seqs"] * (case["new"] + 64) * case["value_heads"] * (case["value_dim"] + 256) > 8e8:
                continue
        if _seconds(case) <= _MOST[op]:
            del case["name"]
            return case


def _lens(case):
    """(new, past) tokens of each sequence; the first has the case's own lengths."""
    r = random.Random(case["lens"])
    new, past = [case["new"]], [case["past"]]
    for _ in range(case["seqs"] - 1):
        new.append(_log(r, 1, case["new"]) if case["ragged"] else case["new"])
        past.append(r.choice([0, _log(r, 1, case["past"] + 1)]) if case["ragged"] else case["past"])
    return new, past


def work(case):
    if case["op"] == "norm":
        n = case["tokens"] * case["heads"] * case["dim"]
        return {"bytes": 2 * n * (2 if case["gate"] == "none" else 3), "flops": 8 * n}
    if case["op"] == "project":
        T, K, N = case["tokens"], case["inputs"], case["outputs"]
        out = 4 if case["out"] == "f32" else 2
        return {"bytes": 2 * (T * K + N * K) + out * T * N * (2 if case["resid"] else 1), "flops": 2 * T * K * N}
    new, past = _lens(case)
    T, KH, VH, DK, DV = sum(new), case["key_heads"], case["value_heads"], case["key_dim"], case["value_dim"]
    states = len(new) + sum(p > 0 for p in past)
    return {"bytes": 4 * T * (KH * DK + VH * DV) + (4 * T * VH if case["decay"] == "token" else 0) + 4 * states * VH * DK * DV,
            "flops": 4 * T * VH * DK * DV}


# ------------------------------------------------------------------------------ inputs --

def _rows(gen, shape, dtype, wide, std):
    """[T, H] values, or H columns cut out of rows of `wide` values."""
    t = torch.randn(shape[0], wide or shape[1], device="cuda", generator=gen) * std
    return t.to(dtype)[:, 8 if wide else 0:][:, :shape[1]]


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    dt = DTYPES[case["dtype"]]
    r = lambda *shape: torch.randn(*shape, device="cuda", generator=gen)  # noqa: E731
    if case["op"] == "norm":
        T, heads, dim = case["tokens"], case["heads"], case["dim"]
        weight = 1 + 0.1 * r(heads if case["each"] else 1, dim)
        return {"case": case, "x": _rows(gen, (T, heads * dim), dt, case["wide"], 0.7), "eps": 1e-6,
                "gate": None if case["gate"] == "none" else _rows(gen, (T, heads * dim), dt, case["wide"], 1.5),
                "weight": weight.to(dt).view(heads, dim) if case["each"] else weight.to(dt).view(dim)}
    if case["op"] == "project":
        T, K, N = case["tokens"], case["inputs"], case["outputs"]
        out = dt if case["out"] == "same" else torch.float32
        return {"case": case, "x": r(T, K).to(dt), "w": (r(N, K) * K ** -0.5).to(dt), "out": out,
                "bias": r(N).to(dt) if case["bias"] else None, "resid": (3 * r(T, N)).to(out) if case["resid"] else None}
    new, past = _lens(case)
    B, T, KH, VH, DK, DV = len(new), sum(new), case["key_heads"], case["value_heads"], case["key_dim"], case["value_dim"]
    # queries and keys of about unit length (a norm made them), values as a product leaves them: columns of one row
    rows = r(T, 2 * KH * DK + VH * DV)
    rows[:, :2 * KH * DK] *= DK ** -0.5
    rows = (rows * torch.exp(0.3 * r(T, 1))).to(dt)
    q, k, v = rows.split([KH * DK, KH * DK, VH * DV], dim=1)
    # log decays: some heads forget within a few tokens, some hardly in thousands
    rate = torch.exp(torch.linspace(math.log(2e-4), math.log(1.0), VH, device="cuda"))
    decay = {"token": lambda: -rate * torch.nn.functional.softplus(1.5 * r(T, VH)), "head": lambda: -rate, "none": lambda: None}[case["decay"]]()
    slots = torch.randperm(B + 2, device="cuda", generator=gen)[:B].to(torch.int32)
    starts = [0]
    for n in new:
        starts.append(starts[-1] + n)
    return {"case": case, "q": q, "k": k, "v": v, "decay": decay, "scale": 1.0, "state": 0.5 * r(B + 2, VH, DK, DV), "slots": slots,
            "new": torch.tensor(new, device="cuda"), "kv_len": torch.tensor([n + p for n, p in zip(new, past)], dtype=torch.int32, device="cuda"),
            "q_start": torch.tensor(starts, dtype=torch.int32, device="cuda"), "tokens": T, "most": max(new)}


# ----------------------------------------------------------------------- the plain form --

def _plain_norm(s):
    c = s["case"]
    x = s["x"].float().reshape(-1, c["heads"], c["dim"])
    if c["center"]:
        x = x - x.mean(dim=2, keepdim=True)
    y = x * torch.rsqrt(x.square().mean(dim=2, keepdim=True) + s["eps"]) * s["weight"].float()
    if s["gate"] is not None:
        g = s["gate"].float().reshape(y.shape)
        y = y / (1 + torch.exp(-g)) * (g if c["gate"] == "silu" else 1)
    return y.to(s["x"].dtype).flatten(1)


def _act(z, act):
    if act == "relu":
        return z.clamp(min=0)
    if act == "gelu":
        return 0.5 * z * (1 + torch.erf(z * math.sqrt(0.5)))
    if act == "sigmoid":
        return 1 / (1 + torch.exp(-z))
    if act == "silu":
        return z / (1 + torch.exp(-z))
    if act == "log_sigmoid":
        return z.clamp(max=0) - torch.log1p(torch.exp(-z.abs()))
    return z


def _plain_project(s):
    z = s["x"].float() @ s["w"].float().T
    if s["bias"] is not None:
        z = z + s["bias"].float()
    z = s["case"]["scale"] * _act(z, s["case"]["act"])
    return (z if s["resid"] is None else s["resid"].float() + z).to(s["out"])


def _plain_mix(s):
    """In chunks: what a chunk's tokens see of one another, what they see of the state at its begin, and these states
    from what every chunk adds, all chunks at once."""
    c = s["case"]
    B, T, VH, DK, DV = len(s["new"]), s["tokens"], c["value_heads"], c["key_dim"], c["value_dim"]
    C = min(64, s["most"])
    N = -(-s["most"] // C)
    seq = torch.repeat_interleave(torch.arange(B, device="cuda"), s["new"], output_size=T)
    row = torch.arange(T, device="cuda") - s["q_start"][seq]

    def chunks(t, heads, dim):  # [T, heads dim] -> [B, VH, N, C, dim], zeros behind a sequence's end
        p = torch.zeros(B, N * C, heads, dim, dtype=t.dtype, device="cuda")
        p[seq, row] = t.reshape(T, heads, dim)
        return p.view(B, N, C, heads, dim).permute(0, 3, 1, 2, 4).repeat_interleave(VH // heads, dim=1)

    q, k = (chunks(s[n].float(), c["key_heads"], DK) for n in "qk")
    v = chunks(s["v"].float(), VH, DV)
    g = torch.zeros(T, VH, dtype=torch.float64, device="cuda")
    if s["decay"] is not None:
        g = g + s["decay"]
    g = chunks(g, VH, 1)[..., 0].cumsum(dim=3)  # [B, VH, N, C]
    end = g[..., -1:]
    low = torch.ones(C, C, dtype=torch.bool, device="cuda").tril()
    apart = torch.where(low, g[..., :, None] - g[..., None, :], -math.inf)
    inside = (q @ k.transpose(3, 4) * torch.exp(apart).float()) @ v
    adds = (k * torch.exp(end - g).float()[..., None]).transpose(3, 4) @ v
    # state at the begin of chunk n: the first one, and what chunks m < n added, each decayed since
    total = end[..., 0].cumsum(dim=2)
    before = torch.cat([torch.zeros_like(total[..., :1]), total], dim=2)  # [B, VH, N + 1]
    later = torch.ones(N + 1, N, dtype=torch.bool, device="cuda").tril(-1)
    since = torch.exp(torch.where(later, before[..., :, None] - total[..., None, :], -math.inf)).float()
    first = torch.where((s["kv_len"] > s["new"])[:, None, None, None], s["state"][s["slots"].long()], 0.0)
    states = (since @ adds.flatten(3)).view(B, VH, N + 1, DK, DV) + torch.exp(before).float()[..., None, None] * first[:, :, None]
    o = s["scale"] * (inside + torch.exp(g).float()[..., None] * (q @ states[:, :, :-1]))
    s["state"][s["slots"].long()] = states[:, :, -1]
    o = o.permute(0, 2, 3, 1, 4).reshape(B, N * C, VH * DV)[seq, row]
    return [o.to(s["q"].dtype), s["state"]]


# ------------------------------------------------------------------------- the library --

def _handles(s):
    """What a program makes once for a layer, a pool of states or a batch layout and keeps."""
    from sparse_moe_router_gb300 import abi
    c = s["case"]
    if c["op"] == "norm":
        cfg = abi.head_norm_config(c["heads"], c["dim"], dtype=s["x"].dtype, center=c["center"], gate=c["gate"], eps=s["eps"])
        return abi, {"cfg": cfg, "y": torch.empty(s["x"].shape, dtype=s["x"].dtype, device="cuda")}
    if c["op"] == "project":
        cfg = abi.project_config(c["inputs"], c["outputs"], dtype=s["x"].dtype, out_dtype=s["out"], act=c["act"], scale=c["scale"])
        return abi, {"cfg": cfg, "y": torch.empty(c["tokens"], c["outputs"], dtype=s["out"], device="cuda"),
                     "ws": abi.alloc_project_workspace(cfg, c["tokens"])}
    cfg = abi.linear_config(c["key_heads"], c["value_heads"], c["key_dim"], c["value_dim"], dtype=s["q"].dtype)
    return abi, {"cfg": cfg, "pool": abi.StatePool(cfg, s["state"]), "batch": abi.StateBatch(s["q_start"], s["kv_len"], s["slots"], s["tokens"]),
                 "ws": abi.alloc_linear_workspace(cfg, len(s["new"]), s["tokens"]),
                 "out": torch.empty(s["v"].shape, dtype=s["v"].dtype, device="cuda")}


def _own(s):
    if "handles" not in s:
        s["handles"] = _handles(s)
    abi, h = s["handles"]
    op = s["case"]["op"]
    if op == "norm":
        abi.moe_head_norm(h["cfg"], s["x"], h["y"], weight=s["weight"], gate=s["gate"])
        return h["y"]
    if op == "project":
        abi.moe_project(h["cfg"], s["x"], s["w"], h["y"], h["ws"], bias=s["bias"], resid=s["resid"])
        return h["y"]
    abi.moe_linear_attention(h["cfg"], h["pool"], h["batch"], s["q"], s["k"], s["v"], s["decay"], h["out"], h["ws"], scale=s["scale"])
    return [h["out"], s["state"]]


def run(state):
    if own:
        return _own(state)
    return {"norm": _plain_norm, "project": _plain_project, "mix": _plain_mix}[state["case"]["op"]](state)


# --------------------------------------------------------------------------- 64 bits --

def _exact_norm(s):
    c = s["case"]
    out = []
    for h in range(c["heads"]):
        at = slice(h * c["dim"], (h + 1) * c["dim"])
        x = s["x"][:, at].double()
        if c["center"]:
            x = x - x.sum(dim=1, keepdim=True) / c["dim"]
        w = s["weight"][h] if c["each"] else s["weight"]
        y = x / (x.pow(2).sum(dim=1, keepdim=True) / c["dim"] + s["eps"]).sqrt() * w.double()
        if s["gate"] is not None:
            g = s["gate"][:, at].double()
            y = y * (torch.sigmoid(g) * g if c["gate"] == "silu" else torch.sigmoid(g))
        out.append(y)
    return torch.cat(out, dim=1)


def _exact_project(s):
    F = torch.nn.functional
    act = {"none": lambda z: z, "relu": F.relu, "gelu": F.gelu, "sigmoid": torch.sigmoid, "silu": F.silu, "log_sigmoid": F.logsigmoid}
    out = []
    for x0 in range(0, s["x"].shape[0], 1024):
        z = F.linear(s["x"][x0:x0 + 1024].double(), s["w"].double(), None if s["bias"] is None else s["bias"].double())
        z = act[s["case"]["act"]](z) * s["case"]["scale"]
        out.append(z if s["resid"] is None else z + s["resid"][x0:x0 + 1024].double())
    return torch.cat(out)


def _exact_mix(s):
    """Token by token: S = e^g S + k v, o = S q."""
    c = s["case"]
    new, past = _lens(c)
    VH, DK, DV = c["value_heads"], c["key_dim"], c["value_dim"]
    G = VH // c["key_heads"]
    state, o = s["state"].double(), torch.zeros(s["tokens"], VH, DV, dtype=torch.float64, device="cuda")
    q, k = (s[n].double().reshape(-1, c["key_heads"], DK).repeat_interleave(G, dim=1) for n in "qk")
    v = s["v"].double().reshape(-1, VH, DV)
    f = torch.ones(s["tokens"], VH, dtype=torch.float64, device="cuda")
    if s["decay"] is not None:
        f = f * torch.exp(s["decay"].double())
    # all sequences that still have tokens take their next one together
    order = sorted(range(len(new)), key=lambda b: -new[b])
    at = torch.tensor([s["q_start"][b].item() for b in order], device="cuda")
    S = torch.stack([state[s["slots"][b].long()] * (past[b] > 0) for b in order])
    for i in range(max(new)):
        n = sum(new[b] > i for b in order)
        t = at[:n] + i
        live = S[:n]
        live.mul_(f[t][:, :, None, None]).add_(k[t][:, :, :, None] * v[t][:, :, None, :])
        o[t] = (q[t][:, :, None, :] @ live)[:, :, 0] * s["scale"]
    for j, b in enumerate(order):
        state[s["slots"][b].long()] = S[j]
    return [o.flatten(1), state]


def exact(case, seed):
    if case["op"] == "mix" and max(_lens(case)[0]) > 40000:
        return None
    s = prepare(case, seed)
    return {"norm": _exact_norm, "project": _exact_project, "mix": _exact_mix}[case["op"]](s)
