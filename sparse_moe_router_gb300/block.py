"""A decoder layer around the MoE layer: block norms, paged 8-bit cache, attention, experts.

    x -> norm -> qkv product -> moe_kv_append -> moe_attention -> output product
      -> norm, gate, residual, norm (moe_block_norm) -> moe_forward -> norm, residual, norm -> ...

A layer may have a recurrent mixer instead of attention, with a state a sequence instead of cached keys and values:

    norm -> moe_project (q, k, v, gate) -> moe_head_norm (q, k) -> moe_linear_attention, its log decays a second
      moe_project -> moe_head_norm with the gate -> moe_project -> norm, gate, residual, norm -> ...

One object holds a stack of layers with their caches and buffers; `prefill` runs a piece of one or more
prompts, `decode` one token a sequence.  Both run the same calls, so a prompt may come in pieces of any
size and a step may mix prompts and single tokens.  All work is asynchronous on the current stream;
`capture` records a decode step as a CUDA graph whose lengths are read from the device.

The attention layers' two projections are plain matrix products (torch.mm); everything else is a call of include/moe.h.

    python -m sparse_moe_router_gb300.block        # a small stack: a prompt in two pieces, then tokens
"""
from __future__ import annotations

import torch

from . import abi


def rope_table(positions, rotary_dim, base=1.0e6, device="cuda"):
    """fp32 [positions, rotary_dim]: cosines, then sines, from 64-bit angles."""
    half = rotary_dim // 2
    inv = base ** (-torch.arange(half, dtype=torch.float64, device=device) / half)
    angle = torch.arange(positions, dtype=torch.float64, device=device)[:, None] * inv
    return torch.cat([angle.cos(), angle.sin()], dim=1).float()


class Pages:
    """Page tables of a fixed set of sequences over one pool, the same for every layer."""

    def __init__(self, n_seqs, max_len, page_size, n_pages, device="cuda"):
        self.page_size, self.n_pages, self.max_len = page_size, n_pages, max_len
        self.max_pages = -(-max_len // page_size)
        self.lens = [0] * n_seqs
        self.pages = [[] for _ in range(n_seqs)]
        self.free = list(range(n_pages - 1, -1, -1))
        self.table = torch.zeros(n_seqs, self.max_pages, dtype=torch.int32, device=device)

    def require(self, new_tokens):
        """Raises, and takes nothing, unless every sequence has room for so many more tokens: a step that fails
        halfway would leave lengths that count tokens which were never written."""
        left = len(self.free)
        for seq, tokens in enumerate(new_tokens):
            need = -(-(self.lens[seq] + tokens) // self.page_size)
            left -= need - len(self.pages[seq])
            if self.lens[seq] + tokens > self.max_len or left < 0:
                raise RuntimeError("no page left for sequence %d at %d tokens" % (seq, self.lens[seq] + tokens))

    def grow(self, seq, tokens):
        """Room for `tokens` more of a sequence; raises when the pool is empty or max_len reached."""
        need = -(-(self.lens[seq] + tokens) // self.page_size)
        if self.lens[seq] + tokens > self.max_len or need - len(self.pages[seq]) > len(self.free):
            raise RuntimeError("no page left for sequence %d at %d tokens" % (seq, self.lens[seq] + tokens))
        new = [self.free.pop() for _ in range(need - len(self.pages[seq]))]
        if new:
            at = len(self.pages[seq])
            self.pages[seq] += new
            self.table[seq, at:need] = torch.tensor(new, dtype=torch.int32, device=self.table.device)
        self.lens[seq] += tokens

    def release(self, seq):
        self.free += reversed(self.pages[seq])
        self.pages[seq], self.lens[seq] = [], 0


def check_recurrent(H, c, layers):
    """Raises unless the recurrent layers' calls can be made with this config and these weights: a step that one of them
    refuses halfway would leave lengths that count tokens which were never written."""
    kd, vd = c.key_heads * c.key_dim, c.value_heads * c.value_dim
    if abi._TORCH_DTYPES[c.dtype] is not torch.bfloat16:
        raise ValueError("linear_cfg is for float16, the stack is bfloat16")
    if max(2 * kd, vd) > 65536:
        raise ValueError("heads of %d and %d values in all, at most 65536 can be normed" % (2 * kd, vd))
    shapes = {"w_mix": [(2 * kd + 2 * vd, H)], "w_decay": [(c.value_heads, H)], "b_decay": [(c.value_heads,)], "w_mix_out": [(H, vd)],
              "mix_norm": [(c.value_dim,), (c.value_heads, c.value_dim)]}
    for i, l in enumerate(layers):
        for name in shapes if "w_mix" in l else ():
            t = l.get(name)
            if t is None or tuple(t.shape) not in shapes[name] or t.dtype is not torch.bfloat16:
                raise ValueError("layer %d: %s is not bfloat16 of shape %s" % (i, name, " or ".join(map(str, shapes[name]))))


class DecoderLayers:
    """layers: a list of dicts with w_qkv [(QH + 2 KH) D, H], w_o [H, QH D], norm_attn, norm_attn_out,
    norm_moe, norm_moe_out [H] (a missing *_out: no norm after that block), attn_gate [H] (optional, layer by layer), and the MoE
    weights of abi.weights.  A recurrent layer (linear_cfg, an abi.LinearConfig) has w_mix [2 KH DK + 2 VH DV, H]: queries, keys,
    values and gates, w_decay [VH, H] and b_decay [VH]: log decays, w_mix_out [H, VH DV] and mix_norm [DV] or [VH, DV]
    in place of w_qkv and w_o.  All bf16 on the device."""

    def __init__(self, moe_cfg, attn_cfg, layers, pages: Pages, max_tokens, rope, eps=1e-6, residual_scale=1.0, linear_cfg=None):
        self.moe, self.attn, self.layers, self.pages, self.rope = moe_cfg, attn_cfg, layers, pages, rope
        if attn_cfg.rotary_dim and rope.shape[0] < pages.max_len:
            raise ValueError("angles for %d positions, sequences of up to %d" % (rope.shape[0], pages.max_len))
        H, dev = moe_cfg.hidden, rope.device
        self.linear = linear_cfg
        if linear_cfg is None and any("w_mix" in l for l in layers):
            raise ValueError("a recurrent layer needs linear_cfg")
        if linear_cfg is not None and linear_cfg.value_heads % 8:
            raise ValueError("the decays' product has a multiple of 8 outputs, not %d value heads" % linear_cfg.value_heads)
        if linear_cfg is not None:
            check_recurrent(H, linear_cfg, layers)
        self.caches = [None if "w_mix" in l else abi.KVCache.alloc(attn_cfg, pages.n_pages, dev) for l in layers]
        self.weights = [abi.weights(l) for l in layers]
        self.moe_ws = abi.alloc_workspace(moe_cfg, max_tokens, dev)
        self.attn_ws = abi.alloc_attn_workspace(attn_cfg, len(pages.lens), max_tokens, dev)
        self.norm_in = abi.norm_config(H, eps=eps)
        self.norm_attn = [abi.norm_config(H, gate="none" if l.get("attn_gate") is None else "channel", eps=eps,
                                          residual_scale=residual_scale) for l in layers]
        self.norm_moe = abi.norm_config(H, eps=eps, residual_scale=residual_scale)
        new = lambda *s: torch.empty(*s, dtype=torch.bfloat16, device=dev)  # noqa: E731
        QD, KD = attn_cfg.q_heads * attn_cfg.head_dim, attn_cfg.kv_heads * attn_cfg.head_dim
        self.resid, self.y, self.block = new(max_tokens, H), new(max_tokens, H), new(max_tokens, H)
        self.qkv, self.ctx = new(max_tokens, QD + 2 * KD), new(max_tokens, QD)
        self.max_tokens = max_tokens
        self.slots = torch.arange(len(pages.lens), dtype=torch.int32, device=dev)
        if linear_cfg is not None:
            c = linear_cfg
            dt = torch.bfloat16
            self.states = [abi.StatePool.alloc(c, len(pages.lens), dev) if "w_mix" in l else None for l in layers]
            self.linear_ws = abi.alloc_linear_workspace(c, len(pages.lens), max_tokens, dev)
            kd, vd = c.key_heads * c.key_dim, c.value_heads * c.value_dim
            self.mix_in = abi.project_config(H, 2 * kd + 2 * vd)
            self.mix_decay = abi.project_config(H, c.value_heads, out_dtype=torch.float32, act="log_sigmoid", scale=1 / 16)
            self.mix_out = abi.project_config(vd, H)
            self.mix_ws = abi.alloc_project_workspace(self.mix_in, max_tokens, dev)
            self.mix_qk = abi.head_norm_config(2 * c.key_heads, c.key_dim, dtype=dt, eps=eps)
            self.mix_norm = abi.head_norm_config(c.value_heads, c.value_dim, dtype=dt, gate="silu", eps=eps)
            self.mix, self.mixed = new(max_tokens, 2 * kd + 2 * vd), new(max_tokens, vd)
            self.decay = torch.empty(max_tokens, c.value_heads, dtype=torch.float32, device=dev)

    def batch(self, new_tokens):
        """The abi.KVBatch of a step with new_tokens[b] new tokens of sequence b; takes their pages, all or none."""
        if len(new_tokens) != len(self.pages.lens) or any(n < 0 for n in new_tokens):
            raise ValueError("new_tokens has to name %d counts" % len(self.pages.lens))
        starts = [0]
        for n in new_tokens:
            starts.append(starts[-1] + n)
        if starts[-1] > self.max_tokens:
            raise ValueError("%d tokens in a step of at most %d" % (starts[-1], self.max_tokens))
        self.pages.require(new_tokens)
        for b, n in enumerate(new_tokens):
            if n:
                self.pages.grow(b, n)
        dev = self.rope.device
        return self.with_states(abi.KVBatch(torch.tensor(starts, dtype=torch.int32, device=dev),
                                            torch.tensor(self.pages.lens, dtype=torch.int32, device=dev), self.pages.table, starts[-1]),
                                new_tokens)

    def with_states(self, batch, new_tokens=None):
        """The batch with what the recurrent layers read of it; a sequence's state has its own number.  Sequences without new
        tokens are left out, where new_tokens tells: a run is cut by how many sequences there are."""
        if self.linear is None:
            return batch
        q_start, kv_len, slots = batch.q_start, batch.kv_len, self.slots
        new_tokens = new_tokens or []
        live = [b for b, n in enumerate(new_tokens) if n]
        if len(live) < len(new_tokens):
            starts = [0]
            for b in live:
                starts.append(starts[-1] + new_tokens[b])
            arrays = torch.tensor(starts + [self.pages.lens[b] for b in live] + live, dtype=torch.int32, device=self.rope.device)
            q_start, kv_len, slots = arrays.split([len(live) + 1, len(live), len(live)])
        batch.states = abi.StateBatch(q_start, kv_len, slots, batch.n_tokens, longest=max(new_tokens, default=0))
        return batch

    def recurrent(self, i, batch, y, out):
        """The mixer of recurrent layer i: y [T, H] -> out [T, H]."""
        l, c, T = self.layers[i], self.linear, batch.n_tokens
        kd, vd = c.key_heads * c.key_dim, c.value_heads * c.value_dim
        mix, mixed, decay = self.mix[:T], self.mixed[:T], self.decay[:T]
        qk, q, k, v, gate = mix[:, :2 * kd], mix[:, :kd], mix[:, kd:2 * kd], mix[:, 2 * kd:2 * kd + vd], mix[:, 2 * kd + vd:]
        abi.moe_project(self.mix_in, y, l["w_mix"], mix, self.mix_ws)
        abi.moe_project(self.mix_decay, y, l["w_decay"], decay, self.mix_ws, bias=l["b_decay"])
        abi.moe_head_norm(self.mix_qk, qk, qk)
        abi.moe_linear_attention(c, self.states[i], batch.states, q, k, v, decay, mixed, self.linear_ws, scale=1 / c.key_dim)
        abi.moe_head_norm(self.mix_norm, mixed, mixed, weight=l["mix_norm"], gate=gate)
        abi.moe_project(self.mix_out, mixed, l["w_mix_out"], out, self.mix_ws)

    def run(self, x, batch):
        """x [T, H] through all layers; returns the residual stream after the last (a view of its buffer)."""
        T, c = batch.n_tokens, self.attn
        QH, KH, D = c.q_heads, c.kv_heads, c.head_dim
        resid, y, block, qkv, ctx = (t[:T] for t in (self.resid, self.y, self.block, self.qkv, self.ctx))
        heads = qkv.view(T, QH + 2 * KH, D)
        q, k, v = heads[:, :QH], heads[:, QH:QH + KH], heads[:, QH + KH:]
        resid.copy_(x)
        abi.moe_block_norm(self.norm_in, None, resid, None, y, w_pre=self.layers[0]["norm_attn"])
        for i, l in enumerate(self.layers):
            if "w_mix" in l:
                self.recurrent(i, batch, y, block)
            else:
                torch.mm(y, l["w_qkv"].T, out=qkv)
                abi.moe_kv_append(c, self.caches[i], batch, q, k, v, self.rope, q, self.attn_ws)
                abi.moe_attention(c, self.caches[i], batch, q, ctx.view(T, QH, D), self.attn_ws)
                torch.mm(ctx, l["w_o"].T, out=block)
            abi.moe_block_norm(self.norm_attn[i], block, resid, resid, y, gate=l.get("attn_gate"), w_post=l.get("norm_attn_out"),
                               w_pre=l["norm_moe"])
            abi.moe_forward(self.moe, self.weights[i], y, T, block, None, self.moe_ws)
            last = i + 1 == len(self.layers)
            abi.moe_block_norm(self.norm_moe, block, resid, resid, None if last else y, w_post=l.get("norm_moe_out"),
                               w_pre=None if last else self.layers[i + 1]["norm_attn"])
        return resid

    def check_rows(self, x, tokens):
        if tuple(x.shape) != (tokens, self.moe.hidden):  # (copying them would broadcast)
            raise ValueError("x has shape %s, not %d rows of %d" % (tuple(x.shape), tokens, self.moe.hidden))

    def prefill(self, x, new_tokens):
        """x [sum(new_tokens), H]: the sequences' new tokens one after another."""
        self.check_rows(x, sum(new_tokens))
        return self.run(x, self.batch(new_tokens))

    def decode(self, x):
        """One token for every sequence: x [sequences, H]."""
        self.check_rows(x, len(self.pages.lens))
        return self.run(x, self.batch([1] * len(self.pages.lens)))

    def check(self):
        """Raises if a kernel recorded an error (waits for the current stream)."""
        spaces = [("attention", self.attn_ws), ("moe", self.moe_ws)]
        if self.linear is not None:
            spaces += [("linear attention", self.linear_ws), ("project", self.mix_ws)]
        for name, ws in spaces:
            st = abi.moe_check_status(ws)
            if st:
                raise abi.MoeError("%s (device status)" % name, st)


class DecodeGraph:
    """A decode step of all sequences, captured once.  step(x) takes the next tokens' pages, writes their
    lengths and rows into the captured buffers and replays."""

    def __init__(self, model: DecoderLayers):
        B, H = len(model.pages.lens), model.moe.hidden
        self.model = model
        self.x = torch.zeros(B, H, dtype=torch.bfloat16, device=model.rope.device)
        self.kv_len = torch.zeros(B, dtype=torch.int32, device=model.rope.device)
        starts = torch.arange(B + 1, dtype=torch.int32, device=model.rope.device)
        self.batch = model.with_states(abi.KVBatch(starts, self.kv_len, model.pages.table, B), [1] * B)
        model.run(self.x, self.batch)  # warms up; with length 0 the tokens' position is negative: nothing is cached, no state changes
        torch.cuda.current_stream().synchronize()
        self.graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(self.graph):
            self.out = model.run(self.x, self.batch)

    def step(self, x):
        self.model.check_rows(x, len(self.model.pages.lens))
        self.model.pages.require([1] * len(self.model.pages.lens))
        for b in range(len(self.model.pages.lens)):
            self.model.pages.grow(b, 1)
        self.x.copy_(x)
        self.kv_len.copy_(torch.tensor(self.model.pages.lens, dtype=torch.int32))
        self.graph.replay()
        return self.out


def random_layers(moe_cfg, attn_cfg, n_layers, seed=0, device="cuda", linear_cfg=None, recurrent=()):
    """Random weights of a stack (a small example, or a benchmark's shapes); the layers numbered in `recurrent` have a
    recurrent mixer of linear_cfg."""
    gen = torch.Generator(device=device).manual_seed(seed)
    r = lambda *s, std=0.02: (torch.randn(*s, device=device, generator=gen) * std).to(torch.bfloat16)  # noqa: E731
    H, E, I, Is = moe_cfg.hidden, moe_cfg.n_experts, moe_cfg.inter, moe_cfg.shared_inter
    QH, KH, D = attn_cfg.q_heads, attn_cfg.kv_heads, attn_cfg.head_dim
    out = []
    for _ in range(n_layers):
        l = {"w_qkv": r((QH + 2 * KH) * D, H), "w_o": r(H, QH * D), "w_router": r(E, H, std=H ** -0.5), "b_router": None,
             "w_gate": r(E, I, H), "w_up": r(E, I, H), "w_down": r(E, H, I), "attn_gate": (1 + r(H, std=0.1))}
        if Is:
            l.update(ws_gate=r(Is, H), ws_up=r(Is, H), ws_down=r(H, Is))
        for n in ("norm_attn", "norm_attn_out", "norm_moe", "norm_moe_out"):
            l[n] = 1 + r(H, std=0.1)
        out.append(l)
    for i in recurrent:
        c, l = linear_cfg, out[i]
        kd, vd = c.key_heads * c.key_dim, c.value_heads * c.value_dim
        del l["w_qkv"], l["w_o"]
        l.update(w_mix=r(2 * kd + 2 * vd, H, std=H ** -0.5), w_decay=r(c.value_heads, H), w_mix_out=r(H, vd), mix_norm=1 + r(c.value_dim, std=0.1),
                 b_decay=torch.linspace(0, 6, c.value_heads, device=device).to(torch.bfloat16))
    return out


def main():
    moe = abi.config(hidden=256, n_experts=16, top_k=4, inter=128, shared_inter=128)
    attn = abi.attn_config(8, 2, 64, 16, rotary_dim=32)
    x = torch.randn(150, 256, device="cuda").to(torch.bfloat16)
    for recurrent in ((), (0, 1, 2)):
        linear = abi.linear_config(4, 8, 64, 64)
        layers = random_layers(moe, attn, 4 if recurrent else 2, linear_cfg=linear, recurrent=recurrent)
        model = DecoderLayers(moe, attn, layers, Pages(2, 512, 16, 80), 256, rope_table(512, 32), residual_scale=0.7, linear_cfg=linear)
        model.prefill(x, [100, 50])
        out = model.prefill(x[:60], [20, 40])
        for _ in range(8):
            out = model.decode(torch.randn(2, 256, device="cuda").to(torch.bfloat16))
        graph = DecodeGraph(model)
        for _ in range(8):
            out = graph.step(torch.randn(2, 256, device="cuda").to(torch.bfloat16))
        model.check()
        print("%d layers, %d of them recurrent: two prompts in two pieces, 16 tokens each: lengths %s, |x| %.3f" %
              (len(layers), len(recurrent), model.pages.lens, float(out.float().abs().mean())))


if __name__ == "__main__":
    main()
