"""The decoder layer that runs norms, cache append, attention and experts together
(sparse_moe_router_gb300/block.py), layer by layer against 64-bit forms, in pieces, token by token and
from a graph."""
import torch

import pytest

from sparse_moe_router_gb300 import abi, block

import layer_ref as ref

pytestmark = pytest.mark.gpu


def make(n_layers=1, max_tokens=256, seqs=2, seed=0):
    moe = abi.config(hidden=256, n_experts=16, top_k=4, inter=128, shared_inter=128)
    attn = abi.attn_config(8, 2, 64, 16, rotary_dim=32)
    layers = block.random_layers(moe, attn, n_layers, seed)
    pages = block.Pages(seqs, 512, 16, 32 * seqs + 4)
    return block.DecoderLayers(moe, attn, layers, pages, max_tokens, block.rope_table(512, 32), residual_scale=0.7)


def plain_layer(l, x, angles, moe, attn, scale):
    """One layer over one whole sequence in 64 bits, keys and values kept exactly (no cache)."""
    d = {k: v.cpu().double() for k, v in l.items() if v is not None}
    T, QH, KH, D = x.shape[0], attn.q_heads, attn.kv_heads, attn.head_dim
    unit = lambda t, w: t / (t.square().mean(-1, keepdim=True) + 1e-6).sqrt() * w  # noqa: E731
    h = (unit(x, d["norm_attn"]) @ d["w_qkv"].T).view(T, QH + 2 * KH, D)
    q, k, v = h.split([QH, KH, KH], dim=1)
    q, k = ref.rotate(q, angles, attn.rotary_dim, False), ref.rotate(k, angles, attn.rotary_dim, False)
    k, v = k.repeat_interleave(QH // KH, 1), v.repeat_interleave(QH // KH, 1)
    z = torch.einsum("qhd,khd->hqk", q, k) * D ** -0.5
    z = z.masked_fill(torch.ones(T, T).triu(1).bool(), -torch.inf)
    o = torch.einsum("hqk,khd->qhd", torch.softmax(z, -1), v).reshape(T, QH * D)
    x = x + scale * d["attn_gate"] * unit(o @ d["w_o"].T, d["norm_attn_out"])
    y = unit(x, d["norm_moe"])
    logits = y @ d["w_router"].T
    w, ids = logits.topk(moe.top_k, -1)
    w = torch.softmax(w, -1)
    silu = lambda t: t / (1 + torch.exp(-t))  # noqa: E731
    out = (silu(y @ d["ws_gate"].T) * (y @ d["ws_up"].T)) @ d["ws_down"].T
    for j in range(moe.top_k):
        g = torch.einsum("th,tih->ti", y, d["w_gate"][ids[:, j]])
        u = torch.einsum("th,tih->ti", y, d["w_up"][ids[:, j]])
        out = out + w[:, j:j + 1] * torch.einsum("ti,thi->th", silu(g) * u, d["w_down"][ids[:, j]])
    return x + scale * unit(out, d["norm_moe_out"]), ids


def test_a_layer_against_its_formula():
    """Two sequences through one layer.  The path rounds to bf16 after every step and keys and values to
    8 bits (2^-4 of each), so rows agree to a few parts in a hundred; a wrong rotation, mask, head
    group, page, gate or norm moves them by their own size.  Rows whose experts differ (a near tie of the
    router's logits) are left out; they are few."""
    m = make()
    gen = torch.Generator().manual_seed(3)
    x = torch.randn(150, 256, generator=gen).to(torch.bfloat16)
    out = m.prefill(x.cuda(), [90, 60]).cpu().double()
    m.check()
    ok = 0
    for a, b in ((0, 90), (90, 150)):
        want, _ = plain_layer(m.layers[0], x[a:b].double(), m.rope.cpu()[:b - a], m.moe, m.attn, 0.7)
        step = (want - x[a:b].double()).norm(dim=1)
        err = (out[a:b] - want).norm(dim=1) / step
        ok += int((err < 0.06).sum())
    assert ok >= 140, ok  # the others: rows routed to another expert


@pytest.mark.parametrize("pieces", [[(150, 0)], [(40, 30), (110, 1), (0, 29)], [(1, 1)] * 5 + [(145, 55)]])
def test_pieces_give_what_one_piece_gives(pieces):
    """The cache holds the same codes however a prompt is cut only while no page's scale had to grow, so
    pieces agree to the 8-bit rounding of a few pages, not bit for bit."""
    gen = torch.Generator().manual_seed(5)
    xs = [torch.randn(150, 256, generator=gen).to(torch.bfloat16).cuda(), torch.randn(60, 256, generator=gen).to(torch.bfloat16).cuda()]
    whole = make(n_layers=1)
    total = [sum(p[0] for p in pieces), sum(p[1] for p in pieces)]
    want = whole.prefill(torch.cat([xs[0][:total[0]], xs[1][:total[1]]]), total).clone()
    want = [want[:total[0]], want[total[0]:]]
    cut = make(n_layers=1)
    at = [0, 0]
    for p in pieces:
        rows = torch.cat([xs[s][at[s]:at[s] + p[s]] for s in (0, 1)])
        got = cut.prefill(rows, list(p)).clone()
        start = 0
        for s in (0, 1):
            g, w = got[start:start + p[s]].double(), want[s][at[s]:at[s] + p[s]].double()
            x = xs[s][at[s]:at[s] + p[s]].double()
            far = (g - w).norm(dim=1) > 0.06 * (w - x).norm(dim=1)
            assert int(far.sum()) <= 0.08 * p[s] + 1, (p, s, int(far.sum()))
            start += p[s]
            at[s] += p[s]
    cut.check()


def test_graph_steps_are_the_eager_steps():
    gen = torch.Generator().manual_seed(6)
    x = torch.randn(100, 256, generator=gen).to(torch.bfloat16).cuda()
    tokens = [torch.randn(2, 256, generator=gen).to(torch.bfloat16).cuda() for _ in range(20)]
    a, b = make(2), make(2)
    a.prefill(x, [70, 30])
    b.prefill(x, [70, 30])
    g = block.DecodeGraph(b)
    for t in tokens:
        u, v = a.decode(t).clone(), g.step(t).clone()
        # two tokens take the decode kernels of the MoE layer, whose atomics may round a value to its neighbour
        assert float((u.double() - v.double()).norm() / u.double().norm()) < 5e-3
    a.check()
    b.check()


def test_pages_run_out_and_come_back():
    p = block.Pages(2, 64, 16, 5)
    p.grow(0, 40)
    p.grow(1, 20)
    with pytest.raises(RuntimeError):
        p.grow(1, 20)
    with pytest.raises(RuntimeError):
        p.grow(0, 30)
    p.release(0)
    p.grow(1, 20)
    assert p.lens == [0, 40] and len(set(p.pages[1])) == 3
