"""Recurrent layers of the decoder stack (sparse_moe_router_gb300/block.py): products, head norms, linear attention and the
experts together, against their formula in 64 bits, in pieces, token by token, beside attention layers, from a graph."""
import pytest
import torch

from sparse_moe_router_gb300 import abi, block

pytestmark = pytest.mark.gpu
LINEAR = (4, 8, 64, 128)


def make(recurrent=(0,), n_layers=1, max_tokens=400, seqs=2, seed=0):
    moe = abi.config(hidden=256, n_experts=16, top_k=4, inter=128, shared_inter=128)
    attn = abi.attn_config(8, 2, 64, 16, rotary_dim=32)
    linear = abi.linear_config(*LINEAR)
    layers = block.random_layers(moe, attn, n_layers, seed, linear_cfg=linear, recurrent=recurrent)
    return block.DecoderLayers(moe, attn, layers, block.Pages(seqs, 512, 16, 32 * seqs + 4), max_tokens, block.rope_table(512, 32),
                               residual_scale=0.7, linear_cfg=linear)


def rows(n, seed=1):
    return torch.randn(n, 256, generator=torch.Generator().manual_seed(seed)).to(torch.bfloat16).cuda()


def plain_layer(l, x, moe, scale):
    """One recurrent layer over one whole sequence in 64 bits."""
    d = {k: v.cpu().double() for k, v in l.items() if v is not None}
    KH, VH, DK, DV = LINEAR
    T, kd, vd = x.shape[0], KH * DK, VH * DV
    unit = lambda t, w=1.0: t / (t.square().mean(-1, keepdim=True) + 1e-6).sqrt() * w  # noqa: E731
    silu = lambda t: t / (1 + torch.exp(-t))  # noqa: E731
    y = unit(x, d["norm_attn"])
    q, k, v, gate = (y @ d["w_mix"].T).split([kd, kd, vd, vd], dim=1)
    q, k = (unit(t.view(T, KH, DK)).repeat_interleave(VH // KH, 1) for t in (q, k))
    v, gate = v.view(T, VH, DV), gate.view(T, VH, DV)
    f = torch.exp(torch.nn.functional.logsigmoid(y @ d["w_decay"].T + d["b_decay"]) / 16)
    S, o = torch.zeros(VH, DK, DV, dtype=torch.float64), []
    for t in range(T):
        S = f[t][:, None, None] * S + k[t][:, :, None] * v[t][:, None, :]
        o.append((q[t][:, None, :] @ S)[:, 0] / DK)
    o = (unit(torch.stack(o), d["mix_norm"]) * silu(gate)).flatten(1)
    x = x + scale * d["attn_gate"] * unit(o @ d["w_mix_out"].T, d["norm_attn_out"])
    y = unit(x, d["norm_moe"])
    w, ids = (y @ d["w_router"].T).topk(moe.top_k, -1)
    w = torch.softmax(w, -1)
    out = (silu(y @ d["ws_gate"].T) * (y @ d["ws_up"].T)) @ d["ws_down"].T
    for j in range(moe.top_k):
        g = torch.einsum("th,tih->ti", y, d["w_gate"][ids[:, j]])
        u = torch.einsum("th,tih->ti", y, d["w_up"][ids[:, j]])
        out = out + w[:, j:j + 1] * torch.einsum("ti,thi->th", silu(g) * u, d["w_down"][ids[:, j]])
    return x + scale * unit(out, d["norm_moe_out"])


@pytest.mark.parametrize("lens", [(150, 90), (300, 1)])
def test_a_layer_against_its_formula(lens):
    """The path rounds to bf16 after every step, ten times on the way (2^-8 of a value at most, a third of that on the
    average), and norms, products and sums pass such errors on: rows agree to a few parts in a hundred; a wrong decay, head,
    chunk, norm or gate moves them by their own size.  Rows whose experts differ (a near tie of the router's logits) are left
    out; they are few."""
    m = make()
    x = rows(sum(lens), 3)
    out = m.prefill(x, list(lens)).cpu().double()
    m.check()
    ok, a = 0, 0
    for n in lens:
        x64 = x[a:a + n].cpu().double()
        want = plain_layer(m.layers[0], x64, m.moe, 0.7)
        err = (out[a:a + n] - want).norm(dim=1) / (want - x64).norm(dim=1)
        ok += int((err < 0.04).sum())
        a += n
    assert ok >= 0.93 * sum(lens), ok


@pytest.mark.parametrize("pieces", [[(150, 0)], [(40, 30), (110, 1), (0, 29)], [(1, 1)] * 5 + [(145, 55)], [(100, 4), (4, 100), (1, 1)]])
def test_pieces_give_what_one_piece_gives(pieces):
    """States are fp32, so a prompt in pieces differs from the whole by roundings to bf16 that fall another way: the path's
    own size of error, and a few rows that go to another expert."""
    total = [sum(p[0] for p in pieces), sum(p[1] for p in pieces)]
    xs = [rows(max(total[0], 1), 5)[:total[0]], rows(max(total[1], 1), 6)[:total[1]]]
    whole, cut = make(), make()
    want = whole.prefill(torch.cat(xs), total).clone()
    want = [want[:total[0]], want[total[0]:]]
    at = [0, 0]
    for p in pieces:
        got = cut.prefill(torch.cat([xs[s][at[s]:at[s] + p[s]] for s in (0, 1)]), list(p)).clone()
        start = 0
        for s in (0, 1):
            g, w = got[start:start + p[s]].double(), want[s][at[s]:at[s] + p[s]].double()
            far = (g - w).norm(dim=1) > 0.02 * (w - xs[s][at[s]:at[s] + p[s]].double()).norm(dim=1)
            assert int(far.sum()) <= 0.06 * p[s] + 1, (p, s, int(far.sum()))
            start += p[s]
            at[s] += p[s]
    cut.check()
    a, b = whole.states[0].states.double(), cut.states[0].states.double()
    # (keys and values of one token pass through another kernel's sums, and may be rounded to a neighbour: 2^-8 of a term)
    assert float((a - b).norm() / a.norm()) < 2.0 ** -8


def test_graph_steps_are_the_eager_steps_of_a_mixed_stack():
    x = rows(100, 6)
    a, b = (make(recurrent=(0, 2), n_layers=3) for _ in range(2))
    assert a.caches[0] is None and a.states[1] is None
    for m in (a, b):
        m.prefill(x, [70, 30])
    g = block.DecodeGraph(b)
    assert torch.equal(a.states[0].states, b.states[0].states)  # the capture's own run changes nothing
    for i in range(12):
        t = rows(2, 20 + i)
        u, v = a.decode(t).clone(), g.step(t).clone()
        assert float((u.double() - v.double()).norm() / u.double().norm()) < 5e-3
    a.check()
    b.check()


def test_a_released_sequence_begins_anew():
    """Its slot still holds the old state, which a prompt from position 0 does not see; the other sequence goes on."""
    a, b = make(), make()
    x, z = rows(80, 2), rows(60, 9)
    a.prefill(x, [50, 30])
    a.pages.release(0)
    got = a.prefill(z, [60, 0]).clone()
    assert torch.equal(got, b.prefill(z, [60, 0]))
    assert torch.equal(a.states[0].states[0], b.states[0].states[0])


def test_configs_that_do_not_fit():
    moe = abi.config(hidden=256, n_experts=16, top_k=4, inter=128, shared_inter=128)
    with pytest.raises(ValueError, match="linear_cfg"):
        block.DecoderLayers(moe, abi.attn_config(8, 2, 64, 16, rotary_dim=32), [{"w_mix": None}], block.Pages(1, 64, 16, 4), 16,
                            block.rope_table(64, 32))
    with pytest.raises(ValueError, match="multiple of 8"):
        block.DecoderLayers(moe, abi.attn_config(8, 2, 64, 16, rotary_dim=32), [], block.Pages(1, 64, 16, 4), 16,
                            block.rope_table(64, 32), linear_cfg=abi.linear_config(2, 4, 64, 64))
