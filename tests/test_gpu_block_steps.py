"""Steps of the decoder stack (sparse_moe_router_gb300/block.py) after one that was refused, and stacks whose
layers differ."""
import pytest
import torch

from sparse_moe_router_gb300 import abi, block

pytestmark = pytest.mark.gpu


def make(n_layers=1, max_tokens=128, seqs=2, n_pages=12, seed=0, layers=None):
    moe = abi.config(hidden=256, n_experts=16, top_k=4, inter=128, shared_inter=128)
    attn = abi.attn_config(8, 2, 64, 16, rotary_dim=32)
    layers = block.random_layers(moe, attn, n_layers, seed) if layers is None else layers
    return block.DecoderLayers(moe, attn, layers, block.Pages(seqs, 512, 16, n_pages), max_tokens, block.rope_table(512, 32),
                               residual_scale=0.7)


def rows(n, seed=1):
    return torch.randn(n, 256, generator=torch.Generator().manual_seed(seed)).to(torch.bfloat16).cuda()


def test_a_step_after_a_refused_one():
    """Prompts, a step that finds the pool too small only at its second sequence, then another: the same as
    without the refused one, bit for bit."""
    a, b = make(), make()
    for m in (a, b):
        m.prefill(rows(100), [60, 40])
    with pytest.raises(RuntimeError):
        a.prefill(rows(120, 2), [20, 100])
    with pytest.raises(ValueError):
        a.prefill(rows(129, 2), [9, 120])
    x = rows(30, 3)
    assert torch.equal(a.prefill(x, [20, 10]), b.prefill(x, [20, 10]))
    assert a.pages.lens == b.pages.lens == [80, 50]
    a.check()


@pytest.mark.parametrize("without", [0, 1, 2])
@pytest.mark.parametrize("none", [False, True])
def test_gates_on_some_layers(without, none):
    """A layer without an attention gate (left out, or None) among gated ones is a layer with a gate of ones."""
    moe = abi.config(hidden=256, n_experts=16, top_k=4, inter=128, shared_inter=128)
    layers = block.random_layers(moe, abi.attn_config(8, 2, 64, 16, rotary_dim=32), 3)
    ones = [dict(l) for l in layers]
    ones[without]["attn_gate"] = torch.ones_like(layers[without]["attn_gate"])
    if none:
        layers[without]["attn_gate"] = None
    else:
        del layers[without]["attn_gate"]
    a, b = make(layers=layers), make(layers=ones)
    x = rows(100)
    assert torch.equal(a.prefill(x, [60, 40]), b.prefill(x, [60, 40]))
    a.check()
