"""Stacks whose recurrent layers could not run are refused when they are made, not by a step that has taken pages; without a GPU."""
import pytest
import torch

from sparse_moe_router_gb300 import abi, block

H, KH, VH, DK, DV = 256, 4, 8, 64, 128


def weights(**other):
    z = lambda *s: torch.zeros(*s, dtype=torch.bfloat16)  # noqa: E731
    l = dict(w_mix=z(2 * KH * DK + 2 * VH * DV, H), w_decay=z(VH, H), b_decay=z(VH), w_mix_out=z(H, VH * DV), mix_norm=z(DV))
    l.update(other)
    return l


def build(layers, cfg=None):
    moe = abi.config(hidden=H, n_experts=16, top_k=4, inter=128, shared_inter=128)
    return block.DecoderLayers(moe, abi.attn_config(8, 2, 64, 16, rotary_dim=32), layers, block.Pages(1, 64, 16, 4, device="cpu"), 16,
                               block.rope_table(64, 32, device="cpu"), linear_cfg=cfg or abi.linear_config(KH, VH, DK, DV))


def test_another_type():
    with pytest.raises(ValueError, match="float16"):
        build([], abi.linear_config(KH, VH, DK, DV, dtype=torch.float16))


@pytest.mark.parametrize("cfg", [(8, 1024, 64, 128), (1024, 1024, 64, 64), (2, 512, 64, 256)])
def test_heads_that_are_too_wide(cfg):
    with pytest.raises(ValueError, match="65536"):
        build([], abi.linear_config(*cfg))


@pytest.mark.parametrize("name,shape", [("w_mix", (2 * KH * DK + VH * DV, H)), ("w_mix", (2 * KH * DK + 2 * VH * DV, H + 8)), ("w_decay", (VH, H - 8)),
                                        ("b_decay", (VH, 1)), ("b_decay", (1,)), ("w_mix_out", (VH * DV, H)), ("mix_norm", (VH * DV,)),
                                        ("mix_norm", (1, DV))])
def test_weights_of_another_shape(name, shape):
    with pytest.raises(ValueError, match="layer 0: " + name):
        build([weights(**{name: torch.zeros(shape, dtype=torch.bfloat16)})])


def test_weights_of_another_type_or_missing():
    for name in weights():
        with pytest.raises(ValueError, match="layer 1: " + name):
            build([weights(), weights(**{name: weights()[name].float()})])
        if name != "w_mix":
            l = weights()
            del l[name]
            with pytest.raises(ValueError, match="layer 0: " + name):
                build([l])


def test_weights_that_fit():
    block.check_recurrent(H, abi.linear_config(KH, VH, DK, DV), [weights(), weights(mix_norm=torch.zeros(VH, DV, dtype=torch.bfloat16)), {}])
