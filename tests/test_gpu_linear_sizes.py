"""moe_linear_attention where value channels, and what is left of their tokens, differ much in size: a channel's state
and output have their own precision, whatever the other channels of the head hold.

Tolerances are those of test_gpu_linear.py: relative to the sizes of the element's own terms.  Where decays reach the end of
fp32's exponents, beside it what a factor below its least normal value 2^-126 may lose, which counts as 0: 2^-126 of the same
terms without their decays."""
import math

import pytest
import torch

from sparse_moe_router_gb300 import abi

import layer_ref
import mixer_ref as ref
from test_gpu_linear import Case

pytestmark = pytest.mark.gpu
BF, F16 = torch.bfloat16, torch.float16


def _pieces(c, n):
    """The same run in pieces of n tokens, each from the state that the last one left."""
    out, states = torch.full((c.T, c.cfg.value_heads * c.cfg.value_dim), 7.0, dtype=c.dtype, device="cuda"), c.states.clone()
    past = c.kv[0] - c.T
    for at in range(0, c.T, n):
        p = Case(c.cfg, [min(n, c.T - at)], [past + at], dtype=c.dtype, n_slots=states.shape[0])
        p.slots, p.scale = c.slots, c.scale
        p.q, p.k, p.v, p.decay = (None if t is None else t[at:at + n] if t.dim() == 2 else t for t in (c.q, c.k, c.v, c.decay))
        p.run(states=states, out=out[at:at + n])
    return out, states


@pytest.mark.parametrize("dtype", [BF, F16])
@pytest.mark.parametrize("span", [20, 26, 32])
@pytest.mark.parametrize("rate", [0.05, 1.0])
@pytest.mark.parametrize("DK,DV", [(64, 128), (128, 64), (128, 256)])
def test_channels_far_apart_in_size(dtype, span, rate, DK, DV):
    for n, past in ((180, 5), (64, 0), (1500, 0)):
        c = Case(abi.linear_config(1, 2, DK, DV, dtype=dtype), [n], [past], seed=span, dtype=dtype, rate=(rate, rate))
        gen = torch.Generator().manual_seed(n)
        sizes = torch.cat([torch.logspace(12, 12 - span, DV, base=2)[torch.randperm(DV, generator=gen)] for _ in range(2)])
        c.v = (c.v.float() * sizes.cuda()).to(dtype)
        c.states = c.states * sizes.view(2, 1, DV).cuda()
        c.check(*c.run(), what=(n, "whole"))
        if n == 180:
            c.check(*_pieces(c, 7), what=(n, "pieces"))


@pytest.mark.parametrize("dtype", [BF, F16])
@pytest.mark.parametrize("rate", [0.5, 1.0])
def test_a_channel_whose_only_value_has_decayed(dtype, rate):
    """Channel 5's one value is the first token's: at the chunk's end it counts e^-31 or e^-63 of itself, beside channels of
    full size."""
    for n in (64, 100, 1500):
        c = Case(abi.linear_config(1, 1, 64, 128, dtype=dtype), [n], [0], seed=n, dtype=dtype)
        c.decay = torch.full((n, 1), -rate, device="cuda")
        c.v = c.v.clone()
        c.v[:, 5] = 0
        at = n - 64 if n > 100 else 0
        c.v[at, 5] = 1000.0
        out, states = c.run()
        o, s, o_size, s_size = c.want()
        _, _, o_whole, s_whole = ref.linear_attention(c.cfg, c.states, c.starts, c.kv, c.slots, c.q, c.k, c.v, None, c.scale)
        steps = 8 * ref.steps(n)
        for got, want, size, whole, room, step, tiny in (
                (out, o.flatten(1), o_size.flatten(1), o_whole.flatten(1), 640, layer_ref.HALF_STEP[dtype], layer_ref.TINY[dtype]),
                (states, s, s_size, s_whole, 192, 0.0, 0.0)):
            bound = step * want.abs() + tiny + (room + steps) * ref.EPS32 * size + 2.0 ** -126 * whole
            assert float(((got.cpu().double() - want).abs() - bound).max()) <= 0, (n, room)
        assert float(states[c.slots[0], 0, :, 5].abs().max()) > 0


@pytest.mark.parametrize("dtype", [BF, F16])
def test_one_large_value_beside_small_ones(dtype):
    """One value of 10^4 in a head of values near 10^-3 costs the other channels nothing."""
    for n, past in ((90, 3), (700, 0)):
        c = Case(abi.linear_config(2, 2, 128, 128, dtype=dtype), [n], [past], seed=n, dtype=dtype, rate=(0.02, 0.02))
        c.v = (c.v.float() * 1e-3).to(dtype)
        c.states = c.states * 1e-3
        c.v[n // 2, 7] = 1e4
        c.check(*c.run(), what=n)


@pytest.mark.parametrize("n", [150, 900])
def test_a_channel_that_is_not_finite_or_zero_beside_others_in_fp16(n):
    """What a channel holds does not show in another one, bit for bit."""
    c = Case(abi.linear_config(1, 1, 64, 128, dtype=F16), [n], [0], seed=n, dtype=F16)
    c.v = c.v.clone()
    clean, clean_states = c.run()
    c.v[n // 2, 3] = math.inf
    c.v[n // 2 + 1, 70] = math.nan
    c.v[:, 9] = 0
    c.v[:, 100] = 6e4
    out, states = c.run()
    left = [i for i in range(128) if i not in (3, 70, 9, 100)]
    assert torch.equal(out[:, left], clean[:, left])
    s, cs = states[c.slots[0], 0], clean_states[c.slots[0], 0]
    assert torch.equal(s[:, left], cs[:, left])
    assert not bool(torch.isfinite(s[:, [3, 70]]).any()) and float(s[:, 9].abs().max()) == 0 and float(out[:, 9].abs().max()) == 0
    assert bool(torch.isfinite(out[:n // 2, 3]).all()) and not bool(torch.isfinite(out[n // 2:, 3]).any())
