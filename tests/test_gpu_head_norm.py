"""moe_head_norm against its 64-bit form: head widths that fill lanes and that do not, gates, mean taken off, weights for
all heads and for each, strided rows, aliased outputs.

Tolerance: one rounding to 16 bits (half a step) and fp32 arithmetic.  Each of the two sums has at most 32 additions a
lane and 5 levels of lanes, its error relative to the sum of sizes at most 37 half steps; square root, division and products
10; __expf (2 + 1.2 |g| ulp, |g| < 12) and the reciprocal 36; so 128 half steps of fp32 relative to the head's root
mean square times weight and gate."""
import pytest
import torch

from sparse_moe_router_gb300 import abi

import layer_ref
import mixer_ref as ref

pytestmark = pytest.mark.gpu
NOISE = 128 * ref.EPS32


def _check(got, want, size, dtype, what=""):
    bound = layer_ref.HALF_STEP[dtype] * want.abs() + layer_ref.TINY[dtype] + NOISE * size
    far = (got.cpu().double() - want).abs() - bound
    assert float(far.max()) <= 0, (what, float(far.max()))


def _make(T, heads, dim, dtype, seed, wide=0, each=False):
    gen = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=gen).to(dtype).cuda()  # noqa: E731
    rows = lambda: r(T, heads * dim + wide)[:, wide // 2:wide // 2 + heads * dim]  # noqa: E731
    return rows(), rows(), (r(heads, dim) if each else r(dim))


def _size(x, weight, gate, heads, dim, center, kind, eps, unit=False):
    """Root mean square (1) times weight and gate, the mean's share of what is left counted."""
    x = x.detach().cpu().double().reshape(-1, heads, dim)
    left = x - x.mean(-1, keepdim=True) if center else x
    rms = (left.square().mean(-1, keepdim=True) + eps).sqrt()
    s = (left.abs() + x.abs().mean(-1, keepdim=True)) / rms
    if weight is not None:
        s = s * (weight.cpu().double() + (1 if unit else 0)).abs()
    if gate is not None:
        g = gate.detach().cpu().double().reshape(s.shape)
        s = s * torch.sigmoid(g) * (g.abs() if kind == "silu" else 1)
    return s.flatten(1)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("T,heads,dim,wide,each", [
    (1, 1, 8, 0, False), (1, 32, 128, 0, False), (3, 5, 64, 16, True), (7, 2, 256, 0, True), (33, 3, 80, 16, False), (129, 7, 120, 0, True),
    (5, 2, 264, 0, False), (9, 1, 1024, 32, False), (2, 3, 520, 0, True), (257, 20, 128, 0, False), (1031, 1, 64, 0, False)])
def test_head_norm(dtype, T, heads, dim, wide, each):
    x, gate, weight = _make(T, heads, dim, dtype, T + dim, wide, each)
    for kind in ("none", "sigmoid", "silu"):
        for center in (False, True):
            cfg = abi.head_norm_config(heads, dim, dtype=dtype, center=center, gate=kind, eps=1e-5)
            y = torch.empty(T, heads, dim, dtype=dtype, device="cuda")
            g = None if kind == "none" else gate
            abi.moe_head_norm(cfg, x, y, weight=weight, gate=g)
            _check(y.flatten(1), ref.head_norm(x, weight, g, heads, dim, center, kind, 1e-5),
                   _size(x, weight, g, heads, dim, center, kind, 1e-5), dtype, (kind, center))


def test_no_weight_unit_offset_and_aliases():
    T, heads, dim, dtype = 21, 4, 128, torch.bfloat16
    x, gate, weight = _make(T, heads, dim, dtype, 3)
    y = torch.empty_like(x)
    abi.moe_head_norm(abi.head_norm_config(heads, dim), x, y)
    _check(y, ref.head_norm(x, None, None, heads, dim, False, "none", 1e-6), _size(x, None, None, heads, dim, False, "none", 1e-6), dtype)
    cfg = abi.head_norm_config(heads, dim, gate="silu", unit_offset=True)
    abi.moe_head_norm(cfg, x, y, weight=weight, gate=gate)
    _check(y, ref.head_norm(x, weight, gate, heads, dim, False, "silu", 1e-6, True),
           _size(x, weight, gate, heads, dim, False, "silu", 1e-6, True), dtype)
    x2, g2 = x.clone(), gate.clone()
    abi.moe_head_norm(cfg, x2, x2, weight=weight, gate=gate)
    abi.moe_head_norm(cfg, x, g2, weight=weight, gate=g2)
    assert torch.equal(x2, y) and torch.equal(g2, y)


def test_a_large_mean_and_odd_values_stay_in_their_head():
    T, heads, dim = 4, 3, 128
    x, gate, weight = _make(T, heads, dim, torch.float16, 9)
    x[0] += 500
    x[1, :dim] = 0
    x[2, dim + 3] = float("nan")
    gate[3, 0] = float("inf")
    cfg = abi.head_norm_config(heads, dim, dtype=torch.float16, center=True, gate="sigmoid")
    y = torch.empty_like(x)
    abi.moe_head_norm(cfg, x, y, weight=weight, gate=gate)
    want = ref.head_norm(x, weight, gate, heads, dim, True, "sigmoid", 1e-6)
    size = _size(x, weight, gate, heads, dim, True, "sigmoid", 1e-6)
    bad = want.isnan()
    assert bool(bad[2, dim:2 * dim].all()) and int(bad.sum()) == dim and torch.equal(y.cpu().isnan(), bad)
    keep = [0, 1, 3]
    _check(y[keep], want[keep], size[keep], torch.float16)
    assert float(y[1, :dim].abs().max()) == 0


def test_other_stream_graph_replay_and_no_rows():
    x, gate, weight = _make(50, 8, 64, torch.bfloat16, 1)
    cfg = abi.head_norm_config(8, 64, gate="silu")
    a, b = torch.empty_like(x), torch.empty_like(x)
    abi.moe_head_norm(cfg, x, a, weight=weight, gate=gate)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    abi.moe_head_norm(cfg, x, b, weight=weight, gate=gate, stream=s)
    s.synchronize()
    assert torch.equal(a, b)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        abi.moe_head_norm(cfg, x, b, weight=weight, gate=gate)
    x.copy_(x.flip(0))
    gate.copy_(gate.flip(0))
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(a.flip(0), b)
    abi.moe_head_norm(cfg, x[:0], b[:0], weight=weight, gate=gate[:0])


def test_rows_past_32_bits():
    T, heads, dim, ld = 33000, 2, 64, 66048
    x = torch.empty((T - 1) * ld + heads * dim, dtype=torch.bfloat16, device="cuda").as_strided((T, heads * dim), (ld, 1))
    x.copy_(torch.randn(T, heads * dim, device="cuda"))
    assert (T - 1) * ld > 2 ** 31
    cfg = abi.head_norm_config(heads, dim)
    y = torch.empty(T, heads * dim, dtype=torch.bfloat16, device="cuda")
    abi.moe_head_norm(cfg, x, y)
    z = torch.empty_like(y)
    abi.moe_head_norm(cfg, x.contiguous(), z)
    assert torch.equal(y, z)
    abi.moe_head_norm(cfg, x, x)
    assert torch.equal(x.contiguous(), z)
