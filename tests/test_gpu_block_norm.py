"""moe_block_norm against its 64-bit form: every gate, weights given or not, odd row counts and widths,
strided rows, aliased outputs, rows of zeros and of large values.

Tolerance: one rounding to 16 bits (half a step), and fp32 arithmetic: the sums of squares (at most 26
additions a thread and a tree of 10), square root, division, products and __expf (at most
2 + 1.2 |x| ulp, |x| < 12) stay below 128 * 2^-24 of the sum of the terms' sizes."""
import pytest
import torch

from sparse_moe_router_gb300 import abi

import layer_ref as ref

pytestmark = pytest.mark.gpu
NOISE = 128 * 2.0 ** -24


def _check(got, want, size, dtype, what):
    bound = ref.HALF_STEP[dtype] * want.abs() + ref.TINY[dtype] + NOISE * (1 + 2 * ref.HALF_STEP[dtype]) * size
    far = (got.cpu().double() - want).abs() - bound
    assert float(far.max()) <= 0, (what, float(far.max()))


def _make(T, H, dtype, gate, seed, wide=0):
    gen = torch.Generator().manual_seed(seed)
    r = lambda *s, std=1.0: (torch.randn(*s, generator=gen) * std).to(dtype).cuda()  # noqa: E731
    rows = lambda std: r(T, H + wide, std=std)[:, wide // 2:wide // 2 + H]  # noqa: E731
    g = {"none": None, "channel": r(H), "token": r(T, 1), "element": rows(1.0)}[gate]
    return rows(0.7), rows(3.0), g, r(H), r(H)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("T,H,gate,sigmoid,wide", [
    (1, 2048, "none", False, 0), (1, 8, "element", True, 0), (3, 264, "channel", False, 16), (7, 2048, "token", True, 0),
    (33, 1024, "element", False, 16), (2, 16384, "element", True, 0), (5, 8200, "channel", True, 0), (129, 2056, "none", False, 8 * 16),
    (1031, 4096, "token", False, 0), (4000, 128, "element", True, 0), (700, 768, "element", True, 768)])
def test_block_norm(dtype, T, H, gate, sigmoid, wide):
    x, resid, g, w_post, w_pre = _make(T, H, dtype, gate, T + H, wide)
    for post in (True, False):
        for pre in (True, False):
            cfg = abi.norm_config(H, dtype=dtype, gate=gate, sigmoid=sigmoid, eps=1e-5, residual_scale=0.75)
            out = torch.empty(T, H, dtype=dtype, device="cuda")
            y = torch.empty_like(out) if pre else None
            abi.moe_block_norm(cfg, x, resid, out, y, gate=g, w_post=w_post if post else None, w_pre=w_pre if pre else None)
            r, n, rs, ns = ref.block_norm(x, resid, g, w_post if post else None, w_pre if pre else None, 1e-5, 0.75, sigmoid)
            _check(out, r, rs, dtype, "resid_out")
            if pre:
                _check(y, n, ns, dtype, "y")


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_parts_left_out_and_unit_offset(dtype):
    T, H = 19, 512
    x, resid, _, w_post, w_pre = _make(T, H, dtype, "none", 5)
    cfg = abi.norm_config(H, dtype=dtype, unit_offset=True, eps=1e-6)
    y = torch.empty(T, H, dtype=dtype, device="cuda")
    abi.moe_block_norm(cfg, None, resid, None, y, w_pre=w_pre)                  # the norm before the first block
    _, n, _, ns = ref.block_norm(None, resid, None, None, w_pre, 1e-6, 1.0, unit_offset=True)
    _check(y, n, ns, dtype, "no block")
    out = torch.empty_like(y)
    abi.moe_block_norm(cfg, x, None, out, y, w_post=w_post, w_pre=w_pre)         # no residual
    r, n, rs, ns = ref.block_norm(x, None, None, w_post, w_pre, 1e-6, 1.0, unit_offset=True)
    _check(out, r, rs, dtype, "no residual")
    _check(y, n, ns, dtype, "no residual, y")
    abi.moe_block_norm(cfg, x, resid, None, y, w_post=w_post, w_pre=w_pre)       # only y
    _, n, _, ns = ref.block_norm(x, resid, None, w_post, w_pre, 1e-6, 1.0, unit_offset=True)
    _check(y, n, ns, dtype, "only y")


def test_outputs_may_be_the_inputs():
    T, H = 37, 1024
    x, resid, g, w_post, w_pre = _make(T, H, torch.bfloat16, "element", 8)
    cfg = abi.norm_config(H, gate="element", sigmoid=True)
    a, b = torch.empty_like(x), torch.empty_like(x)
    abi.moe_block_norm(cfg, x, resid, a, b, gate=g, w_post=w_post, w_pre=w_pre)
    x2, r2 = x.clone(), resid.clone()
    abi.moe_block_norm(cfg, x2, r2, r2, x2, gate=g, w_post=w_post, w_pre=w_pre)
    assert torch.equal(r2, a) and torch.equal(x2, b)


def test_rows_of_zeros_large_values_and_nan_stay_in_their_row():
    T, H = 6, 256
    x, resid, _, w_post, w_pre = _make(T, H, torch.bfloat16, "none", 11)
    x[0] = 0
    resid[0] = 0
    x[1] = 1e18
    x[2, 5] = float("nan")
    x[3, 7] = float("inf")
    cfg = abi.norm_config(H, eps=1e-6)
    out, y = torch.empty_like(x), torch.empty_like(x)
    abi.moe_block_norm(cfg, x, resid, out, y, w_post=w_post, w_pre=w_pre)
    assert torch.equal(out[0], torch.zeros_like(out[0])) and torch.equal(y[0], torch.zeros_like(y[0]))
    keep = [0, 1, 4, 5]
    r, n, rs, ns = ref.block_norm(x[keep], resid[keep], None, w_post, w_pre, 1e-6, 1.0)
    _check(out[keep], r, rs, torch.bfloat16, "out")
    _check(y[keep], n, ns, torch.bfloat16, "y")
    assert bool(y[2].isnan().all()) and not bool(y[keep].isnan().any())


def test_other_stream_and_graph_replay():
    T, H = 50, 2048
    x, resid, _, w_post, w_pre = _make(T, H, torch.bfloat16, "none", 3)
    cfg = abi.norm_config(H)
    a, b, c, d = (torch.empty_like(x) for _ in range(4))
    abi.moe_block_norm(cfg, x, resid, a, b, w_post=w_post, w_pre=w_pre)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    abi.moe_block_norm(cfg, x, resid, c, d, w_post=w_post, w_pre=w_pre, stream=s)
    s.synchronize()
    assert torch.equal(a, c) and torch.equal(b, d)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        abi.moe_block_norm(cfg, x, resid, c, d, w_post=w_post, w_pre=w_pre)
    x.copy_(x.flip(0))
    resid.copy_(resid.flip(0))
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(a.flip(0), c) and torch.equal(b.flip(0), d)


def test_no_rows_is_a_no_op():
    cfg = abi.norm_config(256)
    e = torch.empty(0, 256, dtype=torch.bfloat16, device="cuda")
    w = torch.ones(256, dtype=torch.bfloat16, device="cuda")
    abi.moe_block_norm(cfg, e, e, e, e, w_post=w, w_pre=w)
