"""moe_project against its 64-bit form: one row to thousands, odd sizes, both types, fp32 outputs, every activation,
strided rows, residuals that are the output.

Tolerance: one rounding to the output's type, and fp32 sums of exact products: each of the sums of K products is taken in
pieces whose additions are at most K / 16 + 64 in a row (a matrix instruction adds 16 products at once, and may cut what
it adds at 2^-22 of the largest), so (K / 4 + 256) half steps of fp32 relative to the sum of the sizes, times the
activation's slope (at most 1.13); the activation itself and the residual's addition 64 half steps of the result."""
import pytest
import torch

from sparse_moe_router_gb300 import abi

import layer_ref
import mixer_ref as ref

pytestmark = pytest.mark.gpu
BF, F16, F32 = torch.bfloat16, torch.float16, torch.float32
ACTS = ["none", "relu", "gelu", "silu", "sigmoid", "log_sigmoid"]


def _check(y, x, w, bias, resid, act, scale, what=""):
    want, size = ref.project(x, w, bias, resid, act, scale)
    K = x.shape[1]
    step, tiny = (ref.EPS32, 0.0) if y.dtype is F32 else (layer_ref.HALF_STEP[y.dtype], layer_ref.TINY[y.dtype])
    own = want.abs() + (0 if resid is None else resid.cpu().double().abs())
    bound = step * want.abs() + tiny + (1 + step) * ref.EPS32 * (abs(scale) * 1.13 * (K / 4 + 256) * size + 64 * (own + abs(scale)))
    far = (y.cpu().double() - want).abs() - bound
    assert float(far.max()) <= 0, (what, float(far.max()), want.shape)


def _make(T, K, N, dtype, out=None, seed=0, pad=0):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda *s: torch.randn(*s, device="cuda", generator=gen)  # noqa: E731
    x = r(T, K + pad).to(dtype)[:, :K]
    w = (r(N, K + pad) * K ** -0.5).to(dtype)[:, pad:]
    return x, w, r(N).to(dtype), (2 * r(T, N + pad)).to(out or dtype)[:, :N]


def _run(x, w, out=None, act="none", scale=1.0, bias=None, resid=None, y=None):
    cfg = abi.project_config(x.shape[1], w.shape[0], dtype=x.dtype, out_dtype=out, act=act, scale=scale)
    ws = abi.alloc_project_workspace(cfg, x.shape[0])
    y = torch.empty(x.shape[0], w.shape[0], dtype=out or x.dtype, device="cuda") if y is None else y
    abi.moe_project(cfg, x, w, y, ws, bias=bias, resid=resid)
    assert abi.moe_check_status(ws) == 0
    return y


@pytest.mark.parametrize("dtype", [BF, F16])
@pytest.mark.parametrize("T", [1, 2, 3, 4, 5, 7, 8, 15, 16, 17, 48, 64, 100, 128, 129, 200, 256, 257, 400, 700])
def test_rows(dtype, T):
    for K, N, pad in ((256, 136, 0), (1032, 264, 8), (8, 8, 0), (72, 1000, 16)):
        x, w, bias, resid = _make(T, K, N, dtype, seed=T, pad=pad)
        _check(_run(x, w), x, w, None, None, "none", 1.0, (T, K, N))
        _check(_run(x, w, bias=bias, resid=resid, act="silu", scale=0.5), x, w, bias, resid, "silu", 0.5, (T, K, N, "epilogue"))


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("T", [1, 3, 40, 300])
def test_activations(act, T):
    for dtype, out in ((BF, None), (F16, F32)):
        x, w, bias, resid = _make(T, 264, 200, dtype, out, seed=T)
        for b, r, scale in ((bias, None, 1.0), (None, resid, -0.75), (bias, resid, 0.0625)):
            _check(_run(4 * x, w, out, act, scale, b, r), 4 * x, w, b, r, act, scale, (act, T))


@pytest.mark.parametrize("T,K,N", [(1, 4096, 2048), (4, 2048, 4096), (48, 4096, 2048), (33, 8192, 512), (300, 2048, 2048),
                                   (1031, 1032, 1544), (2048, 512, 4096), (2500, 2048, 32), (1500, 4096, 24)])
def test_sizes_of_use(T, K, N):
    x, w, bias, resid = _make(T, K, N, BF, seed=K + N)
    _check(_run(x, w), x, w, None, None, "none", 1.0)
    out = resid.contiguous()
    keep = out.clone()
    _run(x, w, resid=out, y=out, bias=bias)  # in place
    _check(out, x, w, bias, keep, "none", 1.0)


def test_strided_outputs_leave_what_is_between_them():
    for T in (1, 4, 20, 90, 300):
        x, w, bias, _ = _make(T, 520, 72, BF, seed=T)
        wide = torch.full((T + 2, 96), 7.0, dtype=BF, device="cuda")
        y = wide[1:T + 1, 8:80]
        _run(x, w, bias=bias, y=y)
        _check(y, x, w, bias, None, "none", 1.0, T)
        wide[1:T + 1, 8:80] = 7.0
        assert bool((wide == 7.0).all()), T


def test_a_row_does_not_depend_on_others():
    """The same rows alone and among others that hold infinities and NaN, in every form that such a batch takes."""
    for T in (5, 40, 300):
        x, w, _, _ = _make(T, 512, 264, F16, seed=2)
        clean = _run(x, w)
        x2 = x.clone()
        x2[1::3] = float("nan")
        x2[2::3] = float("inf")
        y = _run(x2, w)
        assert torch.equal(y[0::3], clean[0::3]), T
        assert not bool(torch.isfinite(y[1::3]).any()), T


def test_repeats_and_streams_and_graphs_agree():
    for T in (1, 4, 30, 130, 500):
        x, w, bias, resid = _make(T, 1024, 520, BF, seed=5)
        a = _run(x, w, bias=bias, resid=resid, act="gelu")
        assert torch.equal(a, _run(x, w, bias=bias, resid=resid, act="gelu"))
        cfg = abi.project_config(1024, 520, act="gelu")
        ws = abi.alloc_project_workspace(cfg, T)
        b = torch.empty_like(a)
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        abi.moe_project(cfg, x, w, b, ws, bias=bias, resid=resid, stream=s)
        s.synchronize()
        assert torch.equal(a, b)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            abi.moe_project(cfg, x, w, b, ws, bias=bias, resid=resid)
        x.copy_(x.flip(0))
        resid.copy_(resid.flip(0))
        for _ in range(3):
            b.zero_()
            graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(a.flip(0), b), T


def test_rows_past_32_bits():
    """Rows so far apart that the last lie more than 2^32 bytes and 2^31 values behind the first."""
    T, K, N, ld = 33000, 64, 32, 66048
    x = torch.empty((T - 1) * ld + K, dtype=BF, device="cuda").as_strided((T, K), (ld, 1))
    gen = torch.Generator(device="cuda").manual_seed(1)
    x.copy_(torch.randn(T, K, device="cuda", generator=gen))
    w = torch.randn(N, K, device="cuda", generator=gen).to(BF)
    wide = torch.randn(520, K, device="cuda", generator=gen).to(BF)
    assert (T - 1) * ld > 2 ** 31
    for weights in (w, wide):
        y = _run(x, weights)
        _check(y[-300:], x[-300:], weights, None, None, "none", 1.0)
        _check(y[:300], x[:300], weights, None, None, "none", 1.0)
    _check(_run(x[-3:], wide), x[-3:], wide, None, None, "none", 1.0)
    _check(_run(x[-90:], wide), x[-90:], wide, None, None, "none", 1.0)


def test_no_rows_is_a_no_op():
    x, w, _, _ = _make(1, 64, 64, BF)
    cfg = abi.project_config(64, 64)
    abi.moe_project(cfg, x[:0], w, torch.empty(0, 64, dtype=BF, device="cuda"), abi.alloc_project_workspace(cfg, 0))


@pytest.mark.parametrize("T,K,N", [(2, 1024, 4104), (5, 1032, 8200), (16, 2048, 2056), (32, 264, 2008), (33, 2048, 256), (160, 1024, 8200),
                                   (256, 520, 4104), (192, 2048, 1032), (1100, 1032, 96), (520, 2048, 200), (900, 2048, 256), (40, 512, 65536)])
def test_either_side_of_each_choice_of_kernel(T, K, N):
    """Few rows with many and few weights, and short sides of which the long one has few and many tiles."""
    x, w, bias, resid = _make(T, K, N, F16, seed=T + N)
    _check(_run(x, w, act="gelu", bias=bias, resid=resid), x, w, bias, resid, "gelu", 1.0, (T, K, N))
