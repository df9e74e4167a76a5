"""moe_attention over pages whose scales lie far apart: a row's result depends on the pages that it sees
only, and on each page's exact codes (bounds: attention_bound)."""
import pytest
import torch

import attention_bound
from test_gpu_attention import make_q
from test_gpu_attention_windows import run
from test_gpu_kv_append import Setup

pytestmark = pytest.mark.gpu

HEADS = [(8, 1, 64, 16), (8, 2, 128, 64), (16, 2, 256, 32)]


def check(s, q, out, lse, **kw):
    attention_bound.check(s.cfg, s.cache, s.q_start, s.kv_len, s.table, q, out, lse, **kw)


def steps(s, name, exponent):
    """Page column j of every sequence gets the scale 2^exponent(j)."""
    for b in range(s.table.shape[0]):
        for j in range(s.table.shape[1]):
            if int(s.table[b, j]) >= 0:
                s.cache[name + "_scale"][int(s.table[b, j])] = 2.0 ** exponent(j)


LENS = [[(1, 1280), (5, 640)], [(640, 640)], [(700, 1280), (300, 320)], [(140, 9000)]]


@pytest.mark.parametrize("QH,KH,D,P", HEADS)
@pytest.mark.parametrize("lens", LENS, ids=["short", "one", "two", "parts"])
@pytest.mark.parametrize("step", [-1, 1, 3])
def test_value_scales_that_rise_or_fall(QH, KH, D, P, lens, step):
    """Each 64 positions have a value scale of 2^step times the one before: an early causal row sees only small ones."""
    s = Setup(lens, QH, KH, D, P, seed=D)
    steps(s, "v", lambda j: max(min(step * (j * P // 64) - 20, 20), -55))
    q = make_q(s)
    out, lse = run(s, q)
    check(s, q, out, lse)


@pytest.mark.parametrize("QH,KH,D,P", HEADS)
@pytest.mark.parametrize("lens", LENS, ids=["short", "one", "two", "parts"])
@pytest.mark.parametrize("last", [0, 9])
def test_key_scales_that_rise(QH, KH, D, P, lens, last):
    """Key scales of 2^-50 that rise to 2^last: early rows have nearly flat weights, late ones sharp ones."""
    s = Setup(lens, QH, KH, D, P, seed=D)
    for b, kv in enumerate(s.kv_len.tolist()):
        for j in range(-(-kv // P)):
            s.cache["k_scale"][int(s.table[b, j])] = 2.0 ** max(last - 8 - 3 * ((kv - 1) // P - j) * P // 64, -50)
    q = make_q(s)
    out, lse = run(s, q)
    check(s, q, out, lse)


@pytest.mark.parametrize("QH,KH,D,P", HEADS)
@pytest.mark.parametrize("window", [0, 90])
def test_a_page_under_the_largest_scale_that_a_row_does_not_see(QH, KH, D, P, window):
    """The last page (and, where a window hides it from most rows, the first) is stored under 2^120, as an
    infinity is: rows that do not see it are not touched by it."""
    s = Setup([(640, 640)], QH, KH, D, P, seed=D)
    q = make_q(s)
    for name in "kv":
        s.cache[name + "_scale"][int(s.table[0, 639 // P])] = 2.0 ** 120
        if window:
            s.cache[name + "_scale"][int(s.table[0, 0])] = 2.0 ** 120
    out, lse = run(s, q, window=window)
    pos = torch.arange(640)
    rows = pos < 639 // P * P
    if window:
        rows &= pos - window >= P - 1
    check(s, q, out, lse, window=window, rows=rows)


@pytest.mark.parametrize("QH,KH,D,P", HEADS)
@pytest.mark.parametrize("lens", LENS, ids=["short", "one", "two", "parts"])
@pytest.mark.parametrize("most", [7, 8, 9, 14, 15, 16, 30])
def test_pages_of_mixed_scales(QH, KH, D, P, lens, most):
    """Pages whose scales lie up to 2^most apart in any order, one all of zeros (the smallest scale) with the widest."""
    s = Setup(lens, QH, KH, D, P, seed=D + most)
    gen = torch.Generator().manual_seed(most)
    for name in "kv":
        e = torch.randint(-most, 1, s.cache[name + "_scale"].shape, generator=gen)
        s.cache[name + "_scale"][:] = 2.0 ** (e - 7).double()
    if most == 30:
        zero = [int(s.table[0, 1]), int(s.table[0, 5])]
        for name in "kv":
            s.cache[name + "_codes"][zero], s.cache[name + "_scale"][zero] = 0, 2.0 ** -60
    q = make_q(s)
    out, lse = run(s, q)
    check(s, q, out, lse)


@pytest.mark.parametrize("QH,KH,D,P", HEADS)
@pytest.mark.parametrize("lens", [[(640, 700)], [(3, 640), (1, 400)]], ids=["prompt", "tokens"])
@pytest.mark.parametrize("size", [1e-30, 1e-38])
def test_tiny_queries_over_keys_of_the_smallest_scale(QH, KH, D, P, lens, size):
    """Logits that round to 0: the weights are equal, masked places still have none."""
    s = Setup(lens, QH, KH, D, P, seed=D)
    s.cache["k_scale"][:] = 2.0 ** -60
    q = (make_q(s).double() * size).to(torch.bfloat16)
    out, lse = run(s, q)
    check(s, q, out, lse)
    out, lse = run(s, q, window=50)
    check(s, q, out, lse, window=50)
