"""moe_attention with windows up to the largest int, tokens at negative positions (padding in front) among
them.  Bounds: attention_bound."""
import pytest
import torch

from sparse_moe_router_gb300 import abi

import attention_bound
from test_gpu_attention import make_q
from test_gpu_kv_append import Setup

pytestmark = pytest.mark.gpu


def run(s, q, causal=True, window=0):
    cache, batch, ws = s.device()
    out = torch.full((s.T, s.QH, s.cfg.head_dim), 9.0, dtype=q.dtype, device="cuda")
    lse = torch.full((s.T, s.QH), 9.0, device="cuda")
    abi.moe_attention(s.cfg, cache, batch, q, out, ws, lse=lse, causal=causal, window=window)
    assert abi.moe_check_status(ws) == 0
    return out, lse


# (new tokens, cached ones): padding in front; runs of the split kernel, then of the prompt kernel
PADDED = {"short": [(203, 3), (5, 2), (9, 0), (1, 40)], "prompt": [(700, 640)], "prompts": [(700, 640), (300, 1), (260, 900), (3, 2)]}


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("QH,KH,D,P", [(8, 2, 128, 64), (8, 1, 64, 16), (16, 2, 256, 32)])
@pytest.mark.parametrize("lens", PADDED.values(), ids=PADDED)
def test_windows_that_no_position_reaches(causal, QH, KH, D, P, lens):
    """A window of at least the table's length is no window at all, bit for bit."""
    s = Setup(lens, QH, KH, D, P, seed=D)
    q = make_q(s)
    want, want_lse = run(s, q, causal)
    attention_bound.check(s.cfg, s.cache, s.q_start, s.kv_len, s.table, q, want, want_lse, causal=causal)
    table = s.table.shape[1] * P
    for window in (2 ** 31 - 1, 2 ** 31 - 4, 2 ** 31 - 203, 2 ** 30 + 1, 2 ** 30, table + s.T, table):
        out, lse = run(s, q, causal, window)
        assert torch.equal(out, want) and torch.equal(lse, want_lse), window


@pytest.mark.parametrize("QH,KH,D,P", [(8, 2, 128, 64), (8, 1, 64, 16), (16, 2, 256, 32)])
@pytest.mark.parametrize("lens", PADDED.values(), ids=PADDED)
def test_the_longest_window_that_masks(QH, KH, D, P, lens):
    """One less than the table's length: only a row at the table's last position loses a key."""
    lens = [(n, -(-kv // P) * P) for n, kv in lens]
    s = Setup(lens, QH, KH, D, P, seed=D)
    q = make_q(s)
    for window in (s.table.shape[1] * P - 1, max(s.table.shape[1] * P - 3, 1)):
        out, lse = run(s, q, window=window)
        attention_bound.check(s.cfg, s.cache, s.q_start, s.kv_len, s.table, q, out, lse, window=window)


@pytest.mark.parametrize("dead", [-1, 2 ** 31 - 1])
@pytest.mark.parametrize("QH,KH,D,P", [(8, 2, 128, 16), (8, 1, 64, 16), (16, 2, 256, 32)])
@pytest.mark.parametrize("window", [1, 100, 333])
@pytest.mark.parametrize("lens", [[(1, 1000), (3, 777), (1, 130)], [(600, 1300)], [(300, 1300), (1, 999), (260, 700)], [(140, 9000)]],
                         ids=["tokens", "prompt", "prompts", "parts"])
def test_pages_behind_the_window_may_be_gone(dead, QH, KH, D, P, window, lens):
    """Table entries of pages that no row sees are not looked up: they may be given back, and page 0, which bad
    ids read in their place, may hold anything."""
    s = Setup(lens, QH, KH, D, P, seed=D)
    q = make_q(s)
    for b, (n, kv) in enumerate(lens):
        s.table[b, :max(kv - n + 1 - window, 0) // P] = dead
    used = set(s.table.flatten().tolist())
    for name in "kv":
        free = [p for p in range(s.n_pages) if p not in used]
        s.cache[name + "_codes"][free] = 127
        s.cache[name + "_scale"][free] = float("nan")
    out, lse = run(s, q, window=window)
    attention_bound.check(s.cfg, s.cache, s.q_start, s.kv_len, s.table, q, out, lse, window=window)
