"""moe_attention on tables that could name far more tokens than the sequences have, as a server's do: the keys of
a block are shared out by the lengths, not by the table.  Bounds: attention_bound."""
import pytest
import torch

from sparse_moe_router_gb300 import abi

import attention_bound
from test_gpu_attention import make_q
from test_gpu_attention_windows import run
from test_gpu_kv_append import Setup

pytestmark = pytest.mark.gpu

HEADS = [(8, 1, 128, 64), (12, 2, 64, 16), (8, 1, 256, 32)]


def widen(s, tokens):
    wide = torch.full((s.table.shape[0], tokens // s.cfg.page_size), -7, dtype=torch.int32)
    wide[:, :s.table.shape[1]] = s.table
    s.table = wide


@pytest.mark.parametrize("QH,KH,D,P", HEADS)
@pytest.mark.parametrize("causal,window", [(True, 0), (False, 0), (True, 1500)])
@pytest.mark.parametrize("lens", [[(300, 300)], [(600, 1100)], [(257, 2304)], [(560, 9000)], [(300, 40)],
                                  [(300, 300), (200, 5000), (1, 900), (0, 44), (333, 1200), (64, 64)]],
                         ids=["first", "second", "some", "long", "padded", "mixed"])
@pytest.mark.parametrize("tokens", [16384, 131072])
def test_wide_tables(QH, KH, D, P, causal, window, lens, tokens):
    s = Setup(lens, QH, KH, D, P, seed=D)
    widen(s, tokens)
    q = make_q(s)
    out, lse = run(s, q, causal, window)
    attention_bound.check(s.cfg, s.cache, s.q_start, s.kv_len, s.table, q, out, lse, causal=causal, window=window)


@pytest.mark.parametrize("QH,KH,D,P", HEADS)
def test_a_short_sequence_makes_no_parts(QH, KH, D, P):
    """A first piece has too few keys to share out: its blocks write the output themselves, and the part of the
    workspace that parts' rows are kept in (the last but their sums) stays as it was."""
    s = Setup([(500, 500)], QH, KH, D, P, seed=D)
    q = make_q(s)
    want, want_lse = run(s, q)
    widen(s, 131072)
    cache, batch, ws = s.device()
    ws[256:] = 0xAB
    out, lse = torch.empty_like(want), torch.empty_like(want_lse)
    abi.moe_attention(s.cfg, cache, batch, q, out, ws, lse=lse)
    assert abi.moe_check_status(ws) == 0
    assert torch.equal(out, want) and torch.equal(lse, want_lse)
    rows = min(500 * QH * 16, 320 * (128 if D == 256 else 256))
    assert bool((ws[-rows * (D + 1) * 4:-rows * 4] == 0xAB).all())
