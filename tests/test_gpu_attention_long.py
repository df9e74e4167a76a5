"""Forms of moe_attention that only large batches reach: a segment of more than 4096 keys in one block of the
split kernel, and prompts in a batch of more than 32 sequences.  Bounds: attention_bound."""
import pytest
import torch

from sparse_moe_router_gb300 import abi

import attention_bound
from test_gpu_attention import make_q
from test_gpu_attention_windows import run
from test_gpu_kv_append import Setup

pytestmark = pytest.mark.gpu


def check(s, q, out, lse, **kw):
    attention_bound.check(s.cfg, s.cache, s.q_start, s.kv_len, s.table, q, out, lse, **kw)


@pytest.mark.parametrize("seqs,new,QH,D,P,window,sets", [(34, 1, 2, 64, 16, 0, 3), (16, 1, 1, 128, 64, 0, 2), (16, 1, 1, 128, 64, 95_000, 2),
                                                         (8, 1, 2, 256, 128, 0, 2), (16, 2, 3, 64, 32, 0, 2)])
def test_more_than_32_tiles_a_warp(seqs, new, QH, D, P, window, sets):
    """Sequences of 74,000 to 100,000 keys (of the same pages, each in an order of its own): the share of a block is
    more than 4096 (8192) of a sequence's keys, so that a warp goes through more than 32 (64) tiles of 16 and
    takes up a second (and third) set of pages and scales."""
    KH, kv = 1, 100_003
    lens = [kv - 1709 * (i % 16) for i in range(seqs)]
    blocks = torch.cuda.get_device_properties(0).multi_processor_count * (1 if D == 256 else 2)
    assert sum(min(n, window or n) for n in lens) // blocks > 4096 * (sets - 1) + 256
    s = Setup([(new, kv)], QH, KH, D, P, seed=D)
    gen = torch.Generator().manual_seed(D)
    pages = s.table[0]
    s.table = torch.stack([pages[torch.randperm(len(pages), generator=gen)] for _ in range(seqs)])
    s.kv_len = torch.tensor(lens, dtype=torch.int32)
    s.q_start = torch.arange(0, new * seqs + 1, new, dtype=torch.int32)
    s.T = new * seqs
    q = make_q(s)
    out, lse = run(s, q, window=window)
    check(s, q, out, lse, window=window)


@pytest.mark.parametrize("padded", [0, 77])
@pytest.mark.parametrize("causal,window", [(True, 0), (False, 150)])
@pytest.mark.parametrize("QH,KH,D,P", [(8, 2, 64, 16), (4, 1, 128, 64), (6, 2, 256, 32)])
def test_prompts_among_more_than_32_sequences(padded, causal, window, QH, KH, D, P):
    """40 sequences, of which every other one has 128 rows (tokens x q heads of a kv head) or more, among short
    and empty ones, at lengths that are no multiple of a block's rows; rows behind the last sequence too."""
    G = QH // KH
    lens = []
    for i in range(40):
        n = -(-(128 + 37 * i) // G) if i % 2 else (0, 1, 3, 2)[i // 2 % 4]
        lens.append((n, n + (0, 5, 300, 64, 131)[i % 5] if i != 8 else 0))
    lens[13] = (lens[13][0], lens[13][0] - 20)  # padding in front
    s = Setup(lens, QH, KH, D, P, seed=D)
    assert sum(n for n, _ in lens) * G / 40 >= 33 and sum(n for n, _ in lens) * QH >= 4096
    q = make_q(s)
    out, lse = run(s, q, causal, window)
    check(s, q, out, lse, causal=causal, window=window)
    if padded:
        cache, batch, ws = s.device()
        wide = torch.cat([q, torch.randn(padded, QH, D, device="cuda").to(q.dtype)])
        batch = abi.KVBatch(batch.q_start, batch.kv_len, batch.page_table, s.T + padded)
        ws = abi.alloc_attn_workspace(s.cfg, 40, s.T + padded)
        out2 = torch.full_like(wide, 9.0)
        lse2 = torch.full((s.T + padded, QH), 9.0, device="cuda")
        abi.moe_attention(s.cfg, cache, batch, wide, out2, ws, lse=lse2, causal=causal, window=window)
        assert abi.moe_check_status(ws) == 0
        assert torch.equal(out2[:s.T], out) and torch.equal(lse2[:s.T], lse)
        assert bool((out2[s.T:] == 9).all()) and bool((lse2[s.T:] == 9).all())
