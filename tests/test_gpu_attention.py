"""moe_attention against its 64-bit form: head widths and groups, page sizes, ragged batches from empty
sequences on, causal and windowed masks, rows that see nothing, what lies past a sequence's end,
strided rows, streams and graphs, page ids whose bytes lie past 4 GB.  Bounds: layer_ref.attention."""
import pytest
import torch

from sparse_moe_router_gb300 import abi

import layer_ref as ref
from test_gpu_kv_append import Setup

pytestmark = pytest.mark.gpu


def run(s, q, causal=True, window=0, scale=None, spoil=True, out=None):
    """out, lse; before the call every slot that no row may see is filled with NaN codes."""
    if spoil:
        used = torch.zeros(s.n_pages, s.cfg.page_size, dtype=torch.bool)
        for b, kv in enumerate(s.kv_len.tolist()):
            for j in range(0, kv):
                used[int(s.table[b, j // s.cfg.page_size]), j % s.cfg.page_size] = True
        for name in "kv":
            s.cache[name + "_codes"][~used[:, None, :].expand(-1, s.KH, -1)] = 127
            s.cache[name + "_scale"][~used.any(1)] = float("nan")
    cache, batch, ws = s.device()
    if out is None:
        out = torch.full((s.T, s.QH, s.cfg.head_dim), 9.0, dtype=q.dtype, device="cuda")
    lse = torch.full((s.T, s.QH), 9.0, device="cuda")
    abi.moe_attention(s.cfg, cache, batch, q, out, ws, lse=lse, softmax_scale=scale, causal=causal, window=window)
    assert abi.moe_check_status(ws) == 0
    return out, lse


def check(s, q, out, lse, causal=True, window=0, scale=None):
    c = {k: v.clone() for k, v in s.cache.items()}
    want, wl, tol, ltol = ref.attention(s.cfg, c, s.q_start, s.kv_len, s.table, q.cpu(),
                                        s.cfg.head_dim ** -0.5 if scale is None else scale, causal, window)
    half = ref.HALF_STEP[out.dtype]
    far = (out.cpu().double() - want).abs() - (half * want.abs() + (1 + half) * tol + ref.TINY[out.dtype])
    assert not bool(far.isnan().any()) and float(far.max()) <= 0, (float(far.max()), float(far.isnan().sum()))
    empty = wl == -float("inf")
    assert torch.equal(lse.cpu() == -float("inf"), empty)
    if bool((~empty).any()):
        assert float(((lse.cpu().double() - wl).abs() - ltol)[~empty].max()) <= 0
    assert not out.cpu()[empty].any()


def make_q(s, seed=1, std=1.2):
    gen = torch.Generator().manual_seed(seed)
    dt = {0: torch.bfloat16, 1: torch.float16}[s.cfg.dtype]
    return (torch.randn(s.T, s.QH, s.cfg.head_dim, generator=gen) * std).to(dt).cuda()


TOKENS = [(1, 1), (1, 15), (1, 16), (1, 17), (1, 64), (1, 65), (1, 300), (1, 1), (1, 1500), (1, 0)]
RUNS = [(1, 7), (2, 2), (4, 90), (5, 3), (0, 30), (33, 33), (70, 200), (3, 130)]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("QH,KH,D,P", [(16, 2, 128, 64), (8, 8, 64, 16), (6, 2, 64, 32), (4, 1, 256, 128), (24, 2, 128, 16),
                                       (5, 1, 64, 128), (16, 1, 256, 32), (40, 1, 128, 64)])
@pytest.mark.parametrize("lens", [TOKENS, RUNS], ids=["tokens", "runs"])
def test_attention(dtype, QH, KH, D, P, lens):
    s = Setup(lens, QH, KH, D, P, dtype=dtype, seed=QH + D)
    q = make_q(s)
    out, lse = run(s, q)
    check(s, q, out, lse)


@pytest.mark.parametrize("causal,window", [(True, 1), (True, 40), (False, 0), (False, 33), (True, 100000)])
@pytest.mark.parametrize("QH,KH,D,P", [(16, 2, 128, 64), (6, 2, 64, 16), (4, 2, 256, 32)])
def test_masks(causal, window, QH, KH, D, P):
    s = Setup(RUNS + [(1, 400), (2, 129)], QH, KH, D, P, seed=3)
    q = make_q(s)
    out, lse = run(s, q, causal, window)
    check(s, q, out, lse, causal, window)


PROMPTS = [[(300, 300)], [(257, 900), (1, 33), (129, 129), (64, 1000)], [(600, 601)]]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("QH,KH,D,P", [(16, 2, 128, 64), (12, 4, 64, 16), (3, 1, 128, 128), (8, 1, 256, 32), (2, 2, 64, 32)])
@pytest.mark.parametrize("lens", PROMPTS, ids=["one", "mixed", "odd"])
def test_prompts(dtype, QH, KH, D, P, lens):
    s = Setup(lens, QH, KH, D, P, dtype=dtype, seed=QH + D + 1)
    q = make_q(s)
    out, lse = run(s, q)
    check(s, q, out, lse)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("QH,KH,D,P", [(16, 2, 128, 64), (12, 4, 64, 16), (3, 1, 128, 128), (8, 1, 256, 32), (2, 2, 64, 32),
                                       (2, 1, 256, 16), (40, 1, 64, 64)])
@pytest.mark.parametrize("kind", ["one", "mixed", "odd", "short"])
def test_prompts_of_many_rows(dtype, QH, KH, D, P, kind):
    """4300 rows (tokens x q heads) and more in all, the tensor cores' share of the work."""
    n = 4300 // QH + 3
    lens = {"one": [(n, n)], "mixed": [(n, n + 643), (1, 33), (129, 129), (64, 1000)], "odd": [(n // 2 + 1, n), (n // 2 + 3, 2 * n + 5)],
            "short": [(n, 9), (n // 3, n // 2)]}[kind]
    s = Setup(lens, QH, KH, D, P, dtype=dtype, seed=QH)
    q = make_q(s)
    out, lse = run(s, q)
    check(s, q, out, lse)


@pytest.mark.parametrize("causal,window", [(True, 0), (False, 0), (True, 3000), (False, 5)])
@pytest.mark.parametrize("QH,KH,D,P", [(8, 1, 128, 64), (12, 2, 64, 16), (8, 1, 256, 32)])
@pytest.mark.parametrize("lens", [[(560, 9000)], [(140, 9001)], [(333, 7001), (1, 40), (300, 2100), (0, 77), (64, 64)]],
                         ids=["one", "few", "mixed"])
def test_prompts_behind_long_caches(causal, window, QH, KH, D, P, lens):
    """Few rows and many keys: the keys of a block are shared out and its parts joined."""
    s = Setup(lens, QH, KH, D, P, seed=D)
    q = make_q(s)
    out, lse = run(s, q, causal, window)
    check(s, q, out, lse, causal, window)


@pytest.mark.parametrize("causal,window", [(True, 100), (False, 0), (False, 200), (True, 1)])
@pytest.mark.parametrize("QH,KH,D,P", [(16, 2, 128, 64), (12, 4, 64, 16), (8, 2, 256, 32)])
def test_prompt_masks(causal, window, QH, KH, D, P):
    s = Setup([(300, 700), (290, 200), (64, 64)], QH, KH, D, P, seed=6)
    q = make_q(s)
    out, lse = run(s, q, causal, window)
    check(s, q, out, lse, causal, window)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("QH,KH,D,P", [(16, 2, 128, 64), (6, 2, 64, 16), (4, 1, 256, 32), (24, 2, 128, 128)])
def test_row_tiles_that_share_keys(dtype, QH, KH, D, P):
    """A few tokens a sequence in a table that could name 2^20 tokens: the form whose row tiles share key
    tiles."""
    s = Setup([(4, 300), (7, 7), (3, 1000), (9, 4), (0, 20), (5, 129)], QH, KH, D, P, dtype=dtype, seed=D)
    pages = (1 << 20) // P
    wide = torch.full((6, pages), -7, dtype=torch.int32)
    wide[:, :s.table.shape[1]] = s.table
    s.table = wide
    q = make_q(s)
    out, lse = run(s, q)
    check(s, q, out, lse)
    out, lse = run(s, q, window=70)
    check(s, q, out, lse, window=70)


@pytest.mark.parametrize("lens", [[(1, 900), (2, 77)], [(300, 700)], [(600, 700)]], ids=["tokens", "run", "prompt"])
def test_sharp_and_shifted_logits(lens):
    """Logits in the hundreds: the running reference moves often, most weights vanish; pages whose scales
    lie far apart; a softmax scale of the caller's."""
    s = Setup(lens, 8, 2, 128, 64, seed=4, amp=2.5)
    q = make_q(s, std=30.0)
    out, lse = run(s, q, scale=0.05)
    check(s, q, out, lse, scale=0.05)


@pytest.mark.parametrize("n", [130, 530])
def test_keys_that_grow_along_the_sequence(n):
    """Each page larger than the one before, values too: every step moves the reference and the unit."""
    s = Setup([(1, 640), (n, 640)], 8, 1, 64, 16, seed=4)
    for b in range(2):
        for j in range(40):
            page = int(s.table[b, j])
            s.cache["k_scale"][page] = 2.0 ** (j // 4 - 14)
            s.cache["v_scale"][page] = 2.0 ** (20 - j)
    q = make_q(s)
    out, lse = run(s, q)
    check(s, q, out, lse)


@pytest.mark.parametrize("n,kv", [(1, 5000), (300, 800)])
def test_the_result_does_not_change_from_run_to_run(n, kv):
    s = Setup([(n, kv), (1, 70)], 16, 2, 128, 64)
    q = make_q(s)
    a, la = run(s, q, spoil=False)
    for _ in range(3):
        b, lb = run(s, q, spoil=False)
        assert torch.equal(a, b) and torch.equal(la, lb)


@pytest.mark.parametrize("n", [1, 300, 560])
def test_strided_rows_other_stream_and_graph(n):
    s = Setup([(n, max(500, n + 40)), (1, 333)], 8, 2, 64, 32, seed=8)
    q0 = make_q(s)
    wide = torch.zeros(s.T, 8 * 64 + 72, dtype=torch.bfloat16, device="cuda")
    wide[:, 8:8 + 512] = q0.flatten(1)
    q = wide[:, 8:8 + 512].unflatten(1, (8, 64))
    o_wide = torch.zeros(s.T, 8 * 64 + 24, dtype=torch.bfloat16, device="cuda")
    out = o_wide[:, 16:16 + 512].unflatten(1, (8, 64))
    out, lse = run(s, q, out=out)
    check(s, q0, out, lse)
    assert not o_wide[:, :16].any() and not o_wide[:, 528:].any()
    cache, batch, ws = s.device()
    other = torch.empty(s.T, 8, 64, dtype=torch.bfloat16, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    abi.moe_attention(s.cfg, cache, batch, q, other, ws, stream=side)
    side.synchronize()
    assert torch.equal(other, out)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        abi.moe_attention(s.cfg, cache, batch, q, other, ws)
    s.kv_len = torch.tensor([450, 100], dtype=torch.int32)  # shorter, in place
    batch.kv_len.copy_(s.kv_len)
    graph.replay()
    torch.cuda.synchronize()
    cache2, batch2, ws2 = s.device()
    again = torch.empty_like(other)
    abi.moe_attention(s.cfg, cache2, batch2, q, again, ws2)
    assert torch.equal(other, again)


@pytest.mark.parametrize("n", [1, 300])
def test_bad_pages_are_reported(n):
    s = Setup([(n, 400), (n, 310)], 8, 1, 64, 16, seed=2)
    cache, batch, ws = s.device()
    q = make_q(s)
    good = torch.empty_like(q)
    abi.moe_attention(s.cfg, cache, batch, q, good, ws)
    assert abi.moe_check_status(ws) == 0
    for bad in (-1, s.n_pages, 2 ** 31 - 1):
        s.table[1, 3] = bad
        batch = abi.KVBatch(batch.q_start, batch.kv_len, s.table.cuda(), s.T)
        out = torch.empty_like(q)
        abi.moe_attention(s.cfg, cache, batch, q, out, ws)
        assert abi.moe_check_status(ws) == 1
        assert torch.equal(out[:n], good[:n])  # the other sequence is not touched by it
    lens = torch.tensor([400, 16 * s.table.shape[1] + 1], dtype=torch.int32, device="cuda")
    s.table[1, 3] = 0
    abi.moe_attention(s.cfg, cache, abi.KVBatch(batch.q_start, lens, s.table.cuda(), s.T), q, out, ws)
    assert abi.moe_check_status(ws) == 1


@pytest.mark.parametrize("n", [1, 300])
def test_many_sequences(n):
    gen = torch.Generator().manual_seed(2)
    if n == 1:
        lens = [(1, int(x)) for x in torch.randint(0, 40, (1100,), generator=gen)]
    else:
        lens = [(int(a), int(a) + int(x)) for a, x in zip(torch.randint(0, 40, (70,), generator=gen), torch.randint(0, 200, (70,), generator=gen))]
    s = Setup(lens, 4, 2, 64, 16)
    q = make_q(s)
    out, lse = run(s, q)
    check(s, q, out, lse)


@pytest.mark.parametrize("used", [0, 5, 30, 31, 299])
@pytest.mark.parametrize("n,seqs", [(300, 1), (300, 2), (600, 1), (600, 2)])
def test_rows_past_the_last_sequence(used, n, seqs):
    """A batch held for more tokens than its sequences have: the rows behind them stay as they are."""
    lens = [(n, 700)] + [(0, 9)] * (seqs - 1)
    s = Setup(lens, 8, 2, 128, 64, seed=4)
    q = make_q(s)
    s.q_start[1:] = used
    cache, batch, ws = s.device()
    out = torch.full_like(q, 9.0)
    lse = torch.full((s.T, 8), 9.0, device="cuda")
    abi.moe_attention(s.cfg, cache, batch, q, out, ws, lse=lse)
    assert abi.moe_check_status(ws) == 0
    assert bool((out[used:] == 9).all()) and bool((lse[used:] == 9).all())
    part = Setup(lens, 8, 2, 128, 64, seed=4)
    part.q_start, part.T = s.q_start, used
    if used:
        check(part, q[:used], out[:used], lse[:used])


@pytest.mark.slow
@pytest.mark.parametrize("n", [1, 260])
def test_pages_past_four_gigabytes(n):
    KH, D, P = 8, 128, 128
    pages = (1 << 32) // (KH * D * P) + 64
    s = Setup([(n, 700)], 16, KH, D, P, seed=5)
    q = make_q(s)
    cache, batch, ws = s.device()
    want = torch.empty_like(q)
    abi.moe_attention(s.cfg, cache, batch, q, want, ws)
    big = abi.KVCache(s.cfg, *(torch.empty((pages, KH, P, D), dtype=torch.uint8, device="cuda") for _ in range(2)),
                      *(torch.ones((pages, KH), device="cuda") for _ in range(2)))
    moved = s.table.clone()
    for j in range(6):
        src, dst = int(s.table[0, j]), pages - 1 - 7 * j
        moved[0, j] = dst
        for a in ("k_codes", "v_codes", "k_scale", "v_scale"):
            getattr(big, a)[dst] = getattr(cache, a)[src]
    out = torch.empty_like(q)
    abi.moe_attention(s.cfg, big, abi.KVBatch(batch.q_start, batch.kv_len, moved.cuda(), s.T), q, out, ws)
    assert torch.equal(out, want)
    # and an append writes there
    k = torch.randn(n, KH, D, device="cuda").bfloat16()
    rope = torch.zeros(1024, D, device="cuda")
    abi.moe_kv_append(s.cfg, big, abi.KVBatch(batch.q_start, batch.kv_len, moved.cuda(), s.T), None, k, k, rope, None, ws)
    abi.moe_kv_append(s.cfg, cache, batch, None, k, k, rope, None, ws)
    for j in range(6):
        assert torch.equal(big.v_codes[int(moved[0, j])], cache.v_codes[int(s.table[0, j])])
    assert abi.moe_check_status(ws) == 0
