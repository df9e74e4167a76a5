"""moe_kv_append against its 64-bit form.  Codes, scales and the rotated q are functions of the exact
rotation (include/moe.h), so they are compared bit for bit: the 64-bit form's own error, 2^-53 of
values whose products are exact in it, would have to cross a border of the 8- or 16-bit grid."""
import pytest
import torch

from sparse_moe_router_gb300 import abi

import layer_ref as ref

pytestmark = pytest.mark.gpu


def rope_table(rows, rot, base=10000.0):
    half = rot // 2
    a = torch.arange(rows, dtype=torch.float64)[:, None] * base ** (-torch.arange(half, dtype=torch.float64) / half)
    return torch.cat([a.cos(), a.sin()], 1).float()


class Setup:
    def __init__(self, lens, QH, KH, D, P, rot=None, interleaved=False, dtype=torch.bfloat16, seed=0, fill=True, strided=True,
                 amp=0.8, extra=2, rope_rows=None):
        gen = torch.Generator().manual_seed(seed)
        self.cfg = abi.attn_config(QH, KH, D, P, rotary_dim=rot, interleaved=interleaved, dtype=dtype)
        rot = self.cfg.rotary_dim
        n = [a for a, _ in lens]
        kv = [b for _, b in lens]
        self.T, B = sum(n), len(lens)
        cols = [max(0, -(-x // P)) for x in kv]
        self.n_pages = sum(cols) + extra
        order = torch.randperm(self.n_pages, generator=gen)
        self.table = torch.full((B, max(max(cols), 1)), -7, dtype=torch.int32)
        at = 0
        for b, c in enumerate(cols):
            self.table[b, :c] = order[at:at + c].int()
            at += c
        self.q_start = torch.tensor([0] + list(torch.tensor(n).cumsum(0)), dtype=torch.int32)
        self.kv_len = torch.tensor(kv, dtype=torch.int32)
        self.rope = rope_table(rope_rows or max(max(kv), 1), rot) if rot else None
        wide = QH + 2 * KH + (1 if strided else 0)
        a = torch.randn(self.T, wide, D, generator=gen) * torch.exp(amp * torch.randn(self.T, wide, 1, generator=gen))
        self.qkv = a.to(dtype)
        shape = (self.n_pages, KH, P, D)
        self.cache = {}
        for name in "kv":
            if fill:
                v = torch.randn(shape, generator=gen, dtype=torch.float64) * torch.exp(amp * torch.randn(shape[:2], generator=gen))[..., None, None]
                s = ref.pow2_scale(v.abs().amax(dim=(2, 3)))
                self.cache[name + "_codes"], self.cache[name + "_scale"] = ref.encode(v / s[..., None, None]), s.float()
            else:
                self.cache[name + "_codes"] = torch.zeros(shape, dtype=torch.uint8)
                self.cache[name + "_scale"] = torch.ones(shape[:2])
        self.QH, self.KH = QH, KH

    def split(self, t):
        return t[:, :self.QH], t[:, self.QH:self.QH + self.KH], t[:, self.QH + self.KH:self.QH + 2 * self.KH]

    def device(self):
        c = {k: v.cuda() for k, v in self.cache.items()}
        cache = abi.KVCache(self.cfg, c["k_codes"], c["v_codes"], c["k_scale"], c["v_scale"])
        batch = abi.KVBatch(self.q_start.cuda(), self.kv_len.cuda(), self.table.cuda(), self.T)
        return cache, batch, abi.alloc_attn_workspace(self.cfg, len(self.kv_len), self.T)

    def append(self, cache, batch, ws, stream=None):
        qkv = self.qkv.cuda()
        q, k, v = self.split(qkv)
        q_out = torch.full((self.T, self.QH, self.cfg.head_dim), 7.0, dtype=qkv.dtype, device="cuda")
        abi.moe_kv_append(self.cfg, cache, batch, q, k, v, None if self.rope is None else self.rope.cuda(), q_out, ws, stream)
        return q_out

    def want(self):
        q, k, v = self.split(self.qkv)
        return ref.kv_append(self.cfg, self.cache, self.q_start, self.kv_len, self.table, q, k, v, self.rope)

    def check(self, cache, q_out, want_q):
        for name in ("k_codes", "v_codes", "k_scale", "v_scale"):
            got, want = getattr(cache, name).cpu(), self.cache[name]
            if name.endswith("codes"):  # the two zeros stand for the same value
                got, want = torch.where(got == 128, 0, got), torch.where(want == 128, 0, want)
            assert torch.equal(got, want), (name, int((got != want).sum()))
        wrong = q_out.cpu().double() != ref.round16(want_q, q_out.dtype)
        assert not bool(wrong.any()), int(wrong.sum())


MIXED = [(1, 1), (5, 5), (1, 64), (1, 65), (3, 66), (17, 100), (70, 70), (64, 128), (130, 200), (1, 16), (40, 2000)]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("QH,KH,D,P,rot,inter", [(16, 2, 128, 64, 128, False), (8, 8, 64, 16, 32, True), (6, 2, 64, 32, 64, False),
                                                 (4, 1, 256, 128, 64, False), (3, 1, 256, 64, 256, True), (2, 2, 128, 16, 0, False),
                                                 (8, 4, 128, 128, 96, True), (1, 1, 64, 128, 16, False)])
def test_append(dtype, QH, KH, D, P, rot, inter):
    s = Setup(MIXED, QH, KH, D, P, rot, inter, dtype, seed=D + P + QH)
    cache, batch, ws = s.device()
    got = s.append(cache, batch, ws)
    s.check(cache, got, s.want())
    assert abi.moe_check_status(ws) == 0


def test_token_by_token_growth_rounds_old_codes_again():
    """A page filled one token at a time, each larger than the one before: every scale the page moves
    through re-rounds its codes."""
    s = Setup([(1, 1)], 2, 2, 64, 16, 64, False, fill=False, strided=False)
    cache, _, ws = s.device()
    gen = torch.Generator().manual_seed(9)
    s.rope = rope_table(64, 64)
    for i in range(40):
        s.qkv = (torch.randn(1, 6, 64, generator=gen) * 2.0 ** ((i * 7) % 13 - 6)).to(torch.bfloat16)
        s.kv_len = torch.tensor([i + 1], dtype=torch.int32)
        s.table = torch.tensor([[1, 2, 0]], dtype=torch.int32)
        batch = abi.KVBatch(s.q_start.cuda(), s.kv_len.cuda(), s.table.cuda(), 1)
        got = s.append(cache, batch, ws)
        s.check(cache, got, s.want())


def test_appending_twice_is_appending_once():
    s = Setup([(9, 70), (100, 130)], 4, 2, 128, 64)
    cache, batch, ws = s.device()
    s.append(cache, batch, ws)
    got = s.append(cache, batch, ws)
    s.check(cache, got, s.want())


def test_padding_in_front_and_sequences_without_new_tokens():
    s = Setup([(8, 3), (0, 50), (4, 0), (2, 40), (0, 0)], 4, 2, 64, 16, 64)
    cache, batch, ws = s.device()
    got = s.append(cache, batch, ws)
    want = s.want()
    s.check(cache, got, want)
    assert not got[:5].any() and not got[8:12].any()
    assert abi.moe_check_status(ws) == 0


def test_extreme_values():
    """Zeros (the smallest scale), the largest bf16, values on the scale's borders, exact ties."""
    s = Setup([(64, 64)], 1, 1, 64, 16, 0, fill=False, strided=False)
    s.qkv.zero_()
    s.qkv[16:32, 1:] = 448.0 * 2.0 ** -7
    s.qkv[20, 1:, 3] = 450.0 * 2.0 ** -7
    s.qkv[32:48, 1:] = torch.finfo(torch.bfloat16).max
    s.qkv[33, 1:] = torch.finfo(torch.bfloat16).tiny
    ties = torch.tensor([(16 + 2 * i + 1) * 2.0 ** -4 for i in range(64)])  # between neighbours with 3 fraction bits
    s.qkv[48:, 1:] = ties.to(torch.bfloat16)
    s.qkv[50, 1:] = 256.0
    cache, batch, ws = s.device()
    got = s.append(cache, batch, ws)
    s.check(cache, got, s.want())
    assert abi.moe_check_status(ws) == 0


def test_values_that_are_not_finite_are_reported():
    s = Setup([(20, 30)], 2, 2, 64, 16, 0, strided=False)
    s.qkv[3, 2, 5] = float("nan")
    s.qkv[4, 5, 6] = float("-inf")
    cache, batch, ws = s.device()
    got = s.append(cache, batch, ws)
    s.check(cache, got, s.want())
    assert abi.moe_check_status(ws) == 1


def test_bad_pages_and_positions_are_reported_and_leave_the_rest_alone():
    s = Setup([(1, 33), (2, 20), (1, 5)], 2, 1, 64, 16, 64, rope_rows=32)
    s.table[1, 1] = s.n_pages  # outside the cache
    cache, batch, ws = s.device()
    s.append(cache, batch, ws)
    assert abi.moe_check_status(ws) == 1
    # sequence 2 is as it should be, every page that nobody owns is untouched
    page = int(s.table[2, 0])
    before = {k: v.clone() for k, v in s.cache.items()}
    t = Setup([(1, 5)], 2, 1, 64, 16, 64)
    t.cache, t.table, t.qkv, t.rope, t.T = s.cache, s.table[2:], s.qkv[3:], s.rope, 1
    t.want()
    assert torch.equal(cache.k_codes.cpu()[page], t.cache["k_codes"][page])
    owned = {int(x) for x in s.table.flatten()}
    free = [p for p in range(s.n_pages) if p not in owned]
    assert free and torch.equal(cache.v_codes.cpu()[free], before["v_codes"][free])


def test_other_stream_and_graph_replay():
    s = Setup([(1, 40), (1, 129), (1, 17)], 16, 2, 128, 64)
    cache, batch, ws = s.device()
    qkv = s.qkv.cuda()
    q, k, v = s.split(qkv)
    rope = rope_table(300, 128).cuda()
    s.rope = rope.cpu()
    q_out = torch.empty(3, 16, 128, dtype=torch.bfloat16, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    abi.moe_kv_append(s.cfg, cache, batch, q, k, v, rope, q_out, ws, stream=side)
    side.synchronize()
    s.check(cache, q_out, s.want())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        abi.moe_kv_append(s.cfg, cache, batch, q, k, v, rope, q_out, ws)
    for step in range(1, 4):  # the next tokens of the same sequences, lengths changed in place
        s.kv_len += 1
        batch.kv_len.copy_(s.kv_len)
        s.qkv = torch.randn(s.qkv.shape, generator=torch.Generator().manual_seed(step)).to(torch.bfloat16)
        qkv.copy_(s.qkv)
        graph.replay()
        torch.cuda.synchronize()
        s.check(cache, q_out, s.want())


def test_many_sequences():
    gen = torch.Generator().manual_seed(2)
    lens = [(int(n), int(n) + int(x)) for n, x in zip(torch.randint(0, 3, (1500,), generator=gen), torch.randint(0, 90, (1500,), generator=gen))]
    s = Setup(lens, 2, 1, 64, 32, 64)
    cache, batch, ws = s.device()
    got = s.append(cache, batch, ws)
    s.check(cache, got, s.want())
