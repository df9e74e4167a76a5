"""moe_linear_attention against its 64-bit form, token by token: single tokens, short and long runs, shared key heads,
every head width, decays of all strengths, padding, strided rows, states handed from call to call.

Tolerances, in half steps of fp32 (2^-24) relative to the sum of the terms' sizes.  A state that is carried
token by token takes a product and an addition and a factor's exponential (2 ulp) a token, at most 8; in chunks of 64 the
same a chunk, and within one: weights 2^x, |x| < 150, whose argument is rounded once (104) by an exponential of 2 ulp (4), the
split of weighted values (1) and at most 12 additions of a matrix instruction, each cut at 2^-22 (48): 192.
An output adds the splits of the state and of the weighted products in two 16-bit parts (2^-18 each, 128), another exponential
(108) and 36 additions (144): 640.  Then out is rounded once."""
import math

import pytest
import torch

from sparse_moe_router_gb300 import abi

import layer_ref
import mixer_ref as ref

pytestmark = pytest.mark.gpu
BF, F16 = torch.bfloat16, torch.float16


class Case:
    def __init__(self, cfg, new, past, seed=0, dtype=BF, decay="token", wide=0, n_slots=None, rate=(1e-3, 1.0), behind=0):
        gen = torch.Generator().manual_seed(seed)
        r = lambda *s: torch.randn(*s, generator=gen)  # noqa: E731
        self.cfg, self.dtype, self.new, B = cfg, dtype, new, len(new)
        KH, VH, DK, DV = cfg.key_heads, cfg.value_heads, cfg.key_dim, cfg.value_dim
        self.T = sum(new) + behind
        rows = r(self.T, 2 * KH * DK + VH * DV + wide)
        rows[:, :2 * KH * DK] *= DK ** -0.5
        rows = rows.to(dtype).cuda()
        self.q, self.k, self.v = (t[:, :] for t in rows[:, :2 * KH * DK + VH * DV].split([KH * DK, KH * DK, VH * DV], dim=1))
        rates = torch.exp(torch.linspace(math.log(rate[0]), math.log(rate[1]), VH))
        self.decay = {"token": -rates * torch.nn.functional.softplus(1.5 * r(self.T, VH)), "head": -rates, "none": None}[decay]
        if self.decay is not None:
            self.decay = self.decay.cuda()
        n_slots = n_slots or B + 2
        self.slots = torch.randperm(n_slots, generator=gen)[:B].tolist()
        self.kv = [n + p for n, p in zip(new, past)]
        self.starts = [0]
        for n in new:
            self.starts.append(self.starts[-1] + n)
        self.states = (0.5 * r(n_slots, VH, DK, DV)).cuda()
        self.scale = 0.8

    def batch(self):
        i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
        self.kept = abi.StateBatch(i32(self.starts), i32(self.kv), i32(self.slots), self.T)
        return self.kept  # (alive as long as another stream may read it)

    def run(self, states=None, out=None, ws=None, stream=None, status=0):
        states = self.states.clone() if states is None else states
        out = torch.full((self.T, self.cfg.value_heads * self.cfg.value_dim), 7.0, dtype=self.dtype, device="cuda") if out is None else out
        ws = abi.alloc_linear_workspace(self.cfg, len(self.new), self.T) if ws is None else ws
        abi.moe_linear_attention(self.cfg, abi.StatePool(self.cfg, states), self.batch(), self.q, self.k, self.v, self.decay, out, ws,
                                 scale=self.scale, stream=stream)
        if status is not None and stream is None:
            assert abi.moe_check_status(ws) == status
        return out, states

    def want(self):
        return ref.linear_attention(self.cfg, self.states, self.starts, self.kv, self.slots, self.q, self.k, self.v, self.decay, self.scale)

    def check(self, out, states, rows=None, what=""):
        o, s, o_size, s_size = self.want()
        longest = ref.steps(max(self.new))
        o, o_size = o.flatten(1), o_size.flatten(1)
        left = o.isnan()
        got = out.cpu().double()
        assert bool((got[left] == 7.0).all()), what
        o, got = torch.where(left, 7.0, o), torch.where(left, 7.0, got)
        bound = layer_ref.HALF_STEP[self.dtype] * o.abs() + layer_ref.TINY[self.dtype] + (640 + 8 * longest) * ref.EPS32 * o_size
        far = (got - o).abs() - bound
        assert not bool(got.isnan().any()) and float(far.max()) <= 0, (what, "out", float(far.max()))
        far = (states.cpu().double() - s).abs() - (192 + 8 * longest) * ref.EPS32 * s_size
        assert not bool(states.isnan().any()) and float(far.max()) <= 0, (what, "state", float(far.max()))


DIMS = [(64, 64), (64, 128), (128, 64), (128, 128), (128, 256), (64, 256)]


@pytest.mark.parametrize("dtype", [BF, F16])
@pytest.mark.parametrize("DK,DV", DIMS)
def test_single_tokens_and_short_runs(dtype, DK, DV):
    for KH, VH, new, past in ((1, 1, [1], [0]), (2, 4, [1, 1, 1], [5, 0, 70]), (3, 3, [4, 1, 0, 7], [0, 9, 3, 100]), (1, 4, [16, 15], [3, 0])):
        c = Case(abi.linear_config(KH, VH, DK, DV, dtype=dtype), new, past, seed=DK + DV, dtype=dtype)
        c.check(*c.run(), what=(KH, VH, new))


@pytest.mark.parametrize("dtype", [BF, F16])
@pytest.mark.parametrize("DK,DV", DIMS)
@pytest.mark.parametrize("n", [17, 31, 33, 63, 64, 65, 127, 128, 129, 200, 321])
def test_runs_of_many_tokens(dtype, DK, DV, n):
    c = Case(abi.linear_config(2, 2, DK, DV, dtype=dtype), [n], [n % 3 * 50], seed=n, dtype=dtype)
    c.check(*c.run())


@pytest.mark.parametrize("decay", ["token", "head", "none"])
@pytest.mark.parametrize("KH,VH", [(1, 1), (2, 8), (5, 5)])
def test_long_and_mixed_batches(decay, KH, VH):
    c = Case(abi.linear_config(KH, VH, 128, 128), [1, 700, 0, 3, 129, 1, 64, 450], [4, 0, 9, 0, 30, 0, 1, 8], seed=VH, decay=decay, wide=24)
    c.check(*c.run())


def test_a_few_runs_among_many_single_tokens():
    """More heads than SMs, and few tokens a sequence: the chunk kernel's blocks go by tokens, not by sequences."""
    new = [1] * 120
    for at, n in ((0, 15), (7, 200), (8, 16), (30, 0), (31, 17), (64, 64), (119, 130)):
        new[at] = n
    c = Case(abi.linear_config(2, 4, 64, 64), new, [3 * (i % 3) for i in range(120)], seed=3, behind=2)
    assert 120 * 4 > 304 and c.T // 16 < 120
    c.check(*c.run())
    c.starts[60] = 5  # a range that ends before it begins counts as none, the one before it overlaps others' rows
    c.run(status=1)


def test_slots_past_32_bits():
    """The last slots of a pool of more than 2^31 values."""
    cfg = abi.linear_config(2, 8, 128, 256)
    n_slots = 8200
    assert n_slots * 8 * 128 * 256 > 2 ** 31
    states = torch.empty(n_slots, 8, 128, 256, device="cuda")
    for new in ([3, 1], [150, 9]):
        c = Case(cfg, new, [4, 4], seed=1, n_slots=2)
        out, small = c.run()
        far = [n_slots - 1, 8193]
        for b in (0, 1):
            states[far[b]] = c.states[c.slots[b]]
        near = list(c.slots)
        c.slots = far
        got, _ = c.run(states=states)
        assert torch.equal(got, out)
        for b in (0, 1):
            assert torch.equal(states[far[b]], small[near[b]])


def test_many_chunks_over_few_heads():
    """One head of a long prompt: its chunks are shared out over the SMs."""
    for n, VH, past in ((3000, 1, 0), (3001, 2, 17), (2047, 3, 0)):
        c = Case(abi.linear_config(1, VH, 128, 128), [n], [past], seed=n)
        c.check(*c.run(), what=n)


@pytest.mark.parametrize("n", [40, 200, 900])
def test_decays_of_all_strengths(n):
    """Factors of 0 (one token forgets all), decays that leave nothing after a few tokens, and hardly any: in the same run."""
    cfg = abi.linear_config(2, 4, 64, 64)
    c = Case(cfg, [n, n // 2], [10, 0], seed=1, rate=(1e-6, 60.0))
    g = c.decay
    g[5::37] = -math.inf
    g[11::29, 1] = -3e4
    g[13::31, 2] = -1e-30
    c.check(*c.run())


def test_a_first_token_that_forgets():
    cfg = abi.linear_config(1, 2, 64, 64)
    for n in (1, 5, 80):
        c = Case(cfg, [n], [100], seed=n)
        c.decay[0] = -math.inf
        c.check(*c.run(), what=n)


def test_values_far_from_one():
    """Large and tiny queries, keys, values and states: nothing overflows or vanishes that fits fp32."""
    for dtype, q, k, v, state in ((F16, 200.0, 300.0, 2000.0, 1e6), (F16, 1e-2, 1e-2, 1e-3, 1e-8), (BF, 1e10, 1e9, 1e8, 1e17), (BF, 1e-9, 1e-8, 1e-7, 1e-15)):
        c = Case(abi.linear_config(1, 2, 128, 128, dtype=dtype), [150, 1], [5, 5], seed=3, dtype=dtype)
        c.q, c.k, c.v, c.states = (c.q * q).contiguous(), (c.k * k).contiguous(), (c.v * v).contiguous(), c.states * state
        c.scale = 1e-6 if q > 1 else 1.0
        c.check(*c.run(), what=(dtype, q))


def test_channels_and_tokens_of_different_size():
    for dtype in (BF, F16):
        c = Case(abi.linear_config(1, 1, 64, 128, dtype=dtype), [180], [5], seed=4, dtype=dtype, rate=(0.05, 0.05))
        c.v = (c.v * torch.logspace(-6, 6, 128, base=2, device="cuda")).to(dtype)
        c.k = (c.k * torch.logspace(-8, 5, 180, base=2, device="cuda")[:, None]).to(dtype)
        c.q = (c.q * torch.logspace(6, -6, 180, base=2, device="cuda")[:, None]).to(dtype)
        c.check(*c.run(), what=dtype)


def test_a_prompt_in_pieces_and_tokens_is_the_prompt():
    cfg = abi.linear_config(2, 4, 128, 128)
    whole = Case(cfg, [400], [0], seed=8)
    out, states = whole.run()
    whole.check(out, states)
    got, s = torch.empty_like(out), whole.states.clone()
    at = 0
    for n in (130, 1, 64, 5, 199, 1):
        c = Case(cfg, [n], [at], seed=8)
        c.slots, c.scale = whole.slots, whole.scale
        c.q, c.k, c.v, c.decay = (t[at:at + n] for t in (whole.q, whole.k, whole.v, whole.decay))
        c.run(states=s, out=got[at:at + n])
        at += n
    whole.check(got, s)


def test_padding_in_front_and_rows_behind():
    """Rows at negative positions give 0 and do not count; rows behind the last sequence stay untouched."""
    cfg = abi.linear_config(2, 2, 64, 128)
    for new, kv in (([5, 1, 3], [2, 0, 3]), ([200, 70, 1, 90], [100, 0, 1, 90]), ([130], [1])):
        c = Case(cfg, new, [0] * len(new), seed=len(new), behind=4)
        c.kv = kv
        c.check(*c.run(), what=new)


def test_values_that_are_not_finite_stay_where_they_belong():
    """A value of one token makes its own channel not finite from that token on, and nothing else; a key its whole head, from
    that token on."""
    for n in (6, 150):
        cfg = abi.linear_config(2, 2, 64, 64)
        c = Case(cfg, [n, n], [0, 0], seed=n)
        clean, clean_states = c.run()
        at = n // 2 + 1
        c.v = c.v.clone()
        c.v[at, 3] = math.inf
        c.v[at + 1, 64 + 5] = math.nan
        c.k = c.k.clone()
        c.k[n + at, 1] = math.nan
        out, states = c.run()
        bad = torch.zeros_like(out, dtype=torch.bool)
        bad[at:n, 3] = True
        bad[at + 1:n, 69] = True
        bad[n + at:, :64] = True
        assert torch.equal(torch.isfinite(out), ~bad), n
        assert torch.equal(out[~bad], clean[~bad])
        s, cs = states[c.slots[0]], clean_states[c.slots[0]]
        assert not bool(torch.isfinite(s[0, :, 3]).any()) and not bool(torch.isfinite(s[1, :, 5]).any())
        s[0, :, 3], s[1, :, 5] = cs[0, :, 3], cs[1, :, 5]
        assert torch.equal(s, cs)
        s = states[c.slots[1]]
        assert torch.equal(s[1], clean_states[c.slots[1]][1]) and not bool(torch.isfinite(s[0, 1]).any())


def test_other_sequences_rows_do_not_matter():
    """The last chunk of a run reads into the next run's rows: what these hold does not show."""
    cfg = abi.linear_config(1, 2, 128, 64)
    c = Case(cfg, [100, 90, 30], [0, 4, 4], seed=2)
    out, states = c.run()
    c.q, c.k, c.v, c.decay = c.q.clone(), c.k.clone(), c.v.clone(), c.decay.clone()
    for t in (c.q, c.k, c.v):
        t[100:190] = math.nan
    out2, states2 = c.run()
    for rows, slot in ((slice(0, 100), 0), (slice(190, 220), 2)):
        assert torch.equal(out[rows], out2[rows]) and torch.equal(states[c.slots[slot]], states2[c.slots[slot]])


@pytest.mark.parametrize("n", [1, 100])
def test_reported_mistakes(n):
    cfg = abi.linear_config(1, 2, 64, 64)
    for slot in (-1, 4, 2 ** 31 - 1):
        c = Case(cfg, [n, n], [3, 3], seed=1, n_slots=4)
        good = c.slots[1]
        c.slots[0] = slot
        out, states = c.run(status=1)
        others = [s for s in range(4) if s != good]
        assert torch.equal(states[others], c.states[others])
        c.slots[0] = others[0]
        _, want, _, size = c.want()
        assert float(((states[good].cpu().double() - want[good]).abs() - 1e-3 * size[good]).max()) <= 0
    c = Case(cfg, [n], [3], seed=1)
    c.decay[n // 2, 1] = 0.5
    out, states = c.run(status=1)
    c.decay[n // 2, 1] = 0.0
    c.check(out, states)
    c.decay[n // 2, 0] = math.nan
    out, states = c.run(status=1)
    c.decay[n // 2, 0] = 0.0
    c.check(out, states)
    # a range of rows outside the batch counts as none
    c = Case(cfg, [n, n], [3, 3], seed=5)
    c.starts = [0, n, 2 * n + 9]
    out, states = c.run(status=1)
    assert bool((out[n:] == 7.0).all()) and torch.equal(states[c.slots[1]], c.states[c.slots[1]])


def test_streams_graphs_and_repeats():
    cfg = abi.linear_config(2, 4, 128, 128)
    for new, past in (([1, 1, 1], [3, 0, 9]), ([200, 1, 70], [0, 5, 64]), ([1500], [10])):
        c = Case(cfg, new, past, seed=len(new))
        out, states = c.run()
        again = c.run()
        assert torch.equal(out, again[0]) and torch.equal(states, again[1])
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        o2, s2 = torch.full_like(out, 7.0), c.states.clone()
        ws = abi.alloc_linear_workspace(cfg, len(new), c.T)
        torch.cuda.synchronize()
        c.run(states=s2, out=o2, ws=ws, stream=s)
        s.synchronize()
        assert torch.equal(out, o2) and torch.equal(states, s2)
        # captured: the lengths are read when it is replayed
        batch, pool = c.batch(), abi.StatePool(cfg, s2)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            abi.moe_linear_attention(cfg, pool, batch, c.q, c.k, c.v, c.decay, o2, ws, scale=c.scale)
        for _ in range(2):
            s2.copy_(c.states)
            graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, o2) and torch.equal(states, s2)
        batch.kv_len.copy_(torch.tensor(c.new, dtype=torch.int32))
        s2.copy_(c.states)
        graph.replay()
        torch.cuda.synchronize()
        c.kv = list(c.new)
        c.check(o2, s2)
        assert abi.moe_check_status(ws) == 0


def test_two_calls_at_once():
    """Two streams, each with its workspace and pool."""
    cfg = abi.linear_config(2, 4, 128, 128)
    cases = [Case(cfg, [900, 1], [0, 3], seed=s) for s in (1, 2)]
    want = [c.run() for c in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    args = [(c.states.clone(), torch.full_like(w[0], 7.0), abi.alloc_linear_workspace(cfg, 2, c.T)) for c, w in zip(cases, want)]
    torch.cuda.synchronize()
    batches = [c.batch() for c in cases]
    torch.cuda.synchronize()
    for _ in range(3):
        for c, b, s, (st, o, ws) in zip(cases, batches, streams, args):
            with torch.cuda.stream(s):
                st.copy_(c.states)
                abi.moe_linear_attention(cfg, abi.StatePool(cfg, st), b, c.q, c.k, c.v, c.decay, o, ws, scale=c.scale)
    torch.cuda.synchronize()
    for (o, s), (st, got, _) in zip(want, args):
        assert torch.equal(o, got) and torch.equal(s, st)


def test_no_tokens_is_a_no_op():
    cfg = abi.linear_config(1, 1, 64, 64)
    c = Case(cfg, [0, 0], [3, 0], seed=1)
    out, states = c.run()
    assert torch.equal(states, c.states)
