"""moe_kv_append at its edges."""
import pytest
import torch

from sparse_moe_router_gb300 import abi

from test_gpu_kv_append import Setup

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("used", [0, 1, 40])
@pytest.mark.parametrize("seqs", [1, 3])
def test_rows_behind_the_last_sequence_are_no_error(used, seqs):
    """A batch held for more tokens than its sequences have: the rows behind them give 0 and reach no page, and
    the status word stays clear, as moe_attention leaves it."""
    s = Setup([(40, 100)] + [(0, 9)] * (seqs - 1), 4, 2, 64, 16, 64)
    s.q_start[1:] = used
    cache, batch, ws = s.device()
    before = {k: v.clone() for k, v in s.cache.items()}
    got = s.append(cache, batch, ws)
    assert abi.moe_check_status(ws) == 0
    assert not got[used:].any()
    s.check(cache, got, s.want())
    if used == 0:
        assert all(torch.equal(getattr(cache, k).cpu(), v) for k, v in before.items())


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("inter", [False, True])
def test_infinities_under_a_rotation(dtype, inter):
    """An infinite key turns into infinities of the signs that the formula gives, stored as +-448 of the largest
    scale; where it gives inf - inf or inf * 0 (position 0: a sine of 0), NaN, stored as 0."""
    s = Setup([(20, 30), (3, 3)], 2, 2, 64, 16, 64, inter, dtype, strided=False)
    s.qkv[3, 2, 5] = float("inf")
    s.qkv[4, 3, 40] = float("-inf")
    s.qkv[5, 2, 6], s.qkv[5, 2, 38 if not inter else 7] = float("inf"), float("inf")
    s.qkv[20, 2, 9] = float("inf")   # at position 0
    s.qkv[21, 3, 9] = float("nan")
    cache, batch, ws = s.device()
    got = s.append(cache, batch, ws)
    s.check(cache, got, s.want())
    assert abi.moe_check_status(ws) == 1
