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
