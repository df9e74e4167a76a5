"""moe_linear_attention for a long run among sequences without new tokens (conversations that wait): it goes chunk by chunk,
as it does alone, whether the caller says how long the runs are or not."""
import pytest
import torch

from sparse_moe_router_gb300 import abi

from test_gpu_linear import Case

pytestmark = pytest.mark.gpu


def _chunk_launches(c, longest=0):
    abi.timing_read("linear_chunks")
    plain = c.batch
    c.batch = lambda: _told(plain(), longest)
    abi.timing_enable(True)
    out = c.run()
    abi.timing_enable(False)
    return abi.timing_read("linear_chunks")[0], out


def _told(batch, longest):
    batch.c.longest = longest
    return batch


@pytest.mark.parametrize("B,at,n", [(256, 17, 300), (1000, 999, 1050), (100, 0, 150), (300, 299, 200)])
@pytest.mark.parametrize("known", [False, True])
def test_a_run_among_empty_sequences(B, at, n, known):
    new = [0] * B
    new[at] = n
    c = Case(abi.linear_config(1, 2, 64, 64), new, [3] * B, seed=n)
    launches, got = _chunk_launches(c, n if known else 0)
    assert launches == 1
    c.check(*got)


@pytest.mark.parametrize("longest", [0, 170])
def test_a_run_among_single_tokens_and_empty_sequences(longest):
    new = [i % 2 for i in range(400)]
    new[30] = 170
    c = Case(abi.linear_config(1, 4, 64, 64), new, [i % 3 for i in range(400)], seed=2)
    launches, got = _chunk_launches(c, longest)
    assert launches == 1
    c.check(*got)


@pytest.mark.parametrize("B,longest", [(48, 0), (48, 1), (300, 1)])
def test_single_tokens_alone_need_no_chunks(B, longest):
    c = Case(abi.linear_config(1, 4, 64, 64), [1] * B, [3] * B, seed=2)
    launches, got = _chunk_launches(c, longest)
    assert launches == 0
    c.check(*got)


def test_single_tokens_of_which_the_caller_says_nothing():
    c = Case(abi.linear_config(2, 4, 64, 128), [1] * 200, [i % 2 for i in range(200)], seed=4)
    c.check(*_chunk_launches(c)[1])


@pytest.mark.parametrize("longest", [1, 20, 5000])
def test_a_caller_who_is_wrong_gets_the_same(longest):
    """Too short or too long: every token counts all the same."""
    new = [0, 150, 1, 9, 64, 0, 1]
    c = Case(abi.linear_config(2, 2, 64, 64), new, [3] * 7, seed=5)
    c.check(*_chunk_launches(c, longest)[1])
    c = Case(abi.linear_config(2, 2, 64, 64), [150], [3], seed=6)
    c.check(*_chunk_launches(c, longest)[1])
