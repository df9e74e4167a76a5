"""Recurrent layers of a stack in which most conversations wait: a prompt piece gives what it gives alone, and theirs stay as
they are."""
import pytest
import torch

from test_gpu_block_recurrent import make, rows

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("pieces", [[300], [200, 1, 150], [3, 66]])
def test_a_prompt_among_waiting_conversations(pieces):
    alone, among = make(recurrent=(0, 1), n_layers=2, seqs=1), make(recurrent=(0, 1), n_layers=2, seqs=200)
    x = rows(200, 4)
    among.prefill(x, [1] * 200)
    alone.prefill(x[130:131], [1])
    before = [s.states.clone() for s in among.states]
    first = among.states[0].states[130].clone()
    alone.states[0].states[0].copy_(first)
    alone.states[1].states[0].copy_(among.states[1].states[130])
    for n in pieces:
        x = rows(n, n)
        want = alone.prefill(x, [n]).clone()
        got = among.prefill(x, [0] * 130 + [n] + [0] * 69)
        assert torch.equal(got, want)
    for i in (0, 1):
        assert torch.equal(among.states[i].states[130], alone.states[i].states[0])
        left = [s for s in range(200) if s != 130]
        assert torch.equal(among.states[i].states[left], before[i][left])
    among.check()
    alone.check()
