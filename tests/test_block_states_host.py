"""Which sequences a step hands to the recurrent layers, without a GPU: those with new tokens, and how long the longest run is."""
import pytest
import torch

from sparse_moe_router_gb300 import abi, block


class Handed:
    def __init__(self, q_start, kv_len, slots, n_tokens, longest=0):
        self.q_start, self.kv_len, self.slots, self.n_tokens, self.longest = q_start.tolist(), kv_len.tolist(), slots.tolist(), n_tokens, longest
        assert all(t.dtype is torch.int32 and t.is_contiguous() for t in (q_start, kv_len, slots))


class HandedKV:
    def __init__(self, q_start, kv_len, page_table, n_tokens):
        self.q_start, self.kv_len, self.n_tokens = q_start, kv_len, n_tokens


def stack(monkeypatch, linear=True, seqs=4):
    monkeypatch.setattr(abi, "StateBatch", Handed)
    monkeypatch.setattr(abi, "KVBatch", HandedKV)
    m = object.__new__(block.DecoderLayers)
    m.pages = block.Pages(seqs, 512, 16, 100, device="cpu")
    m.max_tokens, m.rope, m.slots = 400, torch.zeros(512, 8), torch.arange(seqs, dtype=torch.int32)
    m.linear = abi.linear_config(2, 2, 64, 64) if linear else None
    return m


@pytest.mark.parametrize("new,starts,lens,slots,longest", [
    ([0, 300, 0, 0], [0, 300], [305], [1], 300), ([1, 1, 1, 1], [0, 1, 2, 3, 4], [1, 6, 1, 1], [0, 1, 2, 3], 1),
    ([0, 2, 0, 7], [0, 2, 9], [7, 7], [1, 3], 7), ([0, 0, 0, 0], [0], [], [], 0), ([30, 40, 50, 60], [0, 30, 70, 120, 180], [30, 45, 50, 60], [0, 1, 2, 3], 60)])
def test_sequences_without_new_tokens_are_left_out(monkeypatch, new, starts, lens, slots, longest):
    m = stack(monkeypatch)
    m.pages.grow(1, 5)
    b = m.batch(new)
    s = b.states
    assert (s.q_start, s.kv_len, s.slots, s.n_tokens, s.longest) == (starts, lens, slots, sum(new), longest)
    assert len(b.kv_len) == 4  # attention's batch keeps them


def test_a_stack_without_recurrent_layers_has_no_states(monkeypatch):
    assert not hasattr(stack(monkeypatch, linear=False).batch([1, 0, 0, 2]), "states")


def test_a_batch_of_which_only_the_device_knows(monkeypatch):
    """All sequences are handed over, and nothing is said of the longest run."""
    m = stack(monkeypatch)
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32)  # noqa: E731
    s = m.with_states(HandedKV(i32(0, 1, 1, 5, 5), i32(3, 4, 5, 6), m.pages.table, 5)).states
    assert (s.q_start, s.kv_len, s.slots, s.n_tokens, s.longest) == ([0, 1, 1, 5, 5], [3, 4, 5, 6], [0, 1, 2, 3], 5, 0)
