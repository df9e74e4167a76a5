"""What a decoder stack checks before it takes pages, without a GPU: a step that is refused leaves the pages, the
lengths and the pool as they were."""
import pytest
import torch

from sparse_moe_router_gb300 import abi, block


def stack(seqs=3, max_len=64, n_pages=8, max_tokens=50, hidden=16):
    """DecoderLayers with what a step's checks read, and nothing on a device."""
    m = object.__new__(block.DecoderLayers)
    m.moe = abi.config(hidden=hidden, n_experts=16, top_k=4, inter=128, shared_inter=128)
    m.pages = block.Pages(seqs, max_len, 16, n_pages, device="cpu")
    m.max_tokens, m.rope = max_tokens, torch.zeros(max_len, 8)
    return m


def state(p):
    return list(p.lens), [list(x) for x in p.pages], list(p.free), p.table.clone()


def unchanged(p, before):
    lens, pages, free, table = before
    return p.lens == lens and p.pages == pages and p.free == free and torch.equal(p.table, table)


@pytest.mark.parametrize("new,error", [([20, 20, 11], ValueError), ([10, 10], ValueError), ([1, 1, 1, 1], ValueError), ([5, -1, 5], ValueError),
                                       ([1, 1, 48], RuntimeError), ([30, 1, 17], RuntimeError), ([1, 47, 1], RuntimeError)])
def test_a_refused_step_takes_nothing(new, error):
    """Too many tokens, a wrong number of sequences, a negative count, a full table, a full pool: each found only
    after sequences that would have room."""
    m = stack()
    for seq, n in enumerate((20, 30, 17)):
        m.pages.grow(seq, n)  # 2 + 2 + 2 of the 8 pages
    before = state(m.pages)
    with pytest.raises(error):
        m.batch(new)
    assert unchanged(m.pages, before)


def test_a_refused_graph_step_takes_nothing():
    m = stack(seqs=2, n_pages=2)
    m.pages.grow(0, 5)
    m.pages.grow(1, 16)
    g = object.__new__(block.DecodeGraph)
    g.model, g.x = m, torch.zeros(2, 16, dtype=torch.bfloat16)
    before = state(m.pages)
    with pytest.raises(RuntimeError):
        g.step(g.x)  # sequence 1 needs a page that is not there
    assert unchanged(m.pages, before)


def test_lengths_end_at_max_len():
    """Not at the end of the page that holds it: the table of angles may end there."""
    p = block.Pages(2, 50, 16, 8, device="cpu")
    p.grow(0, 50)
    before = state(p)
    with pytest.raises(RuntimeError):
        p.grow(0, 1)
    with pytest.raises(RuntimeError):
        p.require([1, 1])
    with pytest.raises(RuntimeError):
        p.grow(1, 51)
    assert unchanged(p, before)
    p.require([0, 50])


def test_a_table_of_angles_shorter_than_the_sequences():
    moe = abi.config(hidden=16, n_experts=16, top_k=4, inter=128, shared_inter=128)
    pages = block.Pages(2, 50, 16, 8, device="cpu")
    with pytest.raises(ValueError, match="angles"):
        block.DecoderLayers(moe, abi.attn_config(8, 2, 64, 16, rotary_dim=32), [], pages, 50, torch.zeros(49, 32))


@pytest.mark.parametrize("shape", [(1, 16), (16,), (4, 16), (5, 8), (5, 1), (1, 5, 16)])
def test_rows_of_another_shape(shape):
    """One row would be broadcast to all tokens; nothing is taken."""
    m = stack()
    before = state(m.pages)
    with pytest.raises(ValueError, match="rows"):
        m.prefill(torch.zeros(shape, dtype=torch.bfloat16), [3, 0, 2])
    with pytest.raises(ValueError, match="rows"):
        m.decode(torch.zeros(shape, dtype=torch.bfloat16))
    g = object.__new__(block.DecodeGraph)
    g.model, g.x = m, torch.zeros(3, 16, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="rows"):
        g.step(torch.zeros(shape, dtype=torch.bfloat16))
    assert unchanged(m.pages, before)
