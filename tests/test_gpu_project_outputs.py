"""moe_project of one row with up to 2^20 outputs, and what a launch that the device refuses leaves behind."""
import pytest
import torch

from sparse_moe_router_gb300 import abi

import layer_ref
import mixer_ref as ref

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


def _make(K, N):
    """Weights whose rows repeat every 8 outputs."""
    gen = torch.Generator(device="cuda").manual_seed(K + N)
    x = torch.randn(1, K, device="cuda", generator=gen).to(BF)
    base = (torch.randn(8, K, device="cuda", generator=gen) * K ** -0.5).to(BF)
    return x, base, base.repeat(N // 8, 1)


def test_a_call_that_fails_leaves_no_error_to_the_next():
    """A launch that the device refuses is reported by its own call alone."""
    x, _, w = _make(4096, 1 << 20)
    cfg, small = abi.project_config(4096, 1 << 20), abi.project_config(4096, 8)
    ws = abi.alloc_project_workspace(cfg, 1)
    try:
        abi.moe_project(cfg, x, w, torch.empty(1, 1 << 20, dtype=BF, device="cuda"), ws)
    except abi.MoeError:
        pass
    y = torch.empty(1, 8, dtype=BF, device="cuda")
    abi.moe_project(small, torch.ones_like(x), torch.ones_like(w[:8]), y, ws)
    assert y.tolist() == [[4096.0] * 8]


@pytest.mark.parametrize("K,N", [(4096, 524280), (4096, 524288), (4096, 1 << 20), (8192, 524296), (8, 1 << 20), (1032, 1 << 20)])
def test_one_row_of_many_outputs(K, N):
    """On either side of 65,535 blocks of 8 outputs: every output is that of the 8 rows it repeats."""
    x, base, w = _make(K, N)
    cfg = abi.project_config(K, N)
    ws = abi.alloc_project_workspace(cfg, 1)
    y = torch.full((1, N), 7.0, dtype=BF, device="cuda")
    abi.moe_project(cfg, x, w, y, ws)
    assert abi.moe_check_status(ws) == 0
    want, size = ref.project(x, base, None, None, "none", 1.0)
    bound = layer_ref.HALF_STEP[BF] * want.abs() + 2 * ref.EPS32 * (K / 4 + 256) * size
    assert float(((y[:, :8].cpu().double() - want).abs() - bound).max()) <= 0
    assert torch.equal(y.view(N // 8, 8), y[:, :8].expand(N // 8, 8))
