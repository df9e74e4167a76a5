"""moe_block_norm where a block takes several rows one after another, the next under way meanwhile: one, two and
four chunks a thread.  Form and tolerance: test_gpu_block_norm."""
import pytest
import torch

from sparse_moe_router_gb300 import abi

import layer_ref as ref
from test_gpu_block_norm import _check, _make

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("T,H,gate,sigmoid,wide", [
    (3001, 2048, "element", True, 0), (6000, 1000, "token", True, 16), (2500, 4096, "channel", False, 0), (11000, 64, "none", False, 16),
    (650, 4096, "element", True, 0), (1300, 7168, "none", False, 0),
    (333, 16384, "channel", True, 0), (700, 8200, "element", False, 16), (401, 12288, "token", False, 0)])
@pytest.mark.parametrize("post,pre", [(True, True), (False, True), (True, False)])
def test_many_rows_a_block(dtype, T, H, gate, sigmoid, wide, post, pre):
    x, resid, g, w_post, w_pre = _make(T, H, dtype, gate, T + H, wide)
    w_post, w_pre = w_post if post else None, w_pre if pre else None
    cfg = abi.norm_config(H, dtype=dtype, gate=gate, sigmoid=sigmoid, eps=1e-5, residual_scale=0.75)
    out = torch.empty(T, H, dtype=dtype, device="cuda")
    y = torch.empty_like(out) if pre else None
    abi.moe_block_norm(cfg, x, resid, out, y, gate=g, w_post=w_post, w_pre=w_pre)
    r, n, rs, ns = ref.block_norm(x, resid, g, w_post, w_pre, 1e-5, 0.75, sigmoid)
    _check(out, r, rs, dtype, "resid_out")
    if pre:
        _check(y, n, ns, dtype, "y")
    # in place, where each row is read before it is written
    if pre and gate != "element":
        x2, r2 = x.clone(), resid.clone()
        abi.moe_block_norm(cfg, x2, r2, r2, x2, gate=g, w_post=w_post, w_pre=w_pre)
        assert torch.equal(r2, out) and torch.equal(x2, y)
