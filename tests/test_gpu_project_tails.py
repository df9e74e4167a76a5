"""Sigmoid and SiLU of moe_project far below 0, where fp32 outputs show the result's own digits.

The arguments are exact (one input of 1 times z).  e^z with 2 ulp (4 half steps), its sum with 1 (1), the reciprocal (2), the
product with e^z (1), SiLU's with z (1) and the scale's (1): 10 half steps of fp32 relative to the result.  Among subnormals
4 and 1 half steps of 2^-149 for e^z and its product, times |z| <= 104, and 2 more."""
import pytest
import torch

from sparse_moe_router_gb300 import abi

import mixer_ref as ref

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("act", ["sigmoid", "silu"])
@pytest.mark.parametrize("T", [1, 3, 40, 700])
def test_far_below_zero(act, T):
    z = torch.cat([-torch.linspace(0, 104, 520), torch.linspace(0, 104, 512)]).to(torch.bfloat16).cuda()
    x, w = (torch.zeros(n, 8, dtype=torch.bfloat16, device="cuda") for n in (T, len(z)))
    x[:, 0], w[:, 0] = 1.0, z
    cfg = abi.project_config(8, len(z), out_dtype=torch.float32, act=act, scale=0.75)
    ws = abi.alloc_project_workspace(cfg, T)
    y = torch.empty(T, len(z), dtype=torch.float32, device="cuda")
    abi.moe_project(cfg, x, w, y, ws)
    assert abi.moe_check_status(ws) == 0
    want, _ = ref.project(x, w, None, None, act, 0.75)
    far = (y.cpu().double() - want).abs() - 10 * ref.EPS32 * want.abs() - 522 * 2.0 ** -150
    at = int(far.argmax()) % len(z)
    assert float(far.max()) <= 0, (float(z[at]), float(far.max()), float(want[0, at]))
