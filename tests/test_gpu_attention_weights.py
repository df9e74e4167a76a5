"""moe_attention where one key holds nearly all of a row's weight and its value is 0: the output is made of
the others' weights, each far below the largest.  They are kept to fp16's 11 bits down to 2^-23 of it (and to
2^-34 at all): the bound of attention_bound with top = 2^9."""
import pytest
import torch

from sparse_moe_router_gb300 import abi

import attention_bound
import layer_ref as ref
from test_gpu_kv_append import Setup

pytestmark = pytest.mark.gpu


def sink(lens, QH, KH, D, P, dtype, logit, spread, seed=0):
    """Every sequence has the same pages.  Key 0 has the given logit for every row and value 0, the others normal
    logits of the given spread and values around 1."""
    gen = torch.Generator().manual_seed(seed)
    s = Setup([(1, max(kv for _, kv in lens))], QH, KH, D, P, dtype=dtype)
    s.T = sum(n for n, _ in lens)
    s.q_start = torch.tensor([0] + list(torch.tensor([n for n, _ in lens]).cumsum(0)), dtype=torch.int32)
    s.kv_len = torch.tensor([kv for _, kv in lens], dtype=torch.int32)
    s.table = s.table.expand(len(lens), -1).contiguous()
    first = int(s.table[0, 0])
    # q is 1 in the first dim and normal in the others, where key 0 is 0; the softmax scale is 1
    q = torch.randn(s.T, QH, D, generator=gen)
    q[..., 0] = 1
    k = torch.randn(s.n_pages, KH, P, D, generator=gen, dtype=torch.float64) * spread / D ** 0.5
    k[..., 0] = 0
    k[first, :, 0] = 0
    k[first, :, 0, 0] = logit
    v = 1 + 0.2 * torch.randn(s.n_pages, KH, P, D, generator=gen, dtype=torch.float64)
    v[first, :, 0] = 0
    for name, x in (("k", k), ("v", v)):
        scale = ref.pow2_scale(x.abs().amax(dim=(2, 3)))
        s.cache[name + "_codes"], s.cache[name + "_scale"] = ref.encode(x / scale[..., None, None]), scale.float()
    return s, q.to(dtype).cuda()


def run_scaled(s, q, scale):
    cache, batch, ws = s.device()
    out = torch.full((s.T, s.QH, s.cfg.head_dim), 9.0, dtype=q.dtype, device="cuda")
    lse = torch.full((s.T, s.QH), 9.0, device="cuda")
    abi.moe_attention(s.cfg, cache, batch, q, out, ws, lse=lse, softmax_scale=scale)
    assert abi.moe_check_status(ws) == 0
    return out, lse


CASES = {"prompt": [(600, 1500)], "piece": [(130, 9000)], "tokens": [(1, 640 + i % 9) for i in range(160)], "runs": [(3, 700)] * 60,
         "mixed": [(700, 1400), (1, 900), (300, 600)]}


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("QH,KH,D,P", [(8, 2, 128, 64), (8, 1, 64, 16), (16, 2, 256, 32)])
@pytest.mark.parametrize("logit,spread", [(4.0, 1.0), (12.0, 1.0), (18.0, 0.3), (20.0, 1.0)])
@pytest.mark.parametrize("lens", CASES.values(), ids=CASES)
def test_a_key_that_holds_most_of_the_weight(dtype, QH, KH, D, P, logit, spread, lens):
    s, q = sink(lens, QH, KH, D, P, dtype, logit, spread)
    out, lse = run_scaled(s, q, 1.0)
    attention_bound.check(s.cfg, s.cache, s.q_start, s.kv_len, s.table, q, out, lse, scale=1.0, top=512.0)


@pytest.mark.parametrize("lens", [[(600, 1500)], [(1, 700)] * 60], ids=["prompt", "tokens"])
@pytest.mark.parametrize("rise", [0.0, 0.01, 0.3, -0.3])
def test_flat_and_slowly_rising_rows(lens, rise):
    """All logits alike, or rising a little with every key, as far as the weights' upper end: nothing overflows."""
    s, q = sink(lens, 8, 2, 128, 64, torch.bfloat16, 0.0, 0.0)
    kv = max(k for _, k in lens)
    for j in range(kv):
        page, slot = int(s.table[0, j // 64]), j % 64
        x = torch.zeros(2, 128, dtype=torch.float64)
        x[:, 0] = rise * j
        s.cache["k_scale"][page] = 2.0
        s.cache["k_codes"][page, :, slot] = ref.encode(x / 2.0)
    out, lse = run_scaled(s, q, 1.0)
    attention_bound.check(s.cfg, s.cache, s.q_start, s.kv_len, s.table, q, out, lse, scale=1.0, top=512.0)
