"""Entry points called from a thread that has made no CUDA call yet: what the library asks of the driver works there as it
does in the program's first thread."""
import threading

import pytest
import torch

from sparse_moe_router_gb300 import abi, inputs

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


def _in_a_new_thread(call):
    stream, errors = torch.cuda.Stream(), []

    def body():
        try:
            call(stream)
        except Exception as e:  # noqa: BLE001
            errors.append(e)

    torch.cuda.synchronize()
    t = threading.Thread(target=body)
    t.start()
    t.join()
    torch.cuda.synchronize()
    assert not errors, errors


def _rand(*shape):
    return torch.randn(*shape, device="cuda", generator=torch.Generator(device="cuda").manual_seed(1)).to(BF)


@pytest.mark.parametrize("T,N", [(1, 64), (48, 1024), (700, 1024), (700, 32)])
def test_project(T, N):
    x, w = _rand(T, 512), _rand(N, 512)
    cfg = abi.project_config(512, N)
    ws, want, got = abi.alloc_project_workspace(cfg, T), torch.empty(T, N, dtype=BF, device="cuda"), torch.empty(T, N, dtype=BF, device="cuda")
    abi.moe_project(cfg, x, w, want, ws)
    _in_a_new_thread(lambda s: abi.moe_project(cfg, x, w, got, ws, stream=s))
    assert torch.equal(got, want)


@pytest.mark.parametrize("T", [3, 200])
def test_linear_attention(T):
    cfg = abi.linear_config(1, 2, 64, 64)
    q, k, v = _rand(T, 64), _rand(T, 64), _rand(T, 128)
    i32 = lambda *a: torch.tensor(a, dtype=torch.int32, device="cuda")  # noqa: E731
    pools, outs = [abi.StatePool.alloc(cfg, 1) for _ in "ab"], [torch.empty_like(v) for _ in "ab"]
    batch, ws = abi.StateBatch(i32(0, T), i32(T), i32(0), T), abi.alloc_linear_workspace(cfg, 1, T)
    call = lambda i, s: abi.moe_linear_attention(cfg, pools[i], batch, q, k, v, None, outs[i], ws, stream=s)  # noqa: E731
    call(0, None)
    _in_a_new_thread(lambda s: call(1, s))
    assert torch.equal(outs[0], outs[1]) and torch.equal(pools[0].states, pools[1].states)


def test_moe_layer():
    wl = inputs.WORKLOADS["tiny"]
    layers, x = inputs.make(wl, device="cuda:0")
    cfg, w = abi.config_of(wl.shape), abi.weights(layers[0])
    ws, want, got = abi.alloc_workspace(cfg, wl.T), torch.empty_like(x), torch.empty_like(x)
    abi.moe_forward(cfg, w, x, wl.T, want, None, ws)
    _in_a_new_thread(lambda s: abi.moe_forward(cfg, w, x, wl.T, got, None, ws, stream=s))
    assert torch.equal(got, want)
