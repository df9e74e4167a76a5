"""CPU-only checks of the recurrent token mixer's entry points: configs, workspace sizes, the refusals that come before
any device work, and of the 64-bit forms the GPU tests compare with."""
import ctypes
import math

import pytest
import torch

from sparse_moe_router_gb300 import abi

import mixer_ref as ref

OK, INVALID, SMALL, UNSUPPORTED = 0, 1, 2, 3
A = 0x10000  # an aligned address that is never dereferenced: the checks fail or the call is empty


def _cfg(**kw):
    return abi.linear_config(**dict(dict(key_heads=4, value_heads=8, key_dim=128, value_dim=64), **kw))


def _linear(cfg=None, pool=None, batch=None, q=A, q_ld=512, k=A, k_ld=512, v=A, v_ld=512, decay=A, decay_ld=8, scale=1.0, out=A,
            out_ld=512, ws=A, ws_bytes=1 << 30):
    cfg = cfg or _cfg()
    b = abi._StateBatch(2, 5, A, A, A)
    for n, x in (batch or {}).items():
        setattr(b, n, x)
    p = abi._StatePool(A, 3)
    for n, x in (pool or {}).items():
        setattr(p, n, x)
    return abi.load().moe_linear_attention(ctypes.byref(cfg), ctypes.byref(p), ctypes.byref(b), q, q_ld, k, k_ld, v, v_ld, decay, decay_ld,
                                           scale, out, out_ld, ws, ws_bytes, None)


def test_linear_configs_and_workspace():
    assert abi.linear_workspace_size(_cfg(), 4, 100) >= 256
    for bad in (dict(key_heads=0), dict(value_heads=0), dict(value_heads=6), dict(key_dim=96), dict(key_dim=256), dict(value_dim=32),
                dict(value_dim=512), dict(value_heads=2048), dict(key_heads=-4)):
        assert abi.linear_workspace_size(_cfg(**bad), 4, 100) == 0, bad
    c = _cfg()
    c.dtype = 2
    assert abi.linear_workspace_size(c, 4, 100) == 0
    assert abi.linear_workspace_size(_cfg(), -1, 1) == 0 and abi.linear_workspace_size(_cfg(), 1, -1) == 0
    assert abi.linear_workspace_size(_cfg(), 1 << 17, 1) == 0 and abi.linear_workspace_size(_cfg(), 1, 1 << 23) == 0
    assert abi.load().moe_linear_workspace_size(None, 1, 1) == 0
    with pytest.raises(abi.MoeError):
        abi.alloc_linear_workspace(_cfg(key_dim=96), 1, 1, device="cpu")


def test_linear_refusals():
    assert _linear(cfg=_cfg(value_heads=6)) == INVALID and _linear(cfg=_cfg(key_dim=96)) == UNSUPPORTED
    for kw in (dict(n_seqs=-1), dict(n_tokens=-1), dict(n_seqs=0), dict(q_start=None), dict(kv_len=None), dict(slots=None)):
        assert _linear(batch=kw) == INVALID, kw
    for kw in (dict(n_seqs=70000), dict(n_tokens=1 << 23)):
        assert _linear(batch=kw) == UNSUPPORTED, kw
    for kw in (dict(states=None), dict(states=A + 8), dict(n_slots=0), dict(n_slots=-1)):
        assert _linear(pool=kw) == INVALID, kw
    for kw in (dict(q=None), dict(k=None), dict(v=None), dict(out=None), dict(q=A + 8), dict(k=A + 2), dict(q_ld=504), dict(k_ld=516),
               dict(v_ld=-512), dict(out_ld=0), dict(decay=A + 2), dict(decay_ld=7), dict(decay_ld=-8), dict(scale=math.nan),
               dict(scale=math.inf)):
        assert _linear(**kw) == INVALID, kw
    assert _linear(ws=None) == INVALID and _linear(ws=A + 16) == INVALID
    assert _linear(ws_bytes=abi.linear_workspace_size(_cfg(), 2, 5) - 1) == SMALL
    # no new tokens: nothing to do, whatever the pointers
    assert _linear(batch=dict(n_tokens=0, q_start=None), pool=dict(states=None, n_slots=0), q=None, ws=None) == OK
    L = abi.load()
    assert L.moe_linear_attention(None, None, None, A, 8, A, 8, A, 8, None, 0, 1.0, A, 8, A, 256, None) == INVALID


def test_head_norm_refusals():
    L = abi.load()

    def call(x=A, x_ld=512, weight=A, gate=None, gate_ld=0, y=A, y_ld=512, T=3, fields=None, **cfg):
        c = abi.head_norm_config(**dict(dict(heads=4, dim=128), **cfg))
        for n, v in (fields or {}).items():
            setattr(c, n, v)
        return L.moe_head_norm(ctypes.byref(c), x, x_ld, weight, gate, gate_ld, y, y_ld, T, None)

    assert call(T=0, x=None, y=None) == OK and call(T=-1) == INVALID
    assert L.moe_head_norm(None, A, 512, None, None, 0, A, 512, 1, None) == INVALID
    for kw in (dict(dim=100), dict(dim=1032), dict(heads=1024)):
        assert call(**kw) == UNSUPPORTED, kw
    for kw in (dict(heads=0), dict(dim=0), dict(eps=-1.0), dict(eps=math.nan), dict(fields=dict(dtype=2)), dict(fields=dict(gate=3)), dict(x=None),
               dict(y=None), dict(x=A + 8), dict(x_ld=504), dict(y_ld=513), dict(weight=A + 4), dict(gate=A), dict(gate="silu")):
        if kw.get("gate") == "silu":  # a gate is asked for and none given
            assert call(fields=dict(gate=2)) == INVALID
        else:
            assert call(**kw) == INVALID, kw
    for kw in (dict(gate=A, gate_ld=504), dict(gate=A + 8, gate_ld=512)):
        assert call(fields=dict(gate=1), **kw) == INVALID, kw


def test_project_refusals():
    L = abi.load()

    def call(T=3, io=None, fields=None, ws=A, ws_bytes=1 << 30, drop_io=False, **cfg):
        c = abi.project_config(**dict(dict(inputs=256, outputs=64), **cfg))
        for n, v in (fields or {}).items():
            setattr(c, n, v)
        d = abi.ProjectIO(A, A, A, A, A, 256, 256, 64, 64)
        for n, v in (io or {}).items():
            setattr(d, n, v)
        return L.moe_project(ctypes.byref(c), None if drop_io else ctypes.byref(d), T, ws, ws_bytes, None)

    assert call(T=0, drop_io=True) == OK and call(T=-1) == INVALID and call(drop_io=True) == INVALID
    assert call(T=(1 << 30) + 1) == UNSUPPORTED
    assert L.moe_project(None, None, 1, A, 256, None) == INVALID
    for kw in (dict(inputs=252), dict(outputs=60), dict(inputs=65544), dict(outputs=(1 << 20) + 8)):
        assert call(**kw) == UNSUPPORTED, kw
        assert abi.project_workspace_size(abi.project_config(**dict(dict(inputs=256, outputs=64), **kw)), 4) == 0
    for kw in (dict(inputs=0), dict(outputs=-8), dict(scale=math.inf), dict(fields=dict(act=6)), dict(fields=dict(act=-1)),
               dict(fields=dict(dtype=2)), dict(fields=dict(out_f32=2)), dict(ws=None), dict(ws=A + 128)):
        assert call(**kw) == INVALID, kw
    for kw in (dict(x=None), dict(w=None), dict(y=None), dict(x=A + 8), dict(w=A + 2), dict(y=A + 4), dict(bias=A + 2), dict(resid=A + 8),
               dict(x_ld=248), dict(w_ld=260), dict(y_ld=56), dict(resid_ld=0)):
        assert call(io=kw) == INVALID, kw
    c = abi.project_config(256, 64)
    assert call(ws_bytes=abi.project_workspace_size(c, 3) - 1) == SMALL
    assert abi.project_workspace_size(c, -1) == 0
    with pytest.raises(abi.MoeError):
        abi.alloc_project_workspace(abi.project_config(250, 64), 1, device="cpu")


def test_binding_refuses_host_tensors_shapes_and_types():
    x = torch.zeros(2, 256, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        abi.moe_head_norm(abi.head_norm_config(2, 128), x, x)
    with pytest.raises(ValueError):
        abi.moe_project(abi.project_config(256, 64), x, x, x, x)
    with pytest.raises(ValueError):
        abi.StatePool.alloc(_cfg(), 2, device="cpu")
    with pytest.raises(ValueError):
        abi.project_config(256, 64, dtype=torch.bfloat16, out_dtype=torch.float16)
    with pytest.raises(KeyError):
        abi.linear_config(4, 4, 64, 64, dtype=torch.float32)
    with pytest.raises(KeyError):
        abi.project_config(8, 8, act="tanh")


@pytest.mark.parametrize("other", [dict(value_heads=16), dict(key_dim=64), dict(value_dim=128)])
def test_a_pool_of_another_layout(other):
    pool = object.__new__(abi.StatePool)
    pool.layout = (8, 128, 64)
    pool.check(_cfg())
    with pytest.raises(ValueError, match="pool"):
        abi.moe_linear_attention(_cfg(**other), pool, None, None, None, None, None, None, None)


# ------------------------------------------------------------------------- the 64-bit forms --

def test_reference_linear_attention_by_hand():
    cfg = abi.linear_config(1, 2, 64, 64)
    q = torch.zeros(3, 64)
    k = torch.zeros(3, 64)
    v = torch.ones(3, 128)
    q[:, 0] = 1.0
    k[:, 0] = torch.tensor([1.0, 2.0, 4.0])
    states = torch.ones(2, 2, 64, 64)
    decay = torch.tensor([math.log(0.5), 0.0], dtype=torch.float64)
    # head 0 halves before every token; the sequence begins at position 0, its slot holds ones that do not count
    out, new, _, size = ref.linear_attention(cfg, states, [0, 3], [3], [1], q, k, v, decay, 2.0)
    assert (out[:, 0, 0] - torch.tensor([2.0, 5.0, 10.5])).abs().max() < 1e-12 and out[:, 1, 5].tolist() == [2.0, 6.0, 14.0]
    assert abs(float(new[1, 0, 0, 0]) - 5.25) < 1e-12 and torch.equal(new[0], states[0].double()) and float(new[1, 0, 1, 0]) == 0
    # one past token: the slot counts
    out, new, _, _ = ref.linear_attention(cfg, states, [0, 3], [4], [1], q, k, v, decay, 2.0)
    assert abs(float(out[0, 0, 0]) - 3.0) < 1e-12 and abs(float(new[1, 1, 7, 0]) - 1.0) < 1e-12
    # two of three rows are padding
    out, new, _, _ = ref.linear_attention(cfg, states, [0, 3], [1], [0], q, k, v, decay, 2.0)
    assert out[:, 1, 0].tolist() == [0.0, 0.0, 8.0] and float(new[0, 1, 0, 0]) == 4.0


def test_reference_head_norm_and_project_by_hand():
    x = torch.tensor([[3.0, 4.0] + [0.0] * 6, [1.0] * 8])
    y = ref.head_norm(x, None, None, 1, 8, False, "none", 0.0)
    assert abs(float(y[0, 0]) - 3 / math.sqrt(25 / 8)) < 1e-12 and abs(float(y[1, 3]) - 1) < 1e-12
    assert float(ref.head_norm(x, None, None, 1, 8, True, "none", 1e-6)[1].abs().max()) == 0
    y, size = ref.project(torch.tensor([[1.0, -2.0]]), torch.tensor([[3.0, 1.0]]), torch.tensor([0.5]), torch.tensor([[10.0]]), "relu", 2.0)
    assert float(y) == 13.0 and float(size) == 5.5
