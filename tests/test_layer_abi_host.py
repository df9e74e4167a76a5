"""CPU-only checks of the decoder layer's entry points: configs, workspace sizes and the refusals that
come before any device work, and of the plain 64-bit forms the GPU tests compare with."""
import ctypes
import math

import pytest
import torch

from sparse_moe_router_gb300 import abi

import layer_ref as ref

OK, INVALID, SMALL, UNSUPPORTED = 0, 1, 2, 3
A = 0x10000  # an aligned address that is never dereferenced: the checks fail or the call is empty


def _attn(**kw):
    d = dict(q_heads=16, kv_heads=2, head_dim=128, page_size=64)
    d.update(kw)
    return abi.attn_config(**d)


def _cache(n_pages=4, **kw):
    c = abi._KVCache(A, A, A, A, n_pages)
    for k, v in kw.items():
        setattr(c, k, v)
    return c


def _batch(**kw):
    b = abi._KVBatch(2, 5, 3, A, A, A)
    for k, v in kw.items():
        setattr(b, k, v)
    return b


def test_workspace_size_and_attn_configs():
    size = abi.attn_workspace_size(_attn(), 4, 100)
    assert size > 256 and size % 4 == 0
    assert abi.attn_workspace_size(_attn(head_dim=256), 4, 100) > 256
    for bad in (dict(q_heads=0), dict(kv_heads=0), dict(q_heads=15), dict(rotary_dim=-16), dict(rotary_dim=144),
                dict(head_dim=96), dict(page_size=48), dict(page_size=256), dict(rotary_dim=24),
                dict(q_heads=258), dict(kv_heads=2048, q_heads=2048)):
        assert abi.attn_workspace_size(_attn(**bad), 4, 100) == 0, bad
    c = _attn()
    c.dtype = 5
    assert abi.attn_workspace_size(c, 1, 1) == 0
    c = _attn()
    c.interleaved = 2
    assert abi.attn_workspace_size(c, 1, 1) == 0
    assert abi.attn_workspace_size(_attn(), -1, 1) == 0 and abi.attn_workspace_size(_attn(), 1, -1) == 0
    assert abi.load().moe_attn_workspace_size(None, 1, 1) == 0
    with pytest.raises(abi.MoeError):
        abi.alloc_attn_workspace(_attn(head_dim=96), 1, 1, device="cpu")


def _attention(cfg=None, cache=None, batch=None, q=A, q_ld=2048, scale=0.1, causal=1, window=0, out=A, out_ld=2048, lse=None,
               ws=A, ws_bytes=1 << 30):
    cfg = cfg or _attn()
    return abi.load().moe_attention(ctypes.byref(cfg), ctypes.byref(cache or _cache()), ctypes.byref(batch or _batch()), q, q_ld,
                                    scale, causal, window, out, out_ld, lse, ws, ws_bytes, None)


def _append(cfg=None, cache=None, batch=None, q=A, q_ld=2048, k=A, k_ld=256, v=A, v_ld=256, rope=A, rows=10, q_out=A,
            q_out_ld=2048, ws=A, ws_bytes=1 << 30):
    cfg = cfg or _attn()
    return abi.load().moe_kv_append(ctypes.byref(cfg), ctypes.byref(cache or _cache()), ctypes.byref(batch or _batch()), q, q_ld,
                                    k, k_ld, v, v_ld, rope, rows, q_out, q_out_ld, ws, ws_bytes, None)


@pytest.mark.parametrize("call", [_attention, _append])
def test_shared_refusals(call):
    assert call(cfg=_attn(head_dim=96)) == UNSUPPORTED
    assert call(cfg=_attn(q_heads=3)) == INVALID
    for kw in (dict(n_seqs=-1), dict(n_tokens=-1), dict(max_pages=-1), dict(n_seqs=0), dict(q_start=None), dict(kv_len=None),
               dict(page_table=None)):
        assert call(batch=_batch(**kw)) == INVALID, kw
    for kw in (dict(n_seqs=70000), dict(n_tokens=1 << 23), dict(max_pages=1 << 25)):
        assert call(batch=_batch(**kw)) == UNSUPPORTED, kw
    for kw in (dict(n_pages=0), dict(n_pages=-1), dict(k_codes=None), dict(v_codes=A + 8), dict(k_scale=None), dict(v_scale=None)):
        assert call(cache=_cache(**kw)) == INVALID, kw
    assert call(ws=None) == INVALID and call(ws=A + 16) == INVALID
    assert call(ws_bytes=abi.attn_workspace_size(_attn(), 2, 5) - 1) == SMALL
    # no new tokens: nothing to do, whatever the pointers
    assert call(batch=_batch(n_tokens=0)) == OK
    empty = abi._KVBatch(0, 0, 0, None, None, None)
    assert call(batch=empty, cache=abi._KVCache(None, None, None, None, 0), ws=None) == OK


def test_attention_refusals():
    for kw in (dict(q=None), dict(out=None), dict(q=A + 8), dict(out=A + 2), dict(q_ld=2040), dict(out_ld=2052), dict(q_ld=-2048),
               dict(scale=0.0), dict(scale=-1.0), dict(scale=math.nan), dict(scale=math.inf), dict(window=-1), dict(lse=A + 2)):
        assert _attention(**kw) == INVALID, kw


def test_append_refusals():
    for kw in (dict(k=None), dict(v=None), dict(k=A + 8), dict(k_ld=248), dict(v_ld=260), dict(q=None), dict(q_out=None),
               dict(q_ld=100), dict(q_out_ld=2049), dict(rope=None), dict(rope=A + 4), dict(rows=0), dict(rows=-3)):
        assert _append(**kw) == INVALID, kw


def test_block_norm_refusals():
    L = abi.load()

    def call(T=4, io=None, drop_io=False, **cfg):
        c = abi.norm_config(**dict(dict(hidden=256), **cfg))
        d = abi.NormIO(x=A, resid=A, w_post=A, w_pre=A, resid_out=A, y=A, x_ld=256, resid_ld=256, resid_out_ld=256, y_ld=256)
        for k, v in (io or {}).items():
            setattr(d, k, v)
        return L.moe_block_norm(ctypes.byref(c), None if drop_io else ctypes.byref(d), T, None)

    assert call(T=0) == OK and call(T=0, drop_io=True) == OK
    assert call(T=-1) == INVALID and call(drop_io=True) == INVALID
    assert L.moe_block_norm(None, None, 4, None) == INVALID
    assert call(hidden=260) == UNSUPPORTED and call(hidden=16392) == UNSUPPORTED and call(hidden=0) == INVALID
    assert call(eps=-1.0) == INVALID and call(eps=math.nan) == INVALID and call(residual_scale=math.inf) == INVALID
    for kw in (dict(x=None, resid=None), dict(x=None), dict(resid_out=None, y=None), dict(w_pre=None), dict(x=A + 8), dict(x_ld=248),
               dict(resid_ld=257), dict(y_ld=0), dict(resid_out=A + 4), dict(w_post=A + 8), dict(w_pre=A + 2), dict(gate=A)):
        assert call(io=kw) == INVALID, kw
    for gate in ("channel", "token", "element"):
        assert call(gate=gate) == INVALID, gate                       # no gate tensor
    assert call(gate="channel", io=dict(gate=A + 2)) == INVALID
    assert call(gate="element", io=dict(gate=A, gate_ld=8)) == INVALID
    assert call(gate="token", io=dict(gate=A + 1, gate_ld=1)) == INVALID
    assert call(gate="token", io=dict(gate=A + 2, gate_ld=0)) == INVALID
    c = abi.norm_config(256)
    c.gate = 4
    assert L.moe_block_norm(ctypes.byref(c), None, 0, None) == INVALID


def test_binding_refuses_host_tensors_shapes_and_types():
    x = torch.zeros(2, 256, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        abi.moe_block_norm(abi.norm_config(256), x, x, x, None)
    with pytest.raises(ValueError):
        abi.KVCache.alloc(_attn(), 2, device="cpu")
    with pytest.raises(ValueError):
        abi.KVBatch(torch.zeros(3, dtype=torch.int32), torch.zeros(2, dtype=torch.int32), torch.zeros(2, 4, dtype=torch.int32), 2)
    with pytest.raises(KeyError):
        abi.attn_config(4, 2, 64, 16, dtype=torch.float32)


# ------------------------------------------------------------------------- the 64-bit forms --

def test_reference_codes():
    codes = torch.arange(256, dtype=torch.uint8)
    values = ref.decode(codes)
    assert bool(values[127].isnan()) and bool(values[255].isnan())
    assert float(values[126]) == 448.0 and float(values[1]) == 2.0 ** -9 and float(values[0x38]) == 1.0
    ok = torch.tensor([c for c in range(256) if c & 127 != 127])
    assert torch.equal(values[ok], codes[ok].view(torch.float8_e4m3fn).double())
    assert torch.equal(ref.encode(values[ok]).long(), ok)
    v = torch.randn(4096, dtype=torch.float64, generator=torch.Generator().manual_seed(1)) * 20
    assert torch.equal(ref.decode(ref.encode(v.float().double())), v.float().to(torch.float8_e4m3fn).double())
    assert ref.encode(torch.tensor([17.0, 19.0, -17.0, 1e9, math.nan], dtype=torch.float64)).tolist() == [
        0x58, 0x5a, 0xd8, 126, 0]  # 17 lies between 16 and 18, 19 between 18 and 20


def test_reference_rounding_to_16_bits():
    v = torch.randn(4096, generator=torch.Generator().manual_seed(1)) * torch.logspace(-9, 9, 4096, base=2)
    for dt in (torch.bfloat16, torch.float16):  # from 32 bits a cast rounds once
        assert torch.equal(ref.round16(v.double(), dt), v.to(dt).double())
    just_above = torch.tensor([1 + 2.0 ** -8 + 2.0 ** -40], dtype=torch.float64)  # a tie in 32 bits only
    assert float(ref.round16(just_above, torch.bfloat16)) == 1 + 2.0 ** -7


def test_reference_scale():
    a = torch.tensor([448.0, 448.1, 224.0, 224.1, 0.0, 3e38, 1e-30], dtype=torch.float64)
    assert ref.pow2_scale(a).tolist() == [1.0, 2.0, 0.5, 1.0, 2.0 ** -60, 2.0 ** 120, 2.0 ** -60]


def test_reference_append_and_attention_by_hand():
    """One head, D = 64, two pages of 16: a cache written in two steps, attention by the definition."""
    cfg = abi.attn_config(1, 1, 64, 16, rotary_dim=0)
    cache = {n + "_codes": torch.zeros(3, 1, 16, 64, dtype=torch.uint8) for n in "kv"}
    cache.update({n + "_scale": torch.ones(3, 1) for n in "kv"})
    table = torch.tensor([[2, 0]], dtype=torch.int32)
    k = torch.full((17, 1, 64), 1.0, dtype=torch.bfloat16)
    k[16] = 2.0
    v = torch.arange(17).view(17, 1, 1).expand(17, 1, 64).to(torch.bfloat16)
    ref.kv_append(cfg, cache, [0, 17], [17], table, None, k, v, None)
    assert cache["k_scale"][2, 0] == 2.0 ** -8 and cache["k_scale"][0, 0] == 2.0 ** -7
    assert float(ref.decode(cache["k_codes"])[2, 0, 0, 0]) == 256.0
    q = torch.zeros(1, 1, 64, dtype=torch.bfloat16)
    out, lse, _, _ = ref.attention(cfg, cache, [0, 1], [17], table, q, 0.125)
    assert abs(float(out[0, 0, 0]) - 8.0) < 1e-12 and abs(float(lse[0, 0]) - math.log(17)) < 1e-12
    out, lse, _, _ = ref.attention(cfg, cache, [0, 1], [17], table, q, 0.125, window=2)
    assert float(out[0, 0, 5]) == 15.5
    # a larger value in the first page: its codes move to the larger scale
    k2 = torch.full((1, 1, 64), 4.0, dtype=torch.bfloat16)
    ref.kv_append(cfg, cache, [0, 1], [9], table, None, k2, k2, None)
    assert cache["k_scale"][2, 0] == 2.0 ** -6 and float(ref.decode(cache["k_codes"])[2, 0, 0, 0]) == 64.0
