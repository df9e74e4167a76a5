"""What the Python binding of the decoder layer's calls refuses by itself, without a GPU."""
import pytest

from sparse_moe_router_gb300 import abi


@pytest.mark.parametrize("other", [dict(kv_heads=4), dict(page_size=128), dict(head_dim=256), dict(head_dim=64, page_size=128)])
def test_a_cache_of_another_layout(other):
    """A config with other heads, pages or widths than the cache was made for would go past its pages (the library
    has no sizes to check): both calls refuse it before they look at anything else."""
    cfg = abi.attn_config(8, 2, 128, 64)
    cache = object.__new__(abi.KVCache)
    cache.layout = (2, 64, 128)
    cache.check(cfg)
    wrong = abi.attn_config(**dict(dict(q_heads=8, kv_heads=2, head_dim=128, page_size=64), **other))
    for call, args in ((abi.moe_attention, (None,) * 4), (abi.moe_kv_append, (None,) * 7)):
        with pytest.raises(ValueError, match="layout|kv_heads"):
            call(wrong, cache, *args)
