"""What a batch of moe_linear_attention says of its runs, without a GPU."""
import ctypes

import pytest

from sparse_moe_router_gb300 import abi

INVALID, SMALL = 1, 2
A = 0x10000  # an aligned address that is never dereferenced


@pytest.mark.parametrize("longest,status", [(-1, INVALID), (-2 ** 31, INVALID), (0, SMALL), (1, SMALL), (5, SMALL), (2 ** 31 - 1, SMALL)])
def test_the_longest_run(longest, status):
    """Any length that is not negative passes this check; the call then ends at its workspace, which is too small."""
    cfg = abi.linear_config(4, 8, 128, 64)
    pool, batch = abi._StatePool(A, 3), abi._StateBatch(2, 5, A, A, A, longest)
    st = abi.load().moe_linear_attention(ctypes.byref(cfg), ctypes.byref(pool), ctypes.byref(batch), A, 512, A, 512, A, 512, None, 0, 1.0, A, 512, A,
                                         256, None)
    assert st == status
