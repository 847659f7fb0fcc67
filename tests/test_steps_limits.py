"""Refusals at the limits of the layer's steps, beyond those of test_steps_abi.py (no GPU needed)."""
import ctypes

import pytest

from global_attention_moe_b200 import build

FAKE = 0x10000  # aligned, never dereferenced: validation fails first


@pytest.fixture(scope="module")
def M():
    build.build()
    from global_attention_moe_b200 import mimo_attn
    return mimo_attn


@pytest.mark.parametrize("total", [2 ** 31 - 16383, 2 ** 31 - 8192, 2 ** 31 - 8191, 2 ** 31 - 4096])
def test_lists_whose_walk_would_pass_2_31(M, total):
    """The eviction's copy loop counts in int and steps by a cluster's 8 x 1024 threads: from 2^31 - 8191 entries on
    its last step would pass 2^31, come out negative and run below the buffers.  With room: 2^31 - 16384 at most."""
    step = 8 * 1024
    most = 2 ** 31 - 16384
    assert max(first + -(-(most - first) // step) * step for first in (0, 1, 5, step - 1)) < 2 ** 31
    assert M.LIB.mimo_kv_evict(FAKE, FAKE, FAKE, 1, total, total, total, 0, 0, FAKE, FAKE, FAKE, FAKE, None) == M.ERR_UNSUPPORTED
    dims = M.make_decode_dims(1, 1, total, 128, 1, 1, 1, 1)
    assert M.LIB.mimo_decode_key_weights(FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, None, ctypes.byref(dims), M.LAYER_GLOBAL, -1, 1e4,
                                         64, FAKE, FAKE, 1 << 60, None) == M.ERR_UNSUPPORTED
