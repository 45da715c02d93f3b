"""Longest sequences that 4-bit decode covers: host checks, no device call (the
calls are of no sequences, so that none could launch)."""
import ctypes

import pytest

from paged_kv_cache_64_gb300 import _lib

P = ctypes.c_void_p(1 << 20)
OK, INVALID = 0, 1


@pytest.fixture(scope="module")
def lib():
    from paged_kv_cache_64_gb300 import build
    build.build()
    return _lib.load()


@pytest.mark.parametrize("block", [16, 32])
@pytest.mark.parametrize("partition", [-1, 0, 4096])
def test_positions_past_two_to_the_30(lib, block, partition):
    """A sequence is at most as long as its table and max_seq_len say; past 2^30
    the kernel's position arithmetic (and a single pass's partial) would not
    hold.  A large max_seq_len over a short table is only a bound."""
    def call(max_blocks, max_len):
        return lib.pa_decode_int4(P, P, P, P, 10, P, max_blocks, P, max_len, 0, 8, 4, 128, block,
                                  ctypes.c_float(1.0), partition, P, 1 << 40, 1, None)
    top = (1 << 30) // block
    assert call(top, 1 << 30) == OK
    assert call(top, 2**31 - 1) == OK
    assert call(4, 2**31 - 1) == OK
    assert call(top + 1, 1 << 30) == OK
    assert call(top + 1, (1 << 30) + 1) == INVALID
    assert call(top + 1, 2**31 - 1) == INVALID
    # a table whose positions pass 2^31, whatever max_seq_len says
    assert call(2 * top - 1, 4096) == OK
    assert call(2 * top, 4096) == INVALID
