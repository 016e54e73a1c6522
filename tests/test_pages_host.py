"""Limits of the operators on the pages of a cache.  No call here launches a kernel; the device pointers are fakes that
nothing reads."""
import ctypes

import pytest

from transformer_rope_positional_gb300 import _capi as C
from transformer_rope_positional_gb300 import build as B

BAD = C.ROPE_ERR_PARAM_INVALID


@pytest.fixture(scope="module")
def lib():
    B.build()
    return C.load()


def d(dtype, shape, i):
    return ctypes.byref(C.describe(i << 40, dtype, shape))


@pytest.mark.parametrize("W,new_W,bs", [(1 << 30, 5, 1), (5, 1 << 30, 1), (1 << 30, 1 << 30, 1), ((1 << 29) + 1, 5, 2),
                                        (5, (1 << 29) + 1, 2)])
def test_rearrange_widest_tables(lib, W, new_W, bs):
    """A row of 2^30 pages would read as one that keeps a page."""
    n = lib.rope_launch_count()
    one = [d(C.I64, (1,), i) for i in range(2, 9)]
    assert lib.rope_rearrange_sequences(d(C.I64, (1, W), 9), one[0], d(C.I32, (3,), 10), one[1], None, d(C.I64, (1, new_W), 11),
                                        one[2], d(C.I32, (3,), 12), one[3], one[4], d(C.I64, (2,), 13), bs, 0, None) == BAD
    assert lib.rope_launch_count() == n
