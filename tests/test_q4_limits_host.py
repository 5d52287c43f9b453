"""Host-side checks of the int4 attention half at the ends of its documented ranges (no call
here reaches a GPU)."""
import ctypes

import pytest

from activation_sparse_ffn_amd import _abi as A

E_SHAPE = -2
GOOD = 0x10000                                     # fake device address (never dereferenced)


@pytest.fixture(scope="module")
def lib():
    return A.load()


def test_attention_scale_limit(lib):
    """A scale from 2^115 on, of either sign, is refused: 2^12 log2(e) times it is not finite."""
    for qdt in (1, 2):
        for scale in (2.0 ** 115, -(2.0 ** 115), 3e38):
            assert lib.sfx_attn_q4(None, qdt, 2, 8, 2, 64, GOOD, 512, 4, GOOD, 16, 5, GOOD, None, GOOD, ctypes.c_float(scale),
                                   GOOD, None, None, 0) == E_SHAPE
