"""Host-side checks of the int4 attention half at the ends of its documented ranges (no call
here reaches a GPU)."""
import ctypes

import pytest
import torch

from activation_sparse_ffn_amd import _abi as A

E_NULL, E_SHAPE, E_ALIGN = -1, -2, -4
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


def test_lens_validation(lib):
    def call(B=2, pos=GOOD, max_pos=0, window=0, max_pages=3, table=GOOD, page=16, pages=5, lens=GOOD, starts=None):
        return lib.sfx_kv_lens_q4(None, B, pos, max_pos, window, max_pages, table, page, pages, lens, starts)
    assert call(B=0) == E_SHAPE and call(B=1 << 24) == E_SHAPE and call(max_pos=-1) == E_SHAPE
    assert call(window=-1, starts=GOOD) == E_SHAPE and call(window=4) == E_SHAPE and call(starts=GOOD) == E_SHAPE
    assert call(page=12) == E_SHAPE and call(max_pages=0) == E_SHAPE and call(max_pages=1 << 27) == E_SHAPE
    assert call(pages=0) == E_SHAPE
    for name in ("pos", "table", "lens"):
        assert call(**{name: None}) == E_NULL, name
        assert call(**{name: GOOD + 2}) == E_ALIGN, name
    assert call(window=4, starts=GOOD + 2) == E_ALIGN


def test_lens_binding_refusals():
    table, pos = torch.zeros(3, 4, dtype=torch.int32), torch.zeros(3, dtype=torch.int32)
    with pytest.raises(ValueError, match="on the GPU"):
        A.sfx_kv_lens_q4(pos, table, 16, 5, pos.clone())
    with pytest.raises(ValueError):
        A.sfx_kv_lens_q4(pos, table.view(12), 16, 5, pos.clone())
    with pytest.raises(TypeError):
        A.sfx_kv_lens_q4(pos, table.long(), 16, 5, pos.clone())


def test_stream_of_another_device_is_refused():
    """A stream belongs to the tensors' device: nothing is called on another one's."""
    class Stream:
        device_index, cuda_stream = 1, 0

    called = []
    with pytest.raises(ValueError, match="stream is on device 1"):
        A._run_on(0, Stream(), lambda *a: called.append(a) or 0, (), "f")
    assert not called
