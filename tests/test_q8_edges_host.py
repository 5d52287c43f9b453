"""Host-side checks of what the 8-bit layer half refuses beyond test_q8_host.py, and of AttnStep8's
buffers (no call here reaches a GPU)."""
import pytest
import torch

from activation_sparse_ffn_amd import _abi as A

E_NULL, E_SHAPE, E_ALIGN = -1, -2, -4
GOOD, ODD2, ODD4 = 0x10000, 0x10002, 0x10004      # fake device addresses (never dereferenced)


def test_blank_validation():
    lib = A.load()

    def call(T=5, n=64, q_start=GOOD, lens=GOOD, max_pos=0, max_q=3, B=2, max_pages=3, table=GOOD, page=16, pages=5, x=GOOD):
        return lib.sfx_kv_blank_q8(None, T, n, q_start, lens, max_pos, max_q, B, max_pages, table, page, pages, x)
    assert call(T=0) == E_SHAPE and call(T=(1 << 20) + 1) == E_SHAPE and call(q_start=None) == E_SHAPE      # T != B
    assert call(n=0) == E_SHAPE and call(n=12) == E_SHAPE and call(n=(1 << 24) + 8) == E_SHAPE
    assert call(max_q=0) == E_SHAPE and call(max_pos=-1) == E_SHAPE
    assert call(B=0) == E_SHAPE and call(B=4097) == E_SHAPE and call(page=8) == E_SHAPE and call(pages=0) == E_SHAPE
    assert call(max_pages=0) == E_SHAPE and call(max_pages=1 << 27) == E_SHAPE
    for name in ("lens", "table", "x"):
        assert call(**{name: None}) == E_NULL, name
    assert call(x=ODD4) == E_ALIGN and call(lens=ODD2) == E_ALIGN and call(table=ODD2) == E_ALIGN and call(q_start=ODD2) == E_ALIGN


def test_blank_binding_refusals():
    x, lens, table = torch.zeros(4, 64).half(), torch.zeros(2, dtype=torch.int32), torch.zeros(2, 3, dtype=torch.int32)
    args = dict(x=x, lens=lens, table=table, page=16, num_pages=5, q_start=torch.zeros(3, dtype=torch.int32), max_q=4)
    with pytest.raises(ValueError, match="on the GPU"):
        A.sfx_kv_blank_q8(**args)
    for bad in (dict(x=x.view(-1)), dict(x=x[:, ::2]), dict(table=table.view(-1))):
        with pytest.raises(ValueError):
            A.sfx_kv_blank_q8(**{**args, **bad})
    for bad in (dict(x=x.float()), dict(table=table.long())):
        with pytest.raises(TypeError):
            A.sfx_kv_blank_q8(**{**args, **bad})
