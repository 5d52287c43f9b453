"""The binding's work per call."""
import pytest
import torch

from activation_sparse_ffn_amd import _abi as A

pytestmark = pytest.mark.gpu
DEV = "cuda"


class Watched:
    """A tensor whose attributes are counted as they are asked for."""

    def __init__(self, t):
        self.t, self.asked = t, []

    def __getattr__(self, name):
        self.asked.append(name)
        return getattr(self.t, name)


@pytest.mark.parametrize("bits", [4, 8])
def test_attention_looks_at_lens_once(bits):
    B, Hq, Hkv, D = 2, 4, 2, 64
    table = torch.zeros(B, 1, dtype=torch.int32, device=DEV)
    q = torch.zeros(B, Hq, D, dtype=torch.float16, device=DEV)
    lens = Watched(torch.zeros(B, dtype=torch.int32, device=DEV))
    out = torch.full_like(q, 7.0)
    make, call, ws = ((A.kv_cache_q4, A.sfx_attn_q4, A.sfx_attn_q4_ws(B, Hq, Hkv, D, 16)) if bits == 4 else
                      (A.kv_cache_q8, A.sfx_attn_q8, A.sfx_attn_q8_ws(B, 1, Hq, Hkv, D, 16)))
    call(q, make(1, Hkv, 16, D), table, lens, out, A.workspace(ws))
    assert (out == 0).all()
    assert len(lens.asked) == len(set(lens.asked)), lens.asked
