"""The int4 attention half at the ends of its documented ranges: the largest token count, the
largest finite numbers, tokens that are not stored, streams of other devices."""
import numpy as np
import pytest
import torch

from activation_sparse_ffn_amd import _abi as A
from gpu_helpers import say
from oracle import q4_oracle as Q

pytestmark = pytest.mark.gpu
DEV = "cuda"
DT = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}


def np64(t):
    return t.detach().cpu().to(torch.float64).numpy()


def test_append_and_read_at_the_largest_token_count():
    """2^24 - 1 tokens, nearly all padding: the launch's last workgroups, with tokens in the
    first and the last 64 stored and read back and zeros for the others."""
    T, D, page = (1 << 24) - 1, 32, 8
    say(f"append and read {T} tokens")
    at = [0, 1, 7, 8, 62, 63, 64, 4096, T - 65, T - 64, T - 63, T - 9, T - 8, T - 2, T - 1]
    table = torch.tensor([[2, 0]], dtype=torch.int32, device=DEV)
    cache = torch.zeros(3, 1, 1, 9 * D, dtype=torch.uint8, device=DEV)
    pos = torch.full((T,), -1, dtype=torch.int32, device=DEV)
    seq = torch.zeros(T, dtype=torch.int32, device=DEV)
    rows = torch.randn(len(at), 1, D, generator=torch.Generator().manual_seed(4)).half()
    kv = torch.ones(T, 1, D, dtype=torch.float16, device=DEV)
    for i, t in enumerate(at):
        pos[t] = i
        kv[t] = rows[i].to(DEV)
    A.sfx_kv_append_q4(None, kv, kv, pos, table, cache, None, seq=seq)
    ko, vo = torch.full_like(kv, 9.0), torch.full_like(kv, 9.0)
    A.sfx_kv_read_q4(pos, table, cache, ko, vo, seq=seq)
    stored = pos >= 0
    for out, top in ((ko, 65504.0), (vo, 8188.0)):
        want = torch.from_numpy(Q.values(*Q.quantise(rows.float().numpy(), top))).to(torch.float16)
        assert torch.equal(out[stored].cpu(), want)
        assert not out[~stored].any()
