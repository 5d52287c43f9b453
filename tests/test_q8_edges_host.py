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


PROMPT_WS = [  # B, Hq, Hkv, D, max_len, max_q
    (1, 1, 1, 64, 1 << 17, 40000), (1, 64, 8, 128, 131072, 5000), (3, 6, 2, 96, 5000, 5000), (16, 128, 8, 64, 4096, 3000),
    (1, 256, 1, 256, 1 << 20, 600), (2, 7, 7, 160, 700, 3000), (64, 32, 32, 128, 8192, 200), (1, 4, 4, 32, 256, 3000), (1, 20, 1, 224, 3000, 97),
    (5, 40, 8, 128, 100000, 1), (1, 96, 1, 128, 9000, 2), (1, 1, 1, 128, 1 << 20, 33000)]


@pytest.mark.parametrize("case", PROMPT_WS, ids=str)
def test_prompt_workspace_fits_every_row_count(case, monkeypatch):
    """The largest of all row counts' workspaces, from a few hundred calls."""
    from activation_sparse_ffn_amd import step
    B, Hq, Hkv, D, max_len, max_q = case
    want = max(A.sfx_attn_q8_ws(B, n, Hq, Hkv, D, max_len) for n in range(1, max_q + 1))
    calls, ask = [0], A.sfx_attn_q8_ws

    def counted(*a):
        calls[0] += 1
        return ask(*a)
    monkeypatch.setattr(A, "sfx_attn_q8_ws", counted)
    assert step._prompt_ws(*case) == want
    assert calls[0] <= 96 + 500
    assert step._prompt_ws(B, Hq, Hkv, D, max_len, 0) == 0


def test_half_asks_for_few_workspaces(monkeypatch):
    from activation_sparse_ffn_amd import AttnStep8
    calls, ask = [0], A.sfx_attn_q8_ws

    def counted(*a):
        calls[0] += 1
        return ask(*a)
    monkeypatch.setattr(A, "sfx_attn_q8_ws", counted)
    table, pos = torch.zeros(1, 64, dtype=torch.int32), torch.zeros(1, dtype=torch.int32)
    s = AttnStep8(64, 8, 2, 64, 1, "f16", table, pos, 64, max_tokens=1024, device="cpu")
    assert calls[0] < 100
    assert s.ws_prompt.numel() >= max(ask(1, n, 8, 2, 64, 1024) for n in range(1, 1025))


def test_half_keeps_steps_and_prompts_apart():
    """No buffer that a decode step writes is one that a prompt writes."""
    from activation_sparse_ffn_amd import AttnStep8
    table, pos = torch.zeros(2, 4, dtype=torch.int32), torch.zeros(2, dtype=torch.int32)
    s = AttnStep8(64, 8, 2, 64, 2, "f16", table, pos, 8, max_tokens=20, device="cpu")
    spans = [[(t.data_ptr(), t.data_ptr() + t.nbytes) for t in side] for side in (s._step, s._prompt)]
    for a0, a1 in spans[0]:
        assert a1 > a0 and all(b1 <= a0 or a1 <= b0 for b0, b1 in spans[1])
