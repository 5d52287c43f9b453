"""Host-side checks of the int4 attention half: every entry point refuses what it does not
take before anything is enqueued (no call here reaches a GPU), the binding refuses tensors of
the wrong kind, and the oracle's pieces are pinned to closed forms and worked examples."""
import ctypes

import numpy as np
import pytest
import torch

from activation_sparse_ffn_amd import _abi as A
from oracle import q4_oracle as Q

E_NULL, E_SHAPE, E_DTYPE, E_ALIGN, E_WORKSPACE = -1, -2, -3, -4, -5
P = ctypes.c_void_p
GOOD, ODD2, ODD4 = 0x10000, 0x10002, 0x10004      # fake device addresses (never dereferenced)


@pytest.fixture(scope="module")
def lib():
    return A.load()


def test_linear_validation(lib):
    def call(xdt=1, group=32, B=1, n=100, d=256, x=GOOD, ldx=None, W=GOOD, s=GOOD, bias=None, y=GOOD, ldy=None):
        return lib.sfx_linear_q4(None, xdt, group, B, n, d, x, d if ldx is None else ldx, W, s, bias, 0, y,
                                 n if ldy is None else ldy)
    assert call(xdt=0) == E_DTYPE and call(xdt=3) == E_DTYPE and call(xdt=9) == E_DTYPE
    assert call(group=16) == E_SHAPE and call(group=256) == E_SHAPE and call(group=0) == E_SHAPE
    assert call(B=0) == E_SHAPE and call(B=65) == E_SHAPE and call(n=0) == E_SHAPE and call(d=0) == E_SHAPE
    assert call(d=240) == E_SHAPE and call(d=192, group=128) == E_SHAPE
    assert call(n=(1 << 24) + 1) == E_SHAPE and call(d=(1 << 24) + 32) == E_SHAPE
    assert call(ldx=255) == E_SHAPE and call(ldy=99) == E_SHAPE
    for name in ("x", "W", "s", "y"):
        assert call(**{name: None}) == E_NULL
    assert call(x=ODD4) == E_ALIGN and call(W=ODD4) == E_ALIGN and call(ldx=260) == E_ALIGN
    assert call(s=GOOD + 1) == E_ALIGN and call(y=ODD2) == E_ALIGN and call(bias=ODD2) == E_ALIGN


def test_cache_bytes(lib):
    assert lib.sfx_kv_cache_bytes(8, 128, 16, 10) == 10 * 8 * 2 * 9 * 128
    assert lib.sfx_kv_cache_bytes(8, 128, 64, 1 << 20) == (1 << 20) * 8 * 8 * 9 * 128       # past 32 bits
    for bad in ((0, 128, 16, 1), (257, 128, 16, 1), (8, 48, 16, 1), (8, 0, 16, 1), (8, 288, 16, 1), (8, 128, 4, 1),
                (8, 128, 24, 1), (8, 128, 2048, 1), (8, 128, 16, 0), (8, 128, 16, 1 << 30)):
        assert lib.sfx_kv_cache_bytes(*bad) == 0, bad


def test_append_validation(lib):
    def call(xdt=1, qdt=1, T=4, Hq=4, Hkv=2, D=64, q=GOOD, ldq=256, k=GOOD, ldk=128, v=GOOD, ldv=128, pos=GOOD, seq=None,
             cs=None, rot=0, max_pos=0, B=2, max_pages=3, table=GOOD, page=16, pages=5, cache=GOOD, q_out=GOOD):
        return lib.sfx_kv_append_q4(None, xdt, qdt, T, Hq, Hkv, D, q, ldq, k, ldk, v, ldv, pos, seq, cs, rot, max_pos, 0,
                                    B, max_pages, table, page, pages, cache, q_out)
    assert call(xdt=3) == E_DTYPE and call(qdt=0) == E_DTYPE and call(qdt=3) == E_DTYPE
    assert call(T=0) == E_SHAPE and call(T=1 << 24) == E_SHAPE
    assert call(Hq=0) == E_SHAPE and call(Hq=257) == E_SHAPE and call(Hkv=0) == E_SHAPE and call(D=40) == E_SHAPE
    assert call(ldq=255) == E_SHAPE and call(ldk=127) == E_SHAPE and call(ldv=127) == E_SHAPE
    assert call(B=0) == E_SHAPE and call(max_pages=0) == E_SHAPE and call(page=12) == E_SHAPE and call(pages=0) == E_SHAPE
    assert call(max_pages=1 << 27) == E_SHAPE
    for rot, n in ((0, 9), (3, 9), (66, 9), (64, 0)):
        assert call(cs=GOOD, rot=rot, max_pos=n) == E_SHAPE, (rot, n)
    for name in ("k", "v", "pos", "table", "cache", "q_out"):
        assert call(**{name: None}) == E_NULL, name
    for name in ("k", "v", "q", "q_out"):
        assert call(**{name: GOOD + 1}) == E_ALIGN, name
    assert call(xdt=0, k=ODD2) == E_ALIGN and call(cache=GOOD + 8) == E_ALIGN and call(pos=ODD2) == E_ALIGN
    assert call(seq=ODD2) == E_ALIGN and call(table=ODD2) == E_ALIGN and call(cs=ODD2, rot=64, max_pos=9) == E_ALIGN


def test_read_validation(lib):
    def call(odt=0, T=4, Hkv=2, D=64, pos=GOOD, B=2, max_pages=3, table=GOOD, page=16, pages=5, cache=GOOD, k=GOOD, v=GOOD):
        return lib.sfx_kv_read_q4(None, odt, T, Hkv, D, pos, None, B, max_pages, table, page, pages, cache, k, v)
    assert call(odt=3) == E_DTYPE and call(T=0) == E_SHAPE and call(D=33) == E_SHAPE and call(page=7) == E_SHAPE
    for name in ("pos", "table", "cache", "k", "v"):
        assert call(**{name: None}) == E_NULL, name
    assert call(k=GOOD + 8) == E_ALIGN and call(v=ODD2) == E_ALIGN and call(table=ODD2) == E_ALIGN


def test_attention_validation(lib):
    def ws_of(B=2, Hq=8, Hkv=2, D=64, n=4800):
        return lib.sfx_attn_q4_ws(B, Hq, Hkv, D, n)

    def call(qdt=1, B=2, Hq=8, Hkv=2, D=64, q=GOOD, ldq=512, max_pages=300, table=GOOD, page=16, pages=5, cache=GOOD,
             starts=None, lens=GOOD, scale=0.1, out=GOOD, lse=None, ws=0x100000, n=None):
        return lib.sfx_attn_q4(None, qdt, B, Hq, Hkv, D, q, ldq, max_pages, table, page, pages, cache, starts, lens,
                               ctypes.c_float(scale), out, lse, ws, ws_of() if n is None else n)
    assert ws_of() > 0 and ws_of(n=64) == 0            # one run: nothing to join
    assert ws_of(B=65) == 0 and ws_of(Hq=7) == 0 and ws_of(D=48) == 0 and ws_of(n=0) == 0
    assert call(qdt=0) == E_DTYPE and call(qdt=3) == E_DTYPE
    assert call(B=0) == E_SHAPE and call(B=65) == E_SHAPE and call(Hq=7) == E_SHAPE and call(Hq=0) == E_SHAPE
    assert call(Hq=512, ldq=1 << 16) == E_SHAPE and call(ldq=511) == E_SHAPE and call(page=1) == E_SHAPE
    for s in (float("nan"), float("inf"), float("-inf")):
        assert call(scale=s) == E_SHAPE
    for name in ("q", "table", "cache", "lens", "out"):
        assert call(**{name: None}) == E_NULL, name
    assert call(q=ODD4) == E_ALIGN and call(ldq=516) == E_ALIGN and call(out=ODD4) == E_ALIGN and call(lens=ODD2) == E_ALIGN
    assert call(starts=ODD2) == E_ALIGN and call(lse=ODD2) == E_ALIGN and call(cache=ODD4) == E_ALIGN
    assert call(ws=None) == E_WORKSPACE and call(ws=0x100010) == E_WORKSPACE and call(n=ws_of() - 1) == E_WORKSPACE


def test_binding_refusals():
    """Shapes and dtypes are refused before the device is looked at, then tensors off the GPU."""
    f = torch.zeros
    x, W, s, y = f(2, 64, dtype=torch.float16), f(8, 32, dtype=torch.uint8), f(8, 2, dtype=torch.float16), f(2, 8)
    with pytest.raises(ValueError, match="on the GPU"):
        A.sfx_linear_q4(x, W, s, y)
    for bad in (dict(x=f(2, 32, dtype=torch.float16)), dict(y=f(2, 9)), dict(W_scales=f(7, 2, dtype=torch.float16)),
                dict(W_scales=f(8, 3, dtype=torch.float16)), dict(x=f(64, dtype=torch.float16))):
        with pytest.raises(ValueError):
            A.sfx_linear_q4(**{**dict(x=x, W=W, W_scales=s, y=y), **bad})
    for bad in (dict(x=x.float()), dict(y=y.half())):
        with pytest.raises(TypeError):
            A.sfx_linear_q4(**{**dict(x=x, W=W, W_scales=s, y=y), **bad})

    k, pos = f(3, 2, 64, dtype=torch.float16), f(3, dtype=torch.int32)
    table, cache = f(3, 4, dtype=torch.int32), f(6, 2, 2, 576, dtype=torch.uint8)
    ap = dict(q=None, k=k, v=k.clone(), pos=pos, table=table, cache=cache, q_out=None)
    with pytest.raises(ValueError, match="on the GPU"):
        A.sfx_kv_append_q4(**ap)
    with pytest.raises(ValueError):
        A.sfx_kv_append_q4(**{**ap, "v": k[:2]})
    with pytest.raises(TypeError):
        A.sfx_kv_append_q4(**{**ap, "k": k.double(), "v": k.double()})
    rd = dict(pos=pos, table=table, cache=cache, k_out=k, v_out=k.clone())
    with pytest.raises(ValueError, match="on the GPU"):
        A.sfx_kv_read_q4(**rd)
    with pytest.raises(ValueError):
        A.sfx_kv_read_q4(**{**rd, "v_out": k.float()})

    at = dict(q=f(3, 4, 64, dtype=torch.float16), cache=cache, table=table, lens=pos, out=f(3, 4, 64, dtype=torch.float16),
              ws=f(256, dtype=torch.uint8))
    with pytest.raises(ValueError, match="on the GPU"):
        A.sfx_attn_q4(**at)
    for bad in (dict(out=f(3, 4, 32, dtype=torch.float16)), dict(cache=f(6, 2, 2, 500, dtype=torch.uint8)),
                dict(table=f(2, 4, dtype=torch.int32)), dict(q=f(3, 64, dtype=torch.float16))):
        with pytest.raises(ValueError):
            A.sfx_attn_q4(**{**at, **bad})
    with pytest.raises(TypeError):
        A.sfx_attn_q4(**{**at, "q": at["q"].float()})
    with pytest.raises(A.SfxError):
        A.kv_cache_q4(4, 2, 12, 64, device="cpu")
    assert A.kv_cache_q4(4, 2, 16, 64, device="cpu").shape == (4, 2, 2, 576)


def test_row_strides():
    """Strides handed on: rows or heads apart, one row, and what is refused."""
    wide = torch.zeros(4, 100)
    assert A._rows(wide, "f", "x") == 100 and A._rows(wide[:, 8:40], "f", "x") == 100
    assert A._rows(wide[:1, 8:40], "f", "x") == 32 and A._rows(wide[::2], "f", "x") == 200
    with pytest.raises(ValueError):
        A._rows(wide[:, ::2], "f", "x")
    h = torch.zeros(5, 6, 16)
    assert A._head_rows(h, "f", "q") == 96 and A._head_rows(h[:, :4], "f", "q") == 96 and A._head_rows(h[:1, :4], "f", "q") == 64
    with pytest.raises(ValueError):
        A._head_rows(h[:, ::2], "f", "q")
    with pytest.raises(ValueError):
        A._head_rows(h.transpose(0, 1), "f", "q")


# ------------------------------------------------------------------------------ oracle pins

def test_oracle_quantise_worked_example():
    w = np.zeros((1, 64), np.float32)
    w[0, :4] = [7.0, -3.4, 0.5, 1.5]                    # scale 1: halves go to the even code
    w[0, 32:35] = [-0.07, 0.01, 0.035]                  # scale fp16(0.01)
    q, s = Q.quantise(w, 65504.0)
    assert s[0, 0] == 1 and list(q[0, :4]) == [7, -3, 0, 2] and not q[0, 4:32].any()
    assert s[0, 1] == np.float16(0.07 / 7) and q[0, 32] == -7 and q[0, 33] == 1
    assert np.array_equal(Q.values(q, s)[0, :4], [7.0, -3.0, 0.0, 2.0])
    # what is too large is clipped to 7 (or 8) scales, what is not finite marks its group
    q, s = Q.quantise(np.full((1, 32), 1e6, np.float32), 8188.0)
    assert s[0, 0] == 8188 and (q == 7).all()
    w = np.ones((1, 32), np.float32)
    w[0, 5] = np.inf
    q, s = Q.quantise(w, 65504.0)
    assert np.isnan(s).all() and not q.any()
    assert not Q.quantise(np.zeros((1, 32), np.float32), 1.0)[0].any()


def test_oracle_rotation_closed_forms():
    rng = np.random.default_rng(0)
    x = rng.standard_normal((3, 2, 8)).astype(np.float32)
    ang = np.arange(5)[:, None] * np.array([1.0, 0.1, 0.01])
    cs = np.concatenate([np.cos(ang), np.sin(ang)], 1).astype(np.float32)
    pos = np.array([0, 2, 4])
    for pairs in (False, True):
        y = Q.rotate(x, pos, cs, pairs)
        assert np.array_equal(y[0], x[0]) and np.array_equal(y[..., 6:], x[..., 6:])      # angle 0; dims past rot
        i, j = (0, 1) if pairs else (0, 3)
        for t in range(3):
            z = (x[t, :, i] + 1j * x[t, :, j]) * np.exp(1j * ang[pos[t], 0])
            assert np.allclose(y[t, :, i], z.real, atol=1e-6) and np.allclose(y[t, :, j], z.imag, atol=1e-6)
        assert np.allclose(np.linalg.norm(y, axis=-1), np.linalg.norm(x, axis=-1), rtol=1e-6)


def test_oracle_attention_closed_forms():
    rng = np.random.default_rng(1)
    q, k, v = rng.standard_normal((4, 32)), rng.standard_normal((9, 2, 32)), rng.standard_normal((9, 2, 32))
    o, lse, ab = Q.attention(np.zeros_like(q), k, v, 1.0)                # equal weights
    assert np.allclose(o[:2], v[:, 0].mean(0)) and np.allclose(o[2:], v[:, 1].mean(0)) and np.allclose(lse, np.log(9))
    assert (ab >= np.abs(o) - 1e-12).all()
    o, lse, _ = Q.attention(q, k[:1], v[:1], 0.7)                        # one position: its value
    assert np.allclose(o[0], v[0, 0]) and np.allclose(lse[3], 0.7 * q[3] @ k[0, 1])
    o, lse, _ = Q.attention(q, k[:0], v[:0], 1.0)
    assert not o.any() and np.isneginf(lse).all()
    # two halves joined by their log-sum-exps
    (o1, l1, _), (o2, l2, _), (o, lse, _) = (Q.attention(q, k[a], v[a], 1.0) for a in (slice(0, 4), slice(4, 9), slice(0, 9)))
    l = np.logaddexp(l1, l2)
    assert np.allclose(l, lse) and np.allclose(o1 * np.exp(l1 - l)[:, None] + o2 * np.exp(l2 - l)[:, None], o)


def test_oracle_linear_and_block_layout():
    codes = np.array([[0x1F, 0x80]], np.uint8)                            # columns -1, 1, 0, -8
    assert list(Q.unpack_rows(codes)[0]) == [-1, 1, 0, -8]
    rng = np.random.default_rng(2)
    codes = rng.integers(0, 256, (3, 32), dtype=np.uint8)
    s = rng.random((3, 2)).astype(np.float16)
    x = rng.standard_normal((2, 64))
    want = [[sum(float(s[i, c // 32]) * Q.unpack_rows(codes)[i, c] * x[b, c] for c in range(64)) for i in range(3)] for b in range(2)]
    assert np.allclose(Q.linear_q4(x, codes, s), want)
    # every code of a block is found once, whatever the position
    D = 64
    block = rng.integers(0, 256, 9 * D, dtype=np.uint8)
    nib = np.sort(np.concatenate([block[:8 * D] & 15, block[:8 * D] >> 4]))
    seen = np.sort(np.concatenate([np.concatenate(Q.read_block(block, D, i)[0::2]) for i in range(8)]) + 8)
    assert np.array_equal(nib, seen)
