"""Host-side checks of the 8-bit layer half: every entry point refuses what it does not take
before anything is enqueued (no call here reaches a GPU), the binding refuses tensors of the
wrong kind, and the oracle's pieces are pinned to closed forms and worked examples."""
import ctypes

import numpy as np
import pytest
import torch

from activation_sparse_ffn_amd import _abi as A
from oracle import q8_oracle as Q

E_NULL, E_SHAPE, E_DTYPE, E_ALIGN, E_WORKSPACE = -1, -2, -3, -4, -5
GOOD, ODD2, ODD4 = 0x10000, 0x10002, 0x10004      # fake device addresses (never dereferenced)


@pytest.fixture(scope="module")
def lib():
    return A.load()


def test_norm_validation(lib):
    def call(xdt=1, rdt=0, ydt=1, T=3, d=64, norm=1, eps=1e-5, x=GOOD, ldx=64, r=GOOD, ldr=64, ro=GOOD, ldro=64, w=None,
             q=GOOD, s=GOOD, y=GOOD, ldy=64):
        return lib.sfx_norm_q8(None, xdt, rdt, ydt, T, d, norm, ctypes.c_float(eps), x, ldx, r, ldr, ro, ldro, w, q, s, y, ldy)
    assert call(xdt=3) == E_DTYPE and call(rdt=3) == E_DTYPE and call(ydt=-1) == E_DTYPE
    assert call(T=0) == E_SHAPE and call(T=(1 << 20) + 1) == E_SHAPE and call(d=0) == E_SHAPE and call(d=(1 << 24) + 1) == E_SHAPE
    for eps in (0.0, -1.0, float("nan"), float("inf")):
        assert call(eps=eps) == E_SHAPE
    assert call(norm=0, w=GOOD) == E_SHAPE and call(r=None) == E_SHAPE and call(q=None) == E_SHAPE and call(s=None) == E_SHAPE
    for name in ("ldx", "ldr", "ldro", "ldy"):
        assert call(**{name: 63}) == E_SHAPE
    assert call(x=None) == E_NULL and call(q=None, s=None, y=None, r=None, ro=None) == E_NULL
    assert call(x=GOOD + 1) == E_ALIGN and call(r=ODD2) == E_ALIGN and call(ro=ODD2) == E_ALIGN and call(y=GOOD + 1) == E_ALIGN
    assert call(w=ODD2) == E_ALIGN and call(q=ODD4) == E_ALIGN and call(s=ODD2) == E_ALIGN


def test_linear_validation(lib):
    def call(ydt=0, T=3, n=10, d=64, x=GOOD, ldx=64, sx=GOOD, W=GOOD, sw=GOOD, bias=None, y=GOOD, ldy=10):
        return lib.sfx_linear_q8(None, ydt, T, n, d, x, ldx, sx, W, sw, bias, 0, y, ldy)
    assert call(ydt=3) == E_DTYPE and call(T=0) == E_SHAPE and call(T=(1 << 20) + 1) == E_SHAPE
    assert call(n=0) == E_SHAPE and call(d=0) == E_SHAPE and call(d=72) == E_SHAPE and call(n=(1 << 24) + 1, ldy=1 << 25) == E_SHAPE
    assert call(d=131072, ldx=131072) == E_SHAPE            # a sum could leave 32 bits
    assert call(ldx=48) == E_SHAPE and call(ldy=9) == E_SHAPE
    for name in ("x", "sx", "W", "sw", "y"):
        assert call(**{name: None}) == E_NULL
    assert call(x=ODD4) == E_ALIGN and call(W=ODD4) == E_ALIGN and call(ldx=72) == E_ALIGN and call(y=ODD2) == E_ALIGN
    assert call(ydt=1, y=GOOD + 1) == E_ALIGN
    assert call(sx=ODD2) == E_ALIGN and call(sw=ODD2) == E_ALIGN and call(bias=ODD2) == E_ALIGN


def test_cache_bytes(lib):
    assert lib.sfx_kv_cache_q8_bytes(8, 128, 16, 10) == 10 * 8 * (32 * 128 + 16)
    assert lib.sfx_kv_cache_q8_bytes(8, 128, 64, 1 << 20) == (1 << 20) * 8 * 4 * (32 * 128 + 16)       # past 32 bits
    for bad in ((0, 128, 16, 1), (257, 128, 16, 1), (8, 48, 16, 1), (8, 0, 16, 1), (8, 288, 16, 1), (8, 128, 8, 1),
                (8, 128, 24, 1), (8, 128, 2048, 1), (8, 128, 16, 0), (8, 128, 16, 1 << 30)):
        assert lib.sfx_kv_cache_q8_bytes(*bad) == 0, bad


def test_append_validation(lib):
    def call(xdt=1, qdt=1, T=4, Hq=4, Hkv=2, D=64, q=GOOD, ldq=256, k=GOOD, ldk=128, v=GOOD, ldv=128, q_start=GOOD, lens=GOOD,
             cs=None, rot=0, max_pos=0, B=2, max_pages=3, table=GOOD, page=16, pages=5, cache=GOOD, q_out=GOOD):
        return lib.sfx_kv_append_q8(None, xdt, qdt, T, Hq, Hkv, D, q, ldq, k, ldk, v, ldv, q_start, lens, cs, rot, max_pos, 0,
                                    B, max_pages, table, page, pages, cache, q_out)
    assert call(xdt=3) == E_DTYPE and call(qdt=0) == E_DTYPE and call(qdt=3) == E_DTYPE
    assert call(T=0) == E_SHAPE and call(T=(1 << 20) + 1) == E_SHAPE and call(q_start=None) == E_SHAPE     # T != B
    assert call(Hq=0) == E_SHAPE and call(Hq=257) == E_SHAPE and call(Hkv=0) == E_SHAPE and call(D=40) == E_SHAPE
    assert call(ldq=255) == E_SHAPE and call(ldk=127) == E_SHAPE and call(ldv=127) == E_SHAPE
    assert call(B=0) == E_SHAPE and call(B=4097) == E_SHAPE and call(max_pages=0) == E_SHAPE and call(page=8) == E_SHAPE
    assert call(pages=0) == E_SHAPE and call(max_pages=1 << 27) == E_SHAPE
    assert call(T=1 << 20, Hkv=256, D=256, ldk=1 << 16, ldv=1 << 16, Hq=256, ldq=1 << 16) == E_SHAPE       # too many blocks
    for rot, n in ((0, 9), (3, 9), (66, 9), (64, 0)):
        assert call(cs=GOOD, rot=rot, max_pos=n) == E_SHAPE, (rot, n)
    for name in ("k", "v", "lens", "table", "cache", "q_out"):
        assert call(**{name: None}) == E_NULL, name
    for name in ("k", "v", "q", "q_out"):
        assert call(**{name: GOOD + 1}) == E_ALIGN, name
    assert call(xdt=0, k=ODD2) == E_ALIGN and call(cache=GOOD + 8) == E_ALIGN and call(lens=ODD2) == E_ALIGN
    assert call(q_start=ODD2) == E_ALIGN and call(table=ODD2) == E_ALIGN and call(cs=ODD2, rot=64, max_pos=9) == E_ALIGN


def test_read_validation(lib):
    def call(odt=0, T=4, Hkv=2, D=64, pos=GOOD, B=2, max_pages=3, table=GOOD, page=16, pages=5, cache=GOOD, k=GOOD, v=GOOD):
        return lib.sfx_kv_read_q8(None, odt, T, Hkv, D, pos, None, B, max_pages, table, page, pages, cache, k, v)
    assert call(odt=3) == E_DTYPE and call(T=0) == E_SHAPE and call(D=33) == E_SHAPE and call(page=8) == E_SHAPE
    for name in ("pos", "table", "cache", "k", "v"):
        assert call(**{name: None}) == E_NULL, name
    assert call(k=GOOD + 8) == E_ALIGN and call(v=ODD2) == E_ALIGN and call(table=ODD2) == E_ALIGN


def test_attention_validation(lib):
    def ws_of(B=2, max_q=1, Hq=8, Hkv=2, D=64, n=4800):
        return lib.sfx_attn_q8_ws(B, max_q, Hq, Hkv, D, n)

    def call(qdt=1, T=5, B=2, max_q=1, Hq=8, Hkv=2, D=64, q=GOOD, ldq=512, q_start=GOOD, max_pages=300, table=GOOD, page=16,
             pages=5, cache=GOOD, starts=None, lens=GOOD, window=0, scale=0.1, out=GOOD, lse=None, ws=0x100000, n=None):
        return lib.sfx_attn_q8(None, qdt, T, B, max_q, Hq, Hkv, D, q, ldq, q_start, max_pages, table, page, pages, cache,
                               starts, lens, window, ctypes.c_float(scale), out, lse, ws, ws_of() if n is None else n)
    assert ws_of() > 0 and ws_of(n=64) == 0            # one run: nothing to join
    assert ws_of(B=4097) == 0 and ws_of(Hq=7) == 0 and ws_of(D=48) == 0 and ws_of(n=0) == 0 and ws_of(max_q=0) == 0
    assert call(qdt=0) == E_DTYPE and call(qdt=3) == E_DTYPE
    assert call(T=0) == E_SHAPE and call(T=(1 << 20) + 1) == E_SHAPE and call(max_q=0) == E_SHAPE
    assert call(q_start=None) == E_SHAPE and call(q_start=None, T=2, max_q=2) == E_SHAPE
    assert call(B=0) == E_SHAPE and call(B=4097) == E_SHAPE and call(Hq=7) == E_SHAPE and call(Hq=0) == E_SHAPE
    # workgroups for rows that no sequence has: 2^12 x 8 x 2^17
    assert call(B=4096, max_q=1 << 20, Hq=128, Hkv=8, ldq=128 * 64, T=1 << 20) == E_SHAPE
    assert ws_of(B=4096, max_q=1 << 20, Hq=128, Hkv=8) == 0
    assert call(max_q=1 << 20, Hq=256, ldq=1 << 16, T=1 << 20) == E_SHAPE and call(window=-1) == E_SHAPE
    assert call(Hq=512, ldq=1 << 16) == E_SHAPE and call(ldq=511) == E_SHAPE and call(page=8) == E_SHAPE
    for s in (float("nan"), float("inf"), float("-inf")):
        assert call(scale=s) == E_SHAPE
    for name in ("q", "table", "cache", "lens", "out"):
        assert call(**{name: None}) == E_NULL, name
    assert call(q=ODD4) == E_ALIGN and call(ldq=516) == E_ALIGN and call(out=ODD4) == E_ALIGN and call(lens=ODD2) == E_ALIGN
    assert call(starts=ODD2) == E_ALIGN and call(lse=ODD2) == E_ALIGN and call(cache=ODD4) == E_ALIGN
    assert call(q_start=ODD2) == E_ALIGN
    assert call(ws=None) == E_WORKSPACE and call(ws=0x100010) == E_WORKSPACE and call(n=ws_of() - 1) == E_WORKSPACE


def test_workspace_stays_small(lib):
    """No workspace passes 64 MiB."""
    for B, m, Hq, Hkv, D, n in ((1, 1, 64, 8, 128, 131072), (64, 1, 128, 8, 64, 4096), (1, 4096, 256, 1, 256, 1 << 30),
                                (3, 7, 160, 8, 256, 1 << 20), (1, 200, 8, 8, 256, 1 << 20), (4096, 1, 1, 1, 32, 1 << 20), (511, 1, 1, 1, 256, 1 << 30)):
        assert lib.sfx_attn_q8_ws(B, m, Hq, Hkv, D, n) <= 64 << 20


def test_binding_refusals():
    """Shapes and dtypes are refused before the device is looked at, then tensors off the GPU."""
    f = torch.zeros
    x, r, q, s = f(3, 64), f(3, 64), f(3, 64, dtype=torch.int8), f(3)
    with pytest.raises(ValueError, match="on the GPU"):
        A.sfx_norm_q8(x, q, s)
    for bad in (dict(x=f(64)),):
        with pytest.raises(ValueError):
            A.sfx_norm_q8(**{**dict(x=x, q=q, s=s, residual=r), **bad})
    with pytest.raises(TypeError):
        A.sfx_norm_q8(x.double(), q, s)
    x8, W, sw, y = f(2, 64, dtype=torch.int8), f(8, 64, dtype=torch.int8), f(8), f(2, 8)
    ln = dict(x=x8, x_scales=f(2), W=W, W_scales=sw, y=y)
    with pytest.raises(ValueError, match="on the GPU"):
        A.sfx_linear_q8(**ln)
    for bad in (dict(x=f(2, 32, dtype=torch.int8)), dict(y=f(2, 9)), dict(W_scales=f(7)), dict(x_scales=f(3)), dict(x=f(64))):
        with pytest.raises(ValueError):
            A.sfx_linear_q8(**{**ln, **bad})
    for bad in (dict(x=f(2, 64)), dict(y=y.double())):
        with pytest.raises(TypeError):
            A.sfx_linear_q8(**{**ln, **bad})

    k, lens = f(3, 2, 64, dtype=torch.float16), f(3, dtype=torch.int32)
    table, cache = f(3, 4, dtype=torch.int32), f(6, 2, 1, 32 * 64 + 16, dtype=torch.uint8)
    ap = dict(q=None, k=k, v=k.clone(), lens=lens, table=table, cache=cache, q_out=None)
    with pytest.raises(ValueError, match="on the GPU"):
        A.sfx_kv_append_q8(**ap)
    with pytest.raises(ValueError):
        A.sfx_kv_append_q8(**{**ap, "v": k[:2]})
    with pytest.raises(TypeError):
        A.sfx_kv_append_q8(**{**ap, "k": k.double(), "v": k.double()})
    rd = dict(pos=lens, table=table, cache=cache, k_out=k, v_out=k.clone())
    with pytest.raises(ValueError, match="on the GPU"):
        A.sfx_kv_read_q8(**rd)
    with pytest.raises(ValueError):
        A.sfx_kv_read_q8(**{**rd, "v_out": k.float()})
    at = dict(q=f(3, 4, 64, dtype=torch.float16), cache=cache, table=table, lens=lens, out=f(3, 4, 64, dtype=torch.float16),
              ws=f(256, dtype=torch.uint8))
    with pytest.raises(ValueError, match="on the GPU"):
        A.sfx_attn_q8(**at)
    for bad in (dict(out=f(3, 4, 32, dtype=torch.float16)), dict(cache=f(6, 2, 2, 500, dtype=torch.uint8)),
                dict(table=f(2, 4, dtype=torch.int32)), dict(q=f(3, 64, dtype=torch.float16))):
        with pytest.raises(ValueError):
            A.sfx_attn_q8(**{**at, **bad})
    with pytest.raises(TypeError):
        A.sfx_attn_q8(**{**at, "q": at["q"].float()})
    with pytest.raises(A.SfxError):
        A.kv_cache_q8(4, 2, 8, 64, device="cpu")
    assert A.kv_cache_q8(4, 2, 32, 64, device="cpu").shape == (4, 2, 2, 2064)


# ------------------------------------------------------------------------------ pins of the oracle

def test_norm_worked():
    """h = (3, 4): mean square 12.5; n = h / sqrt(12.5); the codes are 127 h / 4."""
    h, n = Q.norm_rows(np.array([[1.0, 4.5]]), np.array([[2.0, -0.5]]), None, 0.0, True)
    assert np.array_equal(h, [[3.0, 4.0]]) and np.allclose(n, np.array([[3.0, 4.0]]) / np.sqrt(12.5), rtol=1e-15)
    s, q = Q.row_codes(n)
    assert np.array_equal(q, [[95, 127]]) and abs(s[0] * 127 - 4 / np.sqrt(12.5)) < 1e-7
    s, q = Q.row_codes(np.array([[0.0, 0.0], [np.nan, 1.0], [np.inf, 1.0], [0.5, -127.0], [1.5, 127.0]]))
    assert s[0] == 0 and np.isnan(s[1]) and np.isnan(s[2]) and s[3] == 1
    assert np.array_equal(q, [[0, 0], [0, 0], [0, 0], [0, -127], [2, 127]])      # ties to even


def test_linear_worked():
    p, y = Q.linear(np.array([[1, -2], [127, 127]]), np.array([0.5, 1.0], np.float32), np.array([[3, 4]]),
                    np.array([2.0], np.float32), np.array([1.0], np.float32))
    assert np.array_equal(p, [[-5], [889]]) and np.array_equal(y, [[-4.0], [1779.0]])


def test_block_layout():
    """Each code is found where the layout says, and writing undoes reading."""
    D = 32
    rng = np.random.default_rng(0)
    raw = rng.integers(0, 256, 32 * D + 16).astype(np.uint8)
    raw[32 * D:32 * D + 8] = np.array([0.5, 2.0], np.float32).view(np.uint8)
    k, v, ks, vs = Q.read_block(raw, D)
    assert k[3, 7] == int(raw[3 * D + 7]) - 128 and v[6, 9] == int(raw[16 * D + (D + 9) * 4 + 2]) - 128 and (ks, vs) == (0.5, 2)
    again = raw.copy()
    again[:32 * D + 8] = 0
    Q.write_block(again, D, k, v, ks, vs)
    assert np.array_equal(raw, again)


def test_store_rows_worked():
    q = np.full((16, 2), 99)
    out, s = Q.store_rows(q, np.float32(7), np.array([[127, -63.5]], np.float32), 0)          # started anew
    assert s == 1 and np.array_equal(out[0], [127, -64]) and (out[1:] == 0).all()
    out2, s2 = Q.store_rows(out, s, np.array([[50, 3.5]], np.float32), 1)                     # fits
    assert s2 == 1 and np.array_equal(out2[:2], [[127, -64], [50, 4]])
    out3, s3 = Q.store_rows(out2, s2, np.array([[-254, 0]], np.float32), 2)                   # grows: halves, ties to even
    assert s3 == 2 and np.array_equal(out3[:3], [[64, -32], [25, 2], [-127, 0]])
    out4, s4 = Q.store_rows(out3, s3, np.array([[np.inf, 0]], np.float32), 3)
    assert np.isnan(s4) and (out4 == 0).all()
    assert np.isnan(Q.store_rows(out4, s4, np.array([[1, 0]], np.float32), 4)[1])
    out5, s5 = Q.store_rows(q, np.float32(0), np.zeros((16, 2), np.float32), 0)
    assert s5 == 0 and (out5 == 0).all()


def test_attention_worked():
    """Two positions whose scores differ by ln 3: weights 1/4 and 3/4."""
    q = np.array([[1.0, 0.0]])
    k = np.array([[0.0, 5.0], [np.log(3.0), 1.0]])
    v = np.array([[4.0, 0.0], [0.0, -8.0]])
    o, lse, ab, size = Q.attention(q, k, v, 1.0)
    assert np.allclose(o, [[1.0, -6.0]]) and np.allclose(lse, np.log(4.0)) and np.allclose(ab, [[1.0, 6.0]])
    assert np.allclose(size, np.log(3.0))
    o, lse, _, _ = Q.attention(q, k[:0], v[:0], 1.0)
    assert (o == 0).all() and lse[0] == -np.inf
