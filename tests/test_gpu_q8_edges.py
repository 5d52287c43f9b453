"""The 8-bit layer half at the ends of its ranges."""
import numpy as np
import pytest
import torch

from activation_sparse_ffn_amd import _abi as A
from gpu_helpers import say
from oracle import q8_oracle as Q
from test_gpu_q8 import DEV, DT, HALF_STEP, TINY, check_norm, logical, make_cache, make_table, np64

pytestmark = pytest.mark.gpu


def i32(a):
    return torch.from_numpy(np.asarray(a, np.int32)).to(DEV)


# ------------------------------------------------------------------------------ norm

NORM_SIZES = [  # largest size of x and of the weights: 127 / max |h w| leaves fp32's normal numbers, scales do too
    (1.0, 1.0), (3e37, 1e3), (3e37, 1e5), (3e38, 1e6), (1e30, 1e13), (3e38, 1e8), (3e38, 3e38), (1e10, 1e-36), (1e10, 1e-43),
    (1e20, 1e-40), (1e-30, 1e38), (1e-40, 1e-3), (1e-44, 1e5)]


def sized_rows(T, d, sizes, seed):
    """Rows of which the first len(sizes) have these sizes, with one strong element in a hundred."""
    g = torch.Generator().manual_seed(seed)
    x = torch.rand(T, d, generator=g, dtype=torch.float64) * 2 - 1
    x *= torch.where(torch.rand(T, d, generator=g) < 0.01, 1.0, 0.05)
    x[:, d // 3] = 1.0
    x[:len(sizes)] *= torch.tensor(sizes, dtype=torch.float64)[:, None]
    return x.float()


@pytest.mark.parametrize("d", [40, 1000, 4096, 9000])
def test_norm_codes_of_any_finite_product(d):
    """Rows up to fp32's largest number with weights of any size: every code is the nearest one, where the
    quotient's factors leave fp32's normal numbers too."""
    say(f"norm sizes {d}")
    for xs, ws in NORM_SIZES:
        x = sized_rows(3, d, [xs, xs / 7, xs / 1000], d)
        w = (1 + 0.3 * torch.randn(d, generator=torch.Generator().manual_seed(1)))
        w = (w.double() / w.abs().max() * ws).float()
        q, s = torch.full((3, d), 99, dtype=torch.int8, device=DEV), torch.full((3,), -1.0, device=DEV)
        r = x.roll(1, 1) / 10
        for res in (None, r):
            ro = None if res is None else res.to(DEV)
            A.sfx_norm_q8(x.to(DEV), q, s, weight=w.to(DEV), residual=ro)
            check_norm((3, d, "f32", None if res is None else "f32", None, True, True), x, res, w, q, s, ro, None)


@pytest.mark.parametrize("d,T", [(333, 160000), (1000, 51000), (2041, 25000), (4096, 12400), (8190, 6300), (16384, 3200)])
def test_norm_codes_of_any_finite_product_many_rows(d, T):
    """The same where rows stay in registers (more than the last-level cache holds)."""
    say(f"norm sizes {T}x{d}")
    for ws in (1e3, 1e6, 1e13, 3e38, 1e-36, 1e-43):
        sizes = [3e38, 3e37, 1e30, 1e20, 1e10, 1.0, 1e-3, 1e-20, 1e-38, 1e-44]
        x = sized_rows(len(sizes), d, sizes, d)
        w = (1 + 0.3 * torch.randn(d, generator=torch.Generator().manual_seed(1)))
        w = (w.double() / w.abs().max() * ws).float()
        big = torch.ones(T, d, device=DEV)
        at = torch.linspace(0, T - 1, len(sizes)).long()
        big[at.to(DEV)] = x.to(DEV)
        q, s = torch.full((T, d), 99, dtype=torch.int8, device=DEV), torch.full((T,), -1.0, device=DEV)
        A.sfx_norm_q8(big, q, s, weight=w.to(DEV))
        check_norm((len(sizes), d, "f32", None, None, True, True), x, None, w, q.cpu()[at], s.cpu()[at], None, None)


# ------------------------------------------------------------------------------ attention

def check_rows(Hq, Hkv, D, dt, page, table, cache, lens, counts, window=0, seed=0, q_scale=1.3, rows=None, max_q=None, starts=None):
    """Rows of a call against the oracle; outputs below the type's normal numbers to its last bit.  `rows` of
    a sequence are looked at (None: all); those past max_q are left as they were."""
    g = torch.Generator().manual_seed(seed)
    q_start = np.concatenate([[0], np.cumsum(counts)])
    T, most = int(q_start[-1]), max(counts) if max_q is None else max_q
    q = (torch.randn(T, Hq, D, generator=g) * q_scale).to(DT[dt])
    out, lse = torch.full((T, Hq, D), 7.0, dtype=DT[dt], device=DEV), torch.full((T, Hq), 7.0, device=DEV)
    ws = A.workspace(A.sfx_attn_q8_ws(len(lens), most, Hq, Hkv, D, table.shape[1] * page))
    ws.fill_(255)
    A.sfx_attn_q8(q.to(DEV), cache.to(DEV), table.to(DEV), i32(lens), out, ws, q_start=i32(q_start), max_q=most, window=window, lse=lse,
                  starts=None if starts is None else i32(starts))
    got, gl = np64(out), np64(lse)
    for b, n in enumerate(lens):
        k, v, has = logical(cache, table.numpy(), page, b, n, D)
        some = range(counts[b]) if rows is None else sorted(set(np.linspace(0, counts[b] - 1, rows).astype(int)))
        for i in some:
            t, p = q_start[b] + i, n - counts[b] + i
            if i >= most:
                assert (got[t] == 7).all() and (gl[t] == 7).all(), (b, i)
                continue
            lo = max(0, p + 1 - window) if window else 0
            lo = lo if starts is None else max(lo, starts[b])
            keep = np.arange(lo, p + 1)[has[lo:p + 1]] if p + 1 > lo else np.arange(0)
            for h in range(Hkv):
                hs = slice(h * (Hq // Hkv), (h + 1) * (Hq // Hkv))
                o, l, ab, size = Q.attention(np64(q[t, hs]), k[keep, h], v[keep, h], D ** -0.5)
                if not len(keep):
                    assert (got[t, hs] == 0).all() and (gl[t, hs] == -np.inf).all(), (b, i, h)
                    continue
                tol, ltol = Q.attention_tolerance(o, l, ab, size, np.abs(v[keep, h]).max(), len(keep), D, HALF_STEP[dt])
                top = {"f16": 65520, "bf16": 2.0 ** 128 * (1 - 2.0 ** -9)}[dt]       # what is rounded to an infinity
                over = (np.abs(o) + tol >= top) & np.isinf(got[t, hs]) & (np.sign(got[t, hs]) == np.sign(o))
                err = np.where(over, 0.0, np.abs(got[t, hs] - o))
                assert (err <= tol + TINY[dt]).all(), (b, i, h, err.max(), o, got[t, hs])
                assert (np.abs(gl[t, hs] - l) <= ltol).all(), (b, i, h, gl[t, hs], l)


@pytest.mark.parametrize("dt", ["f16", "bf16"])
def test_attention_fewer_rows_than_a_sequence_has(dt):
    """Rows past max_q are left out; those in front keep their positions."""
    for Hq, Hkv, D, lens, counts, most in ((4, 2, 64, [40, 60, 9], [5, 3, 9], 3), (8, 1, 128, [300], [40], 7), (2, 1, 96, [500, 77], [300, 77], 200),
                                           (1, 1, 256, [3000], [2500], 130), (4, 4, 64, [5000], [30], 1)):
        say(f"max_q {most} of {counts} {dt}")
        table, pages = make_table(lens, 16, 3)
        cache = make_cache(pages, Hkv, 16, D, 4)
        check_rows(Hq, Hkv, D, dt, 16, table, cache, lens, counts, max_q=most, rows=9)
        check_rows(Hq, Hkv, D, dt, 16, table, cache, lens, counts, max_q=most, rows=9, window=30, starts=[2] * len(lens))


def test_attention_windows_past_every_position():
    """The longest window is none, also for calls with rows in front of position 0."""
    D, page = 64, 16
    lens, counts = [3, 40, 7, 0], [9, 5, 120, 6]
    table, pages = make_table(lens, page, 3)
    cache = make_cache(pages, 2, page, D, 4)
    q_start = np.concatenate([[0], np.cumsum(counts)])
    q = torch.randn(int(q_start[-1]), 4, D, generator=torch.Generator().manual_seed(1)).half().to(DEV)
    ws = A.workspace(A.sfx_attn_q8_ws(4, 120, 4, 2, D, table.shape[1] * page))
    outs = []
    for window in (0, 2 ** 31 - 1, 2 ** 31 - 5, 1 << 20):
        outs.append((torch.full_like(q, 7.0), torch.full((len(q), 4), 7.0, device=DEV)))
        A.sfx_attn_q8(q, cache.to(DEV), table.to(DEV), i32(lens), outs[-1][0], ws, q_start=i32(q_start), max_q=120, window=window, lse=outs[-1][1])
    assert (outs[0][0][6:9] != 0).any() and (outs[0][0][:6] == 0).all()
    for o, l in outs[1:]:
        assert torch.equal(o, outs[0][0]) and torch.equal(l, outs[0][1])
