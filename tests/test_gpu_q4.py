"""The int4 attention half of a layer (sfx_linear_q4, sfx_kv_append_q4, sfx_kv_read_q4,
sfx_attn_q4) against the fp64 oracle, at the sizes and masks where it can go wrong."""
import numpy as np
import pytest
import torch

from activation_sparse_ffn_amd import _abi as A
from gpu_helpers import say
from oracle import q4_oracle as Q

pytestmark = pytest.mark.gpu
DEV = "cuda"
DT = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
HALF_STEP = {"f16": 2.0 ** -11, "bf16": 2.0 ** -8, "f32": 2.0 ** -24}


def np64(t):
    return t.detach().cpu().to(torch.float64).numpy()


def assert_same(got, want, where=""):
    """Equal values (NaN where NaN is wanted)."""
    got, want = got.detach().cpu(), want.detach().cpu()
    assert got.shape == want.shape and got.dtype == want.dtype
    bad = ~((got == want) | (got.isnan() & want.isnan()))
    if bad.any():
        at = bad.nonzero()[:5].tolist()
        raise AssertionError((where, int(bad.sum()), at, [(got[tuple(i)].item(), want[tuple(i)].item()) for i in at]))


# ------------------------------------------------------------------------------ linear

def make_linear(B, n, d, group, dt, seed):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(B, d, generator=g).to(DT[dt])
    W = torch.randint(0, 256, (n, d // 2), generator=g, dtype=torch.uint8)
    s = (0.05 * torch.rand(n, d // group, generator=g) + 1e-3).half()
    bias = torch.randn(n, generator=g)
    return x, W, s, bias


LINEAR = [(3, 40, 8192, 64), (2, 20, 40960, 128), (16, 33, 2016, 32), (13, 8200, 1056, 32), (40, 8193, 288, 32),
          (64, 8192, 160, 32), (1, 1, 32, 32), (1, 17, 64, 64), (2, 15, 96, 32), (1, 33, 128, 128), (3, 100, 160, 32), (4, 1003, 1056, 32),
          (5, 48, 192, 64), (8, 130, 4096, 128), (9, 64, 1024, 32), (16, 257, 640, 128), (17, 31, 2048, 64),
          (32, 96, 352, 32), (33, 80, 512, 128), (64, 129, 1152, 64), (1, 4096, 4096, 32), (7, 512, 8192, 32)]


@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("case", LINEAR, ids=lambda c: "x".join(map(str, c)))
def test_linear(case, dt):
    B, n, d, group = case
    say(f"linear {case} {dt}")
    x, W, s, bias = make_linear(B, n, d, group, dt, B * n + d)
    ref = Q.linear_q4(np64(x), W.numpy(), s.numpy(), bias.numpy())
    tol = Q.linear_q4_bound(np64(x), W.numpy(), s.numpy()) + 2.0 ** -22 * (np.abs(ref) + np.abs(bias.numpy()))
    xd, Wd, sd, bd = (t.to(DEV) for t in (x, W, s, bias))
    y = torch.full((B, n), float("nan"), device=DEV)
    A.sfx_linear_q4(xd, Wd, sd, y, bias=bd)
    err = np.abs(np64(y) - ref)
    assert (err <= tol).all(), (err / tol).max()
    # the same numbers again, bit for bit, without the bias and added to what is there
    y2 = torch.full((B, n), float("nan"), device=DEV)
    A.sfx_linear_q4(xd, Wd, sd, y2, bias=bd)
    assert torch.equal(y, y2)
    y0 = torch.randn(B, n, generator=torch.Generator().manual_seed(1))
    y3 = y0.to(DEV)
    A.sfx_linear_q4(xd, Wd, sd, y3, accumulate=True)
    ref3 = y0.numpy() + Q.linear_q4(np64(x), W.numpy(), s.numpy())
    assert (np.abs(np64(y3) - ref3) <= tol + 2.0 ** -23 * np.abs(ref3)).all()
    say("   rel %.2e" % (np.linalg.norm(np64(y) - ref) / np.linalg.norm(ref)))


@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("B", [1, 3, 8, 11, 40])
def test_linear_rows_apart(B, dt):
    """x and y as slices of wider tensors; what lies beside y's rows stays as it was."""
    n, d, group = 203, 288, 32
    say(f"linear strided B={B} {dt}")
    x, W, s, _ = make_linear(B, n, d, group, dt, 5)
    wide = torch.full((B, d + 40), float("nan"), dtype=DT[dt], device=DEV)
    wide[:, 8:8 + d] = x.to(DEV)
    yw = torch.full((B, n + 9), 7.0, device=DEV)
    A.sfx_linear_q4(wide[:, 8:8 + d], W.to(DEV), s.to(DEV), yw[:, 5:5 + n])
    ref = Q.linear_q4(np64(x), W.numpy(), s.numpy())
    assert (np.abs(np64(yw[:, 5:5 + n]) - ref) <= Q.linear_q4_bound(np64(x), W.numpy(), s.numpy())).all()
    assert (yw[:, :5] == 7).all() and (yw[:, 5 + n:] == 7).all()


@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("B", [2, 6, 20])
def test_linear_bad_token_stays_alone(B, dt):
    """A NaN or an infinity in one token's x leaves the other tokens' results as they were,
    and the smallest and largest finite numbers are taken as they are."""
    n, d = 100, 256
    say(f"linear bad token B={B} {dt}")
    x, W, s, _ = make_linear(B, n, d, 64, dt, 9)
    tiny, big = (2.0 ** -24, 60000.0) if dt == "f16" else (2.0 ** -133, 1e30)
    x[0, :] = tiny * torch.arange(d).remainder(7)
    x[0, 3] = tiny
    good = torch.empty(B, n, device=DEV)
    A.sfx_linear_q4(x.to(DEV), W.to(DEV), s.to(DEV), good)
    ref = Q.linear_q4(np64(x), W.numpy(), s.numpy())
    tol = Q.linear_q4_bound(np64(x), W.numpy(), s.numpy())
    assert (np.abs(np64(good) - ref) <= tol).all(), (np.abs(np64(good) - ref) / tol).max()
    for v in (float("nan"), float("inf"), big):
        x[B - 1, 17] = v
        y = torch.empty(B, n, device=DEV)
        A.sfx_linear_q4(x.to(DEV), W.to(DEV), s.to(DEV), y)
        assert torch.equal(y[:B - 1], good[:B - 1])
        if v == big:
            assert torch.isfinite(y).all()
        else:
            q17 = Q.unpack_rows(W.numpy())[:, 17]
            assert not torch.isfinite(y[B - 1].cpu()[torch.from_numpy(q17 != 0)]).any()


# ------------------------------------------------------------------------------ cache

def make_table(lens, page, seed, spare=2, width=None):
    """Shuffled page table for sequences of the given lengths (host tensor) and page count."""
    per = [-(-n // page) for n in lens]
    order = torch.randperm(sum(per) + spare, generator=torch.Generator().manual_seed(seed)).to(torch.int32)
    table = torch.full((len(lens), max(1, max(per)) if width is None else width), -1, dtype=torch.int32)
    at = 0
    for b, k in enumerate(per):
        table[b, :k] = order[at:at + k]
        at += k
    return table, sum(per) + spare


def rope_table(max_pos, rot):
    i = np.arange(rot // 2)
    ang = np.arange(max_pos)[:, None] * 10000.0 ** (-2.0 * i / rot)
    return np.concatenate([np.cos(ang), np.sin(ang)], 1).astype(np.float32)


APPEND = [  # D, Hq, Hkv, page, dtype, rope, rot
    (32, 1, 1, 8, "f32", "half", 32), (64, 4, 2, 16, "f16", "pairs", 64), (96, 3, 3, 8, "bf16", "half", 50),
    (128, 8, 2, 16, "f32", "half", 128), (128, 5, 5, 64, "f16", "none", 0), (160, 2, 1, 32, "bf16", "pairs", 2),
    (192, 2, 2, 8, "f32", "half", 2), (224, 1, 1, 16, "f16", "half", 224), (256, 16, 4, 128, "bf16", "pairs", 130)]


@pytest.mark.parametrize("case", APPEND, ids=lambda c: "-".join(map(str, c)))
def test_append_and_read(case):
    """Tokens of ragged sequences in mixed order with padding, as slices of one projection:
    bytes, values and rotated queries as the oracle has them, everything else untouched."""
    D, Hq, Hkv, page, dt, rope, rot = case
    say(f"append {case}")
    rng = np.random.default_rng(D + Hq)
    lens = [37, 1, 0, 64, 9]
    table, pages = make_table(lens, page, 3)
    seq = np.concatenate([np.full(n, b) for b, n in enumerate(lens)] + [[0, 1, 7, -1, 2]]).astype(np.int32)
    pos = np.concatenate([np.arange(n) for n in lens] + [[-1, 100000, 0, 0, 0]]).astype(np.int32)
    real = np.arange(len(seq)) < sum(lens)
    order = rng.permutation(len(seq))
    seq, pos, real = seq[order], pos[order], real[order]
    T = len(seq)
    g = torch.Generator().manual_seed(D)
    qkv = (torch.randn(T, (Hq + 2 * Hkv) * D + 8, generator=g) * 3).to(DT[dt])
    k_at, v_at = Hq * D, (Hq + Hkv) * D
    qkv[0, k_at:k_at + 32] = 0                         # a group of zeros
    if dt != "f16":
        qkv[1, v_at:v_at + 32] *= 1e5                  # beyond the V scale's range: clipped
    qkv[2, v_at + 1] = float("nan")
    qkv[3, k_at + D - 1] = float("inf")
    cs = rope_table(128, rot) if rope != "none" else None
    dev = qkv.to(DEV)
    cut = lambda a, h: dev[:, a:a + h * D].unflatten(1, (h, D))  # noqa: E731
    q, k, v = cut(0, Hq), cut(k_at, Hkv), cut(v_at, Hkv)
    before = torch.randint(0, 256, (pages, Hkv, page // 8, 9 * D), generator=g, dtype=torch.uint8)
    cache = before.to(DEV)
    odt = "bf16" if dt == "bf16" else "f16"
    q_out = torch.full((T, Hq, D), 5.0, dtype=DT[odt], device=DEV)
    d_pos, d_seq, d_table = (torch.from_numpy(a).to(DEV) for a in (pos, seq, table.numpy()))
    d_cs = None if cs is None else torch.from_numpy(cs).to(DEV)
    A.sfx_kv_append_q4(q, k, v, d_pos, d_table, cache, q_out, seq=d_seq, cos_sin=d_cs, interleaved=rope == "pairs")

    host = lambda t: t.cpu().float().numpy()  # noqa: E731
    at = np.where(real, pos, 0)
    kr, qr = (Q.rotate(host(x), at, cs, rope == "pairs") for x in (k, q))
    want_q = torch.from_numpy(qr).to(DT[odt])
    want_q[~torch.from_numpy(real)] = 5.0
    assert_same(q_out, want_q, "q_out")
    kq, ks = Q.quantise(kr, 65504.0)
    vq, vs = Q.quantise(host(v), 8188.0)

    got = cache.cpu().numpy()
    seen = np.zeros(got.shape[:3] + (8,), bool)          # written positions
    for t in np.flatnonzero(real):
        pg, r = int(table[seq[t], pos[t] // page]), pos[t] % page
        for h in range(Hkv):
            b = Q.read_block(got[pg, h, r // 8], D, r % 8)
            assert np.array_equal(b[0], kq[t, h]) and np.array_equal(b[2], vq[t, h]), (t, h)
            assert np.array_equal(b[1], ks[t, h], equal_nan=True) and np.array_equal(b[3], vs[t, h], equal_nan=True)
            seen[pg, h, r // 8, r % 8] = True
    old = before.numpy()
    for pg, h, o, i in zip(*np.nonzero(~seen)):
        was, now = Q.read_block(old[pg, h, o], D, i), Q.read_block(got[pg, h, o], D, i)
        assert all(np.array_equal(a, b, equal_nan=True) for a, b in zip(was, now)), (pg, h, o, i)

    for rdt in ("f32", "f16", "bf16"):
        ko = torch.full((T, Hkv, D), float("nan"), dtype=DT[rdt], device=DEV)
        vo = torch.full_like(ko, float("nan"))
        A.sfx_kv_read_q4(d_pos, d_table, cache, ko, vo, seq=d_seq)
        for out, q_, s_ in ((ko, kq, ks), (vo, vq, vs)):
            want = torch.from_numpy(np.where(real[:, None, None], Q.values(q_, s_), 0.0)).to(torch.float32).to(DT[rdt])
            assert_same(out, want, rdt)


def test_append_without_queries_and_seq():
    """Keys and values only, token t of sequence t (a decode step); a token past the table's
    rows is padding."""
    D, Hkv, page, T = 64, 3, 8, 5
    table, pages = make_table([9, 20, 1, 8], page, 1)
    pos = torch.tensor([8, 19, 0, 3, 0], dtype=torch.int32, device=DEV)
    g = torch.Generator().manual_seed(2)
    k, v = (torch.randn(T, Hkv, D, generator=g).half().to(DEV) for _ in range(2))
    cache = torch.zeros(pages, Hkv, page // 8, 9 * D, dtype=torch.uint8, device=DEV)
    A.sfx_kv_append_q4(None, k, v, pos, table.to(DEV), cache, None)
    ko, vo = torch.empty(T, Hkv, D, device=DEV), torch.empty(T, Hkv, D, device=DEV)
    A.sfx_kv_read_q4(pos, table.to(DEV), cache, ko, vo)
    for x, out, top in ((k, ko, 65504.0), (v, vo, 8188.0)):
        want = Q.values(*Q.quantise(x.cpu().float().numpy(), top))
        want[4] = 0
        assert np.array_equal(np64(out), want)


# ------------------------------------------------------------------------------ attention

def make_attn(B, Hq, Hkv, D, page, lens, dt, seed, spread=1.0, width=None):
    """A filled cache (random codes, scales NaN where nothing is stored), queries, and the
    oracle's values of every stored position."""
    rng = np.random.default_rng(seed)
    table, pages = make_table(lens, page, seed, width=width)
    T = sum(lens)
    seq = np.concatenate([np.full(n, b) for b, n in enumerate(lens)]).astype(np.int32)
    pos = np.concatenate([np.arange(n) for n in lens]).astype(np.int32)
    cache = torch.full((pages, Hkv, page // 8, 9 * D), 0xFF, dtype=torch.uint8, device=DEV)   # fp16 0xFFFF: NaN
    k = torch.from_numpy((rng.standard_normal((T, Hkv, D)) * spread).astype(np.float32)).to(DEV)
    v = torch.from_numpy(rng.standard_normal((T, Hkv, D)).astype(np.float32)).to(DEV)
    d_table = table.to(DEV)
    if T:
        args = (torch.from_numpy(pos).to(DEV), d_table, cache)
        d_seq = torch.from_numpy(seq).to(DEV)
        A.sfx_kv_append_q4(None, k, v, *args, None, seq=d_seq)
        ko, vo = torch.empty(T, Hkv, D, device=DEV), torch.empty(T, Hkv, D, device=DEV)
        A.sfx_kv_read_q4(*args, ko, vo, seq=d_seq)
        kn, vn = np64(ko), np64(vo)
    else:
        kn = vn = np.zeros((0, Hkv, D))
    q = torch.from_numpy(rng.standard_normal((B, Hq, D)).astype(np.float32)).to(DT[dt])
    at = np.concatenate([[0], np.cumsum(lens)])
    return q, cache, d_table, [(kn[at[b]:at[b + 1]], vn[at[b]:at[b + 1]]) for b in range(B)]


def check_attn(q, kv, lens, starts, scale, dt, out, lse, skip=None):
    worst = 0.0
    got, got_l = np64(out), np64(lse)
    for b, (k, v) in enumerate(kv):
        lo = max(0, starts[b]) if starts is not None else 0
        keep = np.arange(len(k)) >= lo
        keep &= np.arange(len(k)) < lens[b]
        if skip is not None:
            keep &= ~skip[b]
        k, v = k[keep], v[keep]
        qb = np64(q[b])
        o, ls, ab = Q.attention(qb, k, v, scale)
        if len(k) == 0:
            assert (got[b] == 0).all() and np.isneginf(got_l[b]).all()
            continue
        # scores: fp32 error d gives weights off by 2 d; weight and value each rounded once to
        # fp16 (half a step 2^-11), sums in fp32, the result rounded once to its type
        top_scale = np.abs(k).reshape(len(k), k.shape[1], -1, 32).max((0, 1, 3)) / 7
        d = Q.score_bound(qb, top_scale, scale) + 2.0 ** -22 * 40
        tol = (2 * 2.0 ** -11 + 2 * d + 2.0 ** -18) * ab * 1.01 + HALF_STEP[dt] * np.abs(o) + 2.0 ** -25
        err = np.abs(got[b] - o)
        assert (err <= tol).all(), (b, (err / tol).max())
        assert (np.abs(got_l[b] - ls) <= d + 2.0 ** -20 * (1 + np.abs(ls))).all()
        worst = max(worst, float((err / tol).max()))
    say("   largest error / bound %.2f" % worst)


ATTN = [  # Hq, Hkv, D, page, lens, dt
    (1, 1, 32, 8, [1], "f16"), (4, 4, 64, 16, [7, 8, 9, 0], "bf16"), (8, 2, 128, 16, [31, 32, 33, 64], "f16"),
    (6, 2, 96, 8, [100, 1, 127, 129], "bf16"), (16, 1, 128, 64, [257, 5], "f16"), (17, 1, 64, 32, [70, 300], "bf16"),
    (40, 2, 64, 16, [513], "f16"), (5, 5, 160, 8, [50], "f16"), (2, 1, 192, 1024, [1500], "bf16"),
    (3, 3, 224, 128, [200, 130], "f16"), (8, 1, 256, 16, [900, 40], "bf16"), (32, 32, 128, 16, [700, 12], "f16"),
    (8, 8, 128, 32, [3000], "bf16"), (64, 8, 64, 8, [1025, 2, 600], "f16")]


@pytest.mark.parametrize("case", ATTN, ids=lambda c: "-".join(map(str, c)))
def test_attention(case):
    Hq, Hkv, D, page, lens, dt = case
    B = len(lens)
    say(f"attention {case}")
    q, cache, table, kv = make_attn(B, Hq, Hkv, D, page, lens, dt, Hq + D)
    ws = A.workspace(A.sfx_attn_q4_ws(B, Hq, Hkv, D, table.shape[1] * page))
    d_lens = torch.tensor(lens, dtype=torch.int32, device=DEV)
    qd = q.to(DEV)
    out = torch.full((B, Hq, D), float("nan"), dtype=DT[dt], device=DEV)
    lse = torch.full((B, Hq), float("nan"), device=DEV)
    A.sfx_attn_q4(qd, cache, table, d_lens, out, ws, lse=lse)
    check_attn(q, kv, lens, None, D ** -0.5, dt, out, lse)
    # again on the same workspace: the same bits; without lse too
    out2 = torch.full_like(out, float("nan"))
    A.sfx_attn_q4(qd, cache, table, d_lens, out2, ws)
    assert torch.equal(out, out2)
    # a window: starts before, inside, at and past the end
    for starts in ([max(0, n - 5) for n in lens], [n // 2 + 3 for n in lens], [n for n in lens], [-4 for n in lens],
                   [n + 40 for n in lens]):
        d_starts = torch.tensor(starts, dtype=torch.int32, device=DEV)
        A.sfx_attn_q4(qd, cache, table, d_lens, out, ws, starts=d_starts, scale=0.2, lse=lse)
        check_attn(q, kv, lens, starts, 0.2, dt, out, lse)


def test_attention_sharp_and_flat():
    """Scores from all equal to far apart: the running reference is raised early, late and
    never, and one weight carries the row."""
    Hq, Hkv, D, page, lens = 4, 2, 64, 16, [400, 400, 400, 400]
    q, cache, table, kv = make_attn(4, Hq, Hkv, D, page, lens, "f16", 11)
    q[0] = 0
    q[1] *= 30
    q[2] *= 1e-3
    ws = A.workspace(A.sfx_attn_q4_ws(4, Hq, Hkv, D, table.shape[1] * page))
    out, lse = torch.empty(4, Hq, D, dtype=torch.float16, device=DEV), torch.empty(4, Hq, device=DEV)
    for scale in (D ** -0.5, 1.0, -0.5, 0.0):
        say(f"attention scale {scale}")
        A.sfx_attn_q4(q.to(DEV), cache, table, torch.tensor(lens, dtype=torch.int32, device=DEV), out, ws, scale=scale,
                      lse=lse)
        check_attn(q, kv, lens, None, scale, "f16", out, lse)


def test_attention_missing_pages_and_long_tables():
    """Page ids outside the cache leave their positions out; lens are clamped to the table;
    a table far wider than the sequences."""
    Hq, Hkv, D, page, lens = 8, 4, 128, 8, [130, 64, 40]
    q, cache, table, kv = make_attn(3, Hq, Hkv, D, page, lens, "bf16", 21, width=4000)
    skip = [np.zeros(n, bool) for n in lens]
    for b, j, bad in ((0, 0, -1), (0, 7, 10 ** 6), (0, 16, -5), (1, 3, cache.shape[0])):
        table[b, j] = bad
        skip[b][j * page:(j + 1) * page] = True
    table[2, :] = -7
    skip[2][:] = True
    ws = A.workspace(A.sfx_attn_q4_ws(3, Hq, Hkv, D, table.shape[1] * page))
    out, lse = torch.empty(3, Hq, D, dtype=torch.bfloat16, device=DEV), torch.empty(3, Hq, device=DEV)
    A.sfx_attn_q4(q.to(DEV), cache, table, torch.tensor(lens, dtype=torch.int32, device=DEV), out, ws, lse=lse)
    check_attn(q, kv, lens, None, D ** -0.5, "bf16", out, lse, skip)
    cut = table[:, :9].contiguous()
    A.sfx_attn_q4(q.to(DEV), cache, cut, torch.tensor([130, 10 ** 9, -3], dtype=torch.int32, device=DEV), out, ws, lse=lse)
    check_attn(q, [tuple(x[:72] for x in p) for p in kv], [72, 72, 0], None, D ** -0.5, "bf16", out, lse,
               [s[:72] for s in skip])


# ------------------------------------------------------------------------------ together

def make_layer(d, Hq, Hkv, D, seed):
    """Attention weights of one layer in int4 (host)."""
    g = torch.Generator().manual_seed(seed)
    n = (Hq + 2 * Hkv) * D
    w = {"Wqkv": torch.randint(0, 256, (n, d // 2), generator=g, dtype=torch.uint8),
         "Wqkv_s": (torch.rand(n, d // 32, generator=g) * 0.5 / d ** 0.5 + 1e-3).half(),
         "Wo": torch.randint(0, 256, (d, Hq * D // 2), generator=g, dtype=torch.uint8),
         "Wo_s": (torch.rand(d, Hq * D // (64 if Hq * D % 64 == 0 else 32), generator=g) * 0.5 / (Hq * D) ** 0.5 + 1e-3).half(),
         "bqkv": torch.randn(n, generator=g) * 0.1, "bo": torch.randn(d, generator=g)}
    return w


class Reference:
    """The attention half in fp64 on the host: values of the cache by (sequence, position)."""

    def __init__(self, w, Hq, Hkv, D, cs, pairs, dt, scale):
        self.w = {k: v.numpy() for k, v in w.items()}
        self.Hq, self.Hkv, self.D, self.cs, self.pairs, self.dt, self.scale = Hq, Hkv, D, cs, pairs, dt, scale
        self.k, self.v = {}, {}

    def store(self, b, p, k, v):
        """k, v [Hkv][D] fp32, not rotated."""
        at = np.array([p])
        self.k[b, p] = Q.values(*Q.quantise(Q.rotate(k[None], at, self.cs, self.pairs)[0], 65504.0))
        self.v[b, p] = Q.values(*Q.quantise(v.astype(np.float32), 8188.0))

    def step(self, qkv32, pos, window):
        """From the GPU's fp32 projection qkv32: o [B][Hq D] in fp64 and its rounding bound."""
        Hq, Hkv, D = self.Hq, self.Hkv, self.D
        outs, tols = [], []
        for b, p in enumerate(pos):
            q = qkv32[b, :Hq * D].reshape(Hq, D)
            if p < 0:
                outs.append(np.zeros(Hq * D))
                tols.append(np.zeros(Hq * D))
                continue
            self.store(b, p, qkv32[b, Hq * D:(Hq + Hkv) * D].reshape(Hkv, D), qkv32[b, (Hq + Hkv) * D:].reshape(Hkv, D))
            q = np64(torch.from_numpy(Q.rotate(q[None], np.array([p]), self.cs, self.pairs)[0]).to(DT[self.dt]))
            at = range(max(0, p + 1 - window) if window else 0, p + 1)
            k, v = (np.stack([c[b, i] for i in at]) for c in (self.k, self.v))
            o, _, ab = Q.attention(q, k, v, self.scale)
            d = Q.score_bound(q, np.abs(k).reshape(len(k), Hkv, -1, 32).max((0, 1, 3)) / 7, self.scale) + 2.0 ** -22 * 40
            tol = (2 * 2.0 ** -11 + 2 * d + 2.0 ** -18) * ab * 1.01 + HALF_STEP[self.dt] * np.abs(o) + 2.0 ** -25
            outs.append(o.reshape(-1))
            tols.append(tol.reshape(-1))
        return np.stack(outs), np.stack(tols)

    def project_out(self, o, x_tol):
        q = Q.unpack_rows(self.w["Wo"]).astype(np.float64)
        wo = q * np.repeat(self.w["Wo_s"].astype(np.float64), q.shape[1] // self.w["Wo_s"].shape[1], 1)
        y = o @ wo.T + self.w["bo"].astype(np.float64)
        tol = x_tol @ np.abs(wo).T + Q.linear_q4_bound(o, self.w["Wo"], self.w["Wo_s"]) * 1.01 + 2.0 ** -22 * np.abs(y)
        return y, tol


BLOCKS = [(256, 4, 2, 64, 16, "f16", False, 0), (320, 5, 5, 32, 8, "bf16", True, 9)]


@pytest.mark.parametrize("case", BLOCKS, ids=lambda c: "-".join(map(str, c)))
def test_attention_half_over_steps(case):
    """A prompt of ragged lengths, then decode steps: projection, append, attention and output
    projection through AttnStep, each step against the oracle on the same cache."""
    from activation_sparse_ffn_amd import AttnStep
    d, Hq, Hkv, D, page, dt, pairs, window = case
    say(f"attention half {case}")
    B, lens = 3, [19, 0, 7]
    table, pages = make_table([n + 12 for n in lens], page, 5)
    cs = rope_table(64, D)
    w = make_layer(d, Hq, Hkv, D, 3)
    dev_w = {k: v.to(DEV) for k, v in w.items()}
    pos = torch.tensor([n - 1 for n in lens], dtype=torch.int32, device=DEV)
    step = AttnStep(Hq, Hkv, D, B, dt, table.to(DEV), pos, pages, page=page, cos_sin=torch.from_numpy(cs).to(DEV),
                    interleaved=pairs, window=window)
    ref = Reference(w, Hq, Hkv, D, cs, pairs, dt, D ** -0.5)
    g = torch.Generator().manual_seed(1)
    T = sum(lens)
    k, v = (torch.randn(T, Hkv, D, generator=g) for _ in range(2))
    p_seq = np.concatenate([np.full(n, b) for b, n in enumerate(lens)]).astype(np.int32)
    p_pos = np.concatenate([np.arange(n) for n in lens]).astype(np.int32)
    step.prefill(k.to(DEV), v.to(DEV), torch.from_numpy(p_pos).to(DEV), torch.from_numpy(p_seq).to(DEV))
    for t in range(T):
        ref.store(int(p_seq[t]), int(p_pos[t]), k[t].numpy(), v[t].numpy())
    for s in range(5):
        pos += 1
        if s == 3:
            pos[2] = -1                                  # a request that has ended
        x = torch.randn(B, d, generator=g).to(DT[dt])
        y = torch.full((B, d), float("nan"), device=DEV)
        step.run(dev_w, x.to(DEV), y)
        qkv = step.qkv.cpu().numpy()
        want = Q.linear_q4(np64(x), w["Wqkv"].numpy(), w["Wqkv_s"].numpy(), w["bqkv"].numpy())
        tol = Q.linear_q4_bound(np64(x), w["Wqkv"].numpy(), w["Wqkv_s"].numpy()) + 2.0 ** -22 * np.abs(want)
        assert (np.abs(qkv - want) <= tol).all()
        o, o_tol = ref.step(qkv, pos.tolist(), window)
        assert (np.abs(np64(step.o).reshape(B, -1) - o) <= o_tol).all(), s
        yo, y_tol = ref.project_out(o, o_tol)
        assert (np.abs(np64(y) - yo) <= y_tol).all(), s


def test_parallel_block_layer():
    """run_layer with an attention half: the FFN's y and the attention's, added."""
    import synthetic as S
    from activation_sparse_ffn_amd import AttnStep, StepBuffers, run_layer
    cfg = S.scaled(S.CONFIGS["C4"], name="par", d=512, f=1056, h=128)
    B, Hq, Hkv, D, page = 2, 4, 2, 64, 8
    say("parallel block")
    L = S.make_layer(cfg, 0, device=DEV)
    w = {k: v.to(DEV) for k, v in make_layer(cfg.d, Hq, Hkv, D, 8).items()}
    layer = {**L.tensors(), **w}
    x = S.make_tokens(cfg, 0, 1, B, device=DEV)[0]
    table, pages = make_table([10, 10], page, 2)
    outs = []
    for both in (False, True):
        buf = StepBuffers(cfg.d, cfg.f, cfg.h, B, cfg.wdtype, cfg.pred_storage)
        attn = AttnStep(Hq, Hkv, D, B, "f16", table.to(DEV), torch.zeros(B, dtype=torch.int32, device=DEV), pages, page=page)
        run_layer(buf, layer, x, L.threshold, cfg.act, attn=attn if both else None)
        outs.append(np64(buf.y))
    y = torch.empty(B, cfg.d, device=DEV)
    attn.run(layer, x, y)
    ffn, both = outs
    assert (np.abs(both - (ffn + np64(y))) <= 2.0 ** -22 * (np.abs(both) + np.abs(np64(y)) + np.abs(ffn))).all()
    assert np.abs(np64(y)).max() > 0


def test_graph_replays_and_shared_workspace():
    """A captured decode step replayed over moving positions, with eager work between, and two
    captured graphs of different shapes that share one workspace."""
    from activation_sparse_ffn_amd import AttnStep
    d, Hq, Hkv, D, page, B = 256, 8, 2, 64, 16, 2
    table, pages = make_table([900, 900], page, 1)
    w = {k: v.to(DEV) for k, v in make_layer(d, Hq, Hkv, D, 4).items()}
    g = torch.Generator().manual_seed(9)
    steps = []
    for _ in range(2):
        pos = torch.tensor([699, 400], dtype=torch.int32, device=DEV)
        steps.append(AttnStep(Hq, Hkv, D, B, "f16", table.to(DEV), pos, pages, page=page))
    k, v = (torch.randn(1101, Hkv, D, generator=g).to(DEV) for _ in range(2))
    p_seq = torch.tensor([0] * 700 + [1] * 401, dtype=torch.int32, device=DEV)
    p_pos = torch.cat([torch.arange(700), torch.arange(401)]).to(torch.int32).to(DEV)
    for s in steps:
        s.prefill(k, v, p_pos, p_seq)
    graphed, eager = steps
    x = torch.zeros(B, d, dtype=torch.float16, device=DEV)
    y = torch.zeros(B, d, device=DEV)
    # another shape on the same workspace
    q2, cache2, table2, _ = make_attn(3, 4, 4, 32, 8, [600, 1, 300], "f16", 3)
    lens2 = torch.tensor([600, 1, 300], dtype=torch.int32, device=DEV)
    q2 = q2.to(DEV)
    out2, ref2 = torch.zeros_like(q2), torch.zeros_like(q2)
    need = max(graphed.ws.numel(), A.sfx_attn_q4_ws(3, 4, 4, 32, table2.shape[1] * 8))
    graphed.ws = A.workspace(need)
    A.sfx_attn_q4(q2, cache2, table2, lens2, ref2, A.workspace(need))
    for s in steps:                                      # warm; both caches take this token
        s.run(w, x, y)
    torch.cuda.synchronize()
    ga, gb = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(ga):
        graphed.run(w, x, y)
    with torch.cuda.graph(gb):
        A.sfx_attn_q4(q2, cache2, table2, lens2, out2, graphed.ws)
    for rep in range(4):
        say(f"graph replay {rep}")
        xn = torch.randn(B, d, generator=g).half()
        for s in steps:
            s.pos += 1
        x.copy_(xn.to(DEV))
        ga.replay()
        out2.zero_()
        gb.replay()
        ye = torch.empty(B, d, device=DEV)
        eager.run(w, xn.to(DEV), ye)
        torch.cuda.synchronize()
        assert torch.equal(y, ye) and torch.equal(out2, ref2), rep
        _ = torch.randn(1000, device=DEV).sum().item()


def test_two_streams():
    """Two attention calls and two projections at once, on streams and workspaces of their own."""
    cases = [make_attn(2, 8, 2, 128, 16, [3000, 2500], "bf16", s) for s in (1, 2)]
    lens = torch.tensor([3000, 2500], dtype=torch.int32, device=DEV)
    lin = [[t.to(DEV) for t in make_linear(3, 700, 1024, 64, "f16", s)] for s in (5, 6)]
    want = []
    for (q, cache, table, _), (x, W, s, b) in zip(cases, lin):
        out, y = torch.empty(2, 8, 128, dtype=torch.bfloat16, device=DEV), torch.empty(3, 700, device=DEV)
        A.sfx_attn_q4(q.to(DEV), cache, table, lens, out, A.workspace(A.sfx_attn_q4_ws(2, 8, 2, 128, table.shape[1] * 16)))
        A.sfx_linear_q4(x, W, s, y, bias=b)
        want.append((out, y))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cases]
    got = [(torch.empty_like(o), torch.empty_like(y)) for o, y in want]
    qs = [c[0].to(DEV) for c in cases]
    wss = [A.workspace(A.sfx_attn_q4_ws(2, 8, 2, 128, c[2].shape[1] * 16)) for c in cases]
    torch.cuda.synchronize()
    for rep in range(5):
        for i, st in enumerate(streams):
            A.sfx_attn_q4(qs[i], cases[i][1], cases[i][2], lens, got[i][0], wss[i], stream=st)
            with torch.cuda.stream(st):
                A.sfx_linear_q4(lin[i][0], lin[i][1], lin[i][2], got[i][1], bias=lin[i][3])
    torch.cuda.synchronize()
    for (o, y), (wo, wy) in zip(got, want):
        assert torch.equal(o, wo) and torch.equal(y, wy)


def test_cache_beyond_4_gib():
    """Pages whose bytes lie past 32-bit offsets."""
    Hq, Hkv, D, page = 8, 8, 256, 128
    per_page = Hkv * (page // 8) * 9 * D
    pages = (9 << 29) // per_page + 2                     # 4.5 GiB
    say(f"cache of {pages * per_page / 2**30:.2f} GiB")
    cache = torch.empty(pages, Hkv, page // 8, 9 * D, dtype=torch.uint8, device=DEV)
    ids = [pages - 1, 0, pages - 2]
    table = torch.tensor([ids], dtype=torch.int32, device=DEV)
    for i in ids:
        cache[i].fill_(0xFF)
    n = 300
    rng = np.random.default_rng(0)
    k, v = (torch.from_numpy(rng.standard_normal((n, Hkv, D)).astype(np.float32)) for _ in range(2))
    pos = torch.arange(n, dtype=torch.int32, device=DEV)
    seq = torch.zeros(n, dtype=torch.int32, device=DEV)
    A.sfx_kv_append_q4(None, k.to(DEV), v.to(DEV), pos, table, cache, None, seq=seq)
    kn, vn = Q.values(*Q.quantise(k.numpy(), 65504.0)), Q.values(*Q.quantise(v.numpy(), 8188.0))
    ko, vo = torch.empty(n, Hkv, D, device=DEV), torch.empty(n, Hkv, D, device=DEV)
    A.sfx_kv_read_q4(pos, table, cache, ko, vo, seq=seq)
    assert np.array_equal(np64(ko), kn) and np.array_equal(np64(vo), vn)
    q = torch.from_numpy(rng.standard_normal((1, Hq, D)).astype(np.float32)).half()
    out, lse = torch.empty(1, Hq, D, dtype=torch.float16, device=DEV), torch.empty(1, Hq, device=DEV)
    ws = A.workspace(A.sfx_attn_q4_ws(1, Hq, Hkv, D, 3 * page))
    A.sfx_attn_q4(q.to(DEV), cache, table, torch.tensor([n], dtype=torch.int32, device=DEV), out, ws, lse=lse)
    check_attn(q, [(kn, vn)], [n], None, D ** -0.5, "f16", out, lse)


def test_attention_largest_batch():
    """64 sequences and 256 query heads, lengths from none to many, queries apart in memory."""
    B, Hq, Hkv, D, page = 64, 256, 8, 32, 8
    lens = [(b * 37) % 500 for b in range(B)]
    q, cache, table, kv = make_attn(B, Hq, Hkv, D, page, lens, "f16", 77)
    wide = torch.zeros(B, Hq + 1, D, dtype=torch.float16, device=DEV)
    wide[:, :Hq] = q.to(DEV)
    ws = A.workspace(A.sfx_attn_q4_ws(B, Hq, Hkv, D, table.shape[1] * page))
    out, lse = torch.empty(B, Hq, D, dtype=torch.float16, device=DEV), torch.empty(B, Hq, device=DEV)
    say("attention 64 x 256")
    A.sfx_attn_q4(wide[:, :Hq], cache, table, torch.tensor(lens, dtype=torch.int32, device=DEV), out, ws, lse=lse)
    check_attn(q, kv, lens, None, D ** -0.5, "f16", out, lse)


@pytest.mark.parametrize("case", [  # B, Hq, Hkv, D, page, longest: 258, 512, 512, 510, 512 workgroups
    (43, 51, 3, 32, 8, 1100), (64, 16, 8, 64, 16, 1030), (32, 8, 8, 64, 16, 2100), (3, 170, 170, 32, 64, 1024),
    (16, 32, 32, 256, 32, 1050)], ids=lambda c: "-".join(map(str, c)))
def test_attention_order_of_sequences(case):
    """Batches whose sequences the kernel orders by length: ties, empty ones, windows, and any
    order of the caller's gives each sequence the same bits."""
    B, Hq, Hkv, D, page, longest = case
    say(f"attention order {case}")
    rng = np.random.default_rng(B)
    lens = [int(n) for n in rng.integers(0, 40, B)]
    lens[B // 2] = longest
    lens[1] = lens[0]
    q, cache, table, kv = make_attn(B, Hq, Hkv, D, page, lens, "bf16", B + D)
    ws = A.workspace(A.sfx_attn_q4_ws(B, Hq, Hkv, D, table.shape[1] * page))
    qd, d_lens = q.to(DEV), torch.tensor(lens, dtype=torch.int32, device=DEV)
    for starts in (None, [int(n) for n in rng.integers(-5, 45, B)]):
        d_starts = None if starts is None else torch.tensor(starts, dtype=torch.int32, device=DEV)
        out = torch.full((B, Hq, D), float("nan"), dtype=torch.bfloat16, device=DEV)
        lse = torch.full((B, Hq), float("nan"), device=DEV)
        A.sfx_attn_q4(qd, cache, table, d_lens, out, ws, starts=d_starts, lse=lse)
        check_attn(q, kv, lens, starts, D ** -0.5, "bf16", out, lse)
        perm = torch.from_numpy(rng.permutation(B)).to(DEV)
        out2, lse2 = torch.full_like(out, float("nan")), torch.full_like(lse, float("nan"))
        A.sfx_attn_q4(qd[perm].contiguous(), cache, table[perm].contiguous(), d_lens[perm].contiguous(), out2, ws,
                      starts=None if starts is None else d_starts[perm].contiguous(), lse=lse2)
        assert torch.equal(out2, out[perm]) and torch.equal(lse2, lse[perm])
    # lengths and starts at the ends of their type: clamped, nothing to attend to
    ends = torch.tensor([[-2 ** 31, 2 ** 31 - 1], [2 ** 31 - 1, 2 ** 31 - 1], [-1, -2 ** 31]], dtype=torch.int32, device=DEV)
    d_lens[:3], d_starts = ends[:, 0], torch.zeros_like(d_lens)
    d_starts[:3] = ends[:, 1]
    A.sfx_attn_q4(qd, cache, table, d_lens, out, ws, starts=d_starts, lse=lse)
    assert (out[:3] == 0).all() and torch.isneginf(lse[:3]).all()
    if B > 3:
        check_attn(q[3:], kv[3:], lens[3:], None, D ** -0.5, "bf16", out[3:], lse[3:])


def test_attention_bad_query_stays_alone():
    """A NaN or an infinity in one head's query: the other heads and sequences keep their bits."""
    B, Hq, Hkv, D, lens = 4, 16, 2, 64, [300, 40, 700, 5]
    q, cache, table, _ = make_attn(B, Hq, Hkv, D, 16, lens, "f16", 5)
    ws = A.workspace(A.sfx_attn_q4_ws(B, Hq, Hkv, D, table.shape[1] * 16))
    d_lens, qd = torch.tensor(lens, dtype=torch.int32, device=DEV), q.to(DEV)
    out = torch.empty(B, Hq, D, dtype=torch.float16, device=DEV)
    A.sfx_attn_q4(qd, cache, table, d_lens, out, ws)
    bad = torch.zeros(B, Hq, dtype=torch.bool, device=DEV)
    for b, h, value in ((0, 3, float("nan")), (2, 8, float("inf")), (1, 15, float("-inf"))):
        say(f"attention with {value} in query {b}, {h}")
        qd[b, h, 7] = value
        bad[b, h] = True
    out2 = torch.empty_like(out)
    A.sfx_attn_q4(qd, cache, table, d_lens, out2, ws)
    assert torch.equal(out2[~bad], out[~bad])
    assert not torch.isfinite(out2[bad]).any()                 # of 40 keys some have either sign


def test_shared_pages_and_drafted_tokens():
    """Two sequences whose tables share a prefix, and several query tokens of one sequence as
    rows with the same pages and their own lens."""
    Hq, Hkv, D, page = 4, 1, 64, 8
    q, cache, table, kv = make_attn(1, Hq, Hkv, D, page, [50], "bf16", 31)
    rows = table.expand(4, -1).contiguous()
    lens = [50, 49, 48, 1]
    rng = np.random.default_rng(1)
    q = torch.from_numpy(rng.standard_normal((4, Hq, D)).astype(np.float32)).to(torch.bfloat16)
    ws = A.workspace(A.sfx_attn_q4_ws(4, Hq, Hkv, D, rows.shape[1] * page))
    out, lse = torch.empty(4, Hq, D, dtype=torch.bfloat16, device=DEV), torch.empty(4, Hq, device=DEV)
    A.sfx_attn_q4(q.to(DEV), cache, rows, torch.tensor(lens, dtype=torch.int32, device=DEV), out, ws, lse=lse)
    check_attn(q, kv * 4, lens, None, D ** -0.5, "bf16", out, lse)
