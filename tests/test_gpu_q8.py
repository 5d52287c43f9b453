"""The 8-bit layer half (sfx_norm_q8, sfx_linear_q8, sfx_kv_append_q8, sfx_kv_read_q8,
sfx_attn_q8) against the fp64 oracle, at the sizes and masks where it can go wrong."""
import numpy as np
import pytest
import torch

from activation_sparse_ffn_amd import _abi as A
from gpu_helpers import say
from oracle import q4_oracle as Q4
from oracle import q8_oracle as Q

pytestmark = pytest.mark.gpu
DEV = "cuda"
DT = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
HALF_STEP = {"f16": 2.0 ** -11, "bf16": 2.0 ** -8, "f32": 2.0 ** -24}
TINY = {"f16": 2.0 ** -25, "bf16": 2.0 ** -134, "f32": 2.0 ** -150}    # half of the last bit below the normal numbers


def np64(t):
    return t.detach().cpu().to(torch.float64).numpy()


def within(got, want, dt, extra=0.0):
    """Values rounded once (by way of fp32) to `dt` from `want`, which itself may be off by extra."""
    tol = (HALF_STEP[dt] + 2.0 ** -24) * 1.001 * np.abs(want) + TINY[dt] + extra
    return (np.abs(got - want) <= tol) | (np.isnan(got) & np.isnan(want))


# ------------------------------------------------------------------------------ norm

NORM = [  # T, d, x, residual, y, norm, weight
    (1, 1, "f32", None, "f32", True, True), (1, 7, "f16", "f16", "f16", True, False), (2, 16, "bf16", None, None, True, True),
    (3, 63, "f32", "bf16", "bf16", True, True), (5, 64, "bf16", "f32", "f16", True, True), (7, 100, "f16", "f32", None, False, False),
    (3, 256, "f32", "f32", "f32", True, True), (2, 1000, "bf16", "bf16", "f32", True, True), (1, 4096, "f32", "f32", "f16", True, True),
    (9, 4096, "bf16", "bf16", None, True, True), (300, 512, "f16", "f16", "f16", True, True), (2, 5119, "f16", "f16", "bf16", True, True),
    (33, 7168, "bf16", "f32", "bf16", True, True), (4, 8192, "bf16", None, None, False, False), (257, 8200, "bf16", "bf16", "bf16", True, True),
    (2, 16384, "f32", "f16", "f16", True, True), (3, 28672, "f16", "bf16", "f16", True, False), (2, 32768, "f32", "f32", "f32", True, True),
    (2, 40000, "f32", "f32", "bf16", True, True), (1, 70001, "bf16", "f16", "f16", True, True)]


def make_norm(case, seed):
    T, d, xt, rt, yt, norm, weight = case
    g = torch.Generator().manual_seed(seed)
    strong = 1 + 30 * (torch.rand(d, generator=g) < 0.01)
    x = (torch.randn(T, d, generator=g) * strong).to(DT[xt])
    r = (torch.randn(T, d, generator=g) * 3).to(DT[rt]) if rt else None
    w = 1 + 0.3 * torch.randn(d, generator=g) if weight else None
    return x, r, w


def check_norm(case, x, r, w, q, s, ro, y, eps=1e-5):
    T, d, xt, rt, yt, norm, weight = case
    h, n = Q.norm_rows(np64(x), None if r is None else np64(r), None if w is None else w.numpy(), np.float64(np.float32(eps)), norm)
    s64, _ = Q.row_codes(n)
    sg, qg = np64(s), np64(q)                                    # (limits in 64 bits too)
    # 64-bit sums in another order: 2^-50 of s, which then rounds once
    assert (np.abs(sg - np.abs(n).max(1) / 127) <= 2.0 ** -24 * 1.0001 * sg + 2.0 ** -150).all()
    assert np.array_equal(sg == 0, s64 == 0)
    with np.errstate(all="ignore"):
        ratio = np.where((sg > 0)[:, None], n / sg[:, None], 0.0)
    off = np.abs(np.clip(ratio, -127, 127) - qg)
    assert off.max() <= 0.5 + 2.0 ** -40, off.max()              # the nearest code
    tie = np.abs(np.abs(ratio - np.floor(ratio)) - 0.5) < 2.0 ** -44   # ties to even
    assert (qg[tie] % 2 == 0).all()
    if r is not None:
        assert within(np64(ro), h, rt).all()
    if y is not None:
        assert within(np64(y), n, yt, 2.0 ** -48 * np.abs(n)).all()


@pytest.mark.parametrize("case", NORM, ids=lambda c: "-".join(map(str, c)))
def test_norm(case):
    T, d, xt, rt, yt, norm, weight = case
    say(f"norm {case}")
    x, r, w = make_norm(case, d + T)
    dev = [None if t is None else t.to(DEV) for t in (x, r, w)]
    q, s = torch.full((T, d), 99, dtype=torch.int8, device=DEV), torch.full((T,), -1.0, device=DEV)
    ro = None if r is None else torch.full_like(dev[1], 5.0)
    y = torch.full((T, d), 5.0, dtype=DT[yt], device=DEV) if yt else None
    A.sfx_norm_q8(dev[0], q, s, weight=dev[2], residual=dev[1], residual_out=ro, y=y, norm=norm)
    check_norm(case, x, r, w, q, s, ro, y)
    # in place, only y, and rows apart: the same bits
    q2, s2 = torch.empty_like(q), torch.empty_like(s)
    r2 = None if r is None else dev[1].clone()
    A.sfx_norm_q8(dev[0], q2, s2, weight=dev[2], residual=r2, norm=norm)
    assert torch.equal(q, q2) and torch.equal(s, s2) and (r is None or torch.equal(r2, ro))
    if yt:
        def apart(t, fill):
            wide = torch.full((T, d + 13), fill, dtype=t.dtype, device=DEV)
            wide[:, 5:5 + d] = t
            return wide
        xw, rw, yw = apart(dev[0], 9.0), None if r is None else apart(dev[1], 9.0), apart(y, 9.0)
        cut = lambda t: None if t is None else t[:, 5:5 + d]  # noqa: E731
        cut(yw).fill_(0)
        q3, s3 = torch.empty_like(q), torch.empty_like(s)
        A.sfx_norm_q8(cut(xw), q3, s3, weight=dev[2], residual=cut(rw), y=cut(yw), norm=norm)
        assert torch.equal(q, q3) and torch.equal(s, s3) and torch.equal(cut(yw), y) and (r is None or torch.equal(cut(rw), ro))
        for t in (xw, rw, yw):
            assert t is None or ((t[:, :5] == 9).all() and (t[:, 5 + d:] == 9).all())
        y4 = torch.empty_like(y)
        A.sfx_norm_q8(dev[0], weight=dev[2], residual=None if r is None else dev[1].clone(), y=y4, norm=norm)
        assert torch.equal(y, y4)


NORM_MANY = [  # T, d, x, residual, y: more than the last-level cache holds
    (76000, 333, "f32", "f32", "bf16"), (51000, 1000, "f16", "bf16", None), (12400, 2041, "f32", "f32", "f16"),
    (12300, 4096, "bf16", "bf16", "f32"), (8200, 8190, "f32", None, None), (3200, 16384, "f16", "f16", "f16")]


@pytest.mark.parametrize("case", NORM_MANY, ids=lambda c: "-".join(map(str, c)))
def test_norm_many_rows(case):
    """Rows spread over the call against the oracle; codes and scales of all against calls of fewer rows
    (a scale could differ where two orders of a 64-bit sum fall on two sides of a border: about 2^-28 a row)."""
    T, d, xt, rt, yt = case
    say(f"norm {case}")
    g = torch.Generator(device=DEV).manual_seed(d)
    x = (torch.randn(T, d, generator=g, device=DEV) * 2).to(DT[xt])
    r = torch.randn(T, d, generator=g, device=DEV).to(DT[rt]) if rt else None
    w = 1 + 0.3 * torch.randn(d, generator=g, device=DEV)
    q, s = torch.full((T, d), 99, dtype=torch.int8, device=DEV), torch.full((T,), -1.0, device=DEV)
    y = torch.full((T, d), 5.0, dtype=DT[yt], device=DEV) if yt else None
    ro = None if r is None else r.clone()
    A.sfx_norm_q8(x, q, s, weight=w, residual=ro, y=y)
    rows = torch.from_numpy(np.unique(np.linspace(0, T - 1, 37).astype(int)))
    at = lambda t: None if t is None else t.cpu()[rows]  # noqa: E731
    check_norm((len(rows), d, xt, rt, yt, True, True), at(x), at(r), w.cpu(), at(q), at(s), at(ro), at(y))
    for t in range(0, T, 2000):
        q1, s1 = torch.empty_like(q[t:t + 2000]), torch.empty_like(s[t:t + 2000])
        A.sfx_norm_q8(x[t:t + 2000], q1, s1, weight=w, residual=None if r is None else r[t:t + 2000])
        assert torch.equal(q1, q[t:t + 2000]) and torch.equal(s1, s[t:t + 2000]), t


@pytest.mark.parametrize("d", [40, 1000, 4096, 9000])
def test_norm_special_rows(d):
    """Zeros, ties between codes, one value alone, the largest and smallest numbers, and rows with
    a NaN or an infinity, which leave the other rows alone."""
    say(f"norm special {d}")
    x = torch.randn(12, d, generator=torch.Generator().manual_seed(1))
    x[0] = 0
    x[1] = (torch.arange(d) % 255 - 127) / 2 * 2.0 ** -7          # 63.5 2^-7 is the largest: scale 2^-8 exactly
    x[1, :2] = torch.tensor([127.0, -127.0]) * 2.0 ** -8
    x[2] = 0
    x[2, d - 1] = -3.0
    x[3] *= 1e38
    x[3].clamp_(-3e38, 3e38)
    x[4] *= 2.0 ** -140
    x[5, d // 2] = float("nan")
    x[6, 0] = float("inf")
    x[7, d - 1] = -float("inf")
    x[8] = 2.0 ** -149
    for norm in (False, True):
        q, s, y = torch.empty(12, d, dtype=torch.int8, device=DEV), torch.empty(12, device=DEV), torch.empty(12, d, device=DEV)
        A.sfx_norm_q8(x.to(DEV), q, s, y=y, norm=norm)
        bad = [5, 6, 7]
        good = [i for i in range(12) if i not in bad]
        assert s[bad].isnan().all() and (q[bad] == 0).all()
        if norm:
            assert y[5].isnan().all()
        else:
            assert torch.equal(y.cpu()[6:8], x[6:8])
        pick = lambda t: t[good]  # noqa: E731
        check_norm((9, d, "f32", None, "f32", norm, False), pick(x), None, None, pick(q), pick(s), None, pick(y))
        assert s[0] == 0 and (q[0] == 0).all() and (y[0] == 0).all()
        if not norm:
            assert s[1] == 2.0 ** -8 and torch.equal(q[1].cpu().float(), torch.round(x[1] * 256))
    w = torch.ones(d)
    w[3] = float("inf")
    A.sfx_norm_q8(x[9:].to(DEV), q[:3], s[:3], weight=w.to(DEV))
    assert s[:3].isnan().all() and (q[:3] == 0).all()


# ------------------------------------------------------------------------------ linear

LINEAR = [(1, 1, 16), (1, 17, 48), (2, 100, 64), (3, 33, 272), (1, 4096, 4096), (4, 1003, 1056), (8, 130, 4096), (13, 257, 640),
          (16, 64, 1024), (17, 31, 2048), (31, 300, 80), (33, 129, 528), (64, 11008, 1024), (65, 257, 272), (100, 1003, 1056),
          (127, 128, 128), (128, 256, 512), (129, 130, 4112), (200, 511, 96), (255, 1024, 144), (257, 300, 1040), (513, 777, 2064),
          (777, 1003, 1056), (1025, 256, 64), (2, 40, 131056), (70, 20, 65536), (300, 5000, 16), (1, 70000, 32), (1500, 1100, 320),
          (3, 5, 28672), (48, 2048, 8192), (600, 2600, 272)]


def make_linear(T, n, d, seed):
    g = torch.Generator().manual_seed(seed)
    x = torch.randint(-127, 128, (T, d), generator=g, dtype=torch.int8)
    W = torch.randint(-127, 128, (n, d), generator=g, dtype=torch.int8)
    sx, sw = 0.02 * torch.rand(T, generator=g) + 1e-3, 0.05 * torch.rand(n, generator=g) + 1e-3
    return x, sx, W, sw, torch.randn(n, generator=g) * 3


def sums_of(x, W):
    """Exact sums of products [T][n]: fp64 holds every partial sum."""
    return (x.double() @ W.double().t()).numpy()


def linear_tol(p, sx, sw, y, dt):
    """The sum's, the scales' product's and their product's roundings, the bias or accumulation, y's own."""
    a = np.abs(p * sx.double().numpy()[:, None] * sw.double().numpy())
    return 3.01 * 2.0 ** -24 * a + 2.02 * 2.0 ** -24 * np.abs(y) + (HALF_STEP[dt] * 1.001 * np.abs(y) if dt != "f32" else 0) + TINY[dt]


@pytest.mark.parametrize("case", LINEAR, ids=lambda c: "x".join(map(str, c)))
def test_linear(case):
    T, n, d = case
    say(f"linear {case}")
    x, sx, W, sw, bias = make_linear(T, n, d, T * n + d)
    x[-1], W[-1] = -128, -128                            # the codes that the norm does not make
    p = sums_of(x, W)
    base = p * sx.double().numpy()[:, None] * sw.double().numpy()
    dev = [t.to(DEV) for t in (x, sx, W, sw)]
    ref = base + bias.double().numpy()
    for dt in ("f32", "f16", "bf16"):
        y = torch.full((T, n), float("nan"), dtype=DT[dt], device=DEV)
        A.sfx_linear_q8(*dev, y, bias=bias.to(DEV))
        big = np.abs(ref) * 1.01 > (65504 if dt == "f16" else 1e38)
        err = np.abs(np64(y) - ref)
        assert (err <= linear_tol(p, sx, sw, np.abs(ref) + np.abs(bias.numpy()), dt))[~big].all(), dt
        y2 = torch.full((T, n), float("nan"), dtype=DT[dt], device=DEV)
        A.sfx_linear_q8(*dev, y2, bias=bias.to(DEV))
        assert torch.equal(y, y2)
        y0 = torch.randn(T, n, generator=torch.Generator().manual_seed(1)).to(DT[dt])
        y3 = y0.to(DEV)
        A.sfx_linear_q8(*dev, y3, accumulate=True)
        ref3 = y0.double().numpy() + base
        assert (np.abs(np64(y3) - ref3) <= linear_tol(p, sx, sw, np.abs(ref3) + np.abs(y0.double().numpy()), dt))[~big].all(), dt


@pytest.mark.parametrize("case", [(1, 50, 4096), (7, 300, 1024), (40, 100, 512), (130, 200, 1040), (300, 300, 512)], ids=str)
def test_linear_sums_are_exact(case):
    """With scales of 1 every sum below 2^24 comes out as it is."""
    T, n, d = case
    x, _, W, _, _ = make_linear(T, n, d, 3)
    p = sums_of(x, W)
    assert np.abs(p).max() < 2 ** 24
    y = torch.empty(T, n, device=DEV)
    A.sfx_linear_q8(x.to(DEV), torch.ones(T, device=DEV), W.to(DEV), torch.ones(n, device=DEV), y)
    assert np.array_equal(np64(y), p)


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("T", [1, 5, 20, 64, 70, 300])
def test_linear_rows_apart(T, dt):
    """x and y as slices of wider tensors (y at odd elements); what lies beside y stays; and a
    token's result is the same alone and among others."""
    n, d = 203, 288
    say(f"linear strided T={T} {dt}")
    x, sx, W, sw, _ = make_linear(T, n, d, 5)
    wide = torch.full((T, d + 48), 99, dtype=torch.int8, device=DEV)
    wide[:, 16:16 + d] = x.to(DEV)
    yw = torch.full((T, n + 9), 7.0, dtype=DT[dt], device=DEV)
    A.sfx_linear_q8(wide[:, 16:16 + d], sx.to(DEV), W.to(DEV), sw.to(DEV), yw[:, 5:5 + n])
    y = torch.empty(T, n, dtype=DT[dt], device=DEV)
    A.sfx_linear_q8(x.to(DEV), sx.to(DEV), W.to(DEV), sw.to(DEV), y)
    assert torch.equal(yw[:, 5:5 + n], y)
    assert (yw[:, :5] == 7).all() and (yw[:, 5 + n:] == 7).all()
    one = torch.empty(1, n, dtype=DT[dt], device=DEV)
    A.sfx_linear_q8(x[-1:].to(DEV), sx[-1:].to(DEV), W.to(DEV), sw.to(DEV), one)
    assert torch.equal(one[0], y[-1])


@pytest.mark.parametrize("n,d", [(333, 272), (1024, 4096), (9000, 512)])
def test_linear_rows_do_not_depend_on_others(n, d):
    """A token's y has the same bits in calls of any number of tokens, with and without bias and addition."""
    say(f"linear rows alone {n}x{d}")
    x, sx, W, sw, bias = (t.to(DEV) for t in make_linear(3000, n, d, n + d))
    g = torch.Generator(device=DEV).manual_seed(d)
    for dt in DT:
        y0 = torch.randn(3000, n, generator=g, device=DEV).to(DT[dt])
        for b, acc in ((bias, False), (None, True), (bias, True)):
            ys = []
            for T in (3000, 1, 4, 5, 16, 17, 64, 130, 600):
                y = y0[:T].clone()
                A.sfx_linear_q8(x[:T], sx[:T], W, sw, y, bias=b, accumulate=acc)
                ys.append(y)
            for y in ys[1:]:
                assert torch.equal(y, ys[0][:len(y)]), (dt, acc, len(y))


@pytest.mark.parametrize("T", [2, 30, 150, 400])
def test_linear_bad_scales_stay_alone(T):
    """A NaN scale of a token or of a weight row makes its results NaN and no others'."""
    n, d = 150, 256
    x, sx, W, sw, _ = make_linear(T, n, d, 9)
    good, y = torch.empty(T, n, device=DEV), torch.empty(T, n, device=DEV)
    A.sfx_linear_q8(x.to(DEV), sx.to(DEV), W.to(DEV), sw.to(DEV), good)
    sx[1], sw[77] = float("nan"), float("nan")
    A.sfx_linear_q8(x.to(DEV), sx.to(DEV), W.to(DEV), sw.to(DEV), y)
    assert y[1].isnan().all() and y[:, 77].isnan().all()
    y[1], y[:, 77] = good[1], good[:, 77]
    assert torch.equal(y, good)


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


def positions(q_start, lens, T):
    """Sequence and position of each row (-1: none)."""
    seq, pos = np.full(T, -1), np.full(T, -1)
    for b in range(len(lens)):
        n = q_start[b + 1] - q_start[b]
        seq[q_start[b]:q_start[b + 1]] = b
        pos[q_start[b]:q_start[b + 1]] = np.arange(lens[b] - n, lens[b])
    return seq, pos


APPEND = [  # D, Hq, Hkv, page, dtype, rope, rot
    (32, 1, 1, 16, "f32", "half", 32), (32, 6, 6, 16, "f16", "half", 16), (64, 4, 2, 16, "f16", "pairs", 64),
    (96, 3, 3, 32, "bf16", "half", 50), (128, 8, 2, 16, "f32", "half", 128), (128, 5, 5, 64, "f16", "none", 0),
    (160, 2, 1, 32, "bf16", "pairs", 2), (192, 2, 2, 16, "f32", "half", 2), (224, 1, 1, 16, "f16", "half", 224),
    (256, 16, 4, 128, "bf16", "pairs", 130), (64, 9, 3, 1024, "bf16", "half", 64)]


@pytest.mark.parametrize("case", APPEND, ids=lambda c: "-".join(map(str, c)))
def test_append_and_read(case):
    """Calls of ragged sequences one behind the other, as slices of one projection, with rows of no
    sequence, missing pages, positions past the angles, NaN and infinities: every byte of the cache,
    the rotated queries and what is read back as the oracle has them."""
    D, Hq, Hkv, page, dt, rope, rot = case
    say(f"append {case}")
    g = torch.Generator().manual_seed(D + Hq)
    lens = np.array([0, 0, 0, 0, 0, 0])
    table, pages = make_table([120, 1, 16, 90, 40, 64], page, 3)
    if page <= 32:
        table[4, 0] = -1                                     # sequence 4's first page is missing
        table[5, 1] = pages + 5                              # and one of sequence 5's is none
    max_pos = 100 if rope != "none" else 0
    cs = rope_table(max_pos, rot) if max_pos else None
    start = torch.randint(0, 256, (pages, Hkv, page // 16, 32 * D + 16), generator=g, dtype=torch.uint8)
    sc = start[..., 32 * D:].contiguous().view(torch.float32)
    sc[..., 0], sc[..., 1] = 1e30, float("nan")              # an old block's scales do not matter
    start[..., 32 * D:] = sc.view(torch.uint8)
    cache, want = start.to(DEV), start.numpy().copy()
    d_table = table.to(DEV)
    # tokens per call and sequence; a block is entered at its start, inside, and left full or not
    for step, counts in enumerate(([37, 1, 0, 16, 5, 20], [1, 0, 3, 1, 1, 1], [0, 0, 1, 15, 20, 11], [1, 0, 1, 1, 1, 1],
                                   [70, 0, 11, 33, 5, 31])):
        lens = lens + counts
        lead = step % 3                                     # rows of no sequence in front and behind
        q_start = np.concatenate([[0], np.cumsum(counts)]) + lead
        T = int(q_start[-1]) + step % 2
        if T == 0:
            continue
        qkv = (torch.randn(T, (Hq + 2 * Hkv) * D + 8, generator=g) * (1 + step)).to(DT[dt])
        k_at, v_at = Hq * D, (Hq + Hkv) * D
        if step == 0:
            qkv[lead:lead + 16, k_at:k_at + D] = 0            # a block of zeros
            qkv[lead + 20, v_at + 1] = float("nan")
            qkv[lead + 21, k_at + D - 1] = float("inf")
            qkv[lead + 37, v_at:v_at + D] *= 2.0 ** -10       # a block that has to grow later
        dev = qkv.to(DEV)
        cut = lambda a, h: dev[:, a:a + h * D].unflatten(1, (h, D))  # noqa: E731
        q, k, v = cut(0, Hq), cut(k_at, Hkv), cut(v_at, Hkv)
        odt = "bf16" if dt == "bf16" else "f16"
        q_out = torch.full((T, Hq, D), 5.0, dtype=DT[odt], device=DEV)
        i32 = lambda a: torch.from_numpy(np.asarray(a, np.int32)).to(DEV)  # noqa: E731
        A.sfx_kv_append_q8(q, k, v, i32(lens), d_table, cache, q_out, q_start=i32(q_start),
                           cos_sin=None if cs is None else torch.from_numpy(cs).to(DEV), interleaved=rope == "pairs")
        seq, pos = positions(q_start, lens, T)
        at = np.clip(pos, 0, max(max_pos - 1, 0))
        host = lambda t: t.cpu().float().numpy()  # noqa: E731
        kr, qr = (Q4.rotate(host(x), at, cs, rope == "pairs") for x in (k, q))
        stored = Q.append(want, table.numpy(), page, kr, host(v), q_start, lens, max_pos)
        got = cache.cpu().numpy()
        if not np.array_equal(got, want):
            bad = np.argwhere(got != want)
            raise AssertionError((step, len(bad), bad[:4].tolist(), [(got[tuple(i)], want[tuple(i)]) for i in bad[:4]]))
        want_q = torch.from_numpy(qr).to(DT[odt])
        want_q[~torch.from_numpy(stored)] = 5.0
        same = (q_out.cpu() == want_q) | (q_out.cpu().isnan() & want_q.isnan())
        assert same.all(), step
    # read back, in mixed order, with padding
    rng = np.random.default_rng(1)
    seq = np.concatenate([np.full(n, b) for b, n in enumerate(lens)] + [[0, 1, 7, -1, 2]]).astype(np.int32)
    pos = np.concatenate([np.arange(n) for n in lens] + [[-1, 100000, 0, 0, 1 << 30]]).astype(np.int32)
    order = rng.permutation(len(seq))
    seq, pos = seq[order], pos[order]
    kw, vw = np.zeros((len(seq), Hkv, D)), np.zeros((len(seq), Hkv, D))
    for t, (b, p) in enumerate(zip(seq, pos)):
        pg = Q.pages_of(table.numpy(), page, pages, b, p) if 0 <= b < len(lens) else -1
        if pg >= 0:
            for h in range(Hkv):
                kq, vq, ks, vs = Q.read_block(want[pg, h, p % page // 16], D)
                kw[t, h], vw[t, h] = kq[p % 16] * np.float64(ks), vq[p % 16] * np.float64(vs)
    for odt in DT:
        k_out, v_out = (torch.full((len(seq), Hkv, D), 5.0, dtype=DT[odt], device=DEV) for _ in range(2))
        A.sfx_kv_read_q8(i32(pos), d_table, cache, k_out, v_out, seq=i32(seq))
        # 1e30 times a code of blocks that were never started is past fp16
        for a, b in ((np64(k_out), kw), (np64(v_out), vw)):
            fits = np.abs(b) < 65000
            assert within(a, b, odt)[fits | np.isnan(b)].all(), odt


def test_append_single_tokens():
    """Token by token without row offsets, growing and not, against one sequence stored at once:
    what was stored stays within the documented half steps."""
    D, Hkv, page, B, n = 64, 2, 16, 3, 40
    g = torch.Generator().manual_seed(4)
    k, v = (torch.randn(n, B, Hkv, D, generator=g) * torch.linspace(0.2, 2, n).view(n, 1, 1, 1) for _ in range(2))
    table, pages = make_table([n] * B, page, 1)
    cache = A.kv_cache_q8(pages, Hkv, page, D)
    cache.fill_(255)
    want = cache.cpu().numpy()
    for i in range(n):
        lens = np.array([i + 1] * B, np.int32)
        if i == 5:
            lens[1] = 0                                       # no token this time
            k[i:, 1], v[i:, 1] = k[i:, 1].roll(1, 0), v[i:, 1].roll(1, 0)
        if i > 5:
            lens[1] -= 1
        A.sfx_kv_append_q8(None, k[i].to(DEV), v[i].to(DEV), torch.from_numpy(lens).to(DEV), table.to(DEV), cache, None)
        starts = np.arange(B + 1)
        Q.append(want, table.numpy(), page, k[i].numpy(), v[i].numpy(), starts, lens, 0)
        assert np.array_equal(cache.cpu().numpy(), want), i
    for b in (0, 2):
        for h in range(Hkv):
            for blk in range(0, n, 16):
                kq, vq, ks, vs = Q.read_block(want[int(table[b, blk // page]), h, blk % page // 16], D)
                m = min(16, n - blk)
                err = np.abs(kq[:m] * np.float64(ks) - k[blk:blk + m, b, h].double().numpy())
                assert err.max() <= 16 * 0.5 * ks * 1.01


def test_append_far_positions():
    """Blocks whose bytes lie past 32 bits of offset."""
    D, Hkv, page = 128, 8, 1024
    blk = 32 * D + 16
    pages = (1 << 32) // (Hkv * 64 * blk) + 3
    say(f"append far: {pages * Hkv * 64 * blk / 2 ** 30:.1f} GiB")
    cache = torch.zeros(pages, Hkv, page // 16, blk, dtype=torch.uint8, device=DEV)
    table = torch.tensor([[0, pages - 1]], dtype=torch.int32, device=DEV)
    g = torch.Generator().manual_seed(2)
    k, v = torch.randn(20, Hkv, D, generator=g), torch.randn(20, Hkv, D, generator=g)
    i32 = lambda *a: torch.tensor(a, dtype=torch.int32, device=DEV)  # noqa: E731
    A.sfx_kv_append_q8(None, k.to(DEV), v.to(DEV), i32(1044), table, cache, None, q_start=i32(0, 20))
    ko, vo = torch.empty(20, Hkv, D, device=DEV), torch.empty(20, Hkv, D, device=DEV)
    A.sfx_kv_read_q8(torch.arange(1024, 1044, dtype=torch.int32, device=DEV), table, cache, ko, vo,
                     seq=torch.zeros(20, dtype=torch.int32, device=DEV))
    for a, b in ((ko, k), (vo, v)):
        assert (a.cpu() - b).abs().max() <= b.abs().max() / 127 * 0.501
    q = torch.randn(1, 8, D, generator=g).half().to(DEV)
    out, lse = torch.empty_like(q), torch.empty(1, 8, device=DEV)
    ws = A.workspace(A.sfx_attn_q8_ws(1, 1, 8, Hkv, D, 2048))
    A.sfx_attn_q8(q, cache, table, i32(1044), out, ws, starts=i32(1024), lse=lse)
    for h in range(8):
        o, l, ab, size = Q.attention(np64(q[0, h:h + 1]), np64(ko[:, h]), np64(vo[:, h]), D ** -0.5)
        tol, ltol = Q.attention_tolerance(o, l, ab, size, 4.0, 20, D, HALF_STEP["f16"])
        assert (np.abs(np64(out[0, h:h + 1]) - o) <= tol).all() and abs(float(lse[0, h]) - l[0]) <= ltol[0]


# ------------------------------------------------------------------------------ attention

def make_cache(pages, Hkv, page, D, seed, uneven=True):
    """Random blocks: codes -127..127, keys' scales alike, values' of unlike size."""
    g = torch.Generator().manual_seed(seed)
    c = torch.randint(1, 256, (pages, Hkv, page // 16, 32 * D + 16), generator=g, dtype=torch.uint8)
    s = torch.rand(pages, Hkv, page // 16, 4, generator=g) * 0.02 + 0.01
    if uneven:
        s[..., 1] *= torch.exp2(torch.randint(-6, 7, s.shape[:-1], generator=g).float())
    c[..., 32 * D:] = s.view(torch.uint8)
    return c


def logical(cache, table, page, b, n, D):
    """K and V [n][Hkv][D] fp64 of positions 0 .. n - 1, and which have a page."""
    P, H = cache.shape[:2]
    nb = -(-n // 16)
    k, v, has = np.zeros((nb * 16, H, D)), np.zeros((nb * 16, H, D)), np.zeros(nb * 16, bool)
    c = cache.numpy()
    for j in range(nb):
        pg = Q.pages_of(table, page, P, b, j * 16)
        if pg < 0:
            continue
        raw = c[pg, :, j * 16 % page // 16]
        s = np.ascontiguousarray(raw[:, 32 * D:32 * D + 8]).view(np.float32).astype(np.float64)
        kk = raw[:, :16 * D].reshape(H, 16, D).astype(np.float64) - 128
        vv = raw[:, 16 * D:32 * D].reshape(H, 4, D, 4).transpose(0, 1, 3, 2).reshape(H, 16, D).astype(np.float64) - 128
        k[j * 16:j * 16 + 16] = (kk * s[:, 0, None, None]).transpose(1, 0, 2)
        v[j * 16:j * 16 + 16] = (vv * s[:, 1, None, None]).transpose(1, 0, 2)
        has[j * 16:j * 16 + 16] = True
    return k[:n], v[:n], has[:n]


def check_attn(case, dt, lens, counts, page, window=0, starts=None, seed=0, scale=None, cache=None, table=None, lead=0, tail=0,
               q_scale=1.3, rows=None):
    """Every row (or `rows` per sequence, spread) against the oracle."""
    Hq, Hkv, D = case
    g = torch.Generator().manual_seed(seed)
    if table is None:
        table, pages = make_table([max(n, 0) for n in lens], page, seed)
        cache = make_cache(pages, Hkv, page, D, seed)
    pages = cache.shape[0]
    one = counts is None
    counts = [1] * len(lens) if one else counts
    q_start = np.concatenate([[0], np.cumsum(counts)]) + lead
    T = int(q_start[-1]) + tail
    q = (torch.randn(T, Hq, D, generator=g) * q_scale).to(DT[dt])
    sc = D ** -0.5 if scale is None else scale
    i32 = lambda a: torch.from_numpy(np.asarray(a, np.int32)).to(DEV)  # noqa: E731
    out = torch.full((T, Hq, D), 7.0, dtype=DT[dt], device=DEV)
    lse = torch.full((T, Hq), 7.0, device=DEV)
    most = max(1, max(counts))
    ws = A.workspace(A.sfx_attn_q8_ws(len(lens), most, Hq, Hkv, D, table.shape[1] * page))
    ws.fill_(255)
    args = dict(q=q.to(DEV), cache=cache.to(DEV), table=table.to(DEV), lens=i32(lens), ws=ws, max_q=most, window=window,
                starts=None if starts is None else i32(starts), scale=scale, q_start=None if one else i32(q_start))
    A.sfx_attn_q8(out=out, lse=lse, **args)
    out2 = torch.empty_like(out)
    A.sfx_attn_q8(out=out2, **args)
    got, gl = np64(out), np64(lse)
    assert (got[:lead] == 7).all() and (got[T - tail:] == 7).all() and (gl[:lead] == 7).all()
    assert torch.equal(out[lead:T - tail], out2[lead:T - tail])
    worst = 0.0
    for b, n in enumerate(lens):
        if n <= 0:
            assert (got[q_start[b]:q_start[b + 1]] == 0).all() and (gl[q_start[b]:q_start[b + 1]] == -np.inf).all()
            continue
        cap = min(n, table.shape[1] * page)
        k, v, has = logical(cache, table.numpy(), page, b, cap, D)
        pick = range(counts[b]) if rows is None else sorted(set(np.linspace(0, counts[b] - 1, rows).astype(int))) if counts[b] else []
        for i in pick:
            pos, t = n - counts[b] + i, q_start[b] + i
            lo = max(0 if starts is None else starts[b], pos + 1 - window if window else 0, 0)
            hi = min(pos + 1, cap)
            keep = np.arange(lo, hi)[has[lo:hi]] if hi > lo else np.arange(0)
            for h in range(Hkv):
                hs = slice(h * (Hq // Hkv), (h + 1) * (Hq // Hkv))
                o, l, ab, size = Q.attention(np64(q[t, hs]), k[keep, h], v[keep, h], sc)
                top = np.abs(v[keep, h]).max() if len(keep) else 0.0
                tol, ltol = Q.attention_tolerance(o, l, ab, size, top, len(keep), D, HALF_STEP[dt])
                # fp16 rounds what reaches 65520 to an infinity
                over = (np.abs(o) + tol >= 65520) & np.isinf(got[t, hs]) & (np.sign(got[t, hs]) == np.sign(o)) & (dt == "f16")
                err = np.where(over, 0.0, np.abs(got[t, hs] - o))
                assert (err <= tol).all(), (b, i, h, (err / np.maximum(tol, 1e-300)).max())
                if len(keep):
                    assert (np.abs(gl[t, hs] - l) <= ltol).all(), (b, i, h)
                    worst = max(worst, (err / tol).max())
                else:
                    assert (got[t, hs] == 0).all() and (gl[t, hs] == -np.inf).all()
    say(f"   largest error {worst:.2f} of its limit")


HEADS = [(1, 1, 32), (4, 2, 64), (3, 3, 96), (8, 1, 128), (20, 4, 128), (32, 32, 64), (17, 1, 160), (6, 2, 192), (40, 2, 224), (16, 4, 256)]


@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("case", HEADS, ids=lambda c: "-".join(map(str, c)))
def test_attention_one_token(case, dt):
    say(f"attn {case} {dt}")
    check_attn(case, dt, [1, 0, 15, 16, 17, 33, 300, 2, 511, 100], None, 16, seed=case[0])
    check_attn(case, dt, [700, 31, 5000], None, 64, window=129, seed=case[2])


@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("case", HEADS, ids=lambda c: "-".join(map(str, c)))
def test_attention_many_tokens(case, dt):
    """Prompts, drafts and chunks behind a prefix in one call, rows of no sequence around them."""
    say(f"attn {case} {dt} many")
    check_attn(case, dt, [40, 0, 77, 16, 130, 1], [40, 0, 5, 16, 3, 1], 32, seed=case[0], lead=2, tail=3)
    check_attn(case, dt, [150, 200, 9], [150, 33, 0], 16, window=20, seed=case[1], rows=40)
    check_attn(case, dt, [333], [290], 128, starts=[100], seed=case[2], rows=40)


@pytest.mark.parametrize("dt", ["f16", "bf16"])
def test_attention_large(dt):
    """Long caches cut into runs, long prompts, and rows of both in ragged sequences."""
    check_attn((64, 8, 128), dt, [20000], None, 64, seed=1)
    check_attn((8, 8, 64), dt, [9000, 3], [5, 2], 32, seed=2)
    check_attn((16, 4, 128), dt, [1500, 700], [1500, 600], 64, seed=3, rows=25)
    check_attn((8, 1, 64), dt, [3000], [1111], 16, seed=4, rows=25, window=800)
    check_attn((4, 4, 256), dt, [2100, 40], [513, 40], 16, seed=5, rows=12)


def test_attention_odd_lengths():
    """More rows than positions, lengths past the table, starts past the end, all in one."""
    table, pages = make_table([64, 64, 64, 64, 64], 16, 1)
    cache = make_cache(pages, 2, 16, 64, 1)
    check_attn((4, 2, 64), "f16", [3, 100, 64, 50, -5], [7, 9, 4, 3, 2], 16, table=table, cache=cache, starts=[0, 60, 64, 49, 0])
    check_attn((4, 2, 64), "f16", [3, 100, 64, 50, 1], None, 16, table=table, cache=cache, starts=[5, -3, 63, 0, 0])
    # row offsets that leave rows out, and fewer rows allowed than there are
    q = torch.randn(10, 4, 64, device=DEV).half()
    i32 = lambda *a: torch.tensor(a, dtype=torch.int32, device=DEV)  # noqa: E731
    full, part = (torch.full_like(q, 7.0) for _ in range(2))
    ws = A.workspace(1 << 20)
    args = (q, cache.to(DEV), table[:2].contiguous().to(DEV), i32(40, 60))
    A.sfx_attn_q8(*args, full, ws, q_start=i32(1, 6, 9), max_q=5)
    A.sfx_attn_q8(*args, part, ws, q_start=i32(1, 6, 900), max_q=3)
    assert (full[0] == 7).all() and (full[9] == 7).all() and torch.isfinite(full).all()
    assert (part[4:6] == 7).all() and (part[9] == 7).all()


def test_attention_missing_pages_and_nan():
    """Positions without a page are left out; blocks outside what a row covers may hold NaN."""
    D, Hkv, page = 64, 2, 16
    lens, counts = [100, 70, 90], [30, 1, 40]
    table, pages = make_table(lens, page, 2)
    cache = make_cache(pages, Hkv, page, D, 3)
    table[0, 1], table[1, 0], table[2, 2] = -1, pages, pages + 100
    check_attn((6, 2, 64), "f16", lens, counts, page, table=table, cache=cache)
    for pg in range(pages):                               # NaN in all that is behind the window or past the end
        used = any(pg == int(table[b, j]) and (j + 1) * 16 > lens[b] - counts[b] + 1 - 5 for b in range(3) for j in range(-(-lens[b] // 16)))
        if not used:
            cache[pg, :, :, 32 * D:] = torch.full((4,), float("nan")).view(torch.uint8)
    check_attn((6, 2, 64), "bf16", lens, counts, page, table=table, cache=cache, window=5)
    # a NaN block that early rows do not reach: only rows that cover it are NaN
    table, pages = make_table([64], page, 5)
    cache = make_cache(pages, Hkv, page, D, 6)
    cache[int(table[0, 3]), :, :, 32 * D:] = torch.full((4,), float("nan")).view(torch.uint8)
    q = torch.randn(64, 4, D).half()
    out = torch.empty(64, 4, D, dtype=torch.float16, device=DEV)
    i32 = lambda *a: torch.tensor(a, dtype=torch.int32, device=DEV)  # noqa: E731
    A.sfx_attn_q8(q.to(DEV), cache.to(DEV), table.to(DEV), i32(64), out, A.workspace(1 << 20), q_start=i32(0, 64), max_q=64)
    assert torch.isfinite(out[:48]).all() and out[48:].isnan().all()
    ref = torch.empty(48, 4, D, dtype=torch.float16, device=DEV)
    A.sfx_attn_q8(q[:48].to(DEV), cache.to(DEV), table.to(DEV), i32(48), ref, A.workspace(1 << 20), q_start=i32(0, 48), max_q=48)
    # both are within attention_tolerance of the same numbers, where sum w |v| is at most the largest
    # value and a score's sum of products at most |q| max sum |k|
    k, v, _ = logical(cache, table.numpy(), page, 0, 48, D)
    size = D ** -0.5 * (q[:48].double().abs().amax() * np.abs(k).sum(2).max()).item()
    bound = 2.0 ** -11 + 2 * (D * 2.0 ** -23 * size + (2 * size / np.log(2) + 160) * 2.0 ** -22) + 2.0 ** -17
    off = np.abs(np64(out[:48]) - np64(ref))
    assert (off <= 2 * (bound * np.abs(v).max() + 2.0 ** -11 * np.abs(np64(ref))) * 1.01).all()


@pytest.mark.parametrize("dt", ["f16", "bf16"])
def test_attention_extreme_numbers(dt):
    """Values whose scales are 2^40 apart, zero scales, large scores, queries of any size; a NaN or
    an infinity in one row's query stays in that row."""
    D, Hkv, page = 64, 1, 16
    table, pages = make_table([200], page, 7)
    cache = make_cache(pages, Hkv, page, D, 8, uneven=False)
    s = cache[..., 32 * D:].contiguous().view(torch.float32)
    s[..., 1] *= torch.exp2(torch.arange(pages).float() * 4 - 28).view(-1, 1, 1)
    zero = int(table[0, 3])
    s[zero, :, :, :2] = 0
    cache[..., 32 * D:] = s.view(torch.uint8)
    cache[zero, :, :, :32 * D] = 128
    for n in (64, 200):
        check_attn((2, 1, 64), dt, [n], [1], page, table=table, cache=cache)
        check_attn((2, 1, 64), dt, [n], [40], page, table=table, cache=cache)
    tiny = make_cache(pages, Hkv, page, D, 8, uneven=False)
    t = tiny[..., 32 * D:].contiguous().view(torch.float32)
    t[..., 0] *= 2.0 ** -20
    tiny[..., 32 * D:] = t.view(torch.uint8)
    check_attn((2, 1, 64), dt, [200], [20], page, table=table, cache=tiny, q_scale=2.0 ** 12)
    check_attn((2, 1, 64), dt, [200], [20], page, table=table, cache=cache, q_scale=2.0 ** -12)
    check_attn((2, 1, 64), dt, [200], [20], page, table=table, cache=cache, scale=-0.3)
    check_attn((2, 1, 64), dt, [200], [20], page, table=table, cache=cache, scale=0.0)
    i32 = lambda *a: torch.tensor(a, dtype=torch.int32, device=DEV)  # noqa: E731
    for m in (6, 60):
        q = torch.randn(m, 2, D, generator=torch.Generator().manual_seed(1)).to(DT[dt]).to(DEV)
        good, bad = torch.empty_like(q), torch.empty_like(q)
        args = (cache.to(DEV), table.to(DEV), i32(200))
        ws = A.workspace(1 << 22)
        A.sfx_attn_q8(q, *args, good, ws, q_start=i32(0, m), max_q=m)
        q[2, 1, 5], q[m - 1, 0, 63] = float("nan"), float("inf")
        A.sfx_attn_q8(q, *args, bad, ws, q_start=i32(0, m), max_q=m)
        assert not torch.isfinite(bad[2, 1]).any() and not torch.isfinite(bad[m - 1, 0]).any()
        bad[2, 1], bad[m - 1, 0] = good[2, 1], good[m - 1, 0]
        assert torch.equal(good, bad)


def test_attention_rows_apart_and_strides():
    """Queries as slices of a wider tensor, and a table wider than the lengths need."""
    D, Hq, Hkv, page, T = 64, 4, 2, 16, 21
    table, pages = make_table([21], page, 1, width=40)
    cache = make_cache(pages, Hkv, page, D, 2).to(DEV)
    g = torch.Generator().manual_seed(3)
    wide = torch.randn(T, (Hq + 2 * Hkv) * D, generator=g).half().to(DEV)
    i32 = lambda *a: torch.tensor(a, dtype=torch.int32, device=DEV)  # noqa: E731
    ws = A.workspace(A.sfx_attn_q8_ws(1, T, Hq, Hkv, D, 640))
    outs = []
    for q in (wide[:, :Hq * D].unflatten(1, (Hq, D)), wide[:, :Hq * D].reshape(T, Hq, D)):
        outs.append(torch.empty(T, Hq, D, dtype=torch.float16, device=DEV))
        A.sfx_attn_q8(q, cache, table.to(DEV), i32(21), outs[-1], ws, q_start=i32(0, T), max_q=T)
    assert torch.equal(*outs)
