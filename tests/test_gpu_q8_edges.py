"""The 8-bit layer half at the ends of its ranges."""
import numpy as np
import pytest
import torch

from activation_sparse_ffn_amd import _abi as A
from gpu_helpers import say
from oracle import q8_oracle as Q
from test_gpu_q8 import DEV, DT, HALF_STEP, TINY, check_norm, logical, make_cache, make_table, np64, rope_table

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
                # any number of [o - tol, o + tol] may be what is rounded, and both ends round to infinities where tol is
                # past the top: of terms that cancel, either sign
                over = np.isinf(got[t, hs]) & (np.sign(got[t, hs]) * o + tol >= top)
                err = np.where(over, 0.0, np.abs(got[t, hs] - o))
                assert (err <= tol + TINY[dt]).all(), (b, i, h, err.max(), o, got[t, hs])
                assert (np.abs(gl[t, hs] - l) <= ltol).all(), (b, i, h, gl[t, hs], l)


SCALES = {  # values' scales by page, powers of two
    "tiny": [-116], "tiniest": [-127], "subnormal": [-140, -149], "one tiny": [0, 0, 0, -127, 0], "one subnormal": [-145, 0, 0],
    "small beside smaller": [-60, -70, -100, -130], "huge": [120], "huge and tiny": [110, -60, -127], "huge and zero": [100, None],
    "apart": [100, 60, 30, 0, -30, -64, -90, -128, -149], "zero alone": [None], "tiny and zero": [-149, None]}


@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("name", SCALES)
def test_attention_value_scales_of_any_size(name, dt):
    """Blocks whose values are tiny, subnormal, huge or zero, alone and beside others, few rows and many, in
    one run and in several: weights count whatever the size of the values that they weigh."""
    page = 16
    for Hq, Hkv, D, lens, counts in ((2, 1, 64, [150, 33], [1, 1]), (2, 1, 64, [150, 20], [11, 3]), (4, 2, 96, [300], [60]),
                                     (2, 2, 128, [1500], [1]), (2, 1, 32, [700, 200], [140, 70]), (1, 1, 256, [1100], [120]), (1, 1, 64, [9000], [1])):
        say(f"value scales {name} {dt} {Hq}/{Hkv}x{D} {lens}")
        table, pages = make_table(lens, page, 7)
        cache = make_cache(pages, Hkv, page, D, 8, uneven=False)
        s = cache[..., 32 * D:].contiguous().view(torch.float32)
        for b in range(len(lens)):
            for j in range(-(-lens[b] // page)):
                e, pg = SCALES[name][j % len(SCALES[name])], int(table[b, j])
                s[pg, ..., 1] = 0.0 if e is None else torch.ldexp(1 + (s[pg, ..., 1] * 30), torch.tensor(e)) if e > -126 else 2.0 ** e
                if e is None:
                    cache[pg, ..., 16 * D:32 * D] = 128
        cache[..., 32 * D:] = s.view(torch.uint8)
        for q_scale in (1.3, 20.0):
            check_rows(Hq, Hkv, D, dt, page, table, cache, lens, counts, rows=6, q_scale=q_scale)
        check_rows(Hq, Hkv, D, dt, page, table, cache, lens, counts, rows=6, window=50)


@pytest.mark.parametrize("counts", [[1, 1], [9, 3], [90, 40]], ids=str)
def test_attention_blocks_not_covered_change_no_bit(counts):
    """Whatever scales lie in blocks that a row does not cover (behind its window, past its position), its result
    has the same bits; and so have rows beside one that does cover them."""
    Hq, Hkv, D, page, lens = 4, 2, 64, 16, [400, 120]
    table, pages = make_table([448, 192], page, 7)
    plain = make_cache(pages, Hkv, page, D, 8)
    q_start = np.concatenate([[0], np.cumsum(counts)])
    q = torch.randn(int(q_start[-1]), Hq, D, generator=torch.Generator().manual_seed(1)).half().to(DEV)
    ws = A.workspace(A.sfx_attn_q8_ws(2, max(counts), Hq, Hkv, D, table.shape[1] * page))

    def run(cache, window):
        out, lse = torch.empty_like(q), torch.empty(len(q), Hq, device=DEV)
        A.sfx_attn_q8(q, cache.to(DEV), table.to(DEV), i32(lens), out, ws, q_start=i32(q_start), max_q=max(counts), window=window, lse=lse)
        return out, lse
    for window in (0, 40):
        want = run(plain, window)
        for scale in (float("nan"), 0.0, 2.0 ** -140, 2.0 ** -70, 2.0 ** 100):
            for pos in (0, 300, 384, 400, 416):                # the block that takes this scale
                cache = plain.clone()
                for b in range(2):
                    at = min(pos, 448 if b == 0 else 191) // page
                    s = cache[int(table[b, at])][..., 32 * D:].contiguous().view(torch.float32)
                    s[..., 1] = scale
                    cache[int(table[b, at])][..., 32 * D:] = s.view(torch.uint8)
                got = run(cache, window)
                for b in range(2):
                    first = min(pos, 448 if b == 0 else 191) // page * page
                    p = torch.arange(lens[b] - counts[b], lens[b])
                    sees = (first <= p) & ((first + 15 > p - window) if window else (first >= 0))
                    rows = torch.arange(int(q_start[b]), int(q_start[b + 1]))[~sees]
                    for g, w in zip(got, want):
                        assert torch.equal(g[rows.to(DEV)], w[rows.to(DEV)]), (window, scale, pos, b)


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


# ------------------------------------------------------------------------------ AttnStep8

def make_half(d, Hq, Hkv, D, B, dt, lens, page, max_pos, max_tokens, seed):
    """A half on a cache of noise, its weights, and the position tensor."""
    from activation_sparse_ffn_amd import AttnStep8, rows_q8
    g = torch.Generator().manual_seed(seed)
    table, pages = make_table(lens, page, seed)
    pos = torch.full((B,), -1, dtype=torch.int32, device=DEV)
    s = AttnStep8(d, Hq, Hkv, D, B, dt, table.to(DEV), pos, pages, page=page, max_tokens=max_tokens,
                  cos_sin=torch.from_numpy(rope_table(max_pos, D)).to(DEV) if max_pos else None)
    s.cache.copy_(torch.randint(0, 256, s.cache.shape, generator=g, dtype=torch.uint8))
    w = {"wn": (1 + 0.2 * torch.randn(d, generator=g)).to(DEV), "bqkv": None, "bo": torch.randn(d, generator=g).to(DEV)}
    w["Wqkv"], w["Wqkv_s"] = rows_q8((torch.randn((Hq + 2 * Hkv) * D, d, generator=g) * d ** -0.5).to(DEV))
    w["Wo"], w["Wo_s"] = rows_q8((torch.randn(d, Hq * D, generator=g) * (Hq * D) ** -0.5).to(DEV))
    return s, w, pos


@pytest.mark.parametrize("case", [(8, 2, 64, "f16", 16, [40, 12, 60]), (4, 4, 32, "bf16", 32, [70, 5, 300]), (6, 1, 128, "f16", 16, [20, 31, 130])],
                         ids=lambda c: "-".join(map(str, c)))
def test_prompt_rows_that_are_no_token(case):
    """Rows past the table of angles, without a page, in front of position 0 or of no sequence: their y is the
    output bias, whatever earlier calls left in the object, and the other rows do not see them."""
    Hq, Hkv, D, dt, page, counts = case
    d, max_pos, lead, tail = 256, 33, 2, 3
    say(f"no token {case}")
    g = torch.Generator().manual_seed(D)
    lens = list(counts)
    lens[1] -= 2                                         # two rows in front of position 0
    q_start = np.concatenate([[0], np.cumsum(counts)]) + lead
    T = int(q_start[-1]) + tail
    s, w, _ = make_half(d, Hq, Hkv, D, 3, dt, counts, page, max_pos, T, D)
    s.table[2, 0] = -1                                   # the third sequence's first page is missing
    x = torch.randn(T, d, generator=g).to(DEV)
    start, ys = s.cache.clone(), []
    for junk in (0.0, 3.0, float("nan")):
        s.cache.copy_(start)
        for t in (s.q, s.o, s.qkv):
            t.fill_(junk)
        y = torch.full((T, d), 9.0, device=DEV)
        s.prompt(w, x, y, i32(q_start), i32(lens), max(counts))
        ys.append(y)
    assert torch.equal(ys[0], ys[1]) and torch.equal(ys[0], ys[2])
    is_token = np.zeros(T, bool)
    for b in range(3):
        p = np.arange(lens[b] - counts[b], lens[b])
        is_token[q_start[b]:q_start[b + 1]] = (p >= 0) & (p < max_pos) & ((b != 2) | (p >= page))
    is_token = torch.from_numpy(is_token).to(DEV)
    assert torch.equal(ys[0][~is_token], w["bo"].expand(T, -1)[~is_token])
    assert (ys[0][is_token] != w["bo"]).any(1).all()
    # the tokens' attention over what the cache holds
    got, q, cache, table = np64(s.o[:T]), np64(s.q[:T]), s.cache.cpu(), s.table.cpu().numpy()
    for b in range(3):
        k, v, has = logical(cache, table, page, b, min(lens[b], max_pos), D)
        for i in range(counts[b]):
            t, p = int(q_start[b]) + i, lens[b] - counts[b] + i
            if not is_token[t]:
                continue
            keep = np.flatnonzero(has[:p + 1])
            for h in range(Hkv):
                hs = slice(h * (Hq // Hkv), (h + 1) * (Hq // Hkv))
                o, _, ab, size = Q.attention(q[t, hs], k[keep, h], v[keep, h], D ** -0.5)
                tol, _ = Q.attention_tolerance(o, _, ab, size, np.abs(v[keep, h]).max(), len(keep), D, HALF_STEP[dt])
                assert (np.abs(got[t, hs] - o) <= tol + TINY[dt]).all(), (b, i, h)
    y = torch.full((T, d), 9.0, device=DEV)              # added to y: the bias alone
    s.cache.copy_(start)
    s.prompt(w, x, y, i32(q_start), i32(lens), max(counts), accumulate=True)
    assert torch.equal(y[~is_token], (w["bo"] + 9.0).expand(T, -1)[~is_token])
    # rows past max_q are stored, and have no output
    s.cache.copy_(start)
    s.o.fill_(5.0)
    s.prompt(w, x, y, i32(q_start), i32(lens), 8)
    past = torch.cat([torch.arange(T)[int(q_start[b]) + 8:int(q_start[b + 1])] for b in range(3)])
    assert len(past) and torch.equal(y[past.to(DEV)], w["bo"].expand(len(past), -1))


def test_prompt_without_tokens_in_a_graph():
    """The same captured: rows become tokens and stop being tokens between replays."""
    d, Hq, Hkv, D, B, n = 256, 4, 2, 64, 2, 48
    say("no token, captured")
    s, w, _ = make_half(d, Hq, Hkv, D, B, "f16", [64, 64], 16, 64, 2 * n, 1)
    e, _, _ = make_half(d, Hq, Hkv, D, B, "f16", [64, 64], 16, 64, 2 * n, 1)
    x, y = torch.randn(2 * n, d, device=DEV), torch.zeros(2 * n, d, device=DEV)
    q_start, lens = i32([0, n, 2 * n]), i32([n, n])
    s.prompt(w, x, y, q_start, lens, n)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        s.prompt(w, x, y, q_start, lens, n)
    for rep, (at, ln) in enumerate((([0, n, 2 * n], [n, n]), ([0, 5, 9], [5, 70]), ([3, 3, 40], [0, 20]), ([0, n, 2 * n], [64, 80]),
                                    ([0, n, 2 * n], [n, n]))):
        q_start.copy_(i32(at))
        lens.copy_(i32(ln))
        s.cache.zero_()
        e.cache.zero_()
        g.replay()
        ye = torch.zeros_like(y)
        e.prompt(w, x, ye, i32(at), i32(ln), n)
        torch.cuda.synchronize()
        assert torch.equal(y, ye) and torch.equal(s.cache, e.cache), rep
        assert torch.equal(y[at[2]:], w["bo"].expand(2 * n - at[2], -1)), rep


@pytest.mark.parametrize("case", [(1, 16, 70, 0), (3, 32, 5, 40), (70, 16, 200, 33), (200, 64, 3, 100)], ids=str)
def test_blank_rows(case):
    """Rows that the append does not store and rows past max_q become zeros, the others stay."""
    B, page, most, max_pos = case
    say(f"blank {case}")
    rng = np.random.default_rng(B)
    counts, lens = rng.integers(0, 2 * most // (1 + B // 50) + 2, B), rng.integers(-3, 150, B)
    width = 8
    table = rng.integers(-1, 12, (B, width)).astype(np.int32)              # -1 and 10, 11 are no pages
    q_start = np.concatenate([[0], np.cumsum(counts)]) + 2
    T = int(q_start[-1]) + 3
    for n in (8, 520, 4096):
        x = torch.randn(T, n, generator=torch.Generator().manual_seed(n)).to(torch.bfloat16 if n == 520 else torch.float16)
        for starts in (q_start, None):
            rows = T if starts is not None else B
            first = q_start if starts is not None else np.arange(B + 1)
            got = x[:rows].clone().to(DEV) if rows <= T else x.repeat(-(-rows // T), 1)[:rows].to(DEV)
            was = got.cpu()
            A.sfx_kv_blank_q8(got, i32(lens), torch.from_numpy(table).to(DEV), page, 10, q_start=None if starts is None else i32(starts),
                              max_q=most, max_pos=max_pos)
            keep = np.zeros(rows, bool)
            for b in range(B):
                m = int(first[b + 1] - first[b])
                for i in range(min(m, most)):
                    p = int(lens[b]) - m + i if lens[b] > 0 else -1
                    keep[first[b] + i] = (not max_pos or p < max_pos) and Q.pages_of(table, page, 10, b, p) >= 0
            assert torch.equal(got.cpu()[keep], was[keep]) and (got.cpu()[~keep] == 0).all()
            assert B == 1 or (keep.any() and not keep.all())


def test_steps_and_prompts_of_one_object_overlap():
    """A decode step of other sequences that runs while a prompt is between its calls, and a prompt that runs
    while a step is: both give what they give alone, and so does the cache."""
    d, Hq, Hkv, D, B, n = 256, 8, 2, 64, 3, 40
    say("step within prompt, prompt within step")
    g = torch.Generator().manual_seed(2)
    x, xs = torch.randn(n, d, generator=g).to(DEV), torch.randn(B, d, generator=g).to(DEV)
    q_start, lens = i32([0, 0, n, n]), i32([0, n, 0])
    names = ("sfx_norm_q8", "sfx_linear_q8", "sfx_kv_append_q8", "sfx_attn_q8")

    def run(inner, at, monkeypatch):
        """The prompt of sequence 1 and a step of 0 and 2, one whole inside the other before its call `at`."""
        s, w, pos = make_half(d, Hq, Hkv, D, B, "f16", [64] * 3, 16, 64, n, 5)
        pos.copy_(i32([0, -1, 0]))
        yp, ys = torch.zeros(n, d, device=DEV), torch.zeros(B, d, device=DEV)
        other = torch.cuda.Stream()
        calls = {"prompt": lambda st: s.prompt(w, x, yp, q_start, lens, n, stream=st), "step": lambda st: s.run(w, xs, ys, stream=st)}
        if inner is None:
            calls["prompt"](None)
            calls["step"](None)
        else:
            outer = "step" if inner == "prompt" else "prompt"
            seen, busy = [0], [False]
            with monkeypatch.context() as m:
                for name in names:
                    def call(*a, f=getattr(A, name), **k):
                        if not busy[0]:
                            if seen[0] == at:
                                busy[0] = True
                                torch.cuda.synchronize()
                                other.wait_stream(torch.cuda.current_stream())
                                calls[inner](other)
                                other.synchronize()
                                busy[0] = False
                            seen[0] += 1
                        return f(*a, **k)
                    m.setattr(A, name, call)
                calls[outer](None)
            assert seen[0] == 6
        torch.cuda.synchronize()
        return yp, ys, s.cache.clone()

    with pytest.MonkeyPatch.context() as m:
        alone = run(None, 0, m)
        for inner in ("step", "prompt"):
            for at in range(6):
                for a, b in zip(run(inner, at, m), alone):
                    assert torch.equal(a, b), (inner, at)
