"""The limits of the int4 attention half's precision tests, on the CPU: evaluations with the roundings
that the kernels are allowed pass them, and evaluations with a mistake planted do not."""
import numpy as np
import pytest

import q4_exact as E
from oracle import q4_oracle as Q


def rounded(x, dt):
    if dt == "f16":
        return x.astype(np.float16).astype(np.float64)
    u = x.astype(np.float32).view(np.uint32).astype(np.uint64)
    u = (u + 0x7FFF + ((u >> 16) & 1)) >> 16 << 16
    return u.astype(np.uint32).view(np.float32).astype(np.float64)


HALF = {"f16": 2.0 ** -11, "bf16": 2.0 ** -8}


def attend(q, k, v, scale, dt, terms=None, value=lambda x: x.astype(np.float16), keep=None):
    """One query row [Hq][D] as the kernels take it: weights 2^(s - max + 9) as `terms` fp16 terms
    (default as the kernels: two for fp16), values rounded by `value`, everything else in 64 bits."""
    terms = (2 if dt == "f16" else 1) if terms is None else terms
    o, lse = np.zeros(q.shape), np.zeros(q.shape[0])
    keep = np.ones(len(k), bool) if keep is None else keep
    for h in range(q.shape[0]):
        kv = h // (q.shape[0] // k.shape[1])
        s = scale * (k[keep, kv] @ q[h])
        p = np.exp(s - s.max()) * 512
        held = p.astype(np.float16).astype(np.float64)
        if terms == 2:
            held = held + (p - held).astype(np.float16).astype(np.float64)
        o[h] = held @ value(v[keep, kv]).astype(np.float64) / p.sum()
        lse[h] = s.max() + np.log(p.sum() / 512)
    return rounded(o, dt), lse


def test_linear_limit():
    rng = np.random.default_rng(0)
    for B, n, d, G in ((1, 40, 64, 32), (3, 60, 1056, 32), (2, 50, 4096, 128), (1, 1, 4096, 64)):
        x = rng.standard_normal((B, d)).astype(np.float16).astype(np.float64)
        W = rng.integers(0, 256, (n, d // 2), dtype=np.uint8)
        s = (0.05 * rng.random((n, d // G)) + 1e-3).astype(np.float16)
        ref = Q.linear_q4(x, W, s)
        q = Q.unpack_rows(W).reshape(n, -1, G)
        # fp32 sums, one group after the other, as a correct evaluation might take them
        w32, x32 = q.astype(np.float32), x.astype(np.float32).reshape(B, -1, G)
        y = np.zeros((B, n), np.float32)
        for g in range(d // G):
            part = np.zeros((B, n), np.float32)
            for c in range(G):
                part += x32[:, g, c][:, None] * w32[:, g, c][None]
            y += s[:, g].astype(np.float32) * part
        limit16, limitb = Q.linear_q4_rms(x, W, s, False), Q.linear_q4_rms(x, W, s, True)
        assert Q.rms_ratio(y - ref, limit16) < 1 and (limitb > limit16).all()
        # weights rounded to fp16 or bf16, tokens to bf16: within the bound for any data, not within these
        w = q * s.astype(np.float64)[..., None]
        for bad_w, bad_x in ((rounded(w, "f16"), x), (rounded(w, "bf16"), x), (w, rounded(x, "bf16"))):
            bad = bad_x @ bad_w.reshape(n, d).T
            assert (np.abs(bad - ref) <= Q.linear_q4_bound(x, W, s)).mean() > 0.5 or d < 100
            assert Q.rms_ratio(bad - ref, limitb) > 2, (B, n, d, G)


@pytest.mark.parametrize("dt", ["f16", "bf16"])
def test_attention_rms_limit(dt):
    rng = np.random.default_rng(1)
    Hq, Hkv, D, n = 8, 2, 64, 300
    q = rounded(rng.standard_normal((Hq, D)), dt)
    k, v = (Q.values(*Q.quantise(rng.standard_normal((n, Hkv, D)).astype(np.float32), 8188.0)) for _ in range(2))
    wstep = 2.0 ** -22 if dt == "f16" else 2.0 ** -11
    o, rms = Q.attention_rms(q, k, v, D ** -0.5, dt == "bf16", wstep, 2.0 ** -11, HALF[dt])
    got, _ = attend(q, k, v, D ** -0.5, dt)
    assert 0.3 < Q.rms_ratio(got - o, rms) < 1
    # coarser values, the last position left out
    coarse, _ = attend(q, k, v, D ** -0.5, dt, value=lambda x: rounded(x, "bf16"))
    few, _ = attend(q, k, v, D ** -0.5, dt, keep=np.arange(n) < n - 1)
    assert Q.rms_ratio(few - o, rms) > 1.5
    if dt == "f16":
        assert Q.rms_ratio(coarse - o, rms) > 2


@pytest.mark.parametrize("dt", ["f16", "bf16"])
def test_counting_limit(dt):
    """Equal scores: each position counts in a dim of its own, so one more or less shows."""
    for n, D, Hkv in ((33, 32, 1), (400, 96, 3), (3000, 128, 2)):
        rng = np.random.default_rng(n)
        v = E.counting_values(n + 1, Hkv, D, np.arange(n + 1)).astype(np.float64)
        held = Q.values(*Q.quantise(v.astype(np.float32), 8188.0))
        assert np.array_equal(held, v)
        q, k = np.zeros((2 * Hkv, D)), rng.standard_normal((n + 1, Hkv, D))
        want, lse = E.counting_result(5, n, 2 * Hkv, Hkv, D)
        inside = (np.arange(n + 1) >= 5) & (np.arange(n + 1) < n)

        def passes(keep):
            o, ls = attend(q, k, v, 1.0, dt, keep=keep)
            return (np.abs(o - want) <= (HALF[dt] + E.COUNTING_REL) * want).all() and (np.abs(ls - lse) <= E.COUNTING_LSE).all()
        assert passes(inside)
        for p in (4, 5, 31, n - 1, n):
            wrong = inside.copy()
            wrong[p] = ~wrong[p]
            assert not passes(wrong), (n, p)


@pytest.mark.parametrize("dt", ["f16", "bf16"])
def test_exact_score_limits(dt):
    rng = np.random.default_rng(3)
    n, D = 450, 64
    v = E.whole_values(n, 1, D, rng)
    vq, vs = Q.quantise(v, 8188.0)
    assert (vs == 1).all() and np.array_equal(Q.values(vq, vs), v)
    q = np.stack([E.digit_query(D)] * 2).astype(np.float64)
    ln2 = float(np.float32(np.log(2.0)))
    for name, s in E.score_patterns(n, rng).items():
        k = E.digit_keys(s, D, rng)
        kq, ks = Q.quantise(k, 65504.0)
        assert (ks == 1).all() and np.array_equal(Q.values(kq, ks), k)
        k = k[:, None].astype(np.float64)
        assert np.array_equal(k[:, 0] @ q[0], s)
        for scale in (ln2, 0.3, -0.3):
            o, _, ab = Q.attention(q, k, v, scale)
            tol = E.exact_scores_tolerance(o, ab, 112, n, scale, dt == "f16", HALF[dt])
            got, _ = attend(q, k, v, scale, dt)
            assert (np.abs(got - o) <= tol).all(), (name, scale)
            top = int(np.argmax(scale * s))
            if name in ("rising", "falling", "last", "first", "two"):
                bad, _ = attend(q, k, v, scale, dt, keep=np.arange(n) != top)
                assert not (np.abs(bad - o) <= tol).all(), (name, scale)


def test_one_weight_term_is_not_enough_for_fp16():
    """Small integer scores under a scale that gives no powers of two: with whole values the second
    fp16 term of a weight is all that separates the two forms."""
    rng = np.random.default_rng(5)
    n, D = 48, 128
    s = rng.integers(-8, 9, n)
    k = E.digit_keys(s, D, rng)[:, None].astype(np.float64)
    v = E.whole_values(n, 1, D, rng)
    q = np.stack([E.digit_query(D)] * 2).astype(np.float64)
    o, _, ab = Q.attention(q, k, v, 0.3)
    tol = E.exact_scores_tolerance(o, ab, 8, n, 0.3, True, HALF["f16"])
    one, _ = attend(q, k, v, 0.3, "f16", terms=1)
    two, _ = attend(q, k, v, 0.3, "f16", terms=2)
    assert (np.abs(two - o) <= tol).all()
    assert (np.abs(one - o) > tol).sum() > 5
