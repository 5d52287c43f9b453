"""The limits of the int8 attention's precision tests, on the CPU: evaluations with the roundings that
the kernels are allowed pass them, and evaluations with a mistake planted do not."""
import numpy as np
import pytest

import q8_exact as E
from oracle import q4_oracle as Q4
from oracle import q8_oracle as Q
from test_q4_exact_host import HALF, rounded


def attend(s, v, dt, keep, value=lambda x: x):
    """One row of scores s [n] over values v [n][D] as the kernels take it: weights 2^9 e^(s - max) as one fp16 term,
    summed unrounded, everything else in 64 bits."""
    p = np.exp(s[keep] - s[keep].max()) * 512
    o = p.astype(np.float16).astype(np.float64) @ value(v[keep]) / p.sum()
    return rounded(o[None], dt)[0], s[keep].max() + np.log(p.sum() / 512)


def held(x):
    """What a block of positions stands for once it is stored."""
    out = np.zeros(x.shape)
    for b in range(0, len(x), 16):
        for h in range(x.shape[1]):
            q, s = Q.store_rows(np.zeros((16, x.shape[2]), np.int64), np.float32(0), x[b:b + 16, h], 0)
            out[b:b + 16, h] = (q * np.float64(s))[:len(x[b:b + 16])]
    return out


def test_whole_numbers_are_stored_as_they_are():
    rng = np.random.default_rng(0)
    for x in (E.counting_values(50, 2, 32, np.arange(50)), E.whole_values(50, 3, 64, rng),
              E.whole_keys(rng.integers(-112, 113, 50), 96, rng)[:, None]):
        assert np.array_equal(held(x), x)


def test_counting_results_worked():
    """Positions 3 .. 8 of D = 4, second head shifted by five: dims 3 0 1 2 3 0."""
    o, lse = E.counting_results(np.array([3, 5, 0]), np.array([9, 5, 4]), 2, 2, 4)
    assert np.allclose(o[0, 0] * 6 / 127, [2, 1, 1, 2]) and np.allclose(o[0, 1] * 6 / 127, [2, 2, 1, 1])
    assert (o[1] == 0).all() and np.isneginf(lse[1]) and np.allclose(o[2, 0], 127 / 4) and np.allclose(lse[2], np.log(4))


@pytest.mark.parametrize("dt", ["f16", "bf16"])
def test_counting_limit(dt):
    """Equal scores: each position counts in a dim of its own, so one more or less shows."""
    for n, D in ((33, 32), (400, 96), (3000, 128), (9000, 64)):
        v = E.counting_values(n + 1, 1, D, np.arange(n + 1))[:, 0].astype(np.float64)
        want, lse = E.counting_results(np.array([5]), np.array([n]), 1, 1, D)
        p = np.arange(n + 1)
        inside = (p >= 5) & (p < n)

        def passes(keep):
            o, ls = attend(np.zeros(n + 1), v, dt, keep)
            return (np.abs(o - want[0, 0]) <= (HALF[dt] + E.COUNTING_REL) * want[0, 0]).all() and abs(ls - lse[0]) <= E.COUNTING_LSE
        assert passes(inside)
        for at in (4, 5, 31, n // 2, n - 1, n):
            wrong = inside.copy()
            wrong[at] = ~wrong[at]
            assert not passes(wrong), (n, at)
        # one position for another, and one block for another of another phase
        wrong = inside.copy()
        wrong[6], wrong[4] = False, True
        assert not passes(wrong), n


@pytest.mark.parametrize("dt", ["f16", "bf16"])
def test_whole_score_limits(dt):
    rng = np.random.default_rng(3)
    n, D = 450, 64
    v = E.whole_values(n, 1, D, rng)[:, 0].astype(np.float64)
    q = E.whole_query(D).astype(np.float64)
    for name, s in E.score_patterns(n, rng).items():
        assert np.array_equal(E.whole_keys(s, D, rng).astype(np.float64) @ q, s)
        for scale in (float(np.float32(np.log(2.0))), 0.3, -0.3):
            o, ab, lse = E.causal(s, v, scale, np.array([0]), np.array([n]))
            tol = E.whole_tolerance(o, ab, 112, n, scale, HALF[dt])[0]
            got, ls = attend(scale * s, v, dt, np.ones(n, bool))
            assert (np.abs(got - o[0]) <= tol).all() and abs(ls - lse[0]) < 1e-9, (name, scale)
            top = int(np.argmax(scale * s))
            if name in ("rising", "falling", "last", "first", "two"):
                bad, _ = attend(scale * s, v, dt, np.arange(n) != top)
                assert not (np.abs(bad - o[0]) <= tol).all(), (name, scale)


@pytest.mark.parametrize("dt", ["f16", "bf16"])
def test_attention_rms_limit(dt):
    rng = np.random.default_rng(1)
    Hq, Hkv, D, n = 8, 2, 64, 320
    q = rounded(rng.standard_normal((Hq, D)), dt)
    k, v = (held(rng.standard_normal((n, Hkv, D)).astype(np.float32)) for _ in range(2))
    o, rms = E.attention_rms(q, k, v, D ** -0.5, HALF[dt])

    def ratio(keep=np.ones(n, bool), value=lambda x: x, scores=lambda s: s):
        got = np.stack([attend(scores(D ** -0.5 * (k[:, h // 4] @ q[h])), v[:, h // 4], dt, keep, value)[0] for h in range(Hq)])
        return Q4.rms_ratio(got - o, rms)
    assert 0.3 < ratio() < 1
    assert ratio(keep=np.arange(n) < n - 1) > 2 and ratio(keep=np.arange(n) != 100) > 2
    if dt == "f16":                                      # coarser values, coarser scores
        assert ratio(value=lambda x: rounded(x, "bf16")) > 2
        assert ratio(scores=lambda s: rounded(s, "f16")) > 1.1 and ratio(scores=lambda s: rounded(s, "bf16")) > 3
