"""Data of the int4 attention half whose exact results are known in closed form or held by few
bits, so that one position more or less, or one rounding too many, shows."""
import numpy as np


def counting_values(T: int, Hkv: int, D: int, pos: np.ndarray) -> np.ndarray:
    """v [T][Hkv][D]: 7 at dim (p + 5 h) % D, else 0.  Its scales are 1 and 0, its codes 7 and 0."""
    v = np.zeros((T, Hkv, D), np.float16)
    for h in range(Hkv):
        v[np.arange(T), h, (pos + 5 * h) % D] = 7
    return v


def counting_result(lo: int, hi: int, Hq: int, Hkv: int, D: int):
    """o [Hq][D] and lse for equal scores of 0 over positions lo .. hi - 1."""
    n = max(0, hi - lo)
    o = np.zeros((Hq, D))
    if n == 0:
        return o, -np.inf
    base = np.bincount(np.arange(lo, hi) % D, minlength=D)
    for h in range(Hq):
        kv = h // (Hq // Hkv)
        o[h] = 7.0 * np.roll(base, 5 * kv) / n
    return o, np.log(n)


# Weights are all 2^9 and every sum is exact; the result takes a reciprocal, a product (2^-22
# together) and its own rounding.  lse: log2 off by two units of a number below 32 (2^-18 ln 2)
# and two roundings of numbers below 16.
COUNTING_REL, COUNTING_LSE = 2.0 ** -22, 2.0 ** -18


def digit_keys(s: np.ndarray, D: int, rng) -> np.ndarray:
    """k [T][D] of integers -7..7 with scale 1 in every group: k @ digit_query(D) == s for integers
    |s| <= 112."""
    s = np.asarray(s, np.int64)
    k = rng.integers(-7, 8, (len(s), D)).astype(np.float32)
    k[:, 31::32] = 7                                   # fixes the groups' scales at 1
    hi = np.rint(s / 15.0).astype(np.int64)
    k[:, 0], k[:, 1] = s - 15 * hi, hi
    assert np.abs(k).max() == 7
    return k


def digit_query(D: int) -> np.ndarray:
    q = np.zeros(D, np.float32)
    q[0], q[1] = 1, 15
    return q


def whole_values(T: int, Hkv: int, D: int, rng) -> np.ndarray:
    """v of integers -7..7 with scale 1 in every group."""
    v = rng.integers(-7, 8, (T, Hkv, D)).astype(np.float32)
    v[:, :, ::32] = 7
    return v


def exact_scores_tolerance(o, ab, smax, n, scale, two_terms, half_step):
    """What separates a result from 64 bits when scores are integers of at most `smax` and values
    whole: exponents s k2 + 9 - ref with ref = smax k2, k2 = scale log2(e): four roundings of numbers
    up to (smax |scale| + 16) log2(e), on each side of the quotient; a weight's terms (2^-22, or 2^-11
    for one) and what is below fp16's last bit (2^-25 of at least 2^9, |v| <= 7); sums."""
    e = 2.0 ** -24 * 4 * (smax * abs(scale) + 16)
    w = 2 * e + (2.0 ** -22 if two_terms else 2.0 ** -11) + 2.0 ** -20
    return half_step * np.abs(o) * 1.001 + w * ab + n * 7 * 2.0 ** -34


# Scores over positions, by name: integers of at most 112.
def score_patterns(n: int, rng):
    p = np.arange(n)
    return {"rising": np.minimum(p // 4 - 100, 100), "falling": np.maximum(100 - p // 4, -100),
            "steps": np.where(p % 64 < 32, -100 + p // 8 % 60, -112), "last": np.where(p == n - 1, 112, -112),
            "first": np.where(p == 0, 112, -112), "two": np.where((p == 3) | (p == n - 2), 90, 75),
            "random": rng.integers(-112, 113, n), "equal": np.full(n, -37)}
