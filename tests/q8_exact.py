"""Data of the int8 attention whose exact results are known in closed form or held by few bits, so
that one position more or less, or one rounding too many, shows.  Blocks have scale 1: what is
stored is a whole number, and each position of each head holds a 127."""
import numpy as np


def counting_values(T: int, Hkv: int, D: int, pos: np.ndarray) -> np.ndarray:
    """v [T][Hkv][D]: 127 at dim (p + 5 h) % D, else 0."""
    v = np.zeros((T, Hkv, D), np.float32)
    for h in range(Hkv):
        v[np.arange(T), h, (pos + 5 * h) % D] = 127
    return v


def counting_results(lo: np.ndarray, hi: np.ndarray, Hq: int, Hkv: int, D: int):
    """o [T][Hq][D] and lse [T] for equal scores of 0 over positions lo[t] .. hi[t] - 1 (>= 0)."""
    n = np.maximum(hi - lo, 0)
    d = np.arange(D)
    upto = lambda x: (x[:, None] + D - 1 - d) // D                       # positions below x at dim d  # noqa: E731
    base = np.where(n[:, None] > 0, upto(hi) - upto(lo), 0)
    o = np.zeros((len(n), Hq, D))
    for h in range(Hq):
        o[:, h] = 127.0 * np.roll(base, 5 * (h // (Hq // Hkv)), 1) / np.maximum(n, 1)[:, None]
    with np.errstate(divide="ignore"):
        return o, np.log(n)


# Weights are all 2^9 and every sum is exact; the result takes a reciprocal, a product (2^-22
# together) and its own rounding.  lse: log2 off by two units of a number below 32 (2^-18 ln 2)
# and two roundings of numbers below 16.
COUNTING_REL, COUNTING_LSE = 2.0 ** -22, 2.0 ** -18


def whole_keys(s: np.ndarray, D: int, rng) -> np.ndarray:
    """k [T][D] of whole numbers with k @ whole_query(D) == s for integers |s| <= 127."""
    k = rng.integers(-127, 128, (len(s), D)).astype(np.float32)
    k[:, 0], k[:, D - 1] = s, 127
    return k


def whole_query(D: int) -> np.ndarray:
    q = np.zeros(D, np.float32)
    q[0] = 1
    return q


def whole_values(T: int, Hkv: int, D: int, rng) -> np.ndarray:
    v = rng.integers(-127, 128, (T, Hkv, D)).astype(np.float32)
    v[:, :, 0] = 127
    return v


def causal(s, v, scale, lo, hi):
    """o [T][D], sum_p w_p |v_p| and lse [T] (fp64) of rows with scores scale s[p] over p = lo[t] .. hi[t] - 1."""
    p = np.arange(len(s))
    x = np.where((p >= lo[:, None]) & (p < hi[:, None]), scale * s, -np.inf)
    top = x.max(1, keepdims=True)
    e = np.exp(x - top)
    w = e / e.sum(1, keepdims=True)
    return w @ v, w @ np.abs(v), top[:, 0] + np.log(e.sum(1))


def whole_tolerance(o, ab, smax, n, scale, half_step):
    """What separates a result from 64 bits when scores are integers of at most `smax` and values
    whole: exponents s k2 + 9 - ref with ref at most smax k2 in size, k2 = scale log2(e): four roundings of
    numbers up to (smax |scale| + 16) log2(e), on each side of the quotient; a weight's one fp16 term (2^-11), an
    exponential and sums (2^-20), and what is below fp16's last bit (2^-25 of at least 2^9, |v| <= 127)."""
    e = 2.0 ** -24 * 4 * (smax * abs(scale) + 16)
    return half_step * np.abs(o) * 1.001 + (2 * e + 2.0 ** -11 + 2.0 ** -20) * ab + n * 127 * 2.0 ** -34


def attention_rms(q, k, v, scale, half_step):
    """o [Hq][D] and the root mean square error [Hq][D] of an evaluation that rounds each weight once to fp16 (at
    most 2^-11 of it; uniform errors: over sqrt(3)) and the result within `half_step`, with D exact products of a
    score summed in fp32 (D additions, each off by at most 2^-24 of at most their sizes' sum, as a random walk)."""
    Hq, D = q.shape
    o, rms = np.zeros((Hq, D)), np.zeros((Hq, D))
    for h in range(Hq):
        kv = h // (Hq // k.shape[1])
        s = scale * (k[:, kv] @ q[h])
        w = np.exp(s - s.max())
        w /= w.sum()
        o[h] = w @ v[:, kv]
        ds = 2.0 ** -24 * (np.sqrt(D) * abs(scale) * (np.abs(k[:, kv]) @ np.abs(q[h])) + 8 * (np.abs(s) + np.abs(s).max() + 16))
        rms[h] = np.sqrt((w * w * (2.0 ** -22 / 3 + ds ** 2)) @ v[:, kv] ** 2 + (half_step * o[h]) ** 2 / 3)
    return o, rms


def score_patterns(n: int, rng):
    """Scores over positions, by name: integers of at most 112."""
    p = np.arange(n)
    return {"rising": np.minimum(p // 4 - 100, 100), "falling": np.maximum(100 - p // 4, -100),
            "steps": np.where(p % 64 < 32, -100 + p // 8 % 60, -112), "last": np.where(p == n - 1, 112, -112),
            "first": np.where(p == 0, 112, -112), "two": np.where((p == 3) | (p == n - 2), 90, 75),
            "random": rng.integers(-112, 113, n), "equal": np.full(n, -37)}
