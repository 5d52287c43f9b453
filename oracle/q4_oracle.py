"""Plain fp64 forms of the int4 attention half of a layer (numpy, test infrastructure):
the int4 projection, the rotation and quantisation of cached keys and values, the cache's
byte layout, and attention over a list of positions."""
import numpy as np


def unpack_rows(codes: np.ndarray) -> np.ndarray:
    """Two's-complement nibbles uint8 [n][d/2] -> int [n][d] (column 2c in the low nibble)."""
    out = np.empty((codes.shape[0], codes.shape[1] * 2), np.int64)
    out[:, 0::2] = codes & 15
    out[:, 1::2] = codes >> 4
    return np.where(out > 7, out - 16, out)


def linear_q4(x: np.ndarray, codes: np.ndarray, scales: np.ndarray, bias=None) -> np.ndarray:
    """x fp64 [B][d] -> fp64 [B][n]."""
    q = unpack_rows(codes).astype(np.float64)
    group = q.shape[1] // scales.shape[1]
    w = q * np.repeat(scales.astype(np.float64), group, axis=1)
    y = x @ w.T
    return y if bias is None else y + bias.astype(np.float64)


def linear_q4_bound(x: np.ndarray, codes: np.ndarray, scales: np.ndarray) -> np.ndarray:
    """Largest error of an fp32 evaluation [B][n] whose group sums take (16 + u) x terms from
    a start of -24 sum(x): each of the 65 additions of a group of 32 is off by at most one
    unit 2^-23 of a partial sum, which is at most 55 sum|x| of the group; then one fp32
    multiply-add per group of 32 of the partial results' size."""
    B, d = x.shape
    ng = d // 32
    ax = np.abs(x).reshape(B, ng, 32).sum(2)                          # [B][ng]
    s32 = np.repeat(np.abs(scales.astype(np.float64)), scales.shape[1] and d // scales.shape[1] // 32, axis=1)
    group_err = 2.0 ** -23 * 65 * 55 * (ax @ s32.T)
    sums = 2.0 ** -23 * (ng + 16) * 8 * (ax @ s32.T)
    return group_err + sums + 2.0 ** -120


def rotate(x: np.ndarray, pos: np.ndarray, cos_sin, interleaved: bool) -> np.ndarray:
    """x [T][H][D] (exact values) rotated at pos: 64-bit products and sum, rounded to fp32."""
    x = x.astype(np.float64)
    if cos_sin is None:
        return x.astype(np.float32)
    rot = cos_sin.shape[1]
    c = cos_sin[pos].astype(np.float64)[:, None, :rot // 2]
    s = cos_sin[pos].astype(np.float64)[:, None, rot // 2:]
    y = x.copy()
    if interleaved:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        y[..., 0:rot:2], y[..., 1:rot:2] = a * c - b * s, b * c + a * s
    else:
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        y[..., :rot // 2], y[..., rot // 2:rot] = a * c - b * s, b * c + a * s
    return y.astype(np.float32)


def quantise(w: np.ndarray, top: float):
    """fp32 [..., D] -> codes -8..7 [..., D] and fp16 scales [..., D/32] (at most `top`)."""
    with np.errstate(all="ignore"):
        g = w.astype(np.float32).reshape(*w.shape[:-1], -1, 32)
        m = np.abs(g).max(-1)
        bad = ~np.isfinite(g).all(-1)
        s = np.minimum((m / np.float32(7.0)).astype(np.float32), np.float32(top)).astype(np.float16)
        s = np.where(bad, np.float16(np.nan), s)
        sf = s.astype(np.float32)[..., None]
        q = np.where(sf > 0, np.clip(np.rint((g / np.where(sf > 0, sf, np.float32(1))).astype(np.float32)), -8, 7), 0)
    return np.where(bad[..., None], 0, q).astype(np.int64).reshape(w.shape), s


def values(q: np.ndarray, s: np.ndarray) -> np.ndarray:
    return (q.reshape(*q.shape[:-1], -1, 32) * s.astype(np.float64)[..., None]).reshape(q.shape)


K_NIBBLE = (0, 4, 1, 5, 2, 6, 3, 7)            # nibble of dim j of a K word
V_BYTE = (0, 2, 1, 3, 4, 6, 5, 7)              # byte of position i of a V unit


def read_block(block: np.ndarray, D: int, i: int):
    """Codes and scales (kq, ks, vq, vs) of position i of one 9 D-byte block, one element at
    a time."""
    NG = D // 32
    kq, vq = np.zeros(D, np.int64), np.zeros(D, np.int64)
    for g in range(NG):
        for c in range(4):
            at = i * (D // 2) + (c * NG + g) * 4
            for j in range(8):
                nib = K_NIBBLE[j]
                kq[32 * g + 8 * c + j] = ((int(block[at + nib // 2]) >> (4 * (nib % 2))) & 15) - 8
        for n in range(16):
            byte = int(block[4 * D + n * 8 * NG + g * 8 + V_BYTE[i]])
            vq[32 * g + n], vq[32 * g + 16 + n] = (byte & 15) - 8, (byte >> 4) - 8
    sc = block[8 * D:].view(np.float16).reshape(2, NG, 8)
    return kq, sc[0, :, i].copy(), vq, sc[1, :, i].copy()


def attention(q: np.ndarray, k: np.ndarray, v: np.ndarray, scale: float):
    """One query token: q [Hq][D], k and v [n][Hkv][D] fp64 -> o [Hq][D], lse [Hq], and
    sum_p w_p |v_p| [Hq][D] (what roundings of weights and values are relative to)."""
    Hq, D = q.shape
    n, Hkv = k.shape[0], k.shape[1]
    o, ab, lse = np.zeros((Hq, D)), np.zeros((Hq, D)), np.full(Hq, -np.inf)
    if n == 0:
        return o, lse, ab
    for h in range(Hq):
        kv = h // (Hq // Hkv)
        s = scale * (k[:, kv] @ q[h])
        m = s.max()
        e = np.exp(s - m)
        lse[h] = m + np.log(e.sum())
        w = e / e.sum()
        o[h], ab[h] = w @ v[:, kv], w @ np.abs(v[:, kv])
    return o, lse, ab


def score_bound(q: np.ndarray, k_abs_scale: np.ndarray, scale: float) -> float:
    """Largest error of an fp32 score: per group of 32 dims 65 additions of partial sums up to
    55 sum|q|, times the largest key scale; then the sum over groups and two products."""
    aq = np.abs(q).reshape(q.shape[0], -1, 32).sum(2)                   # [Hq][ng]
    return float(2.0 ** -23 * (65 * 55 + 8 * (aq.shape[1] + 8)) * abs(scale) * np.max(aq @ k_abs_scale))


# ---- limits that a loss of precision does not pass.  linear_q4_bound and score_bound hold for
# any data; for data of random signs the roundings are independent, and their root mean
# square over many results is far smaller.

def linear_q4_rms(x: np.ndarray, codes: np.ndarray, scales: np.ndarray, offset: bool) -> np.ndarray:
    """Root mean square error [B][n] of fp32 sums, for x of random signs.  A group of G columns
    takes at most 2 G additions, each off by at most 2^-23 of a partial sum of the size
    |q x| (2-norm over the group), or 31 |x| where the codes' offset is summed too; then one
    multiply-add per group and 16 additions of the size of the result."""
    q = unpack_rows(codes).astype(np.float64)
    n, d = q.shape
    ng = scales.shape[1]
    G, s2 = d // ng, scales.astype(np.float64) ** 2                    # [n][ng]
    x2 = (x ** 2).reshape(x.shape[0], ng, G)
    r2 = np.einsum("bgc,igc->big", x2, (q ** 2).reshape(n, ng, G))      # |q x|^2 [B][n][ng]
    p2 = np.broadcast_to((31.0 ** 2 * x2.sum(2))[:, None], r2.shape) if offset else r2
    return 2.0 ** -23 * np.sqrt(2 * G * (s2 * p2).sum(2) + (ng + 16) * (s2 * r2).sum(2))


def attention_rms(q, k, v, scale, offset: bool, weight_steps, value_step, half_step):
    """o [Hq][D] and the root mean square error [Hq][D] of an evaluation that rounds each weight and
    each value within the given half steps (relative; uniform errors: half step / sqrt(3)) and the
    result within `half_step`, with fp32 scores summed as linear_q4_rms says (scale groups of 32)."""
    Hq, D = q.shape
    n, Hkv = k.shape[0], k.shape[1]
    o, rms = np.zeros((Hq, D)), np.zeros((Hq, D))
    for h in range(Hq):
        kv = h // (Hq // Hkv)
        s = scale * (k[:, kv] @ q[h])
        w = np.exp(s - s.max())
        w /= w.sum()
        o[h] = w @ v[:, kv]
        k32 = k[:, kv].reshape(n, -1, 32)
        top = np.abs(k32).max(2) / 7                                    # at least the scale, unless all codes are small
        q2 = (q[h] ** 2).reshape(-1, 32).sum(1)
        p2 = (top ** 2 * (31.0 ** 2 if offset else 8.0 ** 2) * q2).sum(1)
        ds = 2.0 ** -23 * np.sqrt(64 * p2 + (q2.size + 8) * (s / scale) ** 2) * abs(scale) + 2.0 ** -23 * (np.abs(s) + 2 * np.abs(s).max())
        e2 = (w * w * (weight_steps ** 2 / 3 + value_step ** 2 / 3 + ds ** 2)) @ v[:, kv] ** 2
        rms[h] = np.sqrt(e2 + (half_step * o[h]) ** 2 / 3)
    return o, rms


def rms_ratio(err: np.ndarray, rms: np.ndarray) -> float:
    """Root mean square of err / rms over the results that have an error at all."""
    on = rms > 0
    return float(np.sqrt(np.mean((err[on] / rms[on]) ** 2)))
