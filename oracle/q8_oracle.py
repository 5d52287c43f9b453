"""Plain fp64 forms of the 8-bit layer half (numpy, test infrastructure): residual norm to int8
rows, the int8 projection, the int8 cache's blocks as calls change them, and causal attention over
a list of positions."""
import numpy as np

BLK = 16


def norm_rows(x, res, weight, eps, norm):
    """h and n, fp64 [T][d]."""
    h = x if res is None else x + res
    if not norm:
        return h, h
    with np.errstate(all="ignore"):
        n = h / np.sqrt((h * h).mean(1, keepdims=True) + eps)
        return h, n if weight is None else n * weight.astype(np.float64)


def row_codes(n):
    """fp32 scales [T] and codes [T][d] of fp64 rows."""
    with np.errstate(all="ignore"):
        s = (np.abs(n).max(1) / 127.0).astype(np.float32)
        bad = ~np.isfinite(n).all(1)
        d = np.where(s > 0, s, 1).astype(np.float64)[:, None]
        q = np.where((s > 0)[:, None], np.clip(np.rint(n / d), -127, 127), 0)
    return np.where(bad, np.float32(np.nan), s), np.where(bad[:, None], 0, q).astype(np.int64)


def linear(x, sx, w, sw, bias=None):
    """int codes -> the exact sums [T][n] (int64) and y fp64."""
    p = x.astype(np.int64) @ w.astype(np.int64).T
    y = p * sx.astype(np.float64)[:, None] * sw.astype(np.float64)
    return p, y if bias is None else y + bias.astype(np.float64)


# ---- cache: blocks uint8 [32 D + 16]

def read_block(block, D):
    """Codes K, V [16][D] and scales, one byte at a time."""
    k, v = np.zeros((BLK, D), np.int64), np.zeros((BLK, D), np.int64)
    for i in range(BLK):
        for d in range(D):
            k[i, d] = int(block[i * D + d]) - 128
            v[i, d] = int(block[16 * D + ((i // 4) * D + d) * 4 + i % 4]) - 128
    s = block[32 * D:32 * D + 8].copy().view(np.float32)
    return k, v, s[0], s[1]


def write_block(block, D, k, v, ks, vs):
    block[:16 * D] = (k + 128).astype(np.uint8).reshape(-1)
    block[16 * D:32 * D] = (v + 128).astype(np.uint8).reshape(4, 4, D).transpose(0, 2, 1).reshape(-1)
    block[32 * D:32 * D + 8] = np.array([ks, vs], np.float32).view(np.uint8)


def store_rows(q, s, rows, i0):
    """Codes [16][D] and scale of one half of a block after rows (fp32 [n][D]) are stored at
    positions i0 ..: the definition, step by step."""
    n = len(rows)
    new = np.zeros(BLK, bool)
    new[i0:i0 + n] = True
    old = np.float32(0) if i0 == 0 else s
    with np.errstate(all="ignore"):
        m = np.abs(rows).max()
        if not np.isfinite(rows).all() or np.isnan(old):
            t = np.float32(np.nan)
        else:
            t = max(old, np.float32(m.astype(np.float64) / 127.0))
    out = q.copy()
    if i0 == 0:
        out[~new] = 0
    elif not t == old:
        out[~new] = np.rint(q[~new].astype(np.float64) * np.float64(old) / np.float64(t)) if t > 0 else 0
    out[new] = np.clip(np.rint(rows.astype(np.float64) / np.float64(t)), -127, 127) if t > 0 else 0
    return out, t


def pages_of(table, page, num_pages, b, p):
    """Page id of position p, or -1."""
    j = p // page
    if p < 0 or j >= table.shape[1]:
        return -1
    i = int(table[b, j])
    return i if 0 <= i < num_pages else -1


def append(cache, table, page, k, v, q_start, lens, max_pos):
    """Stores rotated fp32 k and v [T][Hkv][D] in `cache` (changed): what the calls do, block by
    block.  Returns which rows have been stored [T]."""
    P, H, O, size = cache.shape
    D = (size - 16) // 32
    stored = np.zeros(len(k), bool)
    for b in range(table.shape[0]):
        first, n = int(q_start[b]), int(q_start[b + 1] - q_start[b])
        at = {}
        for i in range(n):
            p = int(lens[b]) - n + i
            if p < 0 or (max_pos and p >= max_pos) or pages_of(table, page, P, b, p) < 0:
                continue
            at.setdefault(p // BLK, []).append((p % BLK, first + i))
            stored[first + i] = True
        for blk, rows in at.items():
            i0, t = rows[0][0], [r for _, r in rows]
            pg = pages_of(table, page, P, b, blk * BLK)
            for h in range(H):
                raw = cache[pg, h, (blk * BLK % page) // BLK]
                kq, vq, ks, vs = read_block(raw, D)
                kq, ks = store_rows(kq, ks, k[t, h], i0)
                vq, vs = store_rows(vq, vs, v[t, h], i0)
                write_block(raw, D, kq, vq, ks, vs)
    return stored


def attention(q, k, v, scale):
    """Query rows of one token and kv head q [G][D] over positions k, v [n][D] (fp64): o, lse,
    sum_p w_p |v_p| [G][D] and scale max_p sum_d |q_d k_pd| [G]."""
    G, D = q.shape
    if len(k) == 0:
        return np.zeros((G, D)), np.full(G, -np.inf), np.zeros((G, D)), np.zeros(G)
    s = scale * (q @ k.T)
    m = s.max(1, keepdims=True)
    e = np.exp(s - m)
    w = e / e.sum(1, keepdims=True)
    return w @ v, (m[:, 0] + np.log(e.sum(1))), w @ np.abs(v), abs(scale) * (np.abs(q) @ np.abs(k).T).max(1)


def attention_tolerance(o, lse, ab, size, v_top, n, D, half_step):
    """Largest error of o [G][D] and lse [G].  A score is a sum of D exact products in fp32, each
    addition off by at most 2^-23 of partial sums up to `size` (with scale); with it come products and
    sums in powers of two up to 2 size / ln 2 + 160 (references, scales' logarithms): three roundings of
    2^-24 and logarithms good to 2^-22 of theirs.  A weight takes an exponential (2^-21) and a rounding to
    fp16 (2^-11), or falls below fp16's last bit (2^-25 of at least 2^9 times the largest
    contribution v_top; n of them); fp32 sums over up to 32 + log2(n) levels."""
    ds = D * 2.0 ** -23 * size + (2 * size / np.log(2) + 160) * 2.0 ** -22
    rel = 2.0 ** -11 + 2 * ds + 2.0 ** -17
    return half_step * np.abs(o) * 1.01 + rel[:, None] * ab * 1.01 + n * 2.0 ** -34 * v_top, ds + 2.0 ** -17 + 2.0 ** -22 * np.abs(lse)
