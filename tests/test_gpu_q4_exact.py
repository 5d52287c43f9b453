"""The int4 attention half where results are known closely: every position of a range counted once,
scores that are whole numbers, and the root mean square of the roundings on random data.  The
limits are those of test_q4_exact_host.py, which plants mistakes in them on the CPU."""
import numpy as np
import pytest
import torch

import q4_exact as E
from activation_sparse_ffn_amd import _abi as A
from gpu_helpers import say
from oracle import q4_oracle as Q

pytestmark = pytest.mark.gpu
DEV = "cuda"
DT = {"f16": torch.float16, "bf16": torch.bfloat16}
HALF = {"f16": 2.0 ** -11, "bf16": 2.0 ** -8}


def np64(t):
    return t.detach().cpu().to(torch.float64).numpy()


# ------------------------------------------------------------------------------ projection

@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("case", [(1, 300, 4096, 32), (1, 200, 7168, 128), (3, 257, 1056, 32), (6, 130, 2048, 64), (8, 64, 8192, 32),
                                  (12, 100, 4096, 128), (20, 64, 1088, 64), (32, 48, 4096, 32), (40, 40, 2048, 128), (64, 33, 1056, 32),
                                  (10, 4128, 544, 32), (24, 4128, 512, 64), (37, 4128, 512, 128), (64, 4128, 288, 32)],
                         ids=lambda c: "x".join(map(str, c)))
def test_linear_precision(case, dt):
    B, n, d, group = case
    say(f"linear precision {case} {dt}")
    g = torch.Generator().manual_seed(B + n + d)
    x = torch.randn(B, d, generator=g).to(DT[dt])
    W = torch.randint(0, 256, (n, d // 2), generator=g, dtype=torch.uint8)
    s = (0.05 * torch.rand(n, d // group, generator=g) + 1e-3).half()
    y = torch.empty(B, n, device=DEV)
    A.sfx_linear_q4(x.to(DEV), W.to(DEV), s.to(DEV), y)
    ref, rms = (f(np64(x), W.numpy(), s.numpy(), *a) for f, a in ((Q.linear_q4, ()), (Q.linear_q4_rms, (dt == "bf16",))))
    ratio = Q.rms_ratio(np64(y) - ref, rms)
    say("   error / limit %.2f" % ratio)
    assert ratio <= 1


# ------------------------------------------------------------------------------ attention

def fill(table, page, pages, lens, k, v, Hkv, D):
    """A cache that holds k, v [T][Hkv][D] at the positions of the sequences, NaN scales elsewhere."""
    cache = torch.full((pages, Hkv, page // 8, 9 * D), 0xFF, dtype=torch.uint8, device=DEV)
    seq = torch.from_numpy(np.concatenate([np.full(n, b) for b, n in enumerate(lens)]).astype(np.int32)).to(DEV)
    pos = torch.from_numpy(np.concatenate([np.arange(n) for n in lens]).astype(np.int32)).to(DEV)
    A.sfx_kv_append_q4(None, k.to(DEV), v.to(DEV), pos, table, cache, None, seq=seq)
    return cache


def tables(lens, page, seed):
    per = [-(-n // page) for n in lens]
    order = torch.randperm(sum(per) + 2, generator=torch.Generator().manual_seed(seed)).to(torch.int32)
    table = torch.full((len(lens), max(per)), -1, dtype=torch.int32)
    at = 0
    for b, k in enumerate(per):
        table[b, :k] = order[at:at + k]
        at += k
    return table.to(DEV), sum(per) + 2


COUNT = [  # Hq, Hkv, D, page, lens, dt
    (4, 4, 32, 8, [1, 31, 32, 33, 255, 256, 257, 700], "f16"), (8, 2, 64, 16, [64, 513, 2047, 2049], "bf16"),
    (3, 3, 96, 32, [95, 1000], "f16"), (8, 8, 128, 32, [3000, 17], "bf16"), (32, 32, 128, 16, [1500, 2048], "f16"),
    (17, 1, 64, 8, [5000, 4097], "f16"), (5, 5, 160, 128, [700], "bf16"), (2, 1, 192, 1024, [1500, 1025], "bf16"),
    (6, 2, 224, 8, [260], "f16"), (4, 1, 256, 64, [8191], "f16"), (64, 8, 64, 32, [9000], "f16"),
    (16, 8, 128, 64, [50000], "bf16")]


@pytest.mark.parametrize("case", COUNT, ids=lambda c: "-".join(map(str, c)))
def test_attention_counts_every_position_once(case):
    """Equal scores and values that name their position's dim: the result is a count, wherever tiles,
    pages, runs and the ends of the range lie."""
    Hq, Hkv, D, page, lens, dt = case
    say(f"counting {case}")
    B = len(lens)
    table, pages = tables(lens, page, D)
    pos = np.concatenate([np.arange(n) for n in lens])
    v = torch.from_numpy(E.counting_values(len(pos), Hkv, D, pos))
    k = torch.randn(v.shape, generator=torch.Generator().manual_seed(D)).half()
    cache = fill(table, page, pages, lens, k, v, Hkv, D)
    q = torch.zeros(B, Hq, D, dtype=DT[dt], device=DEV)
    ws = A.workspace(A.sfx_attn_q4_ws(B, Hq, Hkv, D, table.shape[1] * page))
    out, lse = torch.empty(B, Hq, D, dtype=DT[dt], device=DEV), torch.empty(B, Hq, device=DEV)
    for lo, cut in ((lambda n: 0, 0), (lambda n: 1, 0), (lambda n: n - 1, 0), (lambda n: n // 2, 1), (lambda n: 31, 0),
                    (lambda n: 32, 7), (lambda n: n - 257, 0), (lambda n: n // 3 // 32 * 32 + 5, 33)):
        starts, ends = [max(0, lo(n)) for n in lens], [max(0, n - cut) for n in lens]
        A.sfx_attn_q4(q, cache, table, torch.tensor(ends, dtype=torch.int32, device=DEV), out, ws, lse=lse,
                      starts=torch.tensor(starts, dtype=torch.int32, device=DEV))
        for b in range(B):
            want, ls = E.counting_result(starts[b], ends[b], Hq, Hkv, D)
            got, got_l = np64(out[b]), np64(lse[b])
            assert (np.abs(got - want) <= (HALF[dt] + E.COUNTING_REL) * want).all(), (starts[b], ends[b])
            if np.isneginf(ls):
                assert np.isneginf(got_l).all()
            else:
                assert (np.abs(got_l - ls) <= E.COUNTING_LSE).all(), (starts[b], ends[b])


@pytest.mark.parametrize("case", [(32, 2, 1, 8, 450), (64, 4, 2, 16, 450), (128, 8, 1, 32, 700), (160, 2, 2, 16, 300), (256, 17, 1, 64, 330)],
                         ids=lambda c: "-".join(map(str, c)))
@pytest.mark.parametrize("dt", ["f16", "bf16"])
def test_attention_of_whole_scores(case, dt):
    """Scores of whole numbers in every order: the running reference goes up with each tile, once, late or
    never, and what it leaves behind is scaled down exactly."""
    D, Hq, Hkv, page, n = case
    rng = np.random.default_rng(D)
    patterns = E.score_patterns(n, rng)
    table, pages = tables([n] * len(patterns), page, D)
    k = np.stack([np.stack([E.digit_keys(s, D, rng) for _ in range(Hkv)], 1) for s in patterns.values()])
    v = E.whole_values(n * len(patterns), Hkv, D, rng).reshape(len(patterns), n, Hkv, D)
    cache = fill(table, page, pages, [n] * len(patterns), torch.from_numpy(k.reshape(-1, Hkv, D)),
                 torch.from_numpy(v.reshape(-1, Hkv, D)), Hkv, D)
    B = len(patterns)
    q = torch.from_numpy(np.broadcast_to(E.digit_query(D), (B, Hq, D)).copy()).to(DT[dt]).to(DEV)
    ws = A.workspace(A.sfx_attn_q4_ws(B, Hq, Hkv, D, table.shape[1] * page))
    out, lse = torch.empty(B, Hq, D, dtype=DT[dt], device=DEV), torch.empty(B, Hq, device=DEV)
    for scale in (float(np.float32(np.log(2.0))), float(np.float32(0.3)), float(np.float32(-0.3))):
        say(f"whole scores {case} {dt} {scale}")
        A.sfx_attn_q4(q, cache, table, torch.full((B,), n, dtype=torch.int32, device=DEV), out, ws, scale=scale, lse=lse)
        for b, (name, s) in enumerate(patterns.items()):
            o, ls, ab = Q.attention(np64(q[b]), k[b].astype(np.float64), v[b].astype(np.float64), scale)
            tol = E.exact_scores_tolerance(o, ab, 112, n, scale, dt == "f16", HALF[dt])
            err = np.abs(np64(out[b]) - o)
            assert (err <= tol).all(), (name, (err / tol).max())
            # score errors as in the tolerance; log2 and two roundings of numbers up to 128
            assert (np.abs(np64(lse[b]) - ls) <= 2.0 ** -24 * 4 * (112 * abs(scale) + 16) + 2.0 ** -16).all(), name


@pytest.mark.parametrize("D", [32, 64, 128, 256])
def test_attention_keeps_weights_to_two_terms(D):
    """fp16 results of weights that one fp16 term does not hold."""
    Hq, Hkv, page, n, B = 16, 2, 16, 48, 4
    rng = np.random.default_rng(D + 1)
    table, pages = tables([n] * B, page, D)
    k = np.stack([np.stack([E.digit_keys(rng.integers(-8, 9, n), D, rng) for _ in range(Hkv)], 1) for _ in range(B)])
    v = E.whole_values(n * B, Hkv, D, rng).reshape(B, n, Hkv, D)
    cache = fill(table, page, pages, [n] * B, torch.from_numpy(k.reshape(-1, Hkv, D)), torch.from_numpy(v.reshape(-1, Hkv, D)), Hkv, D)
    q = torch.from_numpy(np.broadcast_to(E.digit_query(D), (B, Hq, D)).copy()).half().to(DEV)
    out = torch.empty(B, Hq, D, dtype=torch.float16, device=DEV)
    scale = float(np.float32(0.3))
    say(f"two terms {D}")
    A.sfx_attn_q4(q, cache, table, torch.full((B,), n, dtype=torch.int32, device=DEV), out,
                  A.workspace(A.sfx_attn_q4_ws(B, Hq, Hkv, D, table.shape[1] * page)), scale=scale)
    for b in range(B):
        o, _, ab = Q.attention(np64(q[b]), k[b].astype(np.float64), v[b].astype(np.float64), scale)
        err, tol = np.abs(np64(out[b]) - o), E.exact_scores_tolerance(o, ab, 8, n, scale, True, HALF["f16"])
        assert (err <= tol).all(), (err / tol).max()


@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("case", [(8, 2, 64, 16, [300, 70]), (16, 4, 128, 32, [1000]), (4, 4, 32, 8, [40, 500]), (20, 1, 96, 64, [400]),
                                  (6, 2, 256, 16, [333]), (8, 8, 160, 8, [129])], ids=lambda c: "-".join(map(str, c)))
def test_attention_precision(case, dt):
    """Random data: the root mean square of the error against that of the documented roundings."""
    Hq, Hkv, D, page, lens = case
    B = len(lens)
    g = torch.Generator().manual_seed(D)
    k, v = (torch.randn(sum(lens), Hkv, D, generator=g) for _ in range(2))
    q = torch.randn(B, Hq, D, generator=g).to(DT[dt])
    table, pages = tables(lens, page, D)
    cache = fill(table, page, pages, lens, k, v, Hkv, D)
    kn, vn = Q.values(*Q.quantise(k.numpy(), 65504.0)), Q.values(*Q.quantise(v.numpy(), 8188.0))
    out = torch.empty(B, Hq, D, dtype=DT[dt], device=DEV)
    A.sfx_attn_q4(q.to(DEV), cache, table, torch.tensor(lens, dtype=torch.int32, device=DEV), out,
                  A.workspace(A.sfx_attn_q4_ws(B, Hq, Hkv, D, table.shape[1] * page)))
    at = np.concatenate([[0], np.cumsum(lens)])
    errs, limits = [], []
    for b in range(B):
        o, rms = Q.attention_rms(np64(q[b]), kn[at[b]:at[b + 1]], vn[at[b]:at[b + 1]], D ** -0.5, dt == "bf16",
                                 2.0 ** -22 if dt == "f16" else 2.0 ** -11, 2.0 ** -11, HALF[dt])
        errs.append(np64(out[b]) - o)
        limits.append(rms)
    ratio = Q.rms_ratio(np.concatenate(errs), np.concatenate(limits))
    say(f"attention precision {case} {dt}: error / limit {ratio:.2f}")
    assert ratio <= 1
