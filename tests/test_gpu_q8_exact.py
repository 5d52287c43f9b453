"""The int8 attention where results are known closely: every position of a range counted once, scores that are
whole numbers, and the root mean square of the roundings on random data; steps that give what a prompt gives.  The
limits are those of test_q8_exact_host.py, which plants mistakes in them on the CPU."""
import numpy as np
import pytest
import torch

import q8_exact as E
from activation_sparse_ffn_amd import _abi as A
from gpu_helpers import say
from oracle import q4_oracle as Q4
from test_gpu_q8 import DEV, DT, HALF_STEP, logical, make_table, np64, rope_table

pytestmark = pytest.mark.gpu


def i32(a):
    return torch.from_numpy(np.asarray(a, np.int32)).to(DEV)


def fill(table, page, pages, lens, k, v, Hkv, D):
    """A cache that holds k, v [T][Hkv][D] at the positions of the sequences, NaN scales elsewhere."""
    cache = torch.full((pages, Hkv, page // 16, 32 * D + 16), 0xFF, dtype=torch.uint8, device=DEV)
    q_start = np.concatenate([[0], np.cumsum(lens)])
    A.sfx_kv_append_q8(None, torch.from_numpy(k).to(DEV), torch.from_numpy(v).to(DEV), i32(lens), table, cache, None, q_start=i32(q_start))
    return cache


class Call:
    """Attention of the last `counts` rows of sequences of `lens` positions."""

    def __init__(self, Hq, Hkv, D, page, lens, counts, dt, k, v, seed):
        self.Hq, self.lens, self.counts = Hq, np.asarray(lens), np.asarray(counts)
        table, pages = make_table(lens, page, seed)
        self.table = table
        self.d_table = table.to(DEV)
        self.cache = fill(self.d_table, page, pages, lens, k, v, Hkv, D)
        self.q_start = np.concatenate([[0], np.cumsum(counts)])
        self.T, self.most = int(self.q_start[-1]), int(max(counts))
        self.ws = A.workspace(A.sfx_attn_q8_ws(len(lens), self.most, Hq, Hkv, D, table.shape[1] * page))
        self.seq = np.repeat(np.arange(len(lens)), counts)
        self.pos = np.concatenate([np.arange(n - m, n) for n, m in zip(lens, counts)])
        self.dt = DT[dt]

    def __call__(self, q, window=0, starts=None, scale=None):
        """out, lse (fp64) and each row's first position and end."""
        out = torch.full(q.shape, 7.0, dtype=self.dt, device=DEV)
        lse = torch.full(q.shape[:2], 7.0, device=DEV)
        A.sfx_attn_q8(q, self.cache, self.d_table, i32(self.lens), out, self.ws, q_start=i32(self.q_start), max_q=self.most, window=window,
                      starts=None if starts is None else i32(starts), scale=scale, lse=lse)
        lo = np.maximum(0, self.pos + 1 - window) if window else np.zeros(self.T, np.int64)
        if starts is not None:
            lo = np.maximum(lo, np.asarray(starts)[self.seq])
        return np64(out), np64(lse), lo, self.pos + 1


COUNT = [  # Hq, Hkv, D, page, lens, rows of each, dtype
    (4, 4, 32, 16, [1, 31, 32, 33, 255, 256, 257, 700], [1] * 8, "f16"), (8, 2, 64, 16, [64, 513, 2047, 2049], [1] * 4, "bf16"),
    (17, 1, 64, 64, [5000, 4097], [1, 1], "f16"), (64, 8, 128, 64, [20000], [1], "bf16"), (2, 1, 192, 1024, [1500, 1025], [1, 1], "bf16"),
    (4, 1, 256, 64, [8191], [1], "f16"), (32, 4, 64, 32, [9000, 3000], [3, 2], "bf16"), (6, 2, 96, 16, [1000, 70, 33], [5, 30, 1], "f16"),
    (16, 1, 128, 16, [3000], [6], "f16"), (3, 3, 160, 128, [700, 90], [32, 20], "bf16"),
    (8, 8, 128, 32, [1500, 17, 300], [1500, 17, 200], "f16"), (16, 4, 64, 16, [900, 130], [900, 33], "bf16"), (2, 2, 32, 64, [3000], [2000], "f16"),
    (4, 2, 96, 16, [1111], [777], "bf16"), (2, 1, 256, 32, [800], [513], "f16"), (2, 2, 224, 16, [400, 129], [300, 129], "bf16"),
    (1, 1, 128, 64, [20000], [150], "bf16"), (4, 1, 64, 1024, [9000], [40], "f16")]


@pytest.mark.parametrize("case", COUNT, ids=lambda c: "-".join(map(str, c)))
def test_attention_counts_every_position_once(case):
    """Equal scores and values that name their position's dim: the result is a count, wherever tiles,
    pages, runs, windows and the ends of the rows' ranges lie."""
    Hq, Hkv, D, page, lens, counts, dt = case
    say(f"counting {case}")
    pos = np.concatenate([np.arange(n) for n in lens])
    v = E.counting_values(len(pos), Hkv, D, pos)
    k = np.random.default_rng(D).standard_normal(v.shape).astype(np.float32)
    call = Call(Hq, Hkv, D, page, lens, counts, dt, k, v, D)
    q = torch.zeros(call.T, Hq, D, dtype=DT[dt], device=DEV)
    ends = call.lens
    for window, starts in ((0, None), (1, None), (0, ends - 1), (33, None), (257, ends // 2), (0, np.minimum(31, ends - 1)),
                           (0, np.minimum(32, ends - 1)), (1000, None), (0, ends // 3 // 32 * 32 + 5), (64, ends + 3)):
        got, lse, lo, hi = call(q, window, starts)
        want, ls = E.counting_results(lo, hi, Hq, Hkv, D)
        bad = np.abs(got - want) > (HALF_STEP[dt] + E.COUNTING_REL) * want
        assert not bad.any(), (window, np.argwhere(bad)[:3].tolist())
        none = np.isneginf(ls)
        assert np.isneginf(lse[none]).all()
        assert (np.abs(lse[~none] - ls[~none, None]) <= E.COUNTING_LSE).all(), window


WHOLE = [(32, 2, 1, 16, 450, 1), (64, 40, 2, 16, 450, 1), (128, 8, 1, 32, 700, 1), (256, 17, 1, 64, 330, 1), (64, 8, 2, 16, 450, 20),
         (160, 4, 2, 16, 300, 9), (32, 2, 2, 16, 450, 450), (64, 1, 1, 32, 450, 430), (128, 4, 2, 16, 450, 200), (256, 2, 1, 64, 330, 330),
         (96, 1, 1, 16, 700, 300)]


@pytest.mark.parametrize("case", WHOLE, ids=lambda c: "-".join(map(str, c)))
@pytest.mark.parametrize("dt", ["f16", "bf16"])
def test_attention_of_whole_scores(case, dt):
    """Scores of whole numbers in every order: the running reference goes up with each tile, once, late or
    never, and what it leaves behind is scaled down exactly."""
    D, Hq, Hkv, page, n, rows = case
    rng = np.random.default_rng(D)
    patterns = E.score_patterns(n, rng)
    B = len(patterns)
    k = np.concatenate([np.stack([E.whole_keys(s, D, rng) for _ in range(Hkv)], 1) for s in patterns.values()])
    v = E.whole_values(n * B, Hkv, D, rng)
    call = Call(Hq, Hkv, D, page, [n] * B, [rows] * B, dt, k, v, D)
    q = torch.from_numpy(np.broadcast_to(E.whole_query(D), (call.T, Hq, D)).copy()).to(DT[dt]).to(DEV)
    values = v.reshape(B, n, Hkv, D).astype(np.float64)
    for scale in (float(np.float32(np.log(2.0))), float(np.float32(0.3)), float(np.float32(-0.3))):
        say(f"whole scores {case} {dt} {scale}")
        for window in (0, 100):
            got, lse, lo, hi = call(q, window, scale=scale)
            for b, (name, s) in enumerate(patterns.items()):
                at = slice(b * rows, (b + 1) * rows)
                for h in range(Hkv):
                    hs = slice(h * (Hq // Hkv), (h + 1) * (Hq // Hkv))
                    o, ab, ls = E.causal(s, values[b, :, h], scale, lo[at], hi[at])
                    err = np.abs(got[at, hs] - o[:, None])
                    tol = E.whole_tolerance(o, ab, 112, n, scale, HALF_STEP[dt])[:, None]
                    assert (err <= tol).all(), (name, window, (err / tol).max())
                    # score errors as in the tolerance; log2 and two roundings of numbers up to 128
                    assert (np.abs(lse[at, hs] - ls[:, None]) <= 2.0 ** -24 * 4 * (112 * abs(scale) + 16) + 2.0 ** -16).all(), name


@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("case", [(8, 2, 64, 16, [300, 70], [1, 1]), (16, 4, 128, 32, [1000], [1]), (20, 1, 96, 64, [400], [2]), (6, 2, 256, 16, [333], [3]),
                                  (8, 8, 160, 16, [129], [20]), (4, 1, 128, 16, [500], [60]), (2, 2, 32, 32, [700], [130]), (8, 8, 64, 16, [300, 200], [200, 3])],
                         ids=lambda c: "-".join(map(str, c)))
def test_attention_precision(case, dt):
    """Random data: the root mean square of the error against that of the documented roundings."""
    Hq, Hkv, D, page, lens, counts = case
    rng = np.random.default_rng(D)
    k, v = (rng.standard_normal((sum(lens), Hkv, D)).astype(np.float32) for _ in range(2))
    call = Call(Hq, Hkv, D, page, lens, counts, dt, k, v, D)
    q = torch.from_numpy(rng.standard_normal((call.T, Hq, D))).to(DT[dt])
    got, _, lo, hi = call(q.to(DEV))
    errs, limits = [], []
    for b, n in enumerate(lens):
        kn, vn, has = logical(call.cache.cpu(), call.table.numpy(), page, b, n, D)
        assert has.all()
        for t in range(call.q_start[b], call.q_start[b + 1]):
            o, rms = E.attention_rms(np64(q[t]), kn[:hi[t]], vn[:hi[t]], D ** -0.5, HALF_STEP[dt])
            errs.append(got[t] - o)
            limits.append(rms)
    ratio = Q4.rms_ratio(np.stack(errs), np.stack(limits))
    say(f"attention precision {case} {dt}: error / limit {ratio:.2f}")
    assert ratio <= 1


@pytest.mark.parametrize("case", [(4, 2, 64, "f16", 0), (8, 1, 128, "bf16", 0), (4, 4, 32, "f16", 17)], ids=lambda c: "-".join(map(str, c)))
def test_steps_give_what_a_prompt_gives(case):
    """The same tokens as one prompt, as two chunks and one by one: the outputs agree row by row.  Projections have
    the same bits (a token's row does not depend on the others); a stored number is off by a uniform error of
    a step, 3.5 sigma / 127 where the block's largest is 3.5 sigma: 0.008 sigma each time its block's scale grows, about
    0.016 after a few; that much of V, and of K as a change of the weights, and 0.008 of the attention's rows, on
    either side: 0.035 of a row's length, 0.1 at most.  Rows of other tokens and a chunk without its prefix
    are further off."""
    from activation_sparse_ffn_amd import AttnStep8, rows_q8
    Hq, Hkv, D, dt, window = case
    d, page, n, cut = 256, 16, 50, 21
    say(f"prompt, chunks, steps {case}")
    g = torch.Generator().manual_seed(3)
    w = {"wn": (1 + 0.2 * torch.randn(d, generator=g)).to(DEV), "bqkv": None, "bo": None}
    w["Wqkv"], w["Wqkv_s"] = rows_q8((torch.randn((Hq + 2 * Hkv) * D, d, generator=g) * d ** -0.5).to(DEV))
    w["Wo"], w["Wo_s"] = rows_q8((torch.randn(d, Hq * D, generator=g) * (Hq * D) ** -0.5).to(DEV))
    x = torch.randn(n, d, generator=g).to(DEV)
    table, pages = make_table([n], page, 2)
    cs = torch.from_numpy(rope_table(64, D)).to(DEV)
    outs = []
    for way in ("prompt", "chunks", "steps", "no prefix"):
        pos = torch.zeros(1, dtype=torch.int32, device=DEV)
        s = AttnStep8(d, Hq, Hkv, D, 1, dt, table.to(DEV), pos, pages, page=page, cos_sin=cs, max_tokens=n, window=window)
        y = torch.zeros(n, d, device=DEV)
        if way == "prompt":
            s.prompt(w, x, y, i32([0, n]), i32([n]), n)
        elif way == "steps":
            for t in range(n):
                pos.fill_(t)
                s.run(w, x[t:t + 1], y[t:t + 1])
        else:
            s.prompt(w, x[:cut], y[:cut], i32([0, cut]), i32([cut]), cut)
            s.prompt(w, x[cut:], y[cut:], i32([0, n - cut]), i32([n if way == "chunks" else n - cut]), n - cut)
        outs.append(np64(y))
    prompt, chunks, steps, short = outs
    apart = lambda a, b: np.linalg.norm(a - b, axis=1) / np.linalg.norm(b, axis=1)  # noqa: E731
    say("   chunks %.3f, steps %.3f" % (apart(chunks, prompt).max(), apart(steps, prompt).max()))
    assert apart(chunks, prompt).max() < 0.1 and apart(steps, prompt).max() < 0.1
    # rows whose window holds five or more tokens of the first chunk (one of 17 weighs about 1 / 17)
    reach = n if not window else cut + window - 5
    assert apart(short, prompt)[cut:reach].min() > 0.1
    assert apart(np.roll(prompt, 1, 0), prompt).min() > 0.1
