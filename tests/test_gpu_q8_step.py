"""The 8-bit layer half as it is used: prompts and decode steps through AttnStep8, each stage held
against the fp64 oracle on what the stage before it left; blocks with the sparse FFN; captured steps."""
import numpy as np
import pytest
import torch

from activation_sparse_ffn_amd import _abi as A
from gpu_helpers import say
from oracle import q4_oracle as Q4
from oracle import q8_oracle as Q
from test_gpu_q8 import (DEV, DT, HALF_STEP, TINY, check_norm, linear_tol, logical, make_table, np64, positions, rope_table,
                         sums_of, within)

pytestmark = pytest.mark.gpu


def i32(a):
    return torch.from_numpy(np.asarray(a, np.int32)).to(DEV)


def make_layer(d, Hq, Hkv, D, seed, bias=True, norm=True):
    from activation_sparse_ffn_amd import rows_q8
    g = torch.Generator().manual_seed(seed)
    n = (Hq + 2 * Hkv) * D
    out = {}
    out["Wqkv"], out["Wqkv_s"] = rows_q8((torch.randn(n, d, generator=g) * d ** -0.5).to(DEV))
    out["Wo"], out["Wo_s"] = rows_q8((torch.randn(d, Hq * D, generator=g) * (Hq * D) ** -0.5).to(DEV).half())
    out["bqkv"], out["bo"] = (torch.randn(m, generator=g).to(DEV) * 0.3 if bias else None for m in (n, d))
    out["wn"] = (1 + 0.2 * torch.randn(d, generator=g)).to(DEV) if norm else None
    return out


def check_linear(x, sx, W, sw, bias, y, rows, y0=None):
    x, sx, W, sw = (t.cpu() for t in (x, sx, W, sw))
    p = sums_of(x[rows], W)
    ref = p * sx[rows].double().numpy()[:, None] * sw.double().numpy()
    size = np.abs(ref)
    for t in (None if bias is None else bias, None if y0 is None else y0[rows]):
        if t is not None:
            ref = ref + np64(t)
            size = size + np.abs(np64(t))
    assert (np.abs(np64(y)[rows] - ref) <= linear_tol(p, sx[rows], sw, size, "f32")).all()


def check_half(s, w, x, y, before, counts, lens, lead, dt, page, rope, window, y0=None, add=None, after=None):
    """Every stage of a call of AttnStep8 `s` on rows x that gave y: sequences of `counts` new rows
    behind `lead` others, with `lens` positions; before: the cache as it was; `after`: x
    once `add` has been added."""
    T, a, b = len(x), s.Hq * s.D, s.Hkv * s.D
    q_start = np.concatenate([[0], np.cumsum(counts)]) + lead
    cut = lambda t: t[:T]  # noqa: E731
    xt = {v: k for k, v in DT.items()}[x.dtype]
    norm = w["wn"] is not None
    rows, res, rt = (x, None, None) if add is None else (add, x, xt)
    check_norm((T, s.d, None, rt, None, norm, norm), rows, res, w["wn"].cpu() if norm else None, cut(s.xq), cut(s.xs), after, None)
    check_linear(cut(s.xq), cut(s.xs), w["Wqkv"], w["Wqkv_s"], w["bqkv"], cut(s.qkv), np.arange(T))
    qkv = cut(s.qkv).cpu().numpy()
    cs = None if s.cos_sin is None else s.cos_sin.cpu().numpy()
    seq, pos = positions(q_start, lens, T)
    at = np.clip(pos, 0, 0 if cs is None else len(cs) - 1)
    table = s.table.cpu().numpy()
    heads = lambda lo, h: qkv[:, lo:lo + h * s.D].reshape(T, h, s.D)  # noqa: E731
    kr, qr = Q4.rotate(heads(a, s.Hkv), at, cs, rope == "pairs"), Q4.rotate(heads(0, s.Hq), at, cs, rope == "pairs")
    want = before.numpy().copy()
    stored = Q.append(want, table, page, kr, heads(a + b, s.Hkv), q_start, lens, 0 if cs is None else len(cs))
    assert np.array_equal(s.cache.cpu().numpy(), want)
    assert torch.equal(s.q[:T].cpu()[stored], torch.from_numpy(qr).to(DT[dt])[stored])
    got, cache = np64(cut(s.o)), s.cache.cpu()
    mine = np.zeros(T, bool)
    for i, n in enumerate(lens):
        rows = np.arange(q_start[i], q_start[i + 1])
        mine[rows] = True
        if n <= 0:
            assert (got[rows] == 0).all()
            continue
        k, v, has = logical(cache, table, page, i, n, s.D)
        assert has.all()
        for t in rows:
            p = pos[t]
            lo = max(0, p + 1 - window) if window else 0
            for h in range(s.Hkv):
                hs = slice(h * (s.Hq // s.Hkv), (h + 1) * (s.Hq // s.Hkv))
                o, l, ab, size = Q.attention(np64(s.q[t, hs]), k[lo:p + 1, h], v[lo:p + 1, h], s.D ** -0.5)
                tol, _ = Q.attention_tolerance(o, l, ab, size, np.abs(v[lo:p + 1, h]).max(), p + 1 - lo, s.D, HALF_STEP[dt])
                # an output below fp16's normal numbers (2^-14) is rounded to a multiple of 2^-24: off by up to 2^-25,
                # which half a step relative to it does not hold (0 times one value plus e^-14 times another comes there)
                off = np.abs(got[t, hs] - o) / (tol + TINY[dt])
                assert off.max() <= 1, (i, t, h, off.max(), off.argmax())
    check_norm((T, a, dt, None, None, False, False), cut(s.o).reshape(T, a), None, None, cut(s.oq), cut(s.os), None, None)
    check_linear(cut(s.oq), cut(s.os), w["Wo"], w["Wo_s"], w["bo"], y, np.flatnonzero(mine), y0)


CASES = [  # d, Hq, Hkv, D, page, dtype, rope, window, x, bias and norm
    (256, 8, 2, 64, 16, "f16", "half", 0, "f32", True), (272, 4, 4, 32, 32, "bf16", "pairs", 20, "bf16", True),
    (512, 6, 1, 128, 16, "f16", "none", 0, "f16", False)]


@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(map(str, c)))
def test_prompts_then_steps(case):
    """Ragged prompts (one request without one, rows of none around them), a second chunk behind them, then
    decode steps over block and page ends with a request that pauses."""
    from activation_sparse_ffn_amd import AttnStep8
    d, Hq, Hkv, D, page, dt, rope, window, xt, rich = case
    say(f"8-bit half {case}")
    g = torch.Generator().manual_seed(d)
    B = 4
    table, pages = make_table([100, 100, 60, 100], page, 5)
    cs = torch.from_numpy(rope_table(128, D)).to(DEV) if rope != "none" else None
    pos = torch.full((B,), -1, dtype=torch.int32, device=DEV)
    s = AttnStep8(d, Hq, Hkv, D, B, dt, table.to(DEV), pos, pages, page=page, cos_sin=cs, interleaved=rope == "pairs",
                  window=window, max_tokens=70)
    s.cache.copy_(torch.randint(0, 256, s.cache.shape, generator=g, dtype=torch.uint8))
    w = make_layer(d, Hq, Hkv, D, 7, rich, rich)
    lens = np.zeros(B, np.int64)
    for counts, lead, tail in (([37, 1, 0, 13], 2, 3), ([16, 20, 5, 0], 0, 1)):
        lens = lens + counts
        q_start = np.concatenate([[0], np.cumsum(counts)]) + lead
        x = (torch.randn(int(q_start[-1]) + tail, d, generator=g) * 2).to(DT[xt])
        y = torch.zeros(len(x), d, device=DEV)
        before = s.cache.cpu()
        s.prompt(w, x.to(DEV), y, i32(q_start), i32(lens), max(counts))
        check_half(s, w, x, y, before, counts, lens, lead, dt, page, rope, window)
    for step in range(12):
        go = np.array([1, 1, 1, step % 3 != 1])
        lens = lens + go
        pos.copy_(i32(np.where(go == 1, lens - 1, -1)))
        x = (torch.randn(B, d, generator=g) * 2).to(DT[xt])
        y0 = torch.randn(B, d, generator=g)
        add = torch.randn(B, d, generator=g) if step % 2 else None
        xd, y = x.to(DEV), y0.to(DEV)
        before = s.cache.cpu()
        s.run(w, xd, y, accumulate=True, add=None if add is None else add.to(DEV))
        check_half(s, w, x, y, before, [1] * B, np.where(go == 1, lens, 0), 0, dt, page, rope, window, y0, add, xd)


def test_steps_follow_prompts():
    """The same tokens as one prompt, as two chunks and one by one: the caches agree within the steps of
    their codes."""
    from activation_sparse_ffn_amd import AttnStep8
    d, Hq, Hkv, D, page, n = 256, 4, 2, 64, 16, 50
    say("prompt, chunks, steps")
    g = torch.Generator().manual_seed(3)
    w = make_layer(d, Hq, Hkv, D, 1)
    x = torch.randn(n, d, generator=g).to(DEV)
    table, pages = make_table([n], page, 2)
    cs = torch.from_numpy(rope_table(64, D)).to(DEV)
    held, outs = [], []
    for way in (0, 1, 2):
        pos = torch.zeros(1, dtype=torch.int32, device=DEV)
        s = AttnStep8(d, Hq, Hkv, D, 1, "f16", table.to(DEV), pos, pages, page=page, cos_sin=cs, max_tokens=n)
        y = torch.zeros(n, d, device=DEV)
        if way == 0:
            s.prompt(w, x, y, i32([0, n]), i32([n]), n)
        elif way == 1:
            s.prompt(w, x[:21], y[:21], i32([0, 21]), i32([21]), 21)
            s.prompt(w, x[21:], y[21:], i32([0, n - 21]), i32([n]), n - 21)
        else:
            for t in range(n):
                pos.fill_(t)
                s.run(w, x[t:t + 1], y[t:t + 1])
        k, v, _ = logical(s.cache.cpu(), table.numpy(), page, 0, n, D)
        held.append((k, v))
        outs.append(np64(y))
    for k, v in held[1:]:
        for a, b in ((held[0][0], k), (held[0][1], v)):
            for j in range(0, n, 16):
                # at most 16 grown scales, each half a step of the last
                lim = 17 * 0.5 * np.abs(b[j:j + 16]).max(axis=(0, 2), keepdims=True) / 127 * 1.01
                assert (np.abs(a[j:j + 16] - b[j:j + 16]) <= lim).all()
    assert np.isfinite(np.stack(outs)).all()


def test_parallel_block_layer():
    """run_layer with the half: the FFN's y and the attention's, added."""
    import synthetic as S
    from activation_sparse_ffn_amd import AttnStep8, StepBuffers, run_layer
    cfg = S.scaled(S.CONFIGS["C4"], name="par", d=512, f=1056, h=128)
    B, Hq, Hkv, D, page = 2, 4, 2, 64, 16
    say("parallel block, 8-bit half")
    L = S.make_layer(cfg, 0, device=DEV)
    layer = {**L.tensors(), **make_layer(cfg.d, Hq, Hkv, D, 8, norm=False)}
    x = S.make_tokens(cfg, 0, 1, B, device=DEV)[0]
    table, pages = make_table([10, 10], page, 2)
    outs = []
    for both in (False, True):
        buf = StepBuffers(cfg.d, cfg.f, cfg.h, B, cfg.wdtype, cfg.pred_storage)
        attn = AttnStep8(cfg.d, Hq, Hkv, D, B, "f16", table.to(DEV), torch.zeros(B, dtype=torch.int32, device=DEV), pages, page=page)
        run_layer(buf, layer, x, L.threshold, cfg.act, attn=attn if both else None)
        outs.append(np64(buf.y))
    y = torch.empty(B, cfg.d, device=DEV)
    attn.run(layer, x, y)
    ffn, both = outs
    # the sum's rounding, and those of the half's own value before it is added
    assert (np.abs(both - (ffn + np64(y))) <= 2.0 ** -22 * (np.abs(both) + np.abs(np64(y)) + np.abs(ffn)) + 2.0 ** -22).all()
    assert np.abs(np64(y)).max() > 0


@pytest.mark.parametrize("cfg_name", ["C1", "C3"])
def test_sequential_blocks(cfg_name):
    """Two pre-norm blocks with the sparse FFN, fused as run_block has them and call by call."""
    import synthetic as S
    from activation_sparse_ffn_amd import AttnStep8, StepBuffers, run_block, run_layer
    cfg = S.scaled(S.CONFIGS[cfg_name], name="seq", d=512, f=1056, h=128)
    dt, ft = "bf16" if cfg.wdtype == "bf16" else "f16", "f16" if cfg.wdtype == "q4" else cfg.wdtype
    B, Hq, Hkv, D, page = 3, 8, 2, 64, 16
    say(f"sequential blocks {cfg_name}")
    g = torch.Generator().manual_seed(11)
    layers = [S.make_layer(cfg, i, device=DEV) for i in range(2)]
    ws = [{**L.tensors(), **make_layer(cfg.d, Hq, Hkv, D, 8 + i), "wf": (1 + 0.1 * torch.randn(cfg.d, generator=g)).to(DEV)}
          for i, L in enumerate(layers)]
    table, pages = make_table([10] * B, page, 2)
    pos = i32([0, 0, 0])
    make = lambda: [AttnStep8(cfg.d, Hq, Hkv, D, B, dt, table.to(DEV), pos, pages, page=page, ffn_dtype=ft) for _ in layers]  # noqa: E731
    one, two = make(), make()
    buf, buf2 = (StepBuffers(cfg.d, cfg.f, cfg.h, B, cfg.wdtype, cfg.pred_storage) for _ in range(2))
    for step in range(3):
        pos.copy_(i32([step, step, -1 if step == 1 else step]))
        x = torch.randn(B, cfg.d, generator=g)
        res = x.to(DEV)
        add = None
        for L, w, a in zip(layers, ws, one):
            run_block(buf, w, res, a, L.threshold, cfg.act, add=add)
            add = buf.y
        h, y = x.to(DEV), None
        for L, w, a in zip(layers, ws, two):
            a.run(w, h, h, accumulate=True, add=y)
            n = torch.empty(B, cfg.d, dtype=DT[ft], device=DEV)
            A.sfx_norm_q8(h, weight=w["wf"], y=n)
            _, want = Q.norm_rows(np64(h), None, w["wf"].cpu().numpy(), np.float64(np.float32(1e-5)), True)
            assert within(np64(n), want, ft, 2.0 ** -48 * np.abs(want)).all()
            run_layer(buf2, w, n, L.threshold, cfg.act)
            y = buf2.y
        assert torch.equal(res, h) and torch.equal(buf.y, y)
        assert (np64(y) != 0).any() and (np64(h) != np64(x)).any(1).all()


def test_graph_replays():
    """A captured decode step replayed over moving positions with eager work and a prompt of another object
    between; a second graph on the same workspace; the last call on another stream."""
    from activation_sparse_ffn_amd import AttnStep8
    d, Hq, Hkv, D, page, B = 256, 16, 2, 64, 16, 2
    say("8-bit half, captured")
    table, pages = make_table([1200, 1200], page, 1)
    w = make_layer(d, Hq, Hkv, D, 4)
    g = torch.Generator().manual_seed(9)
    steps = []
    first = torch.randn(1101, d, generator=g).to(DEV)
    y1 = torch.empty(1101, d, device=DEV)
    for _ in range(2):
        s = AttnStep8(d, Hq, Hkv, D, B, "f16", table.to(DEV), i32([699, 400]), pages, page=page, max_tokens=1101)
        s.cache.zero_()                                  # unused bytes and pages, compared below
        s.prompt(w, first, y1, i32([0, 700, 1101]), i32([700, 401]), 700)
        steps.append(s)
    graphed, eager = steps
    assert torch.equal(graphed.cache, eager.cache)
    x, y = torch.zeros(B, d, device=DEV), torch.zeros(B, d, device=DEV)
    # another shape on the same workspace
    n2 = 3
    need = A.sfx_attn_q8_ws(n2, 1, 8, 2, 64, table.shape[1] * page)
    graphed.ws = A.workspace(max(need, graphed.ws.numel()))
    q2 = torch.randn(n2, 8, D, generator=g).half().to(DEV)
    table2 = torch.cat([table, table[:1]]).to(DEV).contiguous()
    lens2 = i32([600, 1, 300])
    out2, ref2 = torch.zeros_like(q2), torch.zeros_like(q2)
    cache2 = graphed.cache.clone()
    A.sfx_attn_q8(q2, cache2, table2, lens2, ref2, A.workspace(need))
    for s in steps:
        s.run(w, x, y)
    torch.cuda.synchronize()
    ga, gb = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(ga):
        graphed.run(w, x, y)
    with torch.cuda.graph(gb):
        A.sfx_attn_q8(q2, cache2, table2, lens2, out2, graphed.ws)
    other = torch.cuda.Stream()
    for rep in range(5):
        say(f"graph replay {rep}")
        xn = torch.randn(B, d, generator=g)
        for s in steps:
            s.pos += 1
        x.copy_(xn.to(DEV))
        ga.replay()
        out2.zero_()
        gb.replay()
        ye = torch.empty(B, d, device=DEV)
        xe = xn.to(DEV)
        if rep == 4:
            torch.cuda.synchronize()
            eager.run(w, xe, ye, stream=other)
            other.synchronize()
        else:
            eager.run(w, xe, ye)
        torch.cuda.synchronize()
        assert torch.equal(y, ye) and torch.equal(out2, ref2) and torch.equal(graphed.cache, eager.cache), rep
        _ = torch.randn(1000, device=DEV).sum().item()


def test_refusals():
    from activation_sparse_ffn_amd import AttnStep8
    say("8-bit half, refusals")
    table, pages = make_table([40], 16, 1)
    w = make_layer(256, 4, 2, 64, 1)
    s = AttnStep8(256, 4, 2, 64, 1, "f16", table.to(DEV), i32([0]), pages, max_tokens=8)
    x, y = torch.zeros(9, 256, device=DEV), torch.zeros(9, 256, device=DEV)
    with pytest.raises(ValueError):
        s.prompt(w, x, y, i32([0, 9]), i32([9]), 8)
    with pytest.raises(ValueError):
        s.prompt(w, x[:8], y[:8], i32([0, 8]), i32([8]), 9)
    with pytest.raises(ValueError):
        s.run(w, x[:2], y[:2])
    with pytest.raises(ValueError):
        s.run(w, x[:1], y[:1, :128])
    with pytest.raises(ValueError):
        AttnStep8(256, 4, 2, 64, 2, "f16", table.to(DEV), i32([0, 0]), pages)
