"""The int4 attention half at the ends of its documented ranges: the largest token count, the
largest finite numbers, tokens that are not stored, streams of other devices."""
import numpy as np
import pytest
import torch

from activation_sparse_ffn_amd import _abi as A
from gpu_helpers import say
from oracle import q4_oracle as Q

pytestmark = pytest.mark.gpu
DEV = "cuda"
DT = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}


def np64(t):
    return t.detach().cpu().to(torch.float64).numpy()


def test_append_and_read_at_the_largest_token_count():
    """2^24 - 1 tokens, nearly all padding: the launch's last workgroups, with tokens in the
    first and the last 64 stored and read back and zeros for the others."""
    T, D, page = (1 << 24) - 1, 32, 8
    say(f"append and read {T} tokens")
    at = [0, 1, 7, 8, 62, 63, 64, 4096, T - 65, T - 64, T - 63, T - 9, T - 8, T - 2, T - 1]
    table = torch.tensor([[2, 0]], dtype=torch.int32, device=DEV)
    cache = torch.zeros(3, 1, 1, 9 * D, dtype=torch.uint8, device=DEV)
    pos = torch.full((T,), -1, dtype=torch.int32, device=DEV)
    seq = torch.zeros(T, dtype=torch.int32, device=DEV)
    rows = torch.randn(len(at), 1, D, generator=torch.Generator().manual_seed(4)).half()
    kv = torch.ones(T, 1, D, dtype=torch.float16, device=DEV)
    for i, t in enumerate(at):
        pos[t] = i
        kv[t] = rows[i].to(DEV)
    A.sfx_kv_append_q4(None, kv, kv, pos, table, cache, None, seq=seq)
    ko, vo = torch.full_like(kv, 9.0), torch.full_like(kv, 9.0)
    A.sfx_kv_read_q4(pos, table, cache, ko, vo, seq=seq)
    stored = pos >= 0
    for out, top in ((ko, 65504.0), (vo, 8188.0)):
        want = torch.from_numpy(Q.values(*Q.quantise(rows.float().numpy(), top))).to(torch.float16)
        assert torch.equal(out[stored].cpu(), want)
        assert not out[~stored].any()


BF16_MAX = 2.0 ** 127 * (2 - 2.0 ** -7)


@pytest.mark.parametrize("case", [(1, 100, 32), (3, 40, 64), (6, 33, 128), (13, 70, 64), (20, 100, 32), (40, 90, 128), (20, 4130, 64),
                                  (64, 4100, 32)], ids=lambda c: "x".join(map(str, c)))
def test_linear_takes_the_largest_bf16_numbers(case):
    """x of the largest finite size: y is finite (its true size is at most 384 * 2^-10 of x's) and
    within the bound of the fp32 sums."""
    B, n, group = case
    d = 384
    say(f"linear largest bf16 {case}")
    g = torch.Generator().manual_seed(n + B)
    sign = lambda *shape: 2.0 * torch.randint(0, 2, shape, generator=g) - 1  # noqa: E731
    x = (sign(B, d) * BF16_MAX).to(torch.bfloat16)
    x[0, ::3] = (0.25 * BF16_MAX * torch.rand(d // 3, generator=g)).to(torch.bfloat16)
    assert torch.isfinite(x).all()
    q = torch.randint(-1, 2, (n, d), generator=g)
    W = ((q[:, 0::2] & 15) | ((q[:, 1::2] & 15) << 4)).to(torch.uint8)
    s = torch.full((n, d // group), 2.0 ** -10).half()
    y = torch.empty(B, n, device=DEV)
    A.sfx_linear_q4(x.to(DEV), W.to(DEV), s.to(DEV), y)
    assert torch.isfinite(y).all()
    ref = Q.linear_q4(np64(x), W.numpy(), s.numpy())
    assert (np.abs(np64(y) - ref) <= Q.linear_q4_bound(np64(x), W.numpy(), s.numpy())).all()


@pytest.mark.parametrize("B", [2, 20])
def test_linear_keeps_small_bf16_numbers(B):
    """x near 2^-110: sums whose terms lie 2^12 lower still keep all but the last bits above
    fp32's subnormal step, 2^-149 * 2^12 per addition, scales of at most 1."""
    n, d, group = 90, 256, 64
    say(f"linear small bf16 {B}")
    g = torch.Generator().manual_seed(B)
    x = (torch.randn(B, d, generator=g) * 2.0 ** -110).to(torch.bfloat16)
    W = torch.randint(0, 256, (n, d // 2), generator=g, dtype=torch.uint8)
    s = (0.5 + 0.5 * torch.rand(n, d // group, generator=g)).half()
    y = torch.empty(B, n, device=DEV)
    A.sfx_linear_q4(x.to(DEV), W.to(DEV), s.to(DEV), y)
    ref = Q.linear_q4(np64(x), W.numpy(), s.numpy())
    # the oracle's bound less its allowance of 2^-120, plus a step for each of two additions per
    # column and 16 more
    tol = Q.linear_q4_bound(np64(x), W.numpy(), s.numpy()) - 2.0 ** -120 + (2 * d + 16) * 2.0 ** -137
    assert (np.abs(np64(y) - ref) <= tol).all(), (np.abs(np64(y) - ref) / tol).max()


@pytest.mark.parametrize("D", [32, 128, 256])
def test_attention_takes_the_largest_bf16_queries(D):
    """Queries of the largest finite size under a small scale: the scores are ordinary."""
    Hq, Hkv, page, n = 6, 2, 16, 90
    say(f"attention largest bf16 {D}")
    g = torch.Generator().manual_seed(D)
    k, v = (torch.randn(n, Hkv, D, generator=g) for _ in range(2))
    q = (torch.randn(1, Hq, D, generator=g).clamp(-1, 1) * BF16_MAX).to(torch.bfloat16)
    assert torch.isfinite(q).all()
    table = torch.arange(6, dtype=torch.int32, device=DEV).view(1, 6)
    pos, seq = torch.arange(n, dtype=torch.int32, device=DEV), torch.zeros(n, dtype=torch.int32, device=DEV)
    cache = torch.full((6, Hkv, page // 8, 9 * D), 0xFF, dtype=torch.uint8, device=DEV)
    A.sfx_kv_append_q4(None, k.to(DEV), v.to(DEV), pos, table, cache, None, seq=seq)
    kn, vn = Q.values(*Q.quantise(k.numpy(), 65504.0)), Q.values(*Q.quantise(v.numpy(), 8188.0))
    out, lse = torch.empty(1, Hq, D, dtype=torch.bfloat16, device=DEV), torch.empty(1, Hq, device=DEV)
    scale = 2.0 ** -130
    A.sfx_attn_q4(q.to(DEV), cache, table, torch.tensor([n], dtype=torch.int32, device=DEV), out,
                  A.workspace(A.sfx_attn_q4_ws(1, Hq, Hkv, D, 96)), scale=scale, lse=lse)
    q64 = np64(q[0])
    o, ls, ab = Q.attention(q64, kn, vn, scale)
    d = Q.score_bound(q64, np.abs(kn).reshape(n, Hkv, -1, 32).max((0, 1, 3)) / 7, scale) + 2.0 ** -22 * 40
    assert d < 2.0 ** -6
    tol = (2 * 2.0 ** -11 + 2 * d + 2.0 ** -18) * ab * 1.01 + 2.0 ** -8 * np.abs(o)
    assert (np.abs(np64(out[0]) - o) <= tol).all() and (np.abs(np64(lse[0]) - ls) <= d + 2.0 ** -20 * (1 + np.abs(ls))).all()


@pytest.mark.parametrize("angles", [0, 40])
def test_lens_follow_what_the_append_stores(angles):
    """Lengths and starts of a step whose positions have a page and an angle, or lack one: the
    append stores exactly the tokens that get a length."""
    page, num_pages, D = 8, 9, 32
    say(f"lens, angles for {angles}")
    table = torch.tensor([[0, 1, 2, 3, 4, 5], [6, -1, 7, 9, 8, -3]], dtype=torch.int32).repeat(40, 1)
    pos = torch.tensor([(5 * i) % 60 - 4 for i in range(80)], dtype=torch.int32)
    pos[:8] = torch.tensor([0, 7, 8, 15, 39, 40, 47, 48], dtype=torch.int32)
    pos[8:10] = torch.tensor([-2 ** 31, 2 ** 31 - 1])
    want = []
    for b, p in enumerate(pos.tolist()):
        ok = 0 <= p < 48 and 0 <= int(table[b, p // page]) < num_pages and not (angles and p >= angles)
        want.append(p + 1 if ok else 0)
    lens, starts = (torch.full((80,), 7, dtype=torch.int32, device=DEV) for _ in range(2))
    for window in (0, 1, 5, 1000):
        A.sfx_kv_lens_q4(pos.to(DEV), table.to(DEV), page, num_pages, lens, starts=starts if window else None, window=window,
                         max_pos=angles)
        assert lens.tolist() == want
        if window:
            assert starts.tolist() == [max(0, n - window) for n in want]
    # one token at a time, into a cache of its own: its bytes change where it has a length
    cs = torch.ones(angles, 2, device=DEV) if angles else None
    k = torch.ones(1, 1, D, device=DEV)
    for b in range(10):
        cache = torch.zeros(num_pages, 1, 1, 9 * D, dtype=torch.uint8, device=DEV)
        A.sfx_kv_append_q4(None, k, k, pos[b:b + 1].to(DEV), table[b:b + 1].to(DEV), cache, None, cos_sin=cs)
        assert bool(cache.any()) == (want[b] > 0), (b, int(pos[b]))


def attn_weights(d, Hq, Hkv, D, seed):
    g = torch.Generator().manual_seed(seed)
    n = (Hq + 2 * Hkv) * D
    rnd = lambda *shape: torch.randint(0, 256, shape, generator=g, dtype=torch.uint8)  # noqa: E731
    return {"Wqkv": rnd(n, d // 2).to(DEV), "Wqkv_s": (torch.rand(n, d // 32, generator=g) * 0.03 + 1e-3).half().to(DEV),
            "Wo": rnd(d, Hq * D // 2).to(DEV), "Wo_s": (torch.rand(d, Hq * D // 64, generator=g) * 0.03 + 1e-3).half().to(DEV),
            "bqkv": torch.randn(n, generator=g).to(DEV), "bo": torch.randn(d, generator=g).to(DEV)}


@pytest.mark.parametrize("window", [0, 6])
def test_step_treats_what_is_not_stored_as_no_token(window):
    """A sequence past the angle table, one whose page is missing, one whose page id is outside the
    cache and one past its table: their rows are the output bias, as for pos = -1, eager and
    captured, whatever the step before left; the other sequence keeps its bits."""
    from activation_sparse_ffn_amd import AttnStep
    d, Hq, Hkv, D, B, page = 256, 4, 2, 64, 5, 8
    say(f"step, tokens that are not stored, window {window}")
    w = attn_weights(d, Hq, Hkv, D, 6)
    table = torch.arange(20, dtype=torch.int32).view(5, 4).to(DEV)
    angles = torch.ones(22, D, device=DEV) * 0.7
    pos = torch.full((B,), 3, dtype=torch.int32, device=DEV)
    step = AttnStep(Hq, Hkv, D, B, "f16", table, pos, 20, page=page, cos_sin=angles, window=window)
    step.cache.zero_()
    g = torch.Generator().manual_seed(2)
    x = torch.randn(B, d, generator=g).half().to(DEV)
    y = torch.empty(B, d, device=DEV)
    step.run(w, x, y)                                    # leaves queries of every sequence
    before = step.cache.clone()
    table[2, 1], table[3, 1] = -1, 20
    bad = [8, 22, 8, 8, 32]                              # sequence 0 is a good one
    outs = []
    for these in (bad, [8, -1, -1, -1, -1]):
        step.cache.copy_(before)
        pos.copy_(torch.tensor(these, dtype=torch.int32))
        step.run(w, x, y)
        outs.append(y.clone())
    assert torch.equal(outs[0], outs[1])
    assert torch.equal(outs[0][1:], w["bo"].expand(B - 1, d)) and not torch.equal(outs[0][0], w["bo"])
    assert not step.o[1:].any()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step.run(w, x, y)
    for these in (bad, [8, 5, 6, 7, 7], bad):
        step.cache.copy_(before)
        pos.copy_(torch.tensor(these, dtype=torch.int32))
        graph.replay()
        if these == bad:
            assert torch.equal(y, outs[0])
        else:
            assert (y != w["bo"]).any(1).all()
        _ = torch.randn(1000, device=DEV).sum().item()


def test_step_refuses_a_negative_window():
    from activation_sparse_ffn_amd import AttnStep
    table, pos = torch.zeros(1, 1, dtype=torch.int32, device=DEV), torch.zeros(1, dtype=torch.int32, device=DEV)
    w = attn_weights(256, 4, 2, 64, 6)
    step = AttnStep(4, 2, 64, 1, "f16", table, pos, 1, page=8, window=-1)
    with pytest.raises(A.SfxError):
        step.run(w, torch.zeros(1, 256, dtype=torch.float16, device=DEV), torch.zeros(1, 256, device=DEV))


def test_streams_of_this_and_of_another_device():
    """Every entry point takes the tensors' device's streams, the default one and others, and
    refuses a stream that says it is on another device before anything is enqueued."""
    class Elsewhere:
        device_index, cuda_stream = 1, torch.cuda.current_stream().cuda_stream

    D, page = 32, 8
    x, W = torch.zeros(1, 64, dtype=torch.float16, device=DEV), torch.zeros(8, 32, dtype=torch.uint8, device=DEV)
    s, y = torch.zeros(8, 2, dtype=torch.float16, device=DEV), torch.full((1, 8), 3.0, device=DEV)
    k, cache = torch.ones(1, 1, D, device=DEV), torch.zeros(1, 1, 1, 9 * D, dtype=torch.uint8, device=DEV)
    at, table = torch.zeros(1, dtype=torch.int32, device=DEV), torch.zeros(1, 1, dtype=torch.int32, device=DEV)
    q, ko, lens = torch.ones(1, 1, D, dtype=torch.float16, device=DEV), torch.full_like(k, 3.0), torch.full_like(at, 3)
    out = torch.full_like(q, 3.0)
    calls = (lambda st: A.sfx_linear_q4(x, W, s, y, stream=st),
             lambda st: A.sfx_kv_append_q4(None, k, k, at, table, cache, None, stream=st),
             lambda st: A.sfx_kv_read_q4(at, table, cache, ko, ko.clone(), stream=st),
             lambda st: A.sfx_kv_lens_q4(at, table, page, 1, lens, stream=st),
             lambda st: A.sfx_attn_q4(q, cache, table, lens, out, None, stream=st))
    for call in calls:
        with pytest.raises(ValueError, match="stream is on device 1"):
            call(Elsewhere())
    torch.cuda.synchronize()
    assert (y == 3).all() and (ko == 3).all() and (out == 3).all() and not cache.any() and lens.item() == 3
    for st in (torch.cuda.default_stream(), torch.cuda.Stream()):
        st.wait_stream(torch.cuda.current_stream())
        for call in calls:
            call(st)
        torch.cuda.current_stream().wait_stream(st)
    # ones are held as 7 fp16(1 / 7) = 1 - 2^-12; the attention rounds a value and its result to fp16
    held = float(7 * np.float64(np.float16(np.float32(1) / np.float32(7))))
    assert held == 1 - 2.0 ** -12
    assert not y.any() and (ko == held).all() and lens.item() == 1 and (out.double() - held).abs().max() <= 2 * 2.0 ** -11


@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("case", [  # B, n, d, group: x of up to 128 KB in LDS and just past it
    (1, 50, 24544, 32), (1, 20, 65504, 32), (1, 20, 65536, 64), (2, 8192, 32704, 64), (2, 8193, 12288, 64), (3, 4096, 21824, 64),
    (3, 4097, 8192, 128), (3, 4097, 8160, 32), (5, 4096, 13088, 32), (8, 31, 8160, 32), (8, 31, 8192, 128), (8, 5000, 3040, 32),
    (8, 5000, 3200, 128), (9, 4100, 96, 32), (16, 16, 1024, 64)], ids=lambda c: "x".join(map(str, c)))
def test_linear_at_the_borders_of_its_kernels(case, dt):
    """Sizes on either side of what decides between keeping x whole in LDS and taking it in blocks."""
    B, n, d, group = case
    say(f"linear border {case} {dt}")
    g = torch.Generator().manual_seed(n + d)
    x = torch.randn(B, d, generator=g).to(DT[dt])
    W = torch.randint(0, 256, (n, d // 2), generator=g, dtype=torch.uint8)
    s = (0.05 * torch.rand(n, d // group, generator=g) + 1e-3).half()
    y = torch.full((B, n), float("nan"), device=DEV)
    args = [t.to(DEV) for t in (x, W, s)]
    A.sfx_linear_q4(*args, y)
    some = np.unique(np.r_[:min(n, 64), n // 2:min(n, n // 2 + 40), max(0, n - 64):n])
    ref = Q.linear_q4(np64(x), W.numpy()[some], s.numpy()[some])
    err = np.abs(np64(y)[:, some] - ref)
    assert (err <= Q.linear_q4_bound(np64(x), W.numpy()[some], s.numpy()[some])).all()
    assert torch.isfinite(y).all()
    y2 = torch.full_like(y, float("nan"))
    A.sfx_linear_q4(*args, y2)
    assert torch.equal(y, y2)
