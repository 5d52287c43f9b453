"""Timed cases of the 8-bit layer half: residual addition with root-mean-square norm and int8
rows, the int8 projection, the append to the paged int8 key/value cache with its read-back,
and attention of one or many query tokens per sequence over that cache.

`run` computes each operator in its plain form (elementary torch operations in 32 or
64 bits) unless `own` is set, and then through the package's entry points.

Cache layout (one layer), uint8 [pages][Hkv][page / 16][32 D + 16]: a block holds 16
consecutive positions of one kv head.  A code is stored as u = q + 128, a value is q * scale:
  16 D bytes   K codes [16 positions][D]
  16 D bytes   V codes [4][D][4]: byte i of dim d in quarter c is position 4 c + i
  16 bytes     fp32 scale of K, fp32 scale of V, 8 bytes unused
Storing a block's first position starts it anew (its other positions are 0); storing another
one keeps the others, whose codes are taken again when the scale has to grow.
"""
import math

import torch

own = False

DT = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
BYTES = {"f16": 2, "bf16": 2, "f32": 4, "none": 0}
BLK = 16                                         # positions of a cache block
EPS = 1e-5
SCRATCH = 64 << 20                               # workspace such a program keeps per stream


# ---------------------------------------------------------------------------- cases

def listed():
    return [
        # one decode token of a d = 4096 layer: fp32 sums into an fp32 residual stream, with the
        # 16-bit row that a sparse FFN reads beside the int8 row; latency counts
        {"name": "norm 1x4096", "op": "norm", "T": 1, "d": 4096, "x": "f32", "res": "f32", "norm": True, "weight": True,
         "y": "f16"},
        # a prompt's rows of a d = 8192 layer, 16-bit residual stream: bytes count
        {"name": "norm 4099x8192", "op": "norm", "T": 4099, "d": 8192, "x": "bf16", "res": "bf16", "norm": True,
         "weight": True, "y": "none"},
        # output projection of a d = 4096 layer at one token: the ordinary decode call
        {"name": "linear 1x4096x4096", "op": "linear", "T": 1, "n": 4096, "d": 4096, "y": "f32", "bias": False, "acc": False},
        # a full decode batch through an FFN-sized projection, added to the fp32 sums
        {"name": "linear 64x11008x4096", "op": "linear", "T": 64, "n": 11008, "d": 4096, "y": "f32", "bias": False,
         "acc": True},
        # a short prompt through a small projection of odd sizes
        {"name": "linear 777x1003x1056", "op": "linear", "T": 777, "n": 1003, "d": 1056, "y": "bf16", "bias": True,
         "acc": False},
        # prompts of a d = 4096 layer with 16384 rows: the matrix cores count
        {"name": "linear 8192x16384x4096", "op": "linear", "T": 8192, "n": 16384, "d": 4096, "y": "f16", "bias": True,
         "acc": False},
        # one decode step's tokens (one of them padding) straight from the fp32 projection,
        # into blocks that hold eight positions already
        {"name": "append 8x1 32/32x128", "op": "append", "dt": "f32", "B": 8, "tokens": 1, "past": 1000, "hq": 32,
         "hkv": 32, "dim": 128, "page": 16, "rope": "half", "rot": 128, "pad": 1},
        # prompts of three requests, partly rotated in neighbouring pairs
        {"name": "append 3x1365 64/8x128", "op": "append", "dt": "bf16", "B": 3, "tokens": 1365, "past": 0, "hq": 64,
         "hkv": 8, "dim": 128, "page": 64, "rope": "pairs", "rot": 64, "pad": 7},
        # one request early in its answer, one head per kv head: latency counts
        {"name": "attn 1x77 32/32x128", "op": "attn", "dt": "f16", "B": 1, "hq": 32, "hkv": 32, "dim": 128, "page": 16,
         "len": 77, "new": 1, "lens": "equal", "window": 0, "lse": False},
        # one request with a very long context, eight heads per kv head
        {"name": "attn 1x131072 64/8x128", "op": "attn", "dt": "bf16", "B": 1, "hq": 64, "hkv": 8, "dim": 128,
         "page": 64, "len": 131072, "new": 1, "lens": "equal", "window": 0, "lse": False},
        # sixteen requests of different ages with up to 5 drafted tokens each, behind a sliding
        # window, with log-sum-exp
        {"name": "attn 16x4096 by 5 128/8x64 window", "op": "attn", "dt": "bf16", "B": 16, "hq": 128, "hkv": 8, "dim": 64,
         "page": 32, "len": 4096, "new": 5, "lens": "ragged", "window": 1500, "lse": True},
        # prompts of requests of different lengths, one of them behind a stored prefix
        {"name": "attn 3x4096 by 3900 64/8x128", "op": "attn", "dt": "f16", "B": 3, "hq": 64, "hkv": 8, "dim": 128,
         "page": 64, "len": 4096, "new": 3900, "lens": "ragged", "window": 0, "lse": False},
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("norm", "linear", "linear", "append", "attn", "attn"))
    dim = rng.choice((32, 64, 64, 96, 128, 128, 128, 256))
    page = rng.choice((16, 16, 32, 64, 128))
    if op == "norm":
        while True:
            c = {"op": op, "T": _log(rng, 1, 8192), "d": rng.choice((16 * _log(rng, 2, 2048), _log(rng, 32, 32768))),
                 "x": rng.choice(("f32", "f16", "bf16")), "res": rng.choice(("none", "f32", "f16", "bf16")),
                 "norm": rng.random() < 0.8, "weight": rng.random() < 0.8, "y": rng.choice(("none", "f16", "bf16", "f32"))}
            c["weight"] = c["weight"] and c["norm"]
            if c["T"] * c["d"] <= 2048 * 8192:
                return c
    if op == "linear":
        while True:
            c = {"op": op, "T": _log(rng, 1, 8192), "n": _log(rng, 48, 32768), "d": 16 * _log(rng, 4, 1024),
                 "y": rng.choice(("f32", "f16", "bf16")), "bias": rng.random() < 0.5, "acc": rng.random() < 0.3}
            if c["T"] * c["n"] * c["d"] <= 8192 * 16384 * 4096 and c["n"] * c["d"] <= 16384 * 8192 and c["T"] * c["n"] <= 8192 * 16384:
                return c
    if op == "append":
        while True:
            hkv = rng.choice((1, 2, 4, 8, 8, 32))
            c = {"op": op, "dt": rng.choice(("f32", "f16", "bf16")), "B": _log(rng, 1, 64), "tokens": _log(rng, 1, 4096),
                 "past": rng.choice((0, 0, 1, 13, 1000, 100000)), "hq": hkv * rng.choice((1, 2, 5, 8)), "hkv": hkv,
                 "dim": dim, "page": page, "rope": rng.choice(("none", "half", "half", "pairs")),
                 "rot": dim if rng.random() < 0.6 else 2 * rng.randint(1, dim // 2), "pad": rng.choice((0, 0, 1, 5))}
            total = (c["B"] * (c["past"] + c["tokens"])) * hkv * dim
            if c["B"] * c["tokens"] * (c["hq"] + 2 * hkv) * dim <= 2048 * 80 * 128 and total <= 131072 * 8 * 128:
                return c
    while True:
        hkv = rng.choice((1, 2, 4, 8, 8, 32))
        c = {"op": op, "dt": rng.choice(("f16", "bf16")), "B": _log(rng, 1, 64), "hq": hkv * rng.choice((1, 1, 2, 4, 5, 7, 8, 16, 20)),
             "hkv": hkv, "dim": dim, "page": page, "len": _log(rng, 1, 131072), "new": rng.choice((1, 1, 2, 8, _log(rng, 1, 4096))),
             "lens": rng.choice(("equal", "ragged", "ragged")), "window": rng.choice((0, 0, 0, 1, 100, 4096)),
             "lse": rng.random() < 0.5}
        c["new"] = min(c["new"], c["len"])
        dense = c["B"] * c["len"] * c["new"] * c["hq"]
        if c["B"] * c["len"] * hkv * dim <= 131072 * 8 * 128 and c["hq"] <= 160 and dense <= 1 << 30 and dense * dim <= 1 << 36:
            return c


def _lens(c):
    if c["lens"] == "equal":
        return [c["len"]] * c["B"]
    # ages spread evenly over the range; the second of several requests has no token yet
    out = [max(1, c["len"] * (b + 1) // c["B"] - (b * 7) % 5) for b in range(c["B"])]
    if c["B"] > 1:
        out[1] = 0
    return out


def _counts(c):
    """Query tokens of each sequence: its last ones."""
    if c["new"] == 1:
        return [1] * c["B"]
    if c["lens"] == "equal":
        return [c["new"]] * c["B"]
    return [min(n, c["new"] - (b * 3) % c["new"]) for b, n in enumerate(_lens(c))]


def _pairs(c):
    """Query token and position pairs that count."""
    w, total = c["window"], 0
    for n, m in zip(_lens(c), _counts(c)):
        for p in range(max(0, n - m), n):
            total += min(p + 1, w or p + 1)
    return total


def work(case):
    c = case
    if c["op"] == "norm":
        T, d = c["T"], c["d"]
        by = T * d * (BYTES[c["x"]] + 2 * BYTES[c["res"]] + BYTES[c["y"]] + 1 + 2) + 4 * T + 4 * d * c["weight"]
        return {"bytes": by, "flops": 8 * T * d}
    if c["op"] == "linear":
        T, n, d = c["T"], c["n"], c["d"]
        by = n * d + T * d + 4 * (T + n) + T * n * BYTES[c["y"]] * (2 if c["acc"] else 1) + 4 * n * c["bias"]
        return {"bytes": by, "flops": 2 * T * n * d}
    per = c["hkv"] * (2 * c["dim"] + 1)                   # cache bytes of a position
    if c["op"] == "attn":
        held = sum(min(n, c["window"] + m - 1 if c["window"] else n) for n, m in zip(_lens(c), _counts(c)))
        by = held * per + sum(_counts(c)) * c["hq"] * (4 * c["dim"] + 4 * c["lse"])
        return {"bytes": by, "flops": 4 * _pairs(c) * c["hq"] * c["dim"]}
    T, heads = c["B"] * c["tokens"], c["hq"] + 2 * c["hkv"]
    by = T * (heads * c["dim"] * BYTES[c["dt"]] + 2 * c["hq"] * c["dim"] + per)
    by += T * per + T * 2 * c["hkv"] * c["dim"] * 2       # the values read back, 16 bits each
    return {"bytes": by, "flops": 8 * T * heads * c["dim"]}


# ---------------------------------------------------------------------------- inputs

def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _out_dt(c):
    return torch.float16 if c["dt"] == "f32" else DT[c["dt"]]


def _val_dt(c):
    """16-bit type of the values that int8 rows stand for."""
    return torch.bfloat16 if "bf16" in (c["x"], c["y"], c["res"]) else torch.float16


def _pages(c, lens, gen):
    """Page table [B][max pages] in shuffled order and the number of pages (some unused)."""
    per = [-(-n // c["page"]) for n in lens]
    total = sum(per) + 3
    order = torch.randperm(total, generator=gen, device="cuda").to(torch.int32)
    table = torch.full((len(lens), max(1, max(per))), -1, dtype=torch.int32, device="cuda")
    at = 0
    for b, k in enumerate(per):
        table[b, :k] = order[at:at + k]
        at += k
    return table, total


def _held(x):
    """Codes (int8) and fp32 scales of blocks [..., 16, D]."""
    s = (x.abs().amax((-2, -1)).double() / 127).float()
    q = torch.round(x.double() / torch.where(s > 0, s, 1.0).double()[..., None, None])
    return q.to(torch.int8), s


def _logical(c, pages, gen):
    """Codes [pages][Hkv][page / 16][16][D] and scales of a whole cache: keys with a few strong
    channels, values of small unequal size."""
    shape = (pages, c["hkv"], c["page"] // BLK, BLK, c["dim"])
    k = torch.randn(shape, generator=gen, device="cuda")
    k *= 1 + 3 * (torch.rand(c["hkv"], 1, 1, c["dim"], generator=gen, device="cuda") < 0.03)
    kq, ks = _held(k)
    del k
    v = torch.randn(shape, generator=gen, device="cuda")
    v *= 0.05 + 0.5 * torch.rand(c["hkv"], 1, 1, c["dim"], generator=gen, device="cuda")
    vq, vs = _held(v)
    return kq, ks, vq, vs


def _pack(kq, ks, vq, vs):
    P, H, O, _, D = kq.shape
    kb = (kq.to(torch.int16) + 128).to(torch.uint8).reshape(P, H, O, BLK * D)
    vb = (vq.to(torch.int16) + 128).to(torch.uint8).view(P, H, O, 4, 4, D).transpose(4, 5).reshape(P, H, O, BLK * D)
    sc = torch.stack([ks, vs, torch.zeros_like(ks), torch.zeros_like(ks)], -1).view(torch.uint8)
    return torch.cat([kb, vb, sc], 3).contiguous()


def _make(case, seed):
    """Everything the plain form, the kernels and the 64-bit form start from."""
    c, gen = case, _gen(seed)
    rnd = lambda *shape: torch.randn(*shape, generator=gen, device="cuda")  # noqa: E731
    if c["op"] == "norm":
        strong = 1 + 19 * (torch.rand(c["d"], generator=gen, device="cuda") < 0.005)
        st = {"x": (rnd(c["T"], c["d"]) * strong).to(DT[c["x"]])}
        st["res"] = (3 * rnd(c["T"], c["d"]) * strong).to(DT[c["res"]]) if c["res"] != "none" else None
        st["w"] = 1 + 0.2 * rnd(c["d"]) if c["weight"] else None
        return st
    if c["op"] == "linear":
        q = lambda r: (rnd(r, c["d"]) * 32).round_().clamp_(-127, 127).to(torch.int8)  # noqa: E731
        pos = lambda r: 0.3 + torch.rand(r, generator=gen, device="cuda")  # noqa: E731
        return {"x": q(c["T"]), "W": q(c["n"]), "sx": pos(c["T"]) / 32, "sw": pos(c["n"]) / (32 * math.sqrt(c["d"])),
                "bias": rnd(c["n"]) if c["bias"] else None, "y0": rnd(c["T"], c["n"]).to(DT[c["y"]]) if c["acc"] else None}
    lens = _lens(c) if c["op"] == "attn" else [c["past"] + c["tokens"]] * c["B"]
    table, pages = _pages(c, lens, gen)
    st = {"table": table, "pages": pages}
    st["kq"], st["ks"], st["vq"], st["vs"] = _logical(c, pages, gen)
    if c["op"] == "attn":
        counts = torch.tensor(_counts(c), dtype=torch.int32, device="cuda")
        st["lens"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
        st["q_start"] = torch.cat([counts.new_zeros(1), counts.cumsum(0).int()])
        st["q"] = (1.3 * rnd(sum(_counts(c)), c["hq"], c["dim"])).to(DT[c["dt"]])
        return st
    T = c["tokens"]
    pos = torch.arange(T, dtype=torch.int32, device="cuda").repeat(c["B"]) + c["past"]
    pad = c["pad"] if c["pad"] < c["B"] * T else 0
    if pad:
        pos[-pad:] = -1                              # padding behind the last request's tokens
    st["pos"] = pos
    counts = (pos >= 0).view(c["B"], T).sum(1).int()
    st["lens"] = counts + c["past"]
    st["q_start"] = torch.cat([counts.new_zeros(1), counts.cumsum(0).int()])
    # what is read back: every position of the blocks written to, up to the last token
    first = c["past"] // BLK * BLK
    n = c["past"] + T - first
    st["rseq"] = torch.arange(c["B"], dtype=torch.int32, device="cuda").repeat_interleave(n)
    st["rpos"] = torch.arange(n, dtype=torch.int32, device="cuda").repeat(c["B"]) + first
    st["rpos"].view(c["B"], n)[:, c["past"] - first:][(pos < 0).view(c["B"], T)] = -1
    st["qkv"] = rnd(c["B"] * T, (c["hq"] + 2 * c["hkv"]) * c["dim"]).to(DT[c["dt"]])   # one projection's rows
    st["cos_sin"] = None
    if c["rope"] != "none":
        i = torch.arange(c["rot"] // 2, dtype=torch.float64, device="cuda")
        ang = torch.arange(max(lens), dtype=torch.float64, device="cuda")[:, None] * 10000.0 ** (-2 * i / c["rot"])
        st["cos_sin"] = torch.cat([ang.cos(), ang.sin()], 1).float()
    return st


def _slices(c, x):
    a, b = c["hq"] * c["dim"], c["hkv"] * c["dim"]
    return (x[:, :a].unflatten(1, (c["hq"], c["dim"])), x[:, a:a + b].unflatten(1, (c["hkv"], c["dim"])),
            x[:, a + b:].unflatten(1, (c["hkv"], c["dim"])))


def prepare(case, seed):
    c, st = case, _make(case, seed)
    st["case"] = c
    if c["op"] == "norm":
        T, d = c["T"], c["d"]
        st["q"] = torch.empty(T, d, dtype=torch.int8, device="cuda")
        st["s"] = torch.empty(T, device="cuda")
        st["res_out"] = torch.empty_like(st["res"]) if c["res"] != "none" else None
        st["y"] = torch.empty(T, d, dtype=DT[c["y"]], device="cuda") if c["y"] != "none" else None
        st["val"] = torch.empty(T, d, dtype=_val_dt(c), device="cuda")
        return st
    if c["op"] == "linear":
        st["y"] = torch.empty(c["T"], c["n"], dtype=DT[c["y"]], device="cuda")
        return st
    st["cache"] = _pack(st.pop("kq"), st.pop("ks"), st.pop("vq"), st.pop("vs"))
    if c["op"] == "append":
        st["q"], st["k"], st["v"] = _slices(c, st["qkv"])
        st["q_out"] = torch.zeros(c["B"] * c["tokens"], c["hq"], c["dim"], dtype=_out_dt(c), device="cuda")
        st["k_out"] = torch.zeros(st["rpos"].numel(), c["hkv"], c["dim"], dtype=_out_dt(c), device="cuda")
        st["v_out"] = torch.zeros_like(st["k_out"])
        return st
    st["out"] = torch.empty_like(st["q"])
    st["lse"] = torch.empty(st["q"].shape[:2], device="cuda") if c["lse"] else None
    st["ws"] = torch.zeros(SCRATCH, dtype=torch.uint8, device="cuda")
    return st


# ---------------------------------------------------------------------------- plain forms

def _plain_norm(st, c):
    h = st["x"].double()                                  # 64 bits: codes next to a border
    out = []
    if st["res"] is not None:
        h = h + st["res"].double()
        out.append(h.to(st["res"].dtype))
    n = h
    if c["norm"]:
        n = h / (h.square().mean(1, keepdim=True) + EPS).sqrt()
        if st["w"] is not None:
            n = n * st["w"].double()
    s = (n.abs().amax(1) / 127).float()
    q = torch.round(n / torch.where(s > 0, s, 1.0).double()[:, None]).clamp(-127, 127)
    out += [s, (q.float() * s[:, None]).to(_val_dt(c))]
    return out + ([n.to(st["y"].dtype)] if st["y"] is not None else [])


def _plain_linear(st, c):
    y = torch.matmul(st["x"].float(), st["W"].float().t())
    y = y * (st["sx"][:, None] * st["sw"])
    if c["bias"]:
        y = y + st["bias"]
    return (st["y0"].float() + y if c["acc"] else y).to(st["y"].dtype)


def _plain_rotate(st, c, x):
    """x [T][H][D] rotated at its positions: 64-bit products of table entries, float32."""
    x = x.double()
    if st["cos_sin"] is None:
        return x.float()
    r = c["rot"]
    cs = st["cos_sin"][st["pos"].long().clamp(min=0)].double()[:, None]
    co, si = cs[..., :r // 2], cs[..., r // 2:]
    if c["rope"] == "half":
        a, b = x[..., :r // 2], x[..., r // 2:r]
        y = torch.cat([a * co - b * si, b * co + a * si, x[..., r:]], -1)
    else:
        a, b = x[..., 0:r:2], x[..., 1:r:2]
        y = torch.cat([torch.stack([a * co - b * si, b * co + a * si], -1).flatten(-2), x[..., r:]], -1)
    return y.float()


def _unpack(blocks, D):
    """Blocks uint8 [..., 32 D + 16]: K and V codes [..., 16][D] and their scales, float32."""
    k = blocks[..., :16 * D].unflatten(-1, (BLK, D)).float() - 128
    v = blocks[..., 16 * D:32 * D].unflatten(-1, (4, D, 4)).transpose(-2, -1).flatten(-3, -2).float() - 128
    s = blocks[..., 32 * D:32 * D + 8].contiguous().view(torch.float32)
    return k, v, s[..., 0], s[..., 1]


def _plain_append(st, c):
    B, H, D, T, page = c["B"], c["hkv"], c["dim"], c["tokens"], c["page"]
    real = st["pos"] >= 0
    st["q_out"][real] = _plain_rotate(st, c, st["q"])[real].to(st["q_out"].dtype)
    first = c["past"] // BLK * BLK
    blocks = (c["past"] + T - 1) // BLK - first // BLK + 1
    lead = c["past"] - first                              # positions that the first block keeps
    b0 = first // BLK + torch.arange(blocks, device="cuda")
    pages = st["table"].long()[:, b0 * BLK // page].clamp(min=0)               # [B][blocks]
    o = b0 % (page // BLK)
    old = st["cache"][pages, :, o.expand(B, -1)]                               # [B][blocks][H][32 D + 16]
    kc, vc, ks, vs = _unpack(old, D)
    new = torch.zeros(B, blocks * BLK, dtype=torch.bool, device="cuda")
    new[:, lead:lead + T] = real.view(B, T)
    new = new.view(B, blocks, 1, BLK, 1)
    touched = new.any(3, keepdim=True)
    keep = torch.zeros(blocks, 1, device="cuda", dtype=torch.bool)
    keep[0] = lead > 0

    def codes(x, held, s_old):
        rows = torch.zeros(B, blocks * BLK, H, D, device="cuda")
        rows[:, lead:lead + T] = x.view(B, T, H, D)
        rows = torch.where(new, rows.view(B, blocks, BLK, H, D).transpose(2, 3), 0.0)
        s = (rows.abs().amax((-2, -1)).double() / 127).float()
        s_old = torch.where(keep, s_old, 0.0)
        s = torch.maximum(s, s_old)
        d = torch.where(s > 0, s, 1.0).double()[..., None, None]
        again = torch.round(held.double() * s_old.double()[..., None, None] / d)
        q = torch.where(new, torch.round(rows.double() / d).clamp(-127, 127), again)
        return q, s

    kq, ks2 = codes(_plain_rotate(st, c, st["k"]), kc, ks)
    vq, vs2 = codes(st["v"].float(), vc, vs)
    u = lambda q: (q + 128).to(torch.uint8)  # noqa: E731
    vb = u(vq).unflatten(3, (4, 4)).transpose(4, 5).flatten(3)
    sc = torch.stack([ks2, vs2, torch.zeros_like(ks2), torch.zeros_like(ks2)], -1).view(torch.uint8)
    block = torch.where(touched[..., 0], torch.cat([u(kq).flatten(3), vb, sc], 3), old)
    at = touched[:, :, 0, 0, 0]
    st["cache"][pages[at], :, o.expand(B, -1)[at]] = block[at]
    return [st["q_out"]] + _plain_read(st, c)


def _plain_read(st, c):
    D, page = c["dim"], c["page"]
    p = st["rpos"].long()
    real = (p >= 0)[:, None, None]
    p = p.clamp(min=0)
    pg = st["table"][st["rseq"].long(), p // page].long().clamp(min=0)
    head = torch.arange(c["hkv"], device="cuda")
    rows = st["cache"][pg[:, None], head, ((p % page) // BLK)[:, None]]        # [T][H][32 D + 16]
    i = (p % BLK)[:, None, None]
    d = torch.arange(D, device="cuda")
    k = rows.gather(2, (i * D + d).expand(-1, c["hkv"], -1)).float() - 128
    v = rows.gather(2, (16 * D + (i // 4 * D + d) * 4 + i % 4).expand(-1, c["hkv"], -1)).float() - 128
    s = rows[..., 32 * D:32 * D + 8].contiguous().view(torch.float32)
    return [torch.where(real, x, 0.0).to(_out_dt(c)) for x in (k * s[..., :1], v * s[..., 1:])]


def _plain_attn(st, c):
    B, D, H, G, M = c["B"], c["dim"], c["hkv"], c["hq"] // c["hkv"], max(_counts(c))
    kc, vc, ks, vs = _unpack(st["cache"][st["table"].long().clamp(min=0)], D)   # [B][pages][H][page / 16][16][D]
    k, v = (x.transpose(1, 2).reshape(B * H, -1, D) for x in (kc * ks[..., None, None], vc * vs[..., None, None]))
    del kc, vc
    q0, lens = st["q_start"].long(), st["lens"].long()
    n = q0[1:] - q0[:-1]
    i = torch.arange(M, device="cuda")
    row = (q0[:-1, None] + i).clamp(max=st["q"].shape[0] - 1)                   # [B][M]
    q = st["q"][row].float().view(B, M, H, G, D).permute(0, 2, 3, 1, 4).reshape(B * H, G * M, D)
    s = torch.matmul(q, k.transpose(1, 2).contiguous()).view(B, H, G, M, -1) / math.sqrt(D)
    at = (lens - n)[:, None] + i                                                # [B][M] positions of the queries
    p = torch.arange(s.shape[-1], device="cuda")
    seen = p <= at[..., None]
    if c["window"]:
        seen = seen & (p > at[..., None] - c["window"])
    s = s.masked_fill_(~seen[:, None, None], -math.inf)
    m = s.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, 0.0, m)
    e = s.sub_(m).exp_()
    l = e.sum(-1, keepdim=True)
    o = torch.matmul(e.view(B * H, G * M, -1), v).view(B, H, G, M, D) / torch.where(l > 0, l, 1.0)
    real = i < n[:, None]                                                       # [B][M]
    out = [o.permute(0, 3, 1, 2, 4).reshape(B, M, c["hq"], D)[real].to(DT[c["dt"]])]
    return out + [(m + l.log()).permute(0, 3, 1, 2, 4).reshape(B, M, c["hq"])[real]] if c["lse"] else out


def run(state):
    st, c = state, state["case"]
    if own:
        return _own(st, c)
    return {"norm": _plain_norm, "linear": _plain_linear, "append": _plain_append, "attn": _plain_attn}[c["op"]](st, c)


def _own(st, c):
    from activation_sparse_ffn_amd import _abi as A
    if c["op"] == "norm":
        A.sfx_norm_q8(st["x"], st["q"], st["s"], weight=st["w"], eps=EPS, residual=st["res"], residual_out=st["res_out"],
                      y=st["y"], norm=c["norm"])
        val = torch.mul(st["q"], st["s"][:, None], out=st["val"])
        return [t for t in (st["res_out"], st["s"], val, st["y"]) if t is not None]
    if c["op"] == "linear":
        if c["acc"]:
            st["y"].copy_(st["y0"])                     # the residual stream as the layer finds it
        A.sfx_linear_q8(st["x"], st["sx"], st["W"], st["sw"], st["y"], bias=st["bias"], accumulate=c["acc"])
        return st["y"]
    if c["op"] == "append":
        A.sfx_kv_append_q8(st["q"], st["k"], st["v"], st["lens"], st["table"], st["cache"], st["q_out"],
                           q_start=st["q_start"], cos_sin=st["cos_sin"], interleaved=c["rope"] == "pairs")
        A.sfx_kv_read_q8(st["rpos"], st["table"], st["cache"], st["k_out"], st["v_out"], seq=st["rseq"])
        return [st["q_out"], st["k_out"], st["v_out"]]
    one = c["new"] == 1
    A.sfx_attn_q8(st["q"], st["cache"], st["table"], st["lens"], st["out"], st["ws"],
                  q_start=None if one else st["q_start"], max_q=max(1, c["new"]), window=c["window"], lse=st["lse"])
    return [st["out"], st["lse"]] if c["lse"] else [st["out"]]


# ---------------------------------------------------------------------------- 64 bits

def exact(case, seed):
    c, st = case, _make(case, seed)
    if c["op"] == "norm":
        h, out = st["x"].double(), []
        if c["res"] != "none":
            h = st["res"].double() + h
            out = [h]
        n = h
        if c["norm"]:
            n = h * torch.rsqrt((h * h).sum(1) / c["d"] + EPS).unsqueeze(1)
            n = n * st["w"].double() if c["weight"] else n
        s = n.abs().max(1).values / 127.0
        held = s.float().double().unsqueeze(1)
        u = torch.clamp(torch.round(n / torch.where(held == 0, 1.0, held)), -127, 127)
        return out + [s, u * held] + ([n] if c["y"] != "none" else [])
    if c["op"] == "linear":
        y = torch.empty(c["T"], c["n"], dtype=torch.float64, device="cuda")
        w = st["W"].double() * st["sw"].double().unsqueeze(1)
        for t in range(0, c["T"], 1024):
            y[t:t + 1024] = (st["x"][t:t + 1024].double() * st["sx"][t:t + 1024].double().unsqueeze(1)) @ w.T
        y = y + st["bias"].double() if c["bias"] else y
        return y + st["y0"].double() if c["acc"] else y
    H, D = c["hkv"], c["dim"]
    if c["op"] == "attn":
        G, outs, lses = c["hq"] // H, [], []
        at = 0
        for b, (n, m) in enumerate(zip(_lens(c), _counts(c))):
            q = st["q"][at:at + m].double()
            at += m
            if n == 0:
                outs.append(torch.zeros(m, c["hq"], D, dtype=torch.float64, device="cuda"))
                lses.append(torch.full((m, c["hq"]), -math.inf, dtype=torch.float64, device="cuda"))
                continue
            ids = st["table"][b][:-(-n // c["page"])].long()
            o = torch.empty(m, c["hq"], D, dtype=torch.float64, device="cuda")
            ls = torch.empty(m, c["hq"], dtype=torch.float64, device="cuda")
            where = torch.arange(n - m, n, device="cuda").unsqueeze(1)
            gap = where - torch.arange(n, device="cuda")
            hidden = (gap < 0) | (gap >= c["window"]) if c["window"] else gap < 0
            for h in range(H):
                k = (st["kq"][ids, h].double() * st["ks"][ids, h].double()[..., None, None]).reshape(-1, D)[:n]
                v = (st["vq"][ids, h].double() * st["vs"][ids, h].double()[..., None, None]).reshape(-1, D)[:n]
                for g in range(h * G, h * G + G):
                    s = (q[:, g] @ k.T / D ** 0.5).masked_fill(hidden, -math.inf)
                    ls[:, g] = torch.logsumexp(s, 1)
                    o[:, g] = torch.exp(s - ls[:, g:g + 1]) @ v
            outs.append(o)
            lses.append(ls)
        return [torch.cat(outs), torch.cat(lses)] if c["lse"] else [torch.cat(outs)]
    T = c["B"] * c["tokens"]
    pos = st["pos"].long()
    real = (pos >= 0).double().reshape(T, 1, 1)
    q, k, v = (x.double() for x in _slices(c, st["qkv"]))
    if c["rope"] != "none":
        r = c["rot"]
        cs = st["cos_sin"].double()[pos.clamp(min=0)]
        z = torch.complex(cs[:, :r // 2], cs[:, r // 2:]).reshape(T, 1, -1)

        def turn(x):
            if c["rope"] == "half":
                y = torch.complex(x[..., :r // 2].contiguous(), x[..., r // 2:r].contiguous()) * z
                return torch.cat((y.real, y.imag, x[..., r:]), 2)
            y = torch.view_as_complex(x[..., :r].reshape(T, -1, r // 2, 2).contiguous()) * z
            return torch.cat((torch.view_as_real(y).reshape(T, -1, r), x[..., r:]), 2)
        q, k = turn(q), turn(k)

    def stored(x, codes, scales):
        """Values of every listed position, a block's worth at a time."""
        first, out = c["past"] // BLK * BLK, []
        end = c["past"] + c["tokens"]
        for b in range(c["B"]):
            rows = x[b * c["tokens"]:(b + 1) * c["tokens"]]
            live = int((pos[b * c["tokens"]:(b + 1) * c["tokens"]] >= 0).sum())
            res = torch.zeros(end - first, H, D, dtype=torch.float64, device="cuda")
            lead = c["past"] - first
            if lead:
                p = st["table"][b, first // c["page"]].long()
                o = (first % c["page"]) // BLK
                qs, so = codes[p, :, o, :lead].double(), scales[p, :, o].double()
                n = min(live, BLK - lead)
                s = so
                if n:
                    s = torch.maximum(so, (rows[:n].float().double().abs().amax((0, 2)) / 127).float().double())
                    qs = torch.round(qs * so[:, None, None] / s[:, None, None])
                    res[lead:lead + n] = torch.round(rows[:n].float().double() / s[:, None]) * s[:, None]
                res[:lead] = (qs * s[:, None, None]).transpose(0, 1)
                rows, live, at = rows[BLK - lead:], max(0, live - (BLK - lead)), BLK
            else:
                at = 0
            if live > 0:
                full = torch.zeros(-(-live // BLK) * BLK, H, D, dtype=torch.float64, device="cuda")
                full[:live] = rows[:live].float().double()
                g = full.view(-1, BLK, H, D)
                s = (g.abs().amax((1, 3), keepdim=True) / 127).float().double()
                res[at:at + live] = (torch.round(g / torch.where(s == 0, 1.0, s)) * s).view(-1, H, D)[:live]
            out.append(res)
        return torch.cat(out) * (st["rpos"] >= 0).double().reshape(-1, 1, 1)
    return [q * real, stored(k, st["kq"], st["ks"]), stored(v, st["vq"], st["vs"])]
