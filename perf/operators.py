"""Timed cases of the int4 attention half of a decode layer: the projection with int4
weights, the append to the paged int4 key/value cache, reading the cache back, and
decode attention over it.

`run` computes each operator in its plain form (elementary torch operations in 32 or
64 bits) unless `own` is set, and then through the package's entry points.

Cache layout (one layer), uint8 [pages][Hkv][page / 8][9 D]: a block of 9 D bytes holds
8 consecutive positions of one kv head.  Codes are u = q + 8 (4 bits), one fp16 scale
per 32 dimensions, value = q * scale:
  bytes 0 .. 4D      K: per position D/2 bytes, words [c = 0..3][g = 0..D/32-1] holding
                     dims 32 g + 8 c + 0..7 as bytes (0,2) (4,6) (1,3) (5,7), first
                     of a pair in the low nibble;
  bytes 4D .. 8D     V: [n = 0..15][g][8 positions in the order 0 2 1 3 4 6 5 7], a byte
                     holds dims 32 g + n (low nibble) and 32 g + 16 + n;
  then fp16 K scales [g][8 positions], then fp16 V scales [g][8 positions].
"""
import math

import torch

own = False

DT = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
K_LO, K_HI = (0, 4, 1, 5), (2, 6, 3, 7)          # dims of a K word's bytes: low, high nibbles
V_POS = (0, 2, 1, 3, 4, 6, 5, 7)                 # position held by byte i of a V unit
SCRATCH = 64 << 20                               # workspace such a program keeps per stream


# ---------------------------------------------------------------------------- cases

def listed():
    return [
        # output projection of a d = 4096 layer at one token: the ordinary decode call
        {"name": "linear 1x4096x4096", "op": "linear", "dt": "f16", "B": 1, "n": 4096, "d": 4096, "group": 32,
         "bias": False, "acc": False},
        # a small, odd-sized projection for a few tokens: latency counts
        {"name": "linear 5x1003x1056", "op": "linear", "dt": "bf16", "B": 5, "n": 1003, "d": 1056, "group": 32,
         "bias": True, "acc": False},
        # the widest single-token product (d = 7168, 4 d rows): bytes of the codes count
        {"name": "linear 1x28672x7168", "op": "linear", "dt": "f16", "B": 1, "n": 28672, "d": 7168, "group": 128,
         "bias": True, "acc": False},
        # a d = 8192 projection for 37 requests, added to the residual stream
        {"name": "linear 37x8192x8192", "op": "linear", "dt": "bf16", "B": 37, "n": 8192, "d": 8192, "group": 64,
         "bias": False, "acc": True},
        # one request early in its answer, one head per kv head: latency counts
        {"name": "attn 1x77 32/32x128", "op": "attn", "dt": "f16", "B": 1, "hq": 32, "hkv": 32, "dim": 128, "page": 16,
         "len": 77, "lens": "equal", "window": 0, "lse": False},
        # one request with a very long context, eight heads per kv head
        {"name": "attn 1x131072 64/8x128", "op": "attn", "dt": "bf16", "B": 1, "hq": 64, "hkv": 8, "dim": 128,
         "page": 64, "len": 131072, "lens": "equal", "window": 0, "lse": False},
        # eight requests of different ages (one of them empty) behind a sliding window, with log-sum-exp
        {"name": "attn 8x2048 32/32x128 window", "op": "attn", "dt": "f16", "B": 8, "hq": 32, "hkv": 32, "dim": 128,
         "page": 16, "len": 2048, "lens": "ragged", "window": 1500, "lse": True},
        # a full batch with 16 heads per kv head of 64
        {"name": "attn 64x4096 128/8x64", "op": "attn", "dt": "bf16", "B": 64, "hq": 128, "hkv": 8, "dim": 64,
         "page": 32, "len": 4096, "lens": "ragged", "window": 0, "lse": False},
        # one decode step's tokens (one of them padding) straight from the fp32 projection
        {"name": "append 8x1 32/32x128", "op": "append", "dt": "f32", "B": 8, "tokens": 1, "past": 1000, "hq": 32,
         "hkv": 32, "dim": 128, "page": 16, "rope": "half", "rot": 128, "pad": 1},
        # prompts of three requests, partly rotated in neighbouring pairs
        {"name": "append 3x1365 64/8x128", "op": "append", "dt": "bf16", "B": 3, "tokens": 1365, "past": 0, "hq": 64,
         "hkv": 8, "dim": 128, "page": 64, "rope": "pairs", "rot": 64, "pad": 7},
        # a short prefix read back
        {"name": "read 333 8x64", "op": "read", "dt": "f16", "B": 1, "tokens": 333, "hkv": 8, "dim": 64, "page": 32},
        # long prefixes of two requests read back as 16-bit rows for the next prompt chunk
        {"name": "read 2x8192 8x128", "op": "read", "dt": "bf16", "B": 2, "tokens": 8192, "hkv": 8, "dim": 128,
         "page": 16},
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("linear", "linear", "attn", "attn", "append", "read"))
    dim = rng.choice((32, 64, 64, 96, 128, 128, 128, 256))
    page = rng.choice((8, 16, 32, 64, 128))
    if op == "linear":
        while True:
            c = {"op": op, "dt": rng.choice(("f16", "bf16")), "B": _log(rng, 1, 64), "n": _log(rng, 48, 32768),
                 "d": 128 * _log(rng, 1, 64), "group": rng.choice((32, 64, 128)), "bias": rng.random() < 0.5,
                 "acc": rng.random() < 0.3}
            if c["B"] * c["n"] * c["d"] <= 37 * 8192 * 8192 and c["n"] * c["d"] <= 28672 * 7168:
                return c
    if op == "attn":
        while True:
            hkv = rng.choice((1, 2, 4, 8, 8, 32))
            c = {"op": op, "dt": rng.choice(("f16", "bf16")), "B": _log(rng, 1, 64),
                 "hq": hkv * rng.choice((1, 1, 2, 4, 5, 7, 8, 16, 20)), "hkv": hkv, "dim": dim, "page": page,
                 "len": _log(rng, 1, 131072), "lens": rng.choice(("equal", "ragged", "ragged")),
                 "window": rng.choice((0, 0, 0, 1, 100, 4096)), "lse": rng.random() < 0.5}
            if c["B"] * c["len"] * hkv * dim <= 131072 * 8 * 128 and c["hq"] <= 160:
                return c
    if op == "append":
        while True:
            hkv = rng.choice((1, 2, 4, 8, 8, 32))
            rope = rng.choice(("none", "half", "half", "pairs"))
            c = {"op": op, "dt": rng.choice(("f32", "f16", "bf16")), "B": _log(rng, 1, 64), "tokens": _log(rng, 1, 4096),
                 "past": rng.choice((0, 1, 13, 1000, 100000)), "hq": hkv * rng.choice((1, 2, 5, 8)), "hkv": hkv,
                 "dim": dim, "page": page, "rope": rope, "rot": dim if rng.random() < 0.6 else 2 * rng.randint(1, dim // 2),
                 "pad": rng.choice((0, 0, 1, 5))}
            if c["B"] * c["tokens"] * (c["hq"] + 2 * hkv) * dim <= 4095 * 80 * 128:
                return c
    while True:
        c = {"op": "read", "dt": rng.choice(("f32", "f16", "bf16")), "B": _log(rng, 1, 16), "tokens": _log(rng, 1, 16384),
             "hkv": rng.choice((1, 2, 4, 8, 8, 32)), "dim": dim, "page": page}
        if c["B"] * c["tokens"] * c["hkv"] * dim <= 2 * 8192 * 8 * 128:
            return c


def _lens(c):
    if c["lens"] == "equal":
        return [c["len"]] * c["B"]
    # ages spread evenly over the range; the second of several requests has no token yet
    out = [max(1, c["len"] * (b + 1) // c["B"] - (b * 7) % 5) for b in range(c["B"])]
    if c["B"] > 1:
        out[1] = 0
    return out


def work(case):
    c = case
    e = {"f32": 4, "f16": 2, "bf16": 2}
    if c["op"] == "linear":
        B, n, d = c["B"], c["n"], c["d"]
        by = n * d / 2 + 2 * n * d / c["group"] + 2 * B * d + 4 * B * n * (2 if c["acc"] else 1) + 4 * n * c["bias"]
        return {"bytes": by, "flops": 2 * B * n * d}
    per = c["hkv"] * (c["dim"] + c["dim"] / 8)             # cache bytes of a position
    if c["op"] == "attn":
        npos = sum(min(n, c["window"] or n) for n in _lens(c))
        return {"bytes": npos * per + 4 * c["B"] * c["hq"] * c["dim"], "flops": 4 * npos * c["hq"] * c["dim"]}
    T = c["B"] * c["tokens"]
    if c["op"] == "append":
        heads = c["hq"] + 2 * c["hkv"]
        by = T * (heads * c["dim"] * e[c["dt"]] + 2 * c["hq"] * c["dim"] + per)
        by += T * per + T * 2 * c["hkv"] * c["dim"] * 2      # the values read back, 16 bits each
        return {"bytes": by, "flops": 6 * T * heads * c["dim"]}
    return {"bytes": T * (per + 2 * c["hkv"] * c["dim"] * e[c["dt"]]), "flops": 2 * T * c["hkv"] * c["dim"]}


# ---------------------------------------------------------------------------- inputs

def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _quant(w):
    """Codes -8..7 (int8) and fp16 scales of groups of 32 along the last dimension."""
    g = w.float().unflatten(-1, (-1, 32))
    s = (g.abs().amax(-1) / torch.full((), 7.0, device=w.device)).half()
    q = torch.where(s[..., None] > 0, g / s[..., None].float(), torch.zeros_like(g))
    return torch.round(q).clamp(-8, 7).to(torch.int8).flatten(-2), s


def _weights(c, gen):
    """Random codes of a normal weight row and fp16 scales of its size."""
    n, d, G = c["n"], c["d"], c["group"]
    q = (torch.randn(n, d, generator=gen, device="cuda", dtype=torch.float16) * 2.7).round_().clamp_(-8, 7).to(torch.int8)
    s = (0.3 + torch.rand(n, d // G, generator=gen, device="cuda")) / (2.7 * math.sqrt(d))
    return q, s.half()


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


def _logical(c, pages, gen):
    """Codes and scales of a whole cache, [pages][Hkv][page][D] and [..][D/32]: keys with a
    few strong channels, values of small unequal size."""
    shape = (pages, c["hkv"], c["page"], c["dim"])
    chan = 1 + 3 * (torch.rand(c["hkv"], 1, c["dim"], generator=gen, device="cuda") < 0.03)
    k = torch.randn(shape, generator=gen, device="cuda") * chan
    kq, ks = _quant(k)
    del k
    v = torch.randn(shape, generator=gen, device="cuda")
    v *= 0.05 + 0.5 * torch.rand(c["hkv"], 1, c["dim"], generator=gen, device="cuda")
    vq, vs = _quant(v)
    return kq, ks, vq, vs


def _pack(c, kq, ks, vq, vs):
    P, H, page, D = kq.shape
    O, NG = page // 8, D // 32
    ku = (kq + 8).to(torch.uint8).view(P, H, O, 8, NG, 4, 8)
    kb = ku[..., list(K_LO)] | (ku[..., list(K_HI)] << 4)                       # [..8][g][c][4]
    kb = kb.transpose(4, 5).reshape(P, H, O, 4 * D)
    vu = (vq + 8).to(torch.uint8).view(P, H, O, 8, NG, 2, 16)
    vb = (vu[..., 0, :] | (vu[..., 1, :] << 4))[:, :, :, list(V_POS)]          # [..8][g][n]
    vb = vb.permute(0, 1, 2, 5, 4, 3).reshape(P, H, O, 4 * D)
    sc = [s.view(P, H, O, 8, NG).transpose(3, 4).contiguous().view(torch.uint8).reshape(P, H, O, D // 2)
          for s in (ks, vs)]
    return torch.cat([kb, vb] + sc, dim=3).contiguous()


def _make(case, seed):
    """Everything the plain form, the kernels and the 64-bit form start from."""
    c, gen = case, _gen(seed)
    rnd = lambda *shape: torch.randn(*shape, generator=gen, device="cuda")  # noqa: E731
    if c["op"] == "linear":
        q, s = _weights(c, gen)
        x = rnd(c["B"], c["d"]) * (1 + 9 * (torch.rand(c["d"], generator=gen, device="cuda") < 0.005))
        st = {"x": x.to(DT[c["dt"]]), "q": q, "s": s, "bias": rnd(c["n"]) if c["bias"] else None, "y0": rnd(c["B"], c["n"])}
        return st
    T = c.get("tokens", 0)
    lens = _lens(c) if c["op"] == "attn" else [c.get("past", 0) + T] * c["B"]
    table, pages = _pages(c, lens, gen)
    st = {"table": table, "pages": pages, "lens": torch.tensor(lens, dtype=torch.int32, device="cuda")}
    if c["op"] != "append":
        st["kq"], st["ks"], st["vq"], st["vs"] = _logical(c, pages, gen)
    if c["op"] == "attn":
        st["q"] = (1.3 * rnd(c["B"], c["hq"], c["dim"])).to(DT[c["dt"]])
        st["starts"] = (st["lens"] - c["window"]).clamp(min=0) if c["window"] else None
        return st
    # tokens of the requests one behind the other: sequence and position of each
    seq = torch.arange(c["B"], dtype=torch.int32, device="cuda").repeat_interleave(T)
    pos = torch.arange(T, dtype=torch.int32, device="cuda").repeat(c["B"]) + c.get("past", 0)
    st["seq"] = seq
    if c["op"] == "append":
        if 0 < c["pad"] < c["B"] * T:
            pos[-c["pad"]:] = -1                        # padding behind the last request's tokens
        x = rnd(c["B"] * T, (c["hq"] + 2 * c["hkv"]) * c["dim"]).to(DT[c["dt"]])
        st["qkv"] = x                                   # one projection's rows: q, k and v are slices
        st["cos_sin"] = None
        if c["rope"] != "none":
            i = torch.arange(c["rot"] // 2, dtype=torch.float64, device="cuda")
            ang = torch.arange(max(lens), dtype=torch.float64, device="cuda")[:, None] * 10000.0 ** (-2 * i / c["rot"])
            st["cos_sin"] = torch.cat([ang.cos(), ang.sin()], 1).float()
    st["pos"] = pos
    return st


def _out_dt(c):
    return torch.float16 if c["dt"] == "f32" and c["op"] == "append" else DT[c["dt"]]


def _slices(c, x):
    a, b = c["hq"] * c["dim"], c["hkv"] * c["dim"]
    return (x[:, :a].unflatten(1, (c["hq"], c["dim"])), x[:, a:a + b].unflatten(1, (c["hkv"], c["dim"])),
            x[:, a + b:].unflatten(1, (c["hkv"], c["dim"])))


def prepare(case, seed):
    c, st = case, _make(case, seed)
    st["case"] = c
    dev = "cuda"
    if c["op"] == "linear":
        nib = (st.pop("q") & 15).to(torch.uint8)
        st["W"] = (nib[:, 0::2] | (nib[:, 1::2] << 4)).contiguous()
        st["y"] = st["y0"].clone()
        return st
    D, out = c["dim"], _out_dt(c)
    if c["op"] == "append":
        st["cache"] = torch.zeros(st["pages"], c["hkv"], c["page"] // 8, 9 * D, dtype=torch.uint8, device=dev)
        st["q"], st["k"], st["v"] = _slices(c, st["qkv"])
        st["q_out"] = torch.zeros(c["B"] * c["tokens"], c["hq"], D, dtype=out, device=dev)
    else:
        st["cache"] = _pack(c, st.pop("kq"), st.pop("ks"), st.pop("vq"), st.pop("vs"))
    if c["op"] == "attn":
        st["out"] = torch.empty(c["B"], c["hq"], D, dtype=out, device=dev)
        st["lse"] = torch.empty(c["B"], c["hq"], device=dev) if c["lse"] else None
        st["ws"] = torch.zeros(SCRATCH, dtype=torch.uint8, device=dev)
    else:
        st["k_out"] = torch.zeros(c["B"] * c["tokens"], c["hkv"], D, dtype=out, device=dev)
        st["v_out"] = torch.zeros_like(st["k_out"])
    return st


# ---------------------------------------------------------------------------- plain forms

def _nibbles(b):
    """uint8 [...] -> int codes -8..7 of the low and the high nibbles, float32."""
    return (b & 15).float() - 8, (b >> 4).float() - 8


def _read_blocks(c, blocks):
    """Values of octet blocks uint8 [..., 9 D]: K and V [..., 8][D], float32."""
    D, NG, lead = c["dim"], c["dim"] // 32, blocks.shape[:-1]
    lo, hi = _nibbles(blocks[..., :4 * D].unflatten(-1, (8, 4, NG, 4)))
    k = torch.empty(*lead, 8, 4, NG, 8, device=blocks.device)
    k[..., list(K_LO)], k[..., list(K_HI)] = lo, hi
    k = k.transpose(-3, -2)                                            # [8][g][c][8]
    lo, hi = _nibbles(blocks[..., 4 * D:8 * D].unflatten(-1, (16, NG, 8)))
    v = torch.empty(*lead, 8, NG, 2, 16, device=blocks.device)
    v[..., list(V_POS), :, 0, :] = lo.transpose(-3, -1)
    v[..., list(V_POS), :, 1, :] = hi.transpose(-3, -1)
    s = blocks[..., 8 * D:].contiguous().view(torch.float16).float().unflatten(-1, (2, NG, 8)).transpose(-2, -1)
    k = k.flatten(-2) * s[..., 0, :, :, None]                           # [8][g][32]
    v = v.flatten(-2) * s[..., 1, :, :, None]
    return k.flatten(-2), v.flatten(-2)


def _where(st, c):
    """Page, octet and place in the octet of each listed token, and whether it is one."""
    page, pos = c["page"], st["pos"].long()
    real = pos >= 0
    p = pos.clamp(min=0)
    return st["table"][st["seq"].long(), p // page].long().clamp(min=0), (p % page) // 8, p % 8, real


def _plain_read(st, c):
    pg, o, i, real = _where(st, c)
    k, v = _read_blocks(c, st["cache"][pg, :, o])                      # [T][H][8][D]
    at = i[:, None, None, None].expand(-1, c["hkv"], 1, c["dim"])
    keep = real[:, None, None]
    return [torch.where(keep, x.gather(2, at)[:, :, 0], 0.0).to(_out_dt(c)) for x in (k, v)]


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


def _plain_append(st, c):
    D, NG, H = c["dim"], c["dim"] // 32, c["hkv"]
    pg, o, i, real = _where(st, c)
    pg, o, i = pg[real], o[real], i[real]
    st["q_out"][real] = _plain_rotate(st, c, st["q"])[real].to(st["q_out"].dtype)
    flat = st["cache"].view(-1)
    base = (pg * H * (c["page"] // 8) + o) * 9 * D
    base = (base[:, None] + torch.arange(H, device=flat.device) * (c["page"] // 8) * 9 * D)[..., None]   # [T][H][1]
    i = i[:, None, None]
    kq, ks = _quant(_plain_rotate(st, c, st["k"])[real])
    vq, vs = _quant(st["v"][real])
    ku = (kq + 8).to(torch.uint8).unflatten(-1, (NG, 4, 8))
    kb = (ku[..., list(K_LO)] | (ku[..., list(K_HI)] << 4)).transpose(-3, -2).flatten(-3)
    flat[base + i * (D // 2) + torch.arange(D // 2, device=flat.device)] = kb
    vu = (vq + 8).to(torch.uint8).unflatten(-1, (NG, 2, 16))
    vb = (vu[..., 0, :] | (vu[..., 1, :] << 4)).transpose(-2, -1).flatten(-2)         # [n][g]
    byte = torch.tensor([V_POS.index(p) for p in range(8)], device=flat.device)[i]
    flat[base + 4 * D + torch.arange(D // 2, device=flat.device) * 8 + byte] = vb
    half = flat.view(torch.float16)
    g8 = torch.arange(NG, device=flat.device) * 8
    half[(base + 8 * D) // 2 + g8 + i] = ks
    half[(base + 8 * D + D // 2) // 2 + g8 + i] = vs
    return [st["q_out"]] + _plain_read(st, c)


def _plain_linear(st, c):
    n, d = c["n"], c["d"]
    w = torch.stack([st["W"] & 15, st["W"] >> 4], -1).view(n, d).float()
    w = torch.where(w > 7, w - 16, w).unflatten(1, (-1, c["group"])) * st["s"].float()[..., None]
    y = st["x"].float() @ w.flatten(1).t()
    if c["bias"]:
        y = y + st["bias"]
    return st["y0"] + y if c["acc"] else y


def _plain_attn(st, c):
    B, D, H, G = c["B"], c["dim"], c["hkv"], c["hq"] // c["hkv"]
    k, v = _read_blocks(c, st["cache"][st["table"].long().clamp(min=0)])   # [B][pages][H][page/8][8][D]
    k, v = (x.transpose(1, 2).reshape(B * H, -1, D) for x in (k, v))
    q = st["q"].float().view(B * H, G, D)
    s = torch.matmul(q, k.transpose(1, 2).contiguous()).view(B, H, G, -1) / math.sqrt(D)
    p = torch.arange(s.shape[-1], device=s.device)
    seen = p < st["lens"][:, None]
    if c["window"]:
        seen = seen & (p >= st["starts"][:, None])
    s = s.masked_fill(~seen[:, None, None], -math.inf)
    m = s.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, 0.0, m)
    e = (s - m).exp()
    l = e.sum(-1, keepdim=True)
    o = torch.matmul(e.view(B * H, G, -1), v).view(B, H, G, D) / torch.where(l > 0, l, 1.0)
    out = [o.reshape(B, c["hq"], D).to(DT[c["dt"]])]
    return out + [(m + l.log()).view(B, c["hq"])] if c["lse"] else out


def run(state):
    st, c = state, state["case"]
    if own:
        return _own(st, c)
    return {"linear": _plain_linear, "attn": _plain_attn, "append": _plain_append, "read": _plain_read}[c["op"]](st, c)


def _own(st, c):
    from activation_sparse_ffn_amd import _abi as A
    if c["op"] == "linear":
        if c["acc"]:
            st["y"].copy_(st["y0"])                     # the residual stream as the layer finds it
        A.sfx_linear_q4(st["x"], st["W"], st["s"], st["y"], bias=st["bias"], accumulate=c["acc"])
        return st["y"]
    if c["op"] == "attn":
        A.sfx_attn_q4(st["q"], st["cache"], st["table"], st["lens"], st["out"], st["ws"], starts=st["starts"],
                      lse=st["lse"])
        return [st["out"], st["lse"]] if c["lse"] else [st["out"]]
    if c["op"] == "append":
        A.sfx_kv_append_q4(st["q"], st["k"], st["v"], st["pos"], st["table"], st["cache"], st["q_out"], seq=st["seq"],
                           cos_sin=st["cos_sin"], interleaved=c["rope"] == "pairs")
    A.sfx_kv_read_q4(st["pos"], st["table"], st["cache"], st["k_out"], st["v_out"], seq=st["seq"])
    return ([st["q_out"]] if c["op"] == "append" else []) + [st["k_out"], st["v_out"]]


# ---------------------------------------------------------------------------- 64 bits

def exact(case, seed):
    c, st = case, _make(case, seed)
    if c["op"] == "linear":
        w = st["q"].double().reshape(c["n"], -1, c["group"]) * st["s"].double().unsqueeze(2)
        y = torch.matmul(st["x"].double(), w.reshape(c["n"], -1).T)
        y = y + st["bias"].double() if c["bias"] else y
        return y + st["y0"].double() if c["acc"] else y
    H, D = c["hkv"], c["dim"]

    def values(q, s):
        return (q.double().reshape(*q.shape[:-1], -1, 32) * s.double().unsqueeze(-1)).reshape(q.shape)

    if c["op"] == "attn":
        G, outs, lses = c["hq"] // H, [], []
        starts = st["starts"].tolist() if c["window"] else [0] * c["B"]
        for b, n in enumerate(st["lens"].tolist()):
            if n <= starts[b]:
                outs.append(torch.zeros(c["hq"], D, dtype=torch.float64, device="cuda"))
                lses.append(torch.full((c["hq"],), -math.inf, dtype=torch.float64, device="cuda"))
                continue
            ids = st["table"][b][:-(-n // c["page"])].long()
            o, ls = [], []
            for h in range(H):
                k = values(st["kq"][ids, h], st["ks"][ids, h]).reshape(-1, D)[starts[b]:n]
                v = values(st["vq"][ids, h], st["vs"][ids, h]).reshape(-1, D)[starts[b]:n]
                s = st["q"][b, h * G:(h + 1) * G].double() @ k.T / D ** 0.5
                ls.append(torch.logsumexp(s, 1))
                o.append(torch.exp(s - ls[-1][:, None]) @ v)
            outs.append(torch.cat(o))
            lses.append(torch.cat(ls))
        return [torch.stack(outs), torch.stack(lses)] if c["lse"] else [torch.stack(outs)]
    T = c["B"] * c["tokens"]
    pos, real = st["pos"].tolist(), (st["pos"] >= 0).double().reshape(T, 1, 1)
    if c["op"] == "read":
        p = st["pos"].long()
        ids = st["table"][st["seq"].long(), p // c["page"]].long()
        return [values(q[ids, :, p % c["page"]], s[ids, :, p % c["page"]])
                for q, s in ((st["kq"], st["ks"]), (st["vq"], st["vs"]))]
    q, k, v = (x.double() for x in _slices(c, st["qkv"]))
    if c["rope"] != "none":
        r = c["rot"]
        cs = st["cos_sin"].double()[torch.tensor([max(p, 0) for p in pos], device="cuda")]
        z = torch.complex(cs[:, :r // 2], cs[:, r // 2:]).reshape(T, 1, -1)

        def turn(x):
            if c["rope"] == "half":
                y = torch.complex(x[..., :r // 2].contiguous(), x[..., r // 2:r].contiguous()) * z
                return torch.cat((y.real, y.imag, x[..., r:]), 2)
            y = torch.view_as_complex(x[..., :r].reshape(T, -1, r // 2, 2).contiguous()) * z
            return torch.cat((torch.view_as_real(y).reshape(T, -1, r), x[..., r:]), 2)
        q, k = turn(q), turn(k)

    def held(x):
        g = x.reshape(T, H, -1, 32)
        s = (g.abs().max(-1, keepdim=True).values / torch.tensor(7.0, dtype=torch.float64, device="cuda")).half().double()
        u = torch.clamp(torch.round(g / torch.where(s == 0, 1.0, s)), -8, 7)
        return (u * s).reshape(T, H, D)
    return [q * real, held(k) * real, held(v) * real]
