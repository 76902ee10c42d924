"""Cases and plain forms of the operators of a paged KV cache, in bf16 and in 4 bits.

What a serving loop does with new tokens: their keys and values go into the
pages of a cache with the rotation applied on the way (``append``; into a cache
of 4 bits, read back as a prompt's next chunk reads it: ``append4``), and the
tokens attend over the pages: over a sliding window and the first tokens, one
token or a few drafted ones at a time (``window``), and over a cache held in 4
bits (``cache4``).

A 4-bit cache holds, per key and KV head, groups of 32 adjacent elements as
e2m1 codes (0, 0.5, 1, 1.5, 2, 3, 4, 6 with a sign) and one bf16 scale a group,
the group's largest magnitude over 6. Byte (d / 16) g + 2 c + b of a row holds
elements 32 c + 4 g + 2 b (low half) and the next one (high half), g < 8, b < 2.

``run`` computes an operator in its plain form, with elementary tensor
operations in float32 (angles in float64), or, with ``own`` set, through the
library. ``exact`` evaluates the same definition in float64, one request at a
time.
"""

import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def listed():
    return [
        # One decode step of 64 requests out of the fused QKV projection.
        {"name": "append_decode_b64", "op": "append", "dtype": "bf16", "B": 64, "Hq": 32, "Hkv": 8,
         "N": 1, "d": 128, "rot": 128, "layout": "half", "fused": True, "ragged": False,
         "before": 512, "page": 16, "shifted": False},
        # Two long prompts into an empty cache.
        {"name": "append_prompt_n8192", "op": "append", "dtype": "bf16", "B": 2, "Hq": 32,
         "Hkv": 8, "N": 8192, "d": 128, "rot": 128, "layout": "half", "fused": True,
         "ragged": False, "before": 0, "page": 16, "shifted": False},
        # A padded batch of float32 chunks behind what is cached, at positions
        # that an eviction has moved away from the rows.
        {"name": "append_f32_n777", "op": "append", "dtype": "f32", "B": 3, "Hq": 6, "Hkv": 2,
         "N": 777, "d": 64, "rot": 32, "layout": "interleaved", "fused": False, "ragged": True,
         "before": 300, "page": 48, "shifted": True},
        # One decode step of 64 short requests into 4 bits.
        {"name": "append4_decode_b64", "op": "append4", "dtype": "bf16", "B": 64, "Hq": 32,
         "Hkv": 8, "N": 1, "d": 128, "rot": 128, "layout": "half", "fused": True, "ragged": False,
         "before": 128, "page": 16, "shifted": False},
        # The next chunk of four long prompts into 4 bits, and all keys so far
        # back for the attention of the chunk.
        {"name": "append4_chunk_n2048", "op": "append4", "dtype": "bf16", "B": 4, "Hq": 32,
         "Hkv": 8, "N": 2048, "d": 128, "rot": 128, "layout": "half", "fused": True,
         "ragged": False, "before": 6144, "page": 16, "shifted": False},
        # A padded batch of short prompts, half of each head turned.
        {"name": "append4_n333_d64", "op": "append4", "dtype": "bf16", "B": 2, "Hq": 16, "Hkv": 4,
         "N": 333, "d": 64, "rot": 32, "layout": "interleaved", "fused": False, "ragged": True,
         "before": 40, "page": 24, "shifted": True},
        # Four requests behind a short window: latency.
        {"name": "window_b4_w128", "op": "window", "B": 4, "Hq": 16, "Hkv": 2, "T": 1, "d": 64,
         "L": 1000, "left": 127, "global": 4, "page": 16},
        # A decode step of 64 long requests that see 1024 keys and four sinks.
        {"name": "window_b64_w1024", "op": "window", "B": 64, "Hq": 32, "Hkv": 8, "T": 1, "d": 128,
         "L": 16384, "left": 1023, "global": 4, "page": 16},
        # Four drafted tokens of 32 long requests over a wide window.
        {"name": "window_t4_b32_w4096", "op": "window", "B": 32, "Hq": 32, "Hkv": 8, "T": 4,
         "d": 128, "L": 32768, "left": 4095, "global": 4, "page": 64},
        # Three short requests with three drafted tokens: latency.
        {"name": "cache4_b3_l500", "op": "cache4", "B": 3, "Hq": 8, "Hkv": 4, "T": 3, "d": 64,
         "L": 500, "left": -1, "global": 0, "page": 24},
        # A decode step of 64 requests of mixed length.
        {"name": "cache4_b64_l8192", "op": "cache4", "B": 64, "Hq": 32, "Hkv": 8, "T": 1, "d": 128,
         "L": 8191, "left": -1, "global": 0, "page": 16},
        # Two requests at the far end of a long context.
        {"name": "cache4_b2_l131072", "op": "cache4", "B": 2, "Hq": 32, "Hkv": 8, "T": 1, "d": 128,
         "L": 131072, "left": -1, "global": 0, "page": 64},
    ]


def _spread(rng, lo, hi):
    """A whole number of [lo, hi], uniform in its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["append", "append4", "window", "cache4"])
    d = rng.choice([64, 128])
    Hkv = rng.choice([1, 2, 4, 8])
    G = rng.choice([1, 2, 4, 8])
    if op in ("append", "append4"):
        top = 8192 if op == "append" else 4096
        N = rng.choice([1, _spread(rng, 1, top)])
        B = _spread(rng, 1, max(1, min(64, 2 * top // N)))
        room = 512 if op == "append" else min(6144, max(40, 16384 // B))
        return {"op": op, "dtype": rng.choice(["bf16", "bf16", "f32"] if Hkv * G <= 16
                                              else ["bf16"]),
                "B": B, "Hq": min(32, Hkv * G), "Hkv": Hkv, "N": N, "d": d,
                "rot": rng.choice([d, d // 2]), "layout": rng.choice(["half", "interleaved"]),
                "fused": rng.random() < 0.5, "ragged": rng.random() < 0.5,
                "before": _spread(rng, 1, room), "page": rng.choice([16, 24, 48, 64]),
                "shifted": rng.random() < 0.5}
    T = rng.choice([1, 1, rng.randint(2, 8)])
    wide = 4096 if op == "window" else 131072
    keys = _spread(rng, 30, wide)
    B = _spread(rng, 1, max(1, min(64, 131072 // keys if op == "window" else 262144 // keys)))
    open_ = rng.random() < (0.3 if op == "window" else 0.6)
    return {"op": op, "B": B, "Hq": min(32, Hkv * G), "Hkv": Hkv, "T": T, "d": d,
            "L": keys if open_ else _spread(rng, keys, 8 * wide if op == "window" else wide),
            "left": -1 if open_ else max(0, keys - 1), "global": rng.choice([0, 1, 4, 20]),
            "page": rng.choice([16, 24, 48, 64])}


# ------------------------------------------------------------------ inputs


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _randn(g, *shape, dtype=torch.bfloat16):
    return torch.randn(*shape, generator=g, device="cuda").to(dtype)


def _lens(g, n, lo, hi):
    return torch.randint(lo, hi + 1, (n,), generator=g, device="cuda", dtype=torch.int32)


def _table(g, first, end, page, longest, total=None):
    """A block table of the pages that hold keys below ``first[0]`` or in
    [first[1], end) of each request, in a random order, -1 elsewhere, wide
    enough for ``longest`` keys, and the number of pages of the pool (three
    spare ones among them where it is not given)."""
    width = -(-longest // page)
    lo = torch.arange(width, device="cuda") * page
    held = (lo < end[:, None]) & ((lo < first[0][:, None]) | (lo + page > first[1][:, None]))
    total = int(held.sum()) + 3 if total is None else total
    order = torch.randperm(total, generator=g, device="cuda")
    at = (held.flatten().cumsum(0) - 1).view_as(held).clamp(min=0)
    return torch.where(held, order[at], -1).to(torch.int32).contiguous(), total


LEVELS = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def _quantise(x):
    """Codes uint8 [..., d / 2] and scales bf16 [..., d / 32] of float32 rows
    [..., d]; nearest, ties to the even code."""
    x = x.unflatten(-1, (-1, 32))
    s = (x.abs().amax(-1) / 6.0).to(torch.bfloat16)
    y = torch.where(s[..., None] == 0, 0.0, x / s.float()[..., None])
    m = y.abs()
    code = sum((m > b if i % 2 == 0 else m >= b).to(torch.uint8)
               for i, b in enumerate((0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0)))
    code = code + torch.signbit(y).to(torch.uint8) * 8
    c = code.unflatten(-1, (8, 2, 2)).movedim(-4, -3).contiguous()     # [..., g, c, b, half]
    return (c[..., 0] + c[..., 1] * 16).flatten(-3), s


def _pool4(g, total, Hkv, page, d):
    codes = torch.empty(total, Hkv, page, d // 2, dtype=torch.uint8, device="cuda")
    scales = torch.empty(total, Hkv, page, d // 32, dtype=torch.bfloat16, device="cuda")
    step = max(1, (1 << 26) // (Hkv * page * d))
    for i in range(0, total, step):
        n = min(step, total - i)
        codes[i:i + n], scales[i:i + n] = _quantise(
            _randn(g, n, Hkv, page, d, dtype=torch.bfloat16).float())
    return codes, scales


def _prepare_append(case, g):
    B, Hq, Hkv, N, d, page = (case[k] for k in ("B", "Hq", "Hkv", "N", "d", "page"))
    dt = DTYPES[case["dtype"]]
    if case["fused"]:
        qkv = _randn(g, B, N, Hq + 2 * Hkv, d, dtype=dt).transpose(1, 2)
        q, k, v = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
    else:
        q, k, v = (_randn(g, B, H, N, d, dtype=dt) for H in (Hq, Hkv, Hkv))
    new = _lens(g, B, max(1, N // 2), N) if case["ragged"] else _lens(g, B, N, N)
    lens = new + _lens(g, B, case["before"] // 2, case["before"])
    row = (lens - new)[:, None] + torch.arange(N, device="cuda", dtype=torch.int32)
    shift = _lens(g, B, 0, 100000)[:, None] if case["shifted"] else 0
    longest = N + case["before"]
    table, total = _table(g, (lens, lens), lens, page, longest, B * -(-longest // page) + 3)
    b, i = torch.nonzero(torch.arange(N, device="cuda") < new[:, None], as_tuple=True)
    r = case["rot"]
    s = {"q": q, "k": k, "v": v, "q_out": torch.zeros(B, Hq, N, d, dtype=dt, device="cuda"),
         "positions": (row + shift).contiguous() if case["shifted"] else None, "row": row,
         "inv_freq": 10000.0 ** (-torch.arange(0, r, 2, dtype=torch.float64, device="cuda") / r),
         "seq_lens": lens, "new_lens": new if case["ragged"] else None, "block_table": table,
         "tokens": (b, i), "longest": longest}
    if case["op"] == "append":
        return {**s, "pools": (_randn(g, total, Hkv, page, d, dtype=dt),
                               _randn(g, total, Hkv, page, d, dtype=dt))}
    shape = (B, Hkv, longest, d)
    return {**s, "pools": _pool4(g, total, Hkv, page, d) + _pool4(g, total, Hkv, page, d),
            "back": tuple(torch.zeros(shape, dtype=torch.bfloat16, device="cuda")
                          for _ in range(2))}


def _prepare_attend(case, g):
    B, Hq, Hkv, T, d, L, page = (case[k] for k in ("B", "Hq", "Hkv", "T", "d", "L", "page"))
    if case["op"] == "window":
        lens = _lens(g, B, max(T, L // 4), max(T, L))
    else:
        lens = _lens(g, B, T, max(T, L))
        lens[0] = max(T, L)
    zero = torch.zeros_like(lens)
    if case["left"] < 0:
        first = (zero, zero)
    else:                       # pages between the first tokens and the window are given back
        first = (zero + case["global"], (lens - T - case["left"]).clamp(min=0))
    table, total = _table(g, first, lens, page, max(T, L))
    s = {"q": _randn(g, B, Hq, T, d), "seq_lens": lens, "block_table": table,
         "longest": max(T, L)}
    if case["op"] == "window":
        return {**s, "pools": (_randn(g, total, Hkv, page, d), _randn(g, total, Hkv, page, d))}
    return {**s, "pools": _pool4(g, total, Hkv, page, d) + _pool4(g, total, Hkv, page, d)}


def prepare(case, seed):
    g = _gen(seed)
    make = _prepare_append if case["op"].startswith("append") else _prepare_attend
    return {"case": case, **make(case, g)}


# ------------------------------------------------------------------ plain forms


def _turned(x, s, case):
    """x [B, H, N, d] rotated by the tokens' positions, float32."""
    r = case["rot"]
    pos = s["row"] if s["positions"] is None else s["positions"]
    ang = pos.double()[:, None, :, None] * s["inv_freq"]
    cos, sin = ang.cos().float(), ang.sin().float()
    y = x.float()
    if case["layout"] == "half":
        a, b = y[..., :r // 2], y[..., r // 2:r]
        z = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    else:
        a, b = y[..., 0:r:2], y[..., 1:r:2]
        z = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    return torch.cat([z, y[..., r:]], -1)


def _plain_append(s):
    case, page = s["case"], s["case"]["page"]
    b, i = s["tokens"]
    q, k = _turned(s["q"], s, case), _turned(s["k"], s, case)
    s["q_out"][b, :, i] = q[b, :, i].to(s["q"].dtype)
    row = s["row"][b, i].long()
    at, slot = s["block_table"][b, row // page].long(), row % page
    k, v = k[b, :, i], s["v"][b, :, i].float()                  # [tokens, Hkv, d]
    if case["op"] == "append":
        kp, vp = s["pools"]
        kp[at, :, slot] = k.to(kp.dtype)
        vp[at, :, slot] = v.to(vp.dtype)
        return {"q": s["q_out"], "k": kp, "v": vp}
    kc, ks, vc, vs = s["pools"]
    kc[at, :, slot], ks[at, :, slot] = _quantise(k)
    vc[at, :, slot], vs[at, :, slot] = _quantise(v)
    j = torch.arange(s["longest"], device="cuda")
    live = (j < s["seq_lens"][:, None])[:, None, :, None]
    pages = s["block_table"][:, j // page].clamp(min=0).long()
    back = [torch.where(live, _values(c[pages, :, j % page], z[pages, :, j % page]).transpose(1, 2)
                        .to(torch.bfloat16), old)
            for c, z, old in ((kc, ks, s["back"][0]), (vc, vs, s["back"][1]))]
    return {"q": s["q_out"], "k": back[0], "v": back[1]}


def _values(codes, scales):
    """float32 rows [..., d] of codes [..., d / 2] and scales [..., d / 32]."""
    level = torch.tensor(LEVELS + tuple(-x for x in LEVELS), device=codes.device)
    x = torch.stack([level[(codes & 15).long()], level[(codes >> 4).long()]], -1)
    x = x.unflatten(-2, (8, -1, 2)).movedim(-4, -3)             # [..., c, g, b, half]
    return (x.flatten(-3) * scales.float()[..., None]).flatten(-2)


def _plain_attend(s):
    case, q = s["case"], s["q"]
    B, Hq, T, d = q.shape
    page, left, first = case["page"], case["left"], case["global"]
    n = s["seq_lens"][:, None].long()
    Hkv = s["pools"][0].shape[1]
    if left < 0:
        j = torch.arange(s["longest"], device="cuda").expand(B, -1)
        held = j < n
    else:                       # the first keys, then the windows of the T tokens
        near = n - T - left + torch.arange(left + T, device="cuda")
        j = torch.cat([torch.arange(first, device="cuda").expand(B, -1), near], 1)
        held = torch.cat([j[:, :first] < n, near >= first], 1)
    j = j.clamp(min=0)
    at = s["block_table"].gather(1, (j // page).clamp(max=s["block_table"].shape[1] - 1))
    at, slot = at.clamp(min=0).long(), j % page
    if case["op"] == "window":
        k, v = (x[at, :, slot].float() for x in s["pools"])
    else:
        kc, ks, vc, vs = (x[at, :, slot] for x in s["pools"])
        k, v = _values(kc, ks), _values(vc, vs)
    k, v = k.transpose(1, 2), v.transpose(1, 2)                 # [B, Hkv, keys, d]
    pos = n - T + torch.arange(T, device="cuda")                # [B, T]
    seen = j[:, None] <= pos[..., None]
    if left >= 0:
        seen = seen & (j[:, None] >= pos[..., None] - left)
    seen = (seen | (j[:, None] < first)) & held[:, None]
    sc = (q.float().view(B, Hkv, -1, d) @ k.transpose(2, 3) / math.sqrt(d)).view(
        B, Hkv, -1, T, j.shape[1]).masked_fill(~seen[:, None, None], -math.inf)
    top = sc.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, 0.0, top)
    e = (sc - top).exp()
    total = e.sum(-1, keepdim=True)
    o = (e.flatten(2, 3) @ v).view(*e.shape[:-1], d) / torch.where(total > 0, total, 1.0)
    return o.view(B, Hq, T, d).to(q.dtype), (top + total.log()).view(B, Hq, T)


def _own(s):
    import online_softmax_tiled_gb300 as ost
    case = s["case"]
    if case["op"] in ("append", "append4"):
        append = ost.cache_append if case["op"] == "append" else ost.cache_append4
        q = append(s["q"], s["k"], s["v"], *s["pools"], s["block_table"], s["seq_lens"],
                   inv_freq=s["inv_freq"], positions=s["positions"], new_lens=s["new_lens"],
                   interleaved=case["layout"] == "interleaved", out=s["q_out"])
        k, v = s["pools"] if case["op"] == "append" else ost.cache_read4(
            *s["pools"], s["block_table"], s["seq_lens"], out=s["back"])
        return {"q": q, "k": k, "v": v}
    decode = ost.decode_window if case["op"] == "window" else ost.decode_cache4
    return decode(s["q"], *s["pools"], s["block_table"], s["seq_lens"],
                  window_left=case["left"], n_global=case["global"])


def run(state):
    if own:
        return _own(state)
    if state["case"]["op"].startswith("append"):
        return _plain_append(state)
    return _plain_attend(state)


# ------------------------------------------------------------------ work


def work(case):
    c = case
    B, Hq, Hkv, d = (c[k] for k in ("B", "Hq", "Hkv", "d"))
    row4 = d // 2 + d // 16                                     # bytes of a 4-bit row
    if c["op"].startswith("append"):
        size = 2 if c["dtype"] == "bf16" else 4
        new = (max(1, c["N"] // 2) + c["N"]) / 2 if c["ragged"] else c["N"]
        n = new + 0.75 * c["before"]
        if c["op"] == "append":
            return {"bytes": B * new * (2 * Hq + 4 * Hkv) * d * size,
                    "flops": 3 * B * new * (Hq + Hkv) * c["rot"]}
        return {"bytes": B * new * ((2 * Hq + 2 * Hkv) * d * size + 2 * Hkv * row4) +
                B * n * 2 * Hkv * (row4 + 2 * d),
                "flops": B * new * (3 * (Hq + Hkv) * c["rot"] + 4 * Hkv * d) + B * n * 2 * Hkv * d}
    T, L = c["T"], c["L"]
    keys = 0.625 * L if c["op"] == "window" else (L + (B - 1) * (L + T) / 2) / B
    if c["left"] >= 0:
        keys = min(keys, c["left"] + T + c["global"])
    row = 2 * d if c["op"] == "window" else row4
    return {"bytes": B * Hkv * keys * 2 * row + B * Hq * T * (4 * d + 4),
            "flops": 4 * d * B * Hq * T * keys}


# ------------------------------------------------------------------ float64


def _exact_rows(s, which, b, h, keys):
    """Rows ``keys`` of request b, KV head h, of K (0) or V (1), float64."""
    keys = torch.as_tensor(keys, device="cuda")
    page = s["case"]["page"]
    at, slot = s["block_table"][b].long()[keys // page], keys % page
    if len(s["pools"]) == 2:
        return s["pools"][which][at, h, slot].double()
    codes, scales = (x[at, h, slot] for x in s["pools"][2 * which:2 * which + 2])
    d = 2 * codes.shape[1]
    e = torch.arange(d, device="cuda")
    byte = d // 16 * (e % 32 // 4) + 2 * (e // 32) + e % 4 // 2
    nib = (codes[:, byte].long() >> (4 * (e % 2))) % 16
    exp, man = nib % 8 // 2, (nib % 2).double()
    mag = torch.where(exp == 0, man / 2, (1 + man / 2) * 2.0 ** (exp - 1).double())
    return torch.where(nib >= 8, -mag, mag) * scales.double()[:, e // 32]


def _exact_turn(x, pos, s):
    """x [H, d] of one token at position pos."""
    r = s["case"]["rot"]
    w = torch.polar(torch.ones_like(s["inv_freq"]), pos * s["inv_freq"])
    half = s["case"]["layout"] == "half"
    z = torch.complex(*((x[..., :r // 2], x[..., r // 2:r]) if half
                        else (x[..., 0:r:2], x[..., 1:r:2]))) * w
    z = torch.cat([z.real, z.imag], -1) if half else torch.view_as_real(z).flatten(-2)
    return torch.cat([z, x[..., r:]], -1)


def _exact_levels(x):
    """The values that 4 bits hold in the place of x [..., d], float64."""
    x = x.unflatten(-1, (-1, 32))
    s = (x.abs().amax(-1, keepdim=True) / 6).to(torch.bfloat16).double()
    m = torch.where(s == 0, s, x.abs() / s).clamp(max=6)
    # the spacing of the levels is a half up to 2, one up to 4, two from there
    step = torch.where(m <= 2, 0.5, torch.where(m <= 4, 1.0, 2.0)).double()
    return (torch.copysign((m / step).round() * step, x) * s).flatten(-2)


def _exact_append(s):
    case, lens = s["case"], s["seq_lens"].tolist()
    N, page = case["N"], case["page"]
    new = [N] * case["B"] if s["new_lens"] is None else s["new_lens"].tolist()
    pos = s["row"] if s["positions"] is None else s["positions"]
    q_out = s["q_out"].double()
    out = [x.double() for x in (s["pools"] if case["op"] == "append" else s["back"])]
    for b, n in enumerate(lens):
        m, at = new[b], pos[b, :new[b], None].double()
        q_out[b, :, :m] = _exact_turn(s["q"][b, :, :m].double(), at, s)
        fresh = (_exact_turn(s["k"][b, :, :m].double(), at, s), s["v"][b, :, :m].double())
        row = torch.arange(n - m, n, device="cuda")
        for which, x in enumerate(fresh):
            if case["op"] == "append":
                out[which][s["block_table"][b].long()[row // page], :, row % page] = \
                    x.transpose(0, 1)
                continue
            for h in range(x.shape[0]):
                if n > m:
                    out[which][b, h, :n - m] = _exact_rows(s, which, b, h, range(n - m))
                out[which][b, h, n - m:n] = _exact_levels(x[h])
    return {"q": q_out, "k": out[0], "v": out[1]}


def _exact_attend(s):
    case, q = s["case"], s["q"].double()
    B, Hq, T, d = q.shape
    Hkv, left, first = s["pools"][0].shape[1], case["left"], case["global"]
    o, lse = torch.zeros_like(q), torch.full((B, Hq, T), -math.inf, dtype=q.dtype, device="cuda")
    for b, n in enumerate(s["seq_lens"].tolist()):
        lo = max(0, n - T - left) if left >= 0 else 0
        keys = torch.cat([torch.arange(min(first, lo)), torch.arange(lo, n)]).to("cuda")
        for h in range(Hkv):
            k, v = (_exact_rows(s, which, b, h, keys) for which in (0, 1))
            rows = slice(h * (Hq // Hkv), (h + 1) * (Hq // Hkv))
            for t in range(T):
                p = n - T + t
                seen = ((keys <= p) & ((keys >= p - left) | (left < 0))) | (keys < first)
                if not bool(seen.any()):
                    continue
                x = q[b, rows, t] @ k[seen].T * d ** -0.5
                lse[b, rows, t] = torch.logsumexp(x, -1)
                o[b, rows, t] = torch.softmax(x, -1) @ v[seen]
    return o, lse


def exact(case, seed):
    s = prepare(case, seed)
    return _exact_append(s) if case["op"].startswith("append") else _exact_attend(s)
