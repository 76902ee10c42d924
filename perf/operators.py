"""Cases and plain forms of the operators around the KV cache.

Four operators, as one serving or training step uses them: the rotation of
queries and keys by their positions (and its transpose for gradients), decode
of a batch whose requests share long prefixes, the attention weight each
cached key has received, and the eviction of the keys that received least.

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
        # One decode step of 64 requests at positions of their own, out of the
        # fused QKV projection; frequencies blended for a 16x longer context.
        {"name": "rope_decode_b64", "op": "rope", "dtype": "bf16", "B": 64, "Hq": 32, "Hkv": 8,
         "N": 1, "d": 128, "rot": 128, "layout": "half", "scaling": "ramp", "fused": True,
         "inverse": False, "max_pos": 131072},
        # Queries and keys of a long prompt out of the fused projection.
        {"name": "rope_prefill_n8192", "op": "rope", "dtype": "bf16", "B": 2, "Hq": 32, "Hkv": 8,
         "N": 8192, "d": 128, "rot": 128, "layout": "half", "scaling": "none", "fused": True,
         "inverse": False, "max_pos": 8192},
        # Backward of a training step: gradients of half-rotated heads turned
        # back, interleaved pairs.
        {"name": "rope_backward_n4096", "op": "rope", "dtype": "bf16", "B": 2, "Hq": 16, "Hkv": 4,
         "N": 4096, "d": 128, "rot": 64, "layout": "interleaved", "scaling": "linear",
         "fused": False, "inverse": True, "max_pos": 32768},
        # A ragged float32 sequence far into a long context.
        {"name": "rope_f32_n777", "op": "rope", "dtype": "f32", "B": 3, "Hq": 6, "Hkv": 2,
         "N": 777, "d": 64, "rot": 32, "layout": "half", "scaling": "base", "fused": False,
         "inverse": False, "max_pos": 1000000},
        # Four samples continuing one short prompt: latency.
        {"name": "shared_b4_p500", "op": "shared", "B": 4, "Hq": 16, "Hkv": 2, "d": 64,
         "prefixes": 1, "P": 500, "own_mean": 20, "page": 16},
        # 64 requests behind one long system prompt.
        {"name": "shared_b64_p8192", "op": "shared", "B": 64, "Hq": 32, "Hkv": 8, "d": 128,
         "prefixes": 1, "P": 8192, "own_mean": 512, "page": 16},
        # 96 requests over three long documents of different length.
        {"name": "shared_b96_3x32768", "op": "shared", "B": 96, "Hq": 32, "Hkv": 8, "d": 128,
         "prefixes": 3, "P": 32768, "own_mean": 257, "page": 64},
        # The weight every cached key received in one decode step, added to
        # what it had, over the paged cache of a large batch.
        {"name": "weights_decode_b64", "op": "weights", "B": 64, "Hq": 32, "Hkv": 8, "T": 1,
         "L": 4096, "d": 128, "page": 16, "decay": 1.0},
        # The last 64 tokens of two long prompts as observers.
        {"name": "weights_window_l16384", "op": "weights", "B": 2, "Hq": 32, "Hkv": 8, "T": 64,
         "L": 16384, "d": 128, "page": 0, "decay": 0.0},
        # Every token of a prompt as an observer.
        {"name": "weights_prompt_n4096", "op": "weights", "B": 1, "Hq": 16, "Hkv": 4, "T": 4096,
         "L": 4096, "d": 128, "page": 0, "decay": 0.0},
        # Three short caches cut to 128 keys: latency.
        {"name": "evict_l1000", "op": "evict", "B": 3, "Hkv": 2, "L": 1000, "d": 64, "keep": 128,
         "sink": 4, "recent": 32, "page": 0},
        # Eight long paged caches cut to an eighth.
        {"name": "evict_l32768", "op": "evict", "B": 8, "Hkv": 8, "L": 32768, "d": 128,
         "keep": 4096, "sink": 4, "recent": 64, "page": 16},
    ]


def _spread(rng, lo, hi):
    """A whole number of [lo, hi], uniform in its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rope", "shared", "weights", "evict"])
    d = rng.choice([64, 128])
    Hkv = rng.choice([1, 2, 4, 8])
    G = rng.choice([1, 2, 4, 8])
    if op == "rope":
        N = _spread(rng, 1, 8192)
        B = _spread(rng, 1, max(1, min(64, 16384 // N)))
        rot = rng.choice([d, d // 2, d // 4])
        return {"op": op, "dtype": rng.choice(["bf16", "bf16", "f32"]), "B": B,
                "Hq": min(32, Hkv * G), "Hkv": Hkv, "N": N, "d": d, "rot": rot,
                "layout": rng.choice(["half", "interleaved"]),
                "scaling": rng.choice(["none", "linear", "base", "ramp"]),
                "fused": rng.random() < 0.5, "inverse": rng.random() < 0.4,
                "max_pos": _spread(rng, 8192, 1000000)}
    if op == "shared":
        P = _spread(rng, 100, 32768)
        B = _spread(rng, 2, 96)
        return {"op": op, "B": B, "Hq": min(32, Hkv * G), "Hkv": Hkv, "d": d,
                "prefixes": rng.randint(1, min(3, B)), "P": P,
                "own_mean": _spread(rng, 10, 500), "page": rng.choice([16, 32, 48, 64])}
    if op == "weights":
        T = rng.choice([1, 1, _spread(rng, 2, 200), _spread(rng, 200, 4000)])
        L = _spread(rng, max(T, 50), 16384 if T <= 200 else 4096)
        B = _spread(rng, 1, 64) if T == 1 else 1 if T > 200 else rng.randint(1, 2)
        if B * L > 64 * 4096:
            B = max(1, 64 * 4096 // L)
        Hq = min(32 if T <= 200 else 16, Hkv * G)
        return {"op": op, "B": B, "Hq": Hq, "Hkv": min(Hkv, Hq), "T": T, "L": L, "d": d,
                "page": rng.choice([0, 16, 64]), "decay": rng.choice([0.0, 1.0, 0.9])}
    L = _spread(rng, 100, 32768)
    keep = _spread(rng, 32, max(33, min(L, 4096)))
    return {"op": op, "B": _spread(rng, 1, 8), "Hkv": Hkv, "L": L, "d": d, "keep": keep,
            "sink": rng.choice([0, 1, 4]), "recent": rng.randint(0, keep // 2),
            "page": rng.choice([0, 16, 48])}


# ------------------------------------------------------------------ inputs


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _randn(g, *shape, dtype=torch.bfloat16):
    return torch.randn(*shape, generator=g, device="cuda").to(dtype)


def _frequencies(case):
    """Angle per position of each pair, float64 [rot / 2]: what the model's
    configuration says once, kept for all calls."""
    r, base = case["rot"], 10000.0
    i = torch.arange(0, r, 2, dtype=torch.float64, device="cuda")
    if case["scaling"] == "base":
        base *= 8.0 ** (r / (r - 2))
    f = base ** (-i / r)
    if case["scaling"] == "linear":
        f = f / 4.0
    if case["scaling"] == "ramp":
        turns = 8192 * f / (2 * math.pi)
        keep = ((turns - 1.0) / (32.0 - 1.0)).clamp(0.0, 1.0)
        f = f * keep + f / 16.0 * (1.0 - keep)
    return f


def _pool(g, counts, width, page, Hkv, d):
    """Pages of K and V for tables of ``counts`` pages, handed out in a
    random order; a table has ``width`` entries, -1 past its own pages."""
    total = sum(counts) + 3
    kp = _randn(g, total, Hkv, page, d)
    vp = _randn(g, total, Hkv, page, d)
    order = torch.randperm(total, generator=g, device="cuda").to(torch.int32)
    n = torch.tensor(counts, device="cuda")
    at = torch.cumsum(n, 0) - n
    col = torch.arange(width, device="cuda")
    table = torch.where(col < n[:, None], order[(at[:, None] + col).clamp(max=total - 1)], -1)
    return kp, vp, table.to(torch.int32).contiguous()


def _lens(g, n, lo, hi):
    return torch.randint(lo, hi + 1, (n,), generator=g, device="cuda", dtype=torch.int32)


def _prepare_rope(case, g):
    B, Hq, Hkv, N, d = (case[k] for k in ("B", "Hq", "Hkv", "N", "d"))
    dt = DTYPES[case["dtype"]]
    if case["fused"]:
        qkv = _randn(g, B, N, Hq + 2 * Hkv, d, dtype=dt)
        q, k = qkv[:, :, :Hq].transpose(1, 2), qkv[:, :, Hq:Hq + Hkv].transpose(1, 2)
    else:
        q, k = _randn(g, B, Hq, N, d, dtype=dt), _randn(g, B, Hkv, N, d, dtype=dt)
    start = torch.randint(0, max(1, case["max_pos"] - N), (B, 1), generator=g, device="cuda")
    pos = (start + torch.arange(N, device="cuda")).to(torch.int32)
    return {"q": q, "k": k, "positions": pos, "inv_freq": _frequencies(case),
            "magnitude": 1.0 + 0.1 * math.log(16.0) if case["scaling"] == "ramp" else 1.0}


def _prepare_shared(case, g):
    B, Hq, Hkv, d, n_p, P, page = (case[k] for k in ("B", "Hq", "Hkv", "d", "prefixes", "P",
                                                     "page"))
    plens = _lens(g, n_p, max(1, P // 2), P)
    plens[0] = P
    lens = _lens(g, B, 0, 2 * case["own_mean"])
    cut = torch.randperm(B - 1, generator=g, device="cuda")[:n_p - 1].sort().values + 1
    start = torch.cat([cut.new_zeros(1), cut, cut.new_full((1,), B)]).to(torch.int32)
    pc = [-(-n // page) for n in plens.tolist()]
    oc = [-(-n // page) for n in lens.tolist()]
    pw, ow = -(-P // page), -(-2 * case["own_mean"] // page)
    kp, vp, table = _pool(g, pc + oc, max(pw, ow), page, Hkv, d)
    return {"q": _randn(g, B, Hq, d), "k_pages": kp, "v_pages": vp,
            "prefix_table": table[:n_p, :pw].contiguous(), "prefix_lens": plens,
            "prefix_start": start, "block_table": table[n_p:, :ow].contiguous(),
            "seq_lens": lens, "largest_group": int((start[1:] - start[:-1]).max())}


def _cache_rows(pages, table):
    """The rows of each request's table in order: [B, Hkv, width * page, d]."""
    B, width = table.shape
    x = pages[table.clamp(min=0).long()]
    return x.permute(0, 2, 1, 3, 4).reshape(B, pages.shape[1], width * pages.shape[2], -1)


def _prepare_weights(case, g):
    B, Hq, Hkv, T, L, d, page = (case[k] for k in ("B", "Hq", "Hkv", "T", "L", "d", "page"))
    if page:
        lens = _lens(g, B, max(T, L // 2), L)
        k, _, table = _pool(g, [-(-n // page) for n in lens.tolist()], -(-L // page), page,
                            Hkv, d)
        rows = table.shape[1] * page
    else:
        lens, table, rows = torch.full((B,), L, dtype=torch.int32, device="cuda"), None, L
        k = _randn(g, B, Hkv, L, d)
    q = _randn(g, B, Hq, T, d)
    lse = torch.empty(B, Hq, T, device="cuda")
    j, i = torch.arange(rows, device="cuda"), torch.arange(T, device="cuda")
    for b in range(B):
        kb = (_cache_rows(k, table[b:b + 1]) if page else k[b:b + 1])[0].float()
        seen = j <= lens[b] - T + i[:, None]
        s = q[b].float().view(Hkv, -1, d) @ kb.transpose(1, 2) / math.sqrt(d)
        lse[b] = s.view(Hq, T, rows).masked_fill(~seen, -math.inf).logsumexp(-1)
    prev = torch.rand(B, Hkv, rows, generator=g, device="cuda") * 4
    return {"q": q, "k": k, "lse": lse, "prev": prev, "out": torch.zeros_like(prev),
            "block_table": table, "seq_lens": lens}


def _prepare_evict(case, g):
    B, Hkv, L, d, page, keep = (case[k] for k in ("B", "Hkv", "L", "d", "page", "keep"))
    if page:
        lens = _lens(g, B, max(1, L // 2), L)
        k, v, table = _pool(g, [-(-n // page) for n in lens.tolist()], -(-L // page), page,
                            Hkv, d)
        rows = table.shape[1] * page
    else:
        lens, table, rows = torch.full((B,), L, dtype=torch.int32, device="cuda"), None, L
        k, v = _randn(g, B, Hkv, L, d), _randn(g, B, Hkv, L, d)
    # accumulated weights: many small ones, few large ones, some never looked at
    s = torch.rand(B, Hkv, rows, generator=g, device="cuda").pow(6) * 30
    s = torch.where(torch.rand(B, Hkv, rows, generator=g, device="cuda") < 0.05, 0.0, s)
    out = {"k": torch.zeros(B, Hkv, keep, d, dtype=k.dtype, device="cuda"),
           "v": torch.zeros(B, Hkv, keep, d, dtype=k.dtype, device="cuda"),
           "scores": torch.zeros(B, Hkv, keep, device="cuda"),
           "indices": torch.zeros(B, Hkv, keep, dtype=torch.int32, device="cuda"),
           "lens": torch.zeros(B, dtype=torch.int32, device="cuda")}
    return {"k": k, "v": v, "scores": s, "block_table": table, "seq_lens": lens, "out": out}


def prepare(case, seed):
    g = _gen(seed)
    make = {"rope": _prepare_rope, "shared": _prepare_shared, "weights": _prepare_weights,
            "evict": _prepare_evict}[case["op"]]
    return {"case": case, **make(case, g)}


# ------------------------------------------------------------------ plain forms


def _plain_rope(s):
    case = s["case"]
    r = case["rot"]
    ang = s["positions"].double()[:, None, :, None] * s["inv_freq"]
    cos = (ang.cos() * s["magnitude"]).float()
    sin = (ang.sin() * (-s["magnitude"] if case["inverse"] else s["magnitude"])).float()

    def turn(x):
        y = x.float()
        if case["layout"] == "half":
            a, b = y[..., :r // 2], y[..., r // 2:r]
            z = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
        else:
            a, b = y[..., 0:r:2], y[..., 1:r:2]
            z = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
        return torch.cat([z, y[..., r:]], -1).to(x.dtype).contiguous()

    return turn(s["q"]), turn(s["k"])


def _plain_shared(s):
    q, d = s["q"], s["q"].shape[-1]
    B, Hq = q.shape[:2]
    Hkv = s["k_pages"].shape[1]
    qs = q.float().view(B, Hkv, Hq // Hkv, d) / math.sqrt(d)
    # the requests of a prefix side by side
    start, M, n_p = s["prefix_start"].long(), s["largest_group"], s["prefix_lens"].numel()
    at = torch.arange(B, device=q.device)
    group = torch.bucketize(at, start[1:], right=True)
    slot = at - start[group]
    qg = qs.new_zeros(n_p, Hkv, M, Hq // Hkv, d)
    qg[group, :, slot] = qs
    kp, vp = (_cache_rows(s[n], s["prefix_table"]).float() for n in ("k_pages", "v_pages"))
    P = kp.shape[2]
    sp = (qg.flatten(2, 3) @ kp.transpose(2, 3)).view(n_p, Hkv, M, -1, P)
    gone = torch.arange(P, device=q.device) >= s["prefix_lens"][:, None]
    sp = sp.masked_fill(gone[:, None, None, None], -math.inf)
    ko, vo = (_cache_rows(s[n], s["block_table"]).float() for n in ("k_pages", "v_pages"))
    so = qs @ ko.transpose(2, 3)
    past = torch.arange(ko.shape[2], device=q.device) >= s["seq_lens"][:, None]
    so = so.masked_fill(past[:, None, None], -math.inf)
    top = torch.maximum(sp.amax(-1)[group, :, slot], so.amax(-1))
    top = torch.where(top == -math.inf, 0.0, top)
    tg = sp.new_zeros(sp.shape[:-1])
    tg[group, :, slot] = top
    ep, eo = (sp - tg[..., None]).exp(), (so - top[..., None]).exp()
    total = ep.sum(-1)[group, :, slot] + eo.sum(-1)
    og = (ep.flatten(2, 3) @ vp).view(n_p, Hkv, M, -1, d)
    o = (og[group, :, slot] + eo @ vo) / torch.where(total > 0, total, 1.0)[..., None]
    return o.view(B, Hq, d).to(q.dtype), (top + total.log()).view(B, Hq)


def _plain_weights(s):
    q, d = s["q"], s["q"].shape[-1]
    B, Hq, T = q.shape[:3]
    k = s["k"] if s["block_table"] is None else _cache_rows(s["k"], s["block_table"])
    Hkv, rows = k.shape[1], k.shape[2]
    sc = q.float().view(B, Hkv, -1, d) @ k.float().transpose(2, 3) / math.sqrt(d)
    j = torch.arange(rows, device=q.device)
    seen = j <= (s["seq_lens"][:, None] - T + torch.arange(T, device=q.device))[..., None]
    p = (sc.view(B, Hkv, -1, T, rows) - s["lse"].view(B, Hkv, -1, T, 1)).exp()
    w = p.masked_fill(~seen[:, None, None], 0.0).sum((2, 3))
    if s["case"]["decay"]:
        w = w + s["case"]["decay"] * s["prev"]
    return torch.where((j < s["seq_lens"][:, None])[:, None], w, s["out"])


def _plain_evict(s):
    case, out = s["case"], s["out"]
    keep = case["keep"]
    k, v = s["k"], s["v"]
    if s["block_table"] is not None:
        k, v = _cache_rows(k, s["block_table"]), _cache_rows(v, s["block_table"])
    rows = k.shape[2]
    n = s["seq_lens"][:, None, None]
    j = torch.arange(rows, device=k.device)
    held = ((j < case["sink"]) | (j >= n - case["recent"])) & (j < n)
    # rank: held rows, then by score; ties and order by index (stable sorts)
    rank = torch.where(held, math.inf, torch.where(j < n, s["scores"], -1.0))
    first = torch.sort(rank, dim=-1, descending=True, stable=True).indices[..., :keep]
    chosen = first.sort(dim=-1).values
    pad = chosen.new_zeros(*chosen.shape[:2], keep - chosen.shape[2])
    m = n.clamp(max=keep)
    slot = torch.arange(keep, device=k.device)
    chosen = torch.cat([chosen, pad], -1)
    live = slot < m

    def rows_of(x, old):
        return torch.where(live[..., None], x.gather(2, chosen[..., None].expand(
            *chosen.shape, x.shape[-1])), old)

    return {"k": rows_of(k, out["k"]), "v": rows_of(v, out["v"]),
            "scores": torch.where(live, s["scores"].gather(2, chosen), out["scores"]),
            "indices": torch.where(live, chosen, -1).to(torch.int32),
            "lens": m[:, 0, 0].to(torch.int32)}


def _own(s):
    import online_softmax_tiled_gb300 as ost
    case = s["case"]
    if case["op"] == "rope":
        return ost.rope(s["q"], s["k"], s["positions"], s["inv_freq"],
                        interleaved=case["layout"] == "interleaved", magnitude=s["magnitude"],
                        inverse=case["inverse"])
    if case["op"] == "shared":
        return ost.decode_shared(s["q"], s["k_pages"], s["v_pages"], s["prefix_table"],
                                 s["prefix_lens"], s["prefix_start"], s["k_pages"], s["v_pages"],
                                 s["block_table"], s["seq_lens"])
    if case["op"] == "weights":
        return ost.key_weights(s["q"], s["k"], s["lse"], out=s["out"],
                               prev=s["prev"] if case["decay"] else None, decay=case["decay"],
                               seq_lens=s["seq_lens"], block_table=s["block_table"])
    out = s["out"]
    ost.evict(s["k"], s["v"], s["scores"], case["keep"], n_sink=case["sink"],
              n_recent=case["recent"], seq_lens=s["seq_lens"], block_table=s["block_table"],
              out=(out["k"], out["v"], out["scores"], out["indices"], out["lens"]))
    return out


def run(state):
    if own:
        return _own(state)
    return {"rope": _plain_rope, "shared": _plain_shared, "weights": _plain_weights,
            "evict": _plain_evict}[state["case"]["op"]](state)


# ------------------------------------------------------------------ work


def work(case):
    c = case
    if c["op"] == "rope":
        size = 2 if c["dtype"] == "bf16" else 4
        rows = c["B"] * (c["Hq"] + c["Hkv"]) * c["N"]
        return {"bytes": 2 * rows * c["d"] * size + 4 * c["B"] * c["N"] + 4 * c["rot"],
                "flops": 3 * rows * c["rot"]}
    if c["op"] == "shared":
        B, Hq, Hkv, d, P, mean = (c[k] for k in ("B", "Hq", "Hkv", "d", "P", "own_mean"))
        held = P + (c["prefixes"] - 1) * 0.75 * P       # expected lengths
        mean_p = held / c["prefixes"]
        return {"bytes": 4 * d * Hkv * (held + B * mean) + B * Hq * (4 * d + 4),
                "flops": 4 * d * B * Hq * (mean_p + mean)}
    if c["op"] == "weights":
        B, Hq, Hkv, T, d = (c[k] for k in ("B", "Hq", "Hkv", "T", "d"))
        n = (max(T, c["L"] // 2) + c["L"]) / 2 if c["page"] else c["L"]
        pairs = T * (n - T) + T * (T + 1) / 2
        return {"bytes": B * Hkv * n * (2 * d + (8 if c["decay"] else 4)) +
                B * Hq * T * (2 * d + 4), "flops": 2 * d * B * Hq * pairs}
    n = (max(1, c["L"] // 2) + c["L"]) / 2 if c["page"] else c["L"]
    kept = min(n, c["keep"])
    return {"bytes": c["B"] * c["Hkv"] * (4 * n + kept * (8 * c["d"] + 8)), "flops": 0}


# ------------------------------------------------------------------ float64


def _row_list(pages, table, n):
    """Rows 0 .. n - 1 behind one table row, float64 [Hkv, n, d]."""
    t = torch.arange(n, device=pages.device)
    size = pages.shape[2]
    return pages[table.long()[t // size], :, t % size].double().transpose(0, 1)


def _exact_rope(s):
    case, r = s["case"], s["case"]["rot"]
    spin = torch.polar(torch.full_like(s["inv_freq"], s["magnitude"]).expand(
        *s["positions"].shape, -1).contiguous(),
        torch.einsum("bn,f->bnf", s["positions"].double(), s["inv_freq"]))[:, None]
    if case["inverse"]:
        spin = spin.conj()

    def turn(x):
        y = x.double()
        if case["layout"] == "half":
            z = torch.complex(y[..., :r // 2].contiguous(), y[..., r // 2:r].contiguous()) * spin
            return torch.cat([z.real, z.imag, y[..., r:]], -1)
        z = torch.view_as_complex(y[..., :r].unflatten(-1, (-1, 2)).contiguous()) * spin
        return torch.cat([torch.view_as_real(z).flatten(-2), y[..., r:]], -1)

    return turn(s["q"]), turn(s["k"])


def _exact_shared(s):
    q, d = s["q"].double(), s["q"].shape[-1]
    B, Hq = q.shape[:2]
    o, lse = torch.zeros_like(q), torch.full((B, Hq), -math.inf, dtype=q.dtype, device=q.device)
    start, plens, lens = (s[n].tolist() for n in ("prefix_start", "prefix_lens", "seq_lens"))
    for p, n_p in enumerate(plens):
        kp, vp = (_row_list(s[n], s["prefix_table"][p], n_p) for n in ("k_pages", "v_pages"))
        for b in range(start[p], start[p + 1]):
            kb, vb = (torch.cat([x, _row_list(s[n], s["block_table"][b], lens[b])], 1)
                      for x, n in ((kp, "k_pages"), (vp, "v_pages")))
            if kb.shape[1] == 0:
                continue
            x = torch.einsum("hgd,hnd->hgn", q[b].view(kb.shape[0], -1, d), kb) * d ** -0.5
            lse[b] = torch.logsumexp(x, -1).flatten()
            o[b] = torch.einsum("hgn,hnd->hgd", torch.softmax(x, -1), vb).reshape(Hq, d)
    return o, lse


def _exact_weights(s):
    q, out = s["q"], s["out"].double()
    T, d = q.shape[2:]
    Hkv = s["k"].shape[1]
    G = q.shape[1] // Hkv
    for b, n in enumerate(s["seq_lens"].tolist()):
        kb = s["k"][b, :, :n].double() if s["block_table"] is None else \
            _row_list(s["k"], s["block_table"][b], n)
        hidden = torch.ones(T, n, device=q.device, dtype=torch.bool).triu(n - T + 1)
        for h in range(q.shape[1]):
            x = q[b, h].double() @ kb[h // G].T * d ** -0.5 - s["lse"][b, h].double()[:, None]
            w = x.masked_fill(hidden, -math.inf).exp().sum(0)
            if h % G == 0:
                w = w + s["case"]["decay"] * s["prev"][b, h // G, :n].double()
                out[b, h // G, :n] = w
            else:
                out[b, h // G, :n] += w
    return out


def _exact_evict(s):
    case, old = s["case"], s["out"]
    keep, lens = case["keep"], s["seq_lens"].tolist()
    res = {n: old[n].double() if n in ("k", "v", "scores") else old[n].clone() for n in old}
    res["indices"].fill_(-1)
    for b, n in enumerate(lens):
        m = min(n, keep)
        res["lens"][b] = m
        rest = torch.arange(n)[case["sink"]:n - case["recent"]] if n > keep else torch.arange(0)
        for h in range(s["scores"].shape[1]):
            sc = s["scores"][b, h, :n].cpu().double()
            want = keep - case["sink"] - case["recent"]
            worst = [(-float(x), int(i)) for x, i in zip(sc[rest], rest)]
            gone = torch.tensor([i for _, i in sorted(worst)[want:]], dtype=torch.long)
            mask = torch.ones(n, dtype=torch.bool)
            mask[gone] = False
            at = mask.nonzero().flatten().to(s["k"].device)
            for name in ("k", "v"):
                x = s[name][b, h, :n] if s["block_table"] is None else \
                    s[name][s["block_table"][b].long()[at // case["page"]], h, at % case["page"]]
                res[name][b, h, :m] = (x[at] if s["block_table"] is None else x).double()
            res["scores"][b, h, :m] = sc[at.cpu()].to(at.device)
            res["indices"][b, h, :m] = at.to(torch.int32)
    return res


def exact(case, seed):
    s = prepare(case, seed)
    return {"rope": _exact_rope, "shared": _exact_shared, "weights": _exact_weights,
            "evict": _exact_evict}[case["op"]](s)
