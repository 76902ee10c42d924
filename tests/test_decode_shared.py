"""Decode behind shared prefixes: oracle pins, refusals on the CPU, and the
GPU path against the float64 oracle.

Tolerance, per element: the output's bf16 rounding (half a step, 2^-8 of the
value); the rounding of each prefix probability to bf16 (2^-8 of p, so
2^-8 · Σ p|v|); and float32 arithmetic: a score is off by at most
(d + 2) · 2^-24 · scale · Σ|q k|, e = 2^-24 · 130 · 10 < 2^-13 for the inputs
here (Σ|q k| · scale below 10 with N(0, 1) inputs), which changes a
probability by 2e relative and LSE by e. With scale times 8 those terms are 8
times as large.
"""

import numpy as np
import pytest
import torch

import oracle
from workloads import random_like_shape, to_f64

DEV = "cuda:0"
INVALID, UNSUPPORTED, MISALIGNED, WORKSPACE = -1, -2, -3, -4


# ------------------------------------------------------------------ oracle


def _np_case(rng, B=3, Hq=4, Hkv=2, d=8, plens=(5, 0), start=(0, 2, 2), lens=(3, 0, 4)):
    q = rng.standard_normal((B, Hq, d))
    pool = rng.standard_normal((2, 12, Hkv, 4, d))
    pt = np.array([[3, 7], [1, 0]])
    bt = np.array([[2], [4], [5]])
    return q, pool[0], pool[1], pt, np.array(plens), np.array(start), bt, np.array(lens)


def test_oracle_equals_decode_of_the_joined_cache():
    rng = np.random.default_rng(0)
    q, kp, vp, pt, plens, start, bt, lens = _np_case(rng)
    o, lse = oracle.decode_shared(q, kp, vp, pt, plens, start, kp, vp, bt, lens, 0.3)
    # request 0: pages 3, 7 (5 keys), then page 2 (3 keys), as one page list of single keys
    rows = [(3, 0), (3, 1), (3, 2), (3, 3), (7, 0), (2, 0), (2, 1), (2, 2)]
    one = np.stack([kp[p, :, r] for p, r in rows])[:, :, None], \
        np.stack([vp[p, :, r] for p, r in rows])[:, :, None]
    want = oracle.decode_paged(q[:1], *one, np.arange(8)[None], np.array([8]), 1, 0.3)
    assert np.allclose(o[0], want[0][0]) and np.allclose(lse[0], want[1][0])
    # request 1: prefix alone; request 2 is in no group
    assert np.isfinite(lse[1]).all()
    want = oracle.decode_paged(q, kp, vp, bt, lens, 4, 0.3)
    assert np.allclose(o[2], want[0][2]) and np.allclose(lse[2], want[1][2])


def test_oracle_without_any_key():
    rng = np.random.default_rng(1)
    q, kp, vp, pt, plens, start, bt, lens = _np_case(rng, plens=(0, 0), lens=(0, 1, 0))
    o, lse = oracle.decode_shared(q, kp, vp, pt, plens, start, kp, vp, bt, lens, 1.0)
    assert np.all(o[[0, 2]] == 0) and np.all(np.isneginf(lse[[0, 2]]))
    assert np.allclose(o[1], np.repeat(vp[4, :, 0], 2, 0))      # one key: its value


# ------------------------------------------------------------------ refusals

P = 1 << 20


@pytest.fixture(scope="module")
def lib():
    import __graft_entry__
    __graft_entry__.build()
    import online_softmax_tiled_gb300 as ost
    return ost.lib()


SIZES = dict(B=4, Hq=8, Hkv=2, d=64, n_prefix=2, npp=9, pps=16, mpp=4, np_=20, ps=16, mp=3)


def _call(lib, ws=P, ws_bytes=None, scale=0.1, sp=0, so=0, ptrs=None, **kw):
    z = {**SIZES, **kw}
    a = [P] * 12
    for i, x in (ptrs or {}).items():
        a[i] = x
    if ws_bytes is None:
        ws_bytes = lib.attn_decode_shared_workspace_size(
            z["B"], z["Hq"], z["Hkv"], z["d"], z["n_prefix"], z["pps"], z["mpp"], z["ps"],
            z["mp"], sp, so)
    return lib.attn_decode_shared(*a, z["B"], z["Hq"], z["Hkv"], z["d"], z["n_prefix"], z["npp"],
                                  z["pps"], z["mpp"], z["np_"], z["ps"], z["mp"], scale, sp, so,
                                  ws, ws_bytes, None)


@pytest.mark.parametrize("kwargs,expected", [
    (dict(B=0), INVALID), (dict(Hkv=0), INVALID), (dict(Hq=7), INVALID), (dict(d=0), INVALID),
    (dict(n_prefix=0), INVALID), (dict(npp=0), INVALID), (dict(pps=0), INVALID),
    (dict(mpp=0), INVALID), (dict(np_=0), INVALID), (dict(ps=0), INVALID), (dict(mp=0), INVALID),
    (dict(sp=-1), INVALID), (dict(so=-1), INVALID), (dict(scale=0.0), INVALID),
    (dict(scale=float("nan")), INVALID), (dict(scale=float("inf")), INVALID),
    *[(dict(ptrs={i: None}), INVALID) for i in range(11)],
    (dict(d=96), UNSUPPORTED), (dict(Hq=6), UNSUPPORTED), (dict(Hq=32), UNSUPPORTED),
    (dict(pps=12), UNSUPPORTED), (dict(B=65536), UNSUPPORTED),
    (dict(pps=1 << 20, mpp=2048), UNSUPPORTED), (dict(ps=1 << 20, mp=2048), UNSUPPORTED),
    (dict(npp=2 ** 30), UNSUPPORTED), (dict(sp=70000), UNSUPPORTED),
    *[(dict(ptrs={i: P + 8}), MISALIGNED) for i in (0, 1, 2, 6, 7, 10)],
    *[(dict(ptrs={i: P + 2}), MISALIGNED) for i in (3, 4, 5, 8, 9, 11)],
    (dict(ws=None), WORKSPACE), (dict(ws_bytes=100), WORKSPACE), (dict(ws=P + 16), MISALIGNED),
])
def test_refusals(lib, kwargs, expected):
    assert _call(lib, **kwargs) == expected


def test_workspace_size(lib):
    def need(sp, so, pps=16, mpp=64, ps=16, mp=32, B=4, d=64):
        return lib.attn_decode_shared_workspace_size(B, 8, 2, d, 1, pps, mpp, ps, mp, sp, so)

    def a256(x):
        return (x + 255) // 256 * 256
    # 1024 prefix keys are 8 tiles of 128: three splits of three tiles at most
    n = 4 * 8 * (3 + 5)
    assert need(3, 5) == a256(n * 64 * 4) + 2 * a256(n * 4)
    assert need(5, 5) == need(4, 5)         # two tiles a split either way
    assert need(0, 0) > 0
    assert need(3, 5, B=0) == 0 and need(3, 5, d=80) == 0 and need(3, 5, pps=12) == 0
    assert need(3, 5, pps=12, mpp=1) > 0    # one page: any size


# ------------------------------------------------------------------ GPU


def _case(B, Hq, Hkv, d, start, plens, ppage, lens, page, seed, one_pool=False):
    """Device tensors; unused page rows, unlisted pages and table entries
    past a request's own hold NaN and -1."""
    g = torch.Generator().manual_seed(seed)

    def pool(lens, page, extra):
        n = [-(-x // page) for x in lens]
        total = sum(n) + extra
        k, v = (random_like_shape((total, Hkv, page, d), torch.bfloat16, seed + i) for i in (1, 2))
        order = torch.randperm(total, generator=g).to(torch.int32)
        width = max(1, max(n))
        table = torch.full((len(lens), width), -1, dtype=torch.int32)
        used = torch.zeros(total, page, dtype=torch.bool)
        at = 0
        for r, x in enumerate(lens):
            table[r, :n[r]] = order[at:at + n[r]]
            for i in range(n[r]):
                used[order[at + i], :min(page, x - i * page)] = True
            at += n[r]
        mask = ~used[:, None, :, None].expand_as(k)
        return k.masked_fill(mask, float("nan")), v.masked_fill(mask, float("nan")), table
    if one_pool:
        assert ppage == page
        k, v, table = pool([*plens, *lens], page, 3)
        kp, vp, pt, bt = k, v, table[:len(plens)].contiguous(), table[len(plens):].contiguous()
    else:
        kp, vp, pt = pool(plens, ppage, 2)
        k, v, bt = pool(lens, page, 2)
    x = {"q": random_like_shape((B, Hq, d), torch.bfloat16, seed), "k_prefix": kp, "v_prefix": vp,
         "prefix_table": pt, "prefix_lens": torch.tensor(plens, dtype=torch.int32),
         "prefix_start": torch.tensor(start, dtype=torch.int32), "k_pages": k, "v_pages": v,
         "block_table": bt, "seq_lens": torch.tensor(lens, dtype=torch.int32)}
    return {n: t.to(DEV) for n, t in x.items()}


ORDER = ("q", "k_prefix", "v_prefix", "prefix_table", "prefix_lens", "prefix_start", "k_pages",
         "v_pages", "block_table", "seq_lens")


def _ref(x, scale, absolute=False):
    a = [to_f64(x[n]) if x[n].is_floating_point() else x[n].cpu().numpy() for n in ORDER]
    if absolute:
        a[2], a[7] = np.abs(a[2]), np.abs(a[7])
    return oracle.decode_shared(*a, scale)


def _check(o, lse, x, scale, rows=slice(None)):
    d = x["q"].shape[-1]
    e = 2.0 ** -13 * max(1.0, scale * d ** 0.5)
    o_ref, lse_ref = (t[rows] for t in _ref(x, scale))
    spread = _ref(x, scale, True)[0][rows]
    err = np.abs(to_f64(o)[rows] - o_ref)
    assert np.all(err <= 2.0 ** -8 * np.abs(o_ref) + (2.0 ** -8 + 2 * e) * spread + 1e-30), err.max()
    empty = np.isneginf(lse_ref)
    got = to_f64(lse)[rows]
    assert np.array_equal(np.isneginf(got), empty)
    assert np.all(np.abs(got[~empty] - lse_ref[~empty]) <= e)


CASES = [  # B, Hq, Hkv, d, start, prefix lengths, prefix page, own lengths, page
    (4, 16, 2, 64, [0, 4], [500], 16, [3, 17, 40, 0], 16),
    (1, 1, 1, 64, [0, 1], [1], 1, [0], 16),                      # one key in all
    (2, 8, 8, 128, [0, 2], [128], 128, [1, 0], 1),               # one full tile; MHA
    (3, 4, 2, 128, [0, 3], [129], 129, [5, 0, 33], 32),          # one odd page, two tiles
    (5, 8, 2, 128, [0, 2, 2, 4], [300, 77, 0], 8, [10, 0, 7, 0, 9], 8),  # empty group and
                                                                 # prefix; one request outside
    (6, 8, 1, 64, [1, 3, 5], [1000, 260], 48, [0, 200, 31, 32, 0, 500], 48),  # first and last
                                                                 # request without a prefix
    (70, 16, 4, 128, [0, 70], [700], 64, [i % 50 for i in range(70)], 16),   # 280 rows: two runs
    (40, 32, 4, 64, [0, 3, 40], [257, 640], 32, [7] * 40, 16),   # a small and a large group
    (40, 2, 2, 64, list(range(41)), [(i * 37) % 200 for i in range(40)], 16,
     [i % 3 for i in range(40)], 16),                            # forty groups of one request
]


@pytest.mark.gpu
@pytest.mark.parametrize("B,Hq,Hkv,d,start,plens,ppage,lens,page", CASES)
@pytest.mark.parametrize("sp,so", [(0, 0), (1, 1), (3, 2)])
def test_parity(ost, B, Hq, Hkv, d, start, plens, ppage, lens, page, sp, so):
    x = _case(B, Hq, Hkv, d, start, plens, ppage, lens, page, seed=B + 7 * Hq + d)
    for scale in (d ** -0.5, 8 * d ** -0.5):
        o, lse = ost.decode_shared(*(x[n] for n in ORDER), sp, so, scale)
        torch.cuda.synchronize()
        _check(o, lse, x, scale)


@pytest.mark.gpu
def test_one_pool_for_prefixes_and_own_keys(ost):
    x = _case(9, 8, 2, 128, [0, 5, 9], [1500, 900], 16, [0, 1, 16, 17, 100, 5, 6, 7, 8], 16, 5,
              one_pool=True)
    o, lse = ost.decode_shared(*(x[n] for n in ORDER))
    torch.cuda.synchronize()
    _check(o, lse, x, 128 ** -0.5)


@pytest.mark.gpu
@pytest.mark.parametrize("B,n_prefix", [(16, 1), (80, 1)])
def test_long_prefix_with_more_pages_than_are_cached(ost, B, n_prefix):
    """One split over 5000 keys in pages of 8: 625 table entries."""
    x = _case(B, 4, 1, 64, [0, B], [5000], 8, [3] * B, 8, 11)
    for sp in (1, 0):
        o, lse = ost.decode_shared(*(x[n] for n in ORDER), sp, 0)
        torch.cuda.synchronize()
        _check(o, lse, x, 0.125)


@pytest.mark.gpu
def test_agrees_with_paged_decode_of_the_joined_tables(ost):
    """Prefix and own pages as one table of decode_paged: the same attention
    (prefix of whole pages)."""
    x = _case(12, 8, 2, 128, [0, 12], [1024], 16, [30] * 12, 16, 3, one_pool=True)
    o, lse = ost.decode_shared(*(x[n] for n in ORDER))
    table = torch.cat([x["prefix_table"].expand(12, -1)[:, :64], x["block_table"]], 1).contiguous()
    o2, lse2 = ost.decode_paged(x["q"], x["k_pages"], x["v_pages"], table, x["seq_lens"] + 1024, 8)
    torch.cuda.synchronize()
    assert np.max(np.abs(to_f64(lse) - to_f64(lse2))) <= 2 * 2.0 ** -13
    assert np.max(np.abs(to_f64(o) - to_f64(o2))) <= 2e-2 * np.max(np.abs(to_f64(o2)))


@pytest.mark.gpu
def test_bad_tables_are_flagged_not_read(ost):
    args = (6, 4, 2, 64, [0, 2, 4, 6], [200, 100, 300], 16, [20, 0, 9, 9, 40, 1], 16, 21)
    good = _case(*args)
    want = _ref(good, 0.125)
    def run(**change):
        x = {n: t.clone() for n, t in good.items()}
        for n, (at, v) in change.items():
            x[n][at] = v
        o, lse = ost.decode_shared(*(x[n] for n in ORDER))
        torch.cuda.synchronize()
        assert ost.attn_sync_status() == -7 and ost.attn_sync_status() == 0
        return to_f64(o), to_f64(lse)

    def close(got, rows):
        assert np.max(np.abs(got[0][rows] - want[0][rows])) <= 2e-2
        assert np.max(np.abs(got[1][rows] - want[1][rows])) <= 1e-3
    close(run(prefix_table=((1, 3), 99)), [0, 1, 4, 5])
    close(run(prefix_table=((1, 3), -5)), [0, 1, 4, 5])
    close(run(prefix_lens=(2, 305)), [0, 1, 2, 3])
    close(run(prefix_lens=(2, -1)), [0, 1, 2, 3])
    close(run(block_table=((4, 1), 50)), [0, 1, 2, 3, 5])
    close(run(seq_lens=(4, 1000)), [0, 1, 2, 3, 5])
    close(run(prefix_start=(3, 7)), [0, 1, 2, 3])
    close(run(prefix_start=(0, -1)), [2, 3, 4, 5])
    run(prefix_start=(1, 5))                     # decreasing: reported, nothing out of bounds


@pytest.mark.gpu
@pytest.mark.parametrize("page", [16, 200])
def test_offsets_past_32_bits(ost, page):
    """Pages past 2^32 bytes (2^31 elements) of their pool give what the same
    pages at its front give; 200 keys: one page a table row."""
    Hkv, d = 8, 128
    total = (1 << 32) // (Hkv * page * d * 2) + 64
    k = torch.zeros(total, Hkv, page, d, dtype=torch.bfloat16, device=DEV)
    v = torch.zeros_like(k)
    g = torch.Generator().manual_seed(3)
    for x in (k, v):
        x[:16] = torch.randn(16, Hkv, page, d, generator=g).to(torch.bfloat16).to(DEV)
        x[-16:] = x[:16]
    q = torch.randn(3, 32, d, generator=g).to(torch.bfloat16).to(DEV)
    n = 1 if page == 200 else 4
    table = torch.arange(16, dtype=torch.int32, device=DEV)
    lens = torch.tensor([page * n - 3, 0, 17], dtype=torch.int32, device=DEV)
    plen = torch.tensor([page * n - 5], dtype=torch.int32, device=DEV)
    start = torch.tensor([0, 3], dtype=torch.int32, device=DEV)

    def run(at):
        t = table + at
        return ost.decode_shared(q, k, v, t[12:12 + n].view(1, n).contiguous(), plen, start, k, v,
                                 t[:3 * n].view(3, n).contiguous(), lens)
    near, far = run(0), run(total - 16)
    torch.cuda.synchronize()
    assert ost.attn_sync_status() == 0
    assert torch.equal(near[0], far[0]) and torch.equal(near[1], far[1])
    assert bool((near[0] != 0).any())


@pytest.mark.gpu
def test_streams_graphs_and_calls_at_once(ost):
    """Two calls at once on two streams (their own workspaces), a captured
    and replayed call, and many calls back to back on one workspace."""
    x = [_case(8, 8, 2, 128, [0, 8], [900], 16, [5 + i] * 8, 16, 30 + i) for i in range(2)]
    want = [ost.decode_shared(*(y[n] for n in ORDER)) for y in x]
    torch.cuda.synchronize()
    side = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = []
    for y, s in zip(x, side):
        with torch.cuda.stream(s):
            got.append([ost.decode_shared(*(y[n] for n in ORDER)) for _ in range(4)])
    torch.cuda.synchronize()
    for w, g in zip(want, got):
        assert all(torch.equal(w[0], o) and torch.equal(w[1], lse) for o, lse in g)
    n = ost.attn_decode_shared_workspace_size(x[0]["q"], x[0]["k_prefix"], x[0]["prefix_table"],
                                              x[0]["k_pages"], x[0]["block_table"])
    ws = torch.full((n,), 255, dtype=torch.uint8, device=DEV)     # NaN everywhere
    outs = [ost.decode_shared(*(x[i % 2][n] for n in ORDER), workspace=ws) for i in range(6)]
    torch.cuda.synchronize()
    assert all(torch.equal(outs[i][0], want[i % 2][0]) for i in range(6))
    o, lse = torch.empty_like(want[0][0]), torch.empty_like(want[0][1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ost.attn_decode_shared(*(x[0][n] for n in ORDER), o, lse, 128 ** -0.5, 0, 0, ws)
    for i in (1, 0):
        for name in ORDER:
            if name in ("q", "k_pages", "v_pages", "seq_lens", "block_table", "k_prefix",
                        "v_prefix", "prefix_table"):
                x[0][name].copy_(_case(8, 8, 2, 128, [0, 8], [900], 16, [5 + i] * 8, 16,
                                       30 + i)[name])
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(o, want[i][0]) and torch.equal(lse, want[i][1])


@pytest.mark.gpu
def test_binding_refusals(ost):
    x = _case(4, 4, 2, 64, [0, 4], [100], 16, [5] * 4, 16, 1)
    for bad in (dict(q=x["q"].float()), dict(seq_lens=x["seq_lens"].long()),
                dict(prefix_start=x["prefix_start"][:1]), dict(seq_lens=x["seq_lens"][:2]),
                dict(v_prefix=x["v_prefix"][:1]), dict(k_pages=x["k_pages"].transpose(1, 2)),
                dict(q=x["q"].cpu())):
        with pytest.raises((ValueError, TypeError)):
            ost.decode_shared(*({**x, **bad}[n] for n in ORDER))
    with pytest.raises(ost.AttnError):
        ost.decode_shared(*(x[n] for n in ORDER), workspace=torch.empty(256, device=DEV,
                                                                        dtype=torch.uint8))


def _exact_scores(x, seed):
    """The case with scores that float32 holds exactly: queries are the first
    unit vector, keys differ in their first element only, between -3 and 0."""
    g = torch.Generator().manual_seed(seed)
    x["q"].zero_()
    x["q"][..., 0] = 1
    for n in ("k_prefix", "k_pages"):
        k0 = -3 * torch.rand(x[n].shape[:-1], generator=g)
        x[n] = torch.zeros_like(x[n])
        x[n][..., 0] = k0.to(DEV)
    return x


@pytest.mark.gpu
@pytest.mark.parametrize("B,Hq,Hkv,d,plen", [(4, 8, 2, 64, 40), (6, 8, 1, 128, 300),
                                             (70, 16, 4, 128, 129), (40, 32, 4, 64, 77)])
@pytest.mark.parametrize("sp", [0, 1])
def test_prefix_probabilities_keep_more_than_bf16(ost, B, Hq, Hkv, d, plen, sp):
    """As accurate as the paged decode of the same keys. Scores s are exact
    here, so beside the output's own rounding (half a step, 2^-8 of the value)
    a probability is off by two bf16 parts' 2^-16, by the scaling to log2
    units (three roundings of a number below 4.5, 2^-22 of the probability
    each) and by the exponential and the division by the sum (2^-21 together),
    and a sum of 300 float32 terms, rounded or cut, by 300 · 2^-23: below
    2^-14 in all."""
    x = _exact_scores(_case(B, Hq, Hkv, d, [0, B], [plen], 8, [i % 3 for i in range(B)], 16,
                            seed=plen), plen)
    o, _ = ost.decode_shared(*(x[n] for n in ORDER), sp, 0, 1.0)
    torch.cuda.synchronize()
    o_ref, spread = _ref(x, 1.0)[0], _ref(x, 1.0, True)[0]
    err = np.abs(to_f64(o) - o_ref)
    assert np.all(err <= 2.0 ** -8 * np.abs(o_ref) + 2.0 ** -14 * spread), \
        (err - 2.0 ** -8 * np.abs(o_ref)).max()


@pytest.mark.gpu
@pytest.mark.parametrize("B,Hq,Hkv,d,start,plens,ppage,lens,page", [
    (5, 32, 4, 128, [0, 2, 5], [300, 150], 16, [7, 0, 33, 64, 5], 16),
    (40, 16, 2, 128, [0, 40], [700], 64, [i % 50 for i in range(40)], 16),   # 320 rows: two runs
])
@pytest.mark.parametrize("sp,so", [(0, 0), (3, 2)])
def test_eight_query_heads_of_128(ost, B, Hq, Hkv, d, start, plens, ppage, lens, page, sp, so):
    x = _case(B, Hq, Hkv, d, start, plens, ppage, lens, page, seed=B)
    o, lse = ost.decode_shared(*(x[n] for n in ORDER), sp, so)
    torch.cuda.synchronize()
    _check(o, lse, x, d ** -0.5)


@pytest.mark.gpu
@pytest.mark.parametrize("B,Hq,Hkv,d,plens", [(16, 8, 2, 64, [4096]), (64, 16, 4, 128, [6400]),
                                              (40, 16, 4, 128, [8192, 1600])])
@pytest.mark.parametrize("wider", [3, 16])
def test_a_wider_table_changes_nothing(ost, B, Hq, Hkv, d, plens, wider):
    """Splits follow each prefix's own length, not what its table could hold:
    the same bits from a table with many unused columns."""
    start = [0, B] if len(plens) == 1 else [0, B // 3, B]
    x = _case(B, Hq, Hkv, d, start, plens, 16, [5] * B, 16, seed=B)
    o, lse = ost.decode_shared(*(x[n] for n in ORDER))
    torch.cuda.synchronize()
    _check(o, lse, x, d ** -0.5)
    pt = x["prefix_table"]
    x["prefix_table"] = torch.cat([pt, torch.full_like(pt, -1).repeat(1, wider - 1)], 1)
    o2, lse2 = ost.decode_shared(*(x[n] for n in ORDER))
    torch.cuda.synchronize()
    assert torch.equal(o, o2) and torch.equal(lse, lse2)


@pytest.mark.gpu
@pytest.mark.parametrize("d", [64, 128])
def test_more_splits_than_a_warp_has_lanes(ost, d):
    """Splits asked for by the caller, more than are ever chosen: a row's
    partials are merged in several rounds, at every remainder of eight."""
    x = _case(5, 8, 2, d, [0, 2, 5], [9000, 4500], 16, [1500, 0, 33, 700, 1100], 16, seed=d)
    for sp, so in ((70, 40), (71, 1), (1, 47), (65535, 3)):
        o, lse = ost.decode_shared(*(x[n] for n in ORDER), sp, so)
        torch.cuda.synchronize()
        _check(o, lse, x, d ** -0.5)
