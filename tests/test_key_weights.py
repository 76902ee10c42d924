"""Attention weight per cached key: oracle pins, refusals on the CPU, and the
GPU kernels against the float64 oracle.

Tolerance, relative to the sum of the (positive) weights of a key: a score is
off by at most (d + 2) · 2^-24 · scale · Σ|q k| < 2^-13 for these inputs
(Σ|q k| · scale below 10, d <= 128); the exponent in log2 units, below 60 in
size, is rounded three times (3 · 60 · 2^-24 < 2^-16), exp2 is good to 2^-22,
and adding R of them one after another loses at most R · 2^-24. decay · prev
adds 2^-23 of its size.
"""

import numpy as np
import pytest
import torch

import oracle
from workloads import random_like_shape, to_f64

DEV = "cuda:0"
INVALID, UNSUPPORTED, MISALIGNED, WORKSPACE = -1, -2, -3, -4


# ------------------------------------------------------------------ oracle


def test_oracle_weights_are_the_probabilities():
    """Summed over all keys, every query that sees a key gives one per head;
    each single weight is the softmax's."""
    rng = np.random.default_rng(0)
    q, k = rng.standard_normal((4, 3, 8)), rng.standard_normal((2, 7, 8))
    s = np.stack([oracle.scores(q[h], k[h // 2], 0.4, True) for h in range(4)])
    lse = oracle.logsumexp_rows(s.reshape(-1, 7)).reshape(4, 3)
    w = oracle.key_weights(q, k, lse, 0.4)
    assert np.allclose(w.sum(1), 2 * 3)
    p = oracle.softmax_rows(s.reshape(-1, 7)).reshape(4, 3, 7)
    assert np.allclose(w, p.sum(1).reshape(2, 2, 7).sum(1))
    one = oracle.key_weights(q[:, -1:], k, lse[:, -1:], 0.4, causal=False)
    assert np.allclose(one, p[:, 2].reshape(2, 2, 7).sum(1))


def test_oracle_rows_without_keys_give_nothing():
    q, k = np.ones((1, 4, 8)), np.ones((1, 2, 8))
    lse = np.array([[-np.inf, -np.inf, 8.0, 8.0 + np.log(2)]])
    assert np.allclose(oracle.key_weights(q, k, lse, 1.0), [[1.5, 0.5]])


# ------------------------------------------------------------------ refusals

P = 1 << 30


@pytest.fixture(scope="module")
def lib():
    import __graft_entry__
    __graft_entry__.build()
    import online_softmax_tiled_gb300 as ost
    return ost.lib()


def _call(lib, q=P, k=2 * P, lse=3 * P, prev=4 * P, out=5 * P, lens=6 * P, table=None, B=2, Hq=4,
          Hkv=2, T=3, L=100, num_pages=0, page=0, mp=0, out_len=100, d=64, scale=0.1, decay=1.0,
          causal=1, ws=None, nb=0):
    return lib.attn_key_weights(q, k, lse, prev, out, lens, table, B, Hq, Hkv, T, L, num_pages,
                                page, mp, out_len, d, scale, decay, causal, ws, nb, None)


PAGED = dict(table=7 * P, num_pages=9, page=16, mp=4)
NAN, INF = float("nan"), float("inf")


@pytest.mark.parametrize("kwargs,expected", [
    (dict(B=0), INVALID), (dict(Hq=3), INVALID), (dict(Hkv=0), INVALID), (dict(T=0), INVALID),
    (dict(L=0), INVALID), (dict(out_len=0), INVALID), (dict(lens=None, out_len=99), INVALID),
    (dict(q=None), INVALID), (dict(k=None), INVALID), (dict(lse=None), INVALID),
    (dict(out=None), INVALID), (dict(scale=NAN), INVALID), (dict(scale=-INF), INVALID),
    (dict(decay=NAN), INVALID), (dict(causal=2), INVALID),
    (dict(prev=5 * P + 16), INVALID), (dict(prev=5 * P - 2 * 2 * 100 * 4 + 4), INVALID),
    ({**PAGED, "lens": None}, INVALID), ({**PAGED, "num_pages": 0}, INVALID),
    ({**PAGED, "page": 0}, INVALID), ({**PAGED, "mp": -1}, INVALID),
    (dict(d=96), UNSUPPORTED), ({**PAGED, "page": 12}, UNSUPPORTED),
    (dict(B=300, Hkv=300, Hq=300), UNSUPPORTED), (dict(T=2 ** 30, Hq=8), UNSUPPORTED),
    ({**PAGED, "mp": 1 << 20, "page": 2048}, UNSUPPORTED),
    ({**PAGED, "num_pages": 2 ** 31 - 1}, UNSUPPORTED),
    (dict(q=P + 8), MISALIGNED), (dict(k=P + 2), MISALIGNED), (dict(lse=P + 2), MISALIGNED),
    (dict(prev=P + 1), MISALIGNED), (dict(out=5 * P + 2), MISALIGNED),
    (dict(lens=P + 2), MISALIGNED), ({**PAGED, "table": P + 2}, MISALIGNED),
    (dict(T=4096, L=4096, out_len=4096), WORKSPACE),
    (dict(T=4096, L=4096, out_len=4096, ws=8 * P, nb=1000), WORKSPACE),
    (dict(T=4096, L=4096, out_len=4096, ws=8 * P + 16, nb=1 << 24), MISALIGNED),
])
def test_refusals(lib, kwargs, expected):
    assert _call(lib, **kwargs) == expected


def test_workspace_size(lib):
    f = lib.attn_key_weights_workspace_size
    assert f(2, 8, 2, 64, 4096, 4096) == 0            # 256 rows stay in shared memory
    assert f(2, 8, 2, 4096, 4096, 4096) % (2 * 2 * 4096 * 4) == 0
    assert f(2, 8, 2, 4096, 4096, 4096) > 0
    assert f(0, 8, 2, 4096, 4096, 4096) == 0 and f(2, 7, 2, 4096, 4096, 4096) == 0


# ------------------------------------------------------------------ GPU


def _check(ost, B, Hq, Hkv, T, L, d, page=0, lens=None, causal=True, decay=None, pad=0, seed=0,
           scale=None, mutate=None, in_place=False):
    scale = d ** -0.5 if scale is None else scale
    g = torch.Generator().manual_seed(seed)
    lens = [L] * B if lens is None else lens
    if page:
        n_pages = [-(-n // page) for n in lens]
        width, total = max(1, -(-L // page)), sum(n_pages) + 2
        k = random_like_shape((total, Hkv, page, d), torch.bfloat16, seed + 1)
        order, at = torch.randperm(total, generator=g).to(torch.int32), 0
        table = torch.full((B, width), -1, dtype=torch.int32)
        used = torch.zeros(total, page, dtype=torch.bool)
        for b, n in enumerate(lens):
            table[b, :n_pages[b]] = order[at:at + n_pages[b]]
            for i in range(n_pages[b]):
                used[order[at + i], :min(page, n - i * page)] = True
            at += n_pages[b]
        k = k.masked_fill(~used[:, None, :, None], float("nan"))
        keys = [oracle.attention.gather_paged(to_f64(k), table[b].numpy(), lens[b], page)
                for b in range(B)]
        cap = width * page
    else:
        k = random_like_shape((B, Hkv, L, d), torch.bfloat16, seed + 1)
        for b, n in enumerate(lens):
            k[b, :, n:] = float("nan")
        keys, table, cap = [to_f64(k[b, :, :n]) for b, n in enumerate(lens)], None, L
    q = random_like_shape((B, Hq, T, d), torch.bfloat16, seed + 2)
    lse = np.full((B, Hq, T), -np.inf)
    for b, n in enumerate(lens):
        for h in range(Hq):
            for i in range(T):
                last = min(n, n - T + i + 1) if causal else n
                if last > 0:
                    x = scale * (keys[b][h // (Hq // Hkv), :last] @ to_f64(q[b, h, i]))
                    lse[b, h, i] = np.logaddexp.reduce(x)
    lse_t = torch.from_numpy(lse).float()
    if mutate:
        mutate(lse_t)
    out_len = cap + pad
    prev = torch.rand(B, Hkv, out_len, generator=g) * 3 if decay is not None else None
    out = torch.full((B, Hkv, out_len), 77.0).to(DEV)
    prev_t = None if prev is None else prev.to(DEV)
    got = ost.key_weights(q.to(DEV), k.to(DEV), lse_t.to(DEV), out=prev_t if in_place else out,
                          prev=prev_t, decay=1.0 if decay is None else decay, causal=causal,
                          scale=scale, seq_lens=torch.tensor(lens, dtype=torch.int32, device=DEV),
                          block_table=None if table is None else table.to(DEV))
    torch.cuda.synchronize()
    assert ost.attn_sync_status() == 0
    got = to_f64(got)
    R = Hq // Hkv * T
    e = (2.0 ** -13 + 2.0 ** -16) * max(1.0, scale * d ** 0.5) + 2.0 ** -22 + R * 2.0 ** -24
    for b, n in enumerate(lens):
        w = oracle.key_weights(to_f64(q[b]), keys[b], to_f64(lse_t[b]), scale, causal)
        p = np.zeros_like(w) if prev is None else decay * to_f64(prev[b, :, :n])
        err = np.abs(got[b, :, :n] - (w + p))
        assert np.all(err <= e * w + 2.0 ** -23 * np.abs(w + p) + 2.0 ** -23 * np.abs(p)), \
            (b, err.max())
        rest = to_f64(prev[b, :, n:]) if in_place else 77.0
        assert np.all(got[b, :, n:] == rest)


@pytest.mark.gpu
@pytest.mark.parametrize("B,Hq,Hkv,T,L,d,page,lens", [
    (3, 8, 2, 1, 300, 128, 16, [300, 129, 0]),        # a decode step; an empty request
    (5, 16, 2, 1, 260, 64, 0, [260, 1, 128, 256, 257]),
    (2, 3, 1, 1, 40, 128, 1000, [40, 7]),             # three heads; one page each, odd
    (2, 64, 1, 1, 200, 64, 48, [200, 150]),           # 64 rows, 48-key pages
    (2, 12, 2, 11, 500, 128, 8, [500, 5]),            # 66 rows; fewer keys than tokens
    (1, 8, 2, 64, 700, 128, 0, [700]),                # 256 rows
    (2, 4, 4, 250, 300, 64, 64, [300, 251]),          # 250 rows of one head
    (40, 2, 1, 2, 130, 64, 0, [(i * 29) % 131 for i in range(40)]),
])
@pytest.mark.parametrize("causal", [True, False])
def test_rows_in_shared_memory(ost, B, Hq, Hkv, T, L, d, page, lens, causal):
    _check(ost, B, Hq, Hkv, T, L, d, page, lens, causal, None, pad=0, seed=B + T)
    _check(ost, B, Hq, Hkv, T, L, d, page, lens, causal, 0.5, pad=5, seed=B + T)


@pytest.mark.gpu
@pytest.mark.parametrize("B,Hq,Hkv,T,L,d,page,lens", [
    (1, 1, 1, 257, 257, 128, 0, [257]),               # one row over the limit
    (2, 4, 2, 300, 400, 64, 16, [400, 100]),          # tokens without keys
    (1, 8, 2, 130, 515, 128, 0, [515]),               # chunks that cross heads
    (1, 40, 1, 9, 130, 64, 0, [130]),                 # forty heads of nine tokens
    (1, 4, 1, 1100, 1100, 64, 48, [1100]),            # split rows
    (3, 2, 2, 600, 600, 128, 0, [600, 0, 256]),       # an empty request among them
])
@pytest.mark.parametrize("causal", [True, False])
def test_rows_that_stream(ost, B, Hq, Hkv, T, L, d, page, lens, causal):
    _check(ost, B, Hq, Hkv, T, L, d, page, lens, causal, 1.0, pad=3, seed=B + T)


@pytest.mark.gpu
def test_in_place_scale_and_dead_rows(ost):
    _check(ost, 2, 8, 2, 1, 300, 128, 16, [300, 77], decay=0.9, in_place=True)
    _check(ost, 1, 4, 1, 400, 400, 64, 0, decay=0.9, in_place=True)
    _check(ost, 1, 4, 1, 100, 400, 64, 0, scale=1.0)              # peaked rows
    _check(ost, 1, 4, 1, 400, 400, 64, 0, scale=1.0)

    def dead(lse):                    # rows that say they saw nothing give nothing
        lse[0, 1, ::3] = -float("inf")
        lse[0, 0, -1] = float("inf")  # and so does an infinite normaliser
    _check(ost, 1, 4, 1, 60, 200, 64, 0, mutate=dead)
    _check(ost, 1, 4, 1, 100, 200, 128, 0, mutate=dead)
    _check(ost, 1, 4, 1, 300, 300, 64, 16, mutate=dead)


@pytest.mark.gpu
@pytest.mark.parametrize("T,L,causal", [(1, 300, True), (60, 200, True), (60, 200, False),
                                        (300, 300, True), (300, 700, False)])
def test_dead_rows_may_hold_anything(ost, T, L, causal):
    """Queries of rows with an infinite normaliser (padding) may be NaN or
    infinite; the others' weights are what they were."""
    q = random_like_shape((2, 4, T, 64), torch.bfloat16, 5).to(DEV)
    k = random_like_shape((2, 2, L, 64), torch.bfloat16, 6).to(DEV)
    lse = torch.full((2, 4, T), 5.0, device=DEV)
    lse[0, 1, ::3] = -float("inf")
    lse[0, 0, -1] = float("inf")
    lse[1, 3] = -float("inf")
    want = ost.key_weights(q, k, lse, causal=causal)
    q[0, 1, ::3] = float("nan")
    q[0, 0, -1] = 3e38
    q[1, 3] = float("inf")
    got = ost.key_weights(q, k, lse, causal=causal)
    torch.cuda.synchronize()
    assert ost.attn_sync_status() == 0
    assert torch.equal(got, want) and bool(torch.isfinite(got).all())


@pytest.mark.gpu
def test_with_the_librarys_own_lse(ost):
    """Decode and prefill LSE in, probabilities out: each head and token
    gives one in all."""
    q = random_like_shape((3, 8, 128), torch.bfloat16, 1).to(DEV)
    k, v = (random_like_shape((3, 2, 500, 128), torch.bfloat16, i).to(DEV) for i in (2, 3))
    _, lse = ost.decode(q, k, v, 4)
    w = ost.key_weights(q, k, lse)
    assert torch.allclose(w.sum(-1), torch.full((3, 2), 4.0, device=DEV), rtol=1e-3)
    qp = random_like_shape((3, 8, 500, 128), torch.bfloat16, 4).to(DEV)
    _, lse = ost.forward(qp, k, v, causal=True)
    w = ost.key_weights(qp, k, lse)
    assert torch.allclose(w.sum(-1), torch.full((3, 2), 2000.0, device=DEV), rtol=1e-3)


@pytest.mark.gpu
@pytest.mark.parametrize("T", [1, 130])
def test_offsets_past_32_bits(ost, T):
    """Pages, and heads of a contiguous cache, past 2^32 bytes (2^31 elements)
    give what the same keys at the front give."""
    Hkv, page, d, lens = 2, 16, 128, [61, 30]
    total = (1 << 32) // (Hkv * page * d * 2) + 64
    k = torch.zeros(total, Hkv, page, d, dtype=torch.bfloat16, device=DEV)
    k[:8] = random_like_shape((8, Hkv, page, d), torch.bfloat16, 1).to(DEV)
    k[-8:] = k[:8]
    q = random_like_shape((2, 4, T, d), torch.bfloat16, 2).to(DEV)
    lse = torch.full((2, 4, T), 4.0, device=DEV)
    sl = torch.tensor(lens, dtype=torch.int32, device=DEV)
    table = torch.arange(8, dtype=torch.int32, device=DEV).view(2, 4)
    near, far = (ost.key_weights(q, k, lse, causal=False, seq_lens=sl, block_table=table + at)
                 for at in (0, total - 8))
    L = total * page // 64 * 64                      # [1, 2, L, d], past 2^32 bytes too
    flat = k.view(-1)[:Hkv * L * d].view(1, Hkv, L, d)
    flat[0, 1, -1000:] = random_like_shape((1000, d), torch.bfloat16, 3).to(DEV)
    w = ost.key_weights(q[:1], flat, lse[:1], causal=False)
    torch.cuda.synchronize()
    assert ost.attn_sync_status() == 0
    assert torch.equal(near, far) and bool((near != 0).any())
    same = ost.key_weights(q[:1, 2:], flat[:, 1:, -1000:].contiguous(), lse[:1, 2:], causal=False)
    # (2 T terms, added in another order where their rows are split over CTAs)
    assert torch.allclose(w[:, 1:, -1000:], same, rtol=4 * T * 2.0 ** -24, atol=0)


@pytest.mark.gpu
def test_bad_lengths_and_pages_are_flagged_not_read(ost):
    k = random_like_shape((9, 1, 16, 64), torch.bfloat16, 1).to(DEV)
    q = random_like_shape((3, 2, 1, 64), torch.bfloat16, 2).to(DEV)
    lse = torch.full((3, 2, 1), 5.0, device=DEV)
    table = torch.tensor([[0, 1, 2], [3, 9, 4], [5, 6, 7]], dtype=torch.int32, device=DEV)
    lens = torch.tensor([49, 48, 40], dtype=torch.int32, device=DEV)
    out = torch.full((3, 1, 48), 7.0, device=DEV)
    prev = torch.ones(3, 1, 48, device=DEV)
    ost.key_weights(q, k, lse, prev, seq_lens=lens, block_table=table, out=out)
    torch.cuda.synchronize()
    assert ost.attn_sync_status() == -7 and ost.attn_sync_status() == 0
    assert torch.all(out[0] == 7.0) and torch.all(out[2, 0, 40:] == 7.0)
    assert torch.all(out[1, 0, 16:32] == 1.0) and torch.all(out[1, 0, :16] > 1.0)
    w = torch.exp(0.125 * (q[2, :, 0].float() @ k[5:8, 0].flatten(0, 1).float().T) - 5).sum(0)[:40]
    assert torch.allclose(out[2, 0, :40], 1 + w, rtol=1e-4)


@pytest.mark.gpu
@pytest.mark.parametrize("T", [1, 300])
def test_streams_graphs_and_calls_at_once(ost, T):
    B, Hq, Hkv, L, d = 2, 8, 2, 1000, 64
    q = [random_like_shape((B, Hq, T, d), torch.bfloat16, i).to(DEV) for i in (1, 2)]
    k = random_like_shape((B, Hkv, L, d), torch.bfloat16, 3).to(DEV)
    lse = torch.full((B, Hq, T), 7.0, device=DEV)
    want = [ost.key_weights(x, k, lse) for x in q]
    torch.cuda.synchronize()
    side, got = [torch.cuda.Stream(), torch.cuda.Stream()], []
    for x, s in zip(q, side):
        with torch.cuda.stream(s):
            got.append([ost.key_weights(x, k, lse) for _ in range(3)])
    torch.cuda.synchronize()
    assert all(torch.equal(w, y) for w, ys in zip(want, got) for y in ys)
    n = ost.attn_key_weights_workspace_size(B, Hq, Hkv, T, L, L)
    ws = torch.full((n,), 255, dtype=torch.uint8, device=DEV) if n else None
    out = torch.zeros_like(want[0])
    x = q[0].clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ost.attn_key_weights(x, k, lse, None, out, d ** -0.5, workspace=ws)
    for i in (1, 0):
        x.copy_(q[i])
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want[i])


@pytest.mark.gpu
def test_binding_refusals(ost):
    q = random_like_shape((2, 4, 1, 64), torch.bfloat16, 1).to(DEV)
    k = random_like_shape((2, 2, 50, 64), torch.bfloat16, 2).to(DEV)
    lse, out = torch.zeros(2, 4, 1, device=DEV), torch.zeros(2, 2, 50, device=DEV)
    for bad in (dict(q=q.float()), dict(lse=lse[:1]), dict(lse=lse.double()), dict(k=k[:1]),
                dict(k=k.transpose(0, 1)), dict(prev=out[:, :, :4].contiguous()),
                dict(out=out.half()), dict(seq_lens=torch.tensor([5, 5], device=DEV)),
                dict(q=q.cpu())):
        with pytest.raises((ValueError, TypeError)):
            ost.key_weights(**{**dict(q=q, k=k, lse=lse, out=out), **bad})
    with pytest.raises(ost.AttnError):
        ost.key_weights(q, k, lse, scale=float("nan"))


@pytest.mark.parametrize("kwargs", [
    dict(out=P), dict(out=P - 2 * 2 * 100 * 4 + 4), dict(out=P + 2 * 4 * 3 * 64 * 2 - 4),   # q
    dict(out=2 * P + 2 * 2 * 100 * 64 * 2 - 4), dict(out=3 * P), dict(out=6 * P + 4),
    {**PAGED, "out": 2 * P + 9 * 2 * 16 * 64 * 2 - 4}, {**PAGED, "out": 7 * P + 2 * 4 * 4 - 4},
])
def test_outputs_on_top_of_inputs_are_refused(lib, kwargs):
    if torch.cuda.is_available():
        pytest.skip("made-up addresses: nothing may launch")
    assert _call(lib, **kwargs) == INVALID


def test_outputs_next_to_inputs_are_not_refused(lib):
    if torch.cuda.is_available():
        pytest.skip("made-up addresses: nothing may launch")
    for kwargs in (dict(), dict(out=P - 2 * 2 * 100 * 4), dict(out=P + 2 * 4 * 3 * 64 * 2),
                   dict(out=2 * P + 2 * 2 * 100 * 64 * 2), dict(out=4 * P), PAGED):
        assert _call(lib, **kwargs) != INVALID


@pytest.mark.gpu
@pytest.mark.parametrize("causal", [True, False])
def test_more_requests_than_threads(ost, causal):
    """Requests are counted by the threads of a CTA, several each past 352 (and
    past 256 where partial sums are joined); lengths of zero among them."""
    lens = [0 if i % 7 == 0 else 1 + (i * 53) % 300 for i in range(800)]
    _check(ost, 800, 2, 1, 1, 300, 64, 0, lens, causal, seed=21)
    lens = [0 if i % 5 == 0 else 300 if i == 399 else 1 + (i * 29) % 40 for i in range(400)]
    _check(ost, 400, 1, 1, 260, 300, 64, 0, lens, causal, 0.5, seed=22)
