"""Cache eviction: the oracle's pins, refusals on the CPU, and the GPU kernels
against the oracle. Everything is selection and copying, so results are equal,
not close."""

import numpy as np
import pytest
import torch

import oracle
from workloads import random_like_shape

DEV = "cuda:0"
INVALID, UNSUPPORTED, MISALIGNED = -1, -2, -3


# ------------------------------------------------------------------ oracle


def test_oracle_keeps_sinks_recents_and_the_best():
    s = np.array([0.1, 5.0, 3.0, 9.0, 3.0, 0.0, 7.0, 0.2])
    assert list(oracle.evict(s, 5, 1, 2)) == [0, 1, 3, 6, 7]
    assert list(oracle.evict(s, 3)) == [1, 3, 6]
    assert list(oracle.evict(s, 4)) == [1, 2, 3, 6]             # tie 2 / 4: the lower index
    assert list(oracle.evict(s, 8)) == list(range(8))
    assert list(oracle.evict(s[:3], 5, 2, 2)) == [0, 1, 2]      # fewer keys than places
    assert list(oracle.evict(s, 3, 1, 2)) == [0, 6, 7]          # no place for the middle
    n = np.array([np.nan, -np.inf, 1.0, np.nan, np.inf])
    assert list(oracle.evict(n, 3)) == [0, 2, 4]                # NaN as -inf, lowest index


def test_oracle_is_the_largest_sum():
    rng = np.random.default_rng(0)
    for _ in range(20):
        s = rng.standard_normal(30)
        at = oracle.evict(s, 10)
        assert np.isclose(s[at].sum(), np.sort(s)[-10:].sum()) and np.all(np.diff(at) > 0)


# ------------------------------------------------------------------ refusals

P = 1 << 30  # an aligned stand-in address; never dereferenced on these paths


@pytest.fixture(scope="module")
def lib():
    import __graft_entry__
    __graft_entry__.build()
    import online_softmax_tiled_gb300 as ost
    return ost.lib()


def _call(lib, k=P, v=2 * P, scores=3 * P, lens=4 * P, table=None, ko=5 * P, vo=6 * P, so=7 * P,
          kept=8 * P, new=9 * P, B=2, Hkv=2, L=100, num_pages=0, page=0, max_pages=0, slen=100,
          d=64, keep=10, sink=1, recent=2, out_len=10, dt=1):
    return lib.attn_cache_evict(k, v, scores, lens, table, ko, vo, so, kept, new, B, Hkv, L,
                                num_pages, page, max_pages, slen, d, keep, sink, recent, out_len,
                                dt, None)


PAGED = dict(table=10 * P, num_pages=8, page=16, max_pages=4)


@pytest.mark.parametrize("kwargs,expected", [
    (dict(B=0), INVALID), (dict(Hkv=0), INVALID), (dict(L=0), INVALID), (dict(slen=0), INVALID),
    (dict(k=None), INVALID), (dict(v=None), INVALID), (dict(scores=None), INVALID),
    (dict(ko=None), INVALID), (dict(vo=None), INVALID), (dict(kept=None), INVALID),
    (dict(new=None), INVALID), (dict(keep=0), INVALID), (dict(sink=-1), INVALID),
    (dict(recent=-1), INVALID), (dict(sink=5, recent=6), INVALID),
    (dict(sink=2 ** 31 - 1, recent=2 ** 31 - 1), INVALID), (dict(out_len=9), INVALID),
    (dict(dt=3), INVALID), (dict(lens=None, slen=99), INVALID),
    ({**PAGED, "lens": None}, INVALID), ({**PAGED, "num_pages": 0}, INVALID),
    ({**PAGED, "page": 0}, INVALID), ({**PAGED, "max_pages": 0}, INVALID),
    (dict(d=96), UNSUPPORTED), (dict(B=256, Hkv=256), UNSUPPORTED),
    ({**PAGED, "max_pages": 1 << 20, "page": 2048}, UNSUPPORTED),
    (dict(k=P + 8), MISALIGNED), (dict(vo=6 * P + 4), MISALIGNED), (dict(lens=P + 2), MISALIGNED),
    (dict(so=7 * P + 2), MISALIGNED), ({**PAGED, "table": P + 1}, MISALIGNED),
    (dict(ko=P), INVALID),                     # in place
    (dict(vo=P + 2 * 2 * 100 * 128 - 16), INVALID),   # the last bytes of k
    (dict(so=3 * P), INVALID), (dict(new=4 * P), INVALID), (dict(ko=6 * P), INVALID),
    (dict(kept=9 * P), INVALID),
])
def test_refusals(lib, kwargs, expected):
    assert _call(lib, **kwargs) == expected


# ------------------------------------------------------------------ GPU


def _scores(kind, shape, seed):
    g = torch.Generator().manual_seed(seed)
    s = torch.rand(shape, generator=g).pow(6) * 30
    if kind == "ties":
        s = torch.randint(0, 4, shape, generator=g).float()
    if kind == "zeros":
        s = torch.zeros(shape)
    if kind == "signed":
        s = torch.randn(shape, generator=g) * 10.0 ** torch.randint(-30, 30, shape, generator=g)
    if kind == "odd":
        special = torch.tensor([float("nan"), float("inf"), -float("inf"), 0.0, -0.0, 1e-45, -1.0,
                                3.4e38])
        s = special[torch.randint(0, 8, shape, generator=g)]
    return s


def _check(ost, B, Hkv, L, d, keep, sink, recent, page=0, lens=None, kind="rand", out_len=None,
           dt=torch.bfloat16, score_pad=0, seed=0, with_scores=True):
    g = torch.Generator().manual_seed(seed)
    out_len = out_len or keep
    if lens is None:
        lens = [L] * B
    lens_t = torch.tensor(lens, dtype=torch.int32, device=DEV)
    if page:
        width = -(-L // page)
        num = B * width + 2
        k, v = (random_like_shape((num, Hkv, page, d), dt, seed + i).to(DEV) for i in (1, 2))
        table = torch.randperm(num, generator=g)[:B * width].view(B, width).to(torch.int32)
        for b, n in enumerate(lens):
            table[b, -(-n // page):] = -1                     # never read
        rows = [[(int(table[b, j // page]), slice(None), j % page) for j in range(lens[b])]
                for b in range(B)]
        kf, vf = ([torch.stack([t[p, :, i] for p, _, i in rows[b]], 1) if lens[b] else None
                   for b in range(B)] for t in (k.cpu(), v.cpu()))
        table = table.to(DEV)
    else:
        k, v = (random_like_shape((B, Hkv, L, d), dt, seed + i).to(DEV) for i in (1, 2))
        kf, vf, table = k.cpu(), v.cpu(), None
    s = _scores(kind, (B, Hkv, L + score_pad), seed).to(DEV)
    out = (torch.full((B, Hkv, out_len, d), 7.0, dtype=dt, device=DEV),
           torch.full((B, Hkv, out_len, d), 8.0, dtype=dt, device=DEV),
           torch.full((B, Hkv, out_len), 9.0, device=DEV) if with_scores else None,
           torch.full((B, Hkv, keep), 55, dtype=torch.int32, device=DEV),
           torch.full((B,), 66, dtype=torch.int32, device=DEV))
    before = [t.clone() for t in (k, v, s)]
    ost.evict(k, v, s, keep, sink, recent, seq_lens=lens_t, block_table=table, out=out)
    torch.cuda.synchronize()
    assert ost.attn_sync_status() == 0
    assert all(torch.equal(a.nan_to_num(), b.nan_to_num()) for a, b in zip((k, v, s), before))
    ko, vo, so, kept, new = (None if t is None else t.cpu() for t in out)
    for b in range(B):
        m = min(lens[b], keep)
        assert new[b] == m
        for h in range(Hkv):
            at = oracle.evict(s[b, h, :lens[b]].cpu().double().numpy(), keep, sink, recent)
            assert np.array_equal(kept[b, h, :m].numpy(), at), (b, h)
            assert torch.all(kept[b, h, m:] == -1)
            if m:
                assert torch.equal(ko[b, h, :m], kf[b][h, at])
                assert torch.equal(vo[b, h, :m], vf[b][h, at])
            assert torch.all(ko[b, h, m:] == 7.0) and torch.all(vo[b, h, m:] == 8.0)
            if with_scores:
                want = s[b, h].cpu()[at]
                assert torch.equal(so[b, h, :m].nan_to_num(1.5), want.nan_to_num(1.5))
                assert torch.all(so[b, h, m:] == 9.0)


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["rand", "ties", "zeros", "signed", "odd"])
@pytest.mark.parametrize("page", [0, 16])
def test_scores_of_every_kind(ost, kind, page):
    _check(ost, 3, 2, 1000, 64, 128, 4, 32, page, [1000, 517, 128], kind, seed=3)


@pytest.mark.gpu
@pytest.mark.parametrize("B,Hkv,L,d,keep,sink,recent,page,lens", [
    (1, 1, 1, 64, 1, 0, 0, 0, [1]),
    (4, 1, 40, 128, 7, 3, 4, 0, [0, 1, 7, 40]),            # nothing ranked; empty; shorter
    (2, 3, 129, 128, 128, 0, 0, 0, [129, 128]),            # one key leaves; none does
    (2, 2, 300, 64, 33, 0, 33, 48, [300, 34]),             # recents alone, 48-key pages
    (2, 1, 77, 128, 5, 5, 0, 1, [77, 4]),                  # sinks alone, one key a page
    (1, 2, 20001, 64, 4099, 4, 64, 16, [19999]),           # a cluster with ragged slices
    (1, 1, 70000, 64, 1000, 1, 1, 0, [69999]),             # eight CTAs a row
])
def test_shapes(ost, B, Hkv, L, d, keep, sink, recent, page, lens):
    for kind in ("rand", "ties"):
        _check(ost, B, Hkv, L, d, keep, sink, recent, page, lens, kind, seed=L)


@pytest.mark.gpu
def test_wide_outputs_float32_and_padded_scores(ost):
    _check(ost, 2, 2, 500, 128, 50, 2, 8, out_len=64, dt=torch.float32, score_pad=3)
    _check(ost, 2, 2, 500, 64, 50, 2, 8, page=16, out_len=51, dt=torch.float32, score_pad=5,
           lens=[499, 20])
    _check(ost, 2, 4, 500, 64, 50, 2, 8, with_scores=False)


@pytest.mark.gpu
def test_offsets_past_32_bits(ost):
    """A cache whose last rows lie past 2^32 bytes (and 2^31 elements): 18
    heads of a million keys."""
    B, Hkv, L, d, keep = 1, 18, 1 << 20, 128, 300
    k = torch.empty(B, Hkv, L, d, dtype=torch.bfloat16, device=DEV)
    k.view(torch.int16).view(-1, d)[:] = torch.arange(Hkv * L, device=DEV)[:, None] % 32749
    v = k.flip(2)
    s = torch.rand(B, Hkv, L, device=DEV)
    ko, vo, so, kept, new = ost.evict(k, v, s, keep)
    for h in (0, Hkv - 1):
        at = torch.sort(torch.topk(s[0, h], keep).indices).values
        assert torch.equal(kept[0, h].long(), at)
        assert torch.equal(ko[0, h].view(torch.int16), k[0, h, at].view(torch.int16))
        assert torch.equal(vo[0, h].view(torch.int16), v[0, h, at].view(torch.int16))
        assert torch.equal(so[0, h], s[0, h, at])


@pytest.mark.gpu
def test_bad_lengths_and_pages_are_flagged_not_read(ost):
    k = random_like_shape((6, 1, 16, 64), torch.bfloat16, 1).to(DEV)
    v = random_like_shape((6, 1, 16, 64), torch.bfloat16, 2).to(DEV)
    table = torch.tensor([[0, 1], [2, 6], [3, 4]], dtype=torch.int32, device=DEV)
    lens = torch.tensor([33, 30, 31], dtype=torch.int32, device=DEV)
    s = torch.rand(3, 1, 32, device=DEV)
    s[1, 0, :20] = 2.0 + s[1, 0, :20]
    out = ost.evict(k, v, s, 18, seq_lens=lens, block_table=table)
    assert ost.attn_sync_status() == -7 and ost.attn_sync_status() == 0
    assert out[4].tolist() == [0, 18, 18] and torch.all(out[3][0] == -1)
    at = out[3][1, 0].long()
    good = at < 16
    assert torch.equal(out[0][1, 0][good], k[2, 0][at[good]])
    assert torch.all(out[0][1, 0][~good] == 0) and (~good).any()   # the bad page's rows stay
    at = out[3][2, 0].long()
    assert torch.equal(out[1][2, 0], torch.cat([v[3, 0], v[4, 0]])[at])


@pytest.mark.gpu
def test_stream_graph_and_binding_refusals(ost):
    k, v = (random_like_shape((2, 2, 600, 64), torch.bfloat16, i).to(DEV) for i in (1, 2))
    s = torch.rand(2, 2, 600, device=DEV)
    want = ost.evict(k, v, s, 40, 2, 5)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = ost.evict(k, v, s, 40, 2, 5, stream=side,
                    out=tuple(torch.zeros_like(t) for t in want))
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    out = tuple(torch.zeros_like(t) for t in want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ost.evict(k, v, s, 40, 2, 5, out=out)
    s.copy_(torch.rand(2, 2, 600, device=DEV))
    graph.replay()
    again = ost.evict(k, v, s, 40, 2, 5)
    assert all(torch.equal(a, b) for a, b in zip(out, again))
    lens = torch.tensor([600, 600], device=DEV)
    for bad in (dict(scores=s.double()), dict(scores=s[:, :1].contiguous()), dict(v=v[:1]),
                dict(v=v.float()), dict(seq_lens=lens), dict(k=k.transpose(0, 1))):
        args = {"k": k, "v": v, "scores": s, "n_keep": 40, **bad}
        with pytest.raises((ValueError, TypeError)):
            ost.evict(**args)
    with pytest.raises(ost.AttnError):
        ost.evict(k, v, s, 40, 30, 11)


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["rand", "ties", "zeros", "signed", "odd"])
def test_rows_that_do_not_stay_in_registers(ost, kind):
    """More than 131072 scores a row are read again for every pass: ties that
    are cut, NaN and infinities, held keys and ragged last segments, beside a
    request short enough to be held."""
    _check(ost, 3, 1, 140001, 64, 4001, 3, 70, 0, [139990, 131500, 5000], kind, seed=7)


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["rand", "ties"])
def test_four_ctas_a_row(ost, kind):
    """32 rows of more than 8192 scores: two CTAs a row would leave SMs idle."""
    _check(ost, 4, 8, 9001, 64, 300, 2, 17, 0, [9001, 8999, 4097, 301], kind, seed=11)


@pytest.mark.gpu
def test_offsets_past_32_bits_in_a_stable_order(ost):
    """As test_offsets_past_32_bits, whose scores tie now and then: here with
    seeded scores and the ties' lower index first."""
    B, Hkv, L, d, keep = 1, 18, 1 << 20, 128, 300
    k = torch.empty(B, Hkv, L, d, dtype=torch.bfloat16, device=DEV)
    k.view(torch.int16).view(-1, d)[:] = torch.arange(Hkv * L, device=DEV)[:, None] % 32749
    v = k.flip(2)
    g = torch.Generator().manual_seed(17)
    s = (torch.rand(Hkv, L, generator=g) * 4096).floor().to(DEV)[None]     # 256 keys a score
    ko, vo, so, kept, new = ost.evict(k, v, s, keep)
    for h in range(Hkv):
        order = torch.sort(s[0, h], descending=True, stable=True).indices
        at = torch.sort(order[:keep]).values
        assert torch.equal(kept[0, h].long(), at)
        assert torch.equal(ko[0, h].view(torch.int16), k[0, h, at].view(torch.int16))
        assert torch.equal(vo[0, h].view(torch.int16), v[0, h, at].view(torch.int16))
        assert torch.equal(so[0, h], s[0, h, at])
