"""Decode of T tokens over paged caches under a window and first tokens, in
bf16 and in 4 bits: the oracle's pins, refusals on the CPU, and the GPU kernels
against the float64 oracle.

Tolerances, with A = Σ p |v| / Σ p the row's weighted mean of |v| per element
(the oracle's `spread`), u = 2^-24, for inputs with scale · Σ|q k| <= 16 and n <=
4000 keys (longer ones: n u more): a score is off by at most (d + 4) u · 16 <
2^-12.9 (products are exact, sums float32, one multiplication by the scale, one
subtraction of the reference), so p by 2^-12.9 + 2^-22 of itself, numerator and
denominator alike; adding n terms loses n u <= 2^-12; P enters the product as two
bf16 parts (2^-17) or, times the scale, in float16 (2^-11). In all below
(2 · 2^-12.9 + 2 · 2^-12 + 2^-17) A < 2^-10 A in bf16, 2^-9.4 A in 4 bits, plus
half a step of the bf16 result, 2^-8 of it. lse: 2^-12.9 + 2^-12 + one rounding of
a value below 32, 2^-20: below 2^-11.
"""

import numpy as np
import pytest
import torch

import oracle
from workloads import random_like_shape, to_f64

DEV = "cuda:0"
INVALID, UNSUPPORTED, MISALIGNED, WORKSPACE = -1, -2, -3, -4
BF = torch.bfloat16


# ------------------------------------------------------------------ oracle


def test_oracle_is_masked_attention():
    """The rule is attn_mask's {window_left, 0, n_global} of the last T rows."""
    rng = np.random.default_rng(0)
    q, k, v = rng.standard_normal((4, 9, 8)), *rng.standard_normal((2, 2, 9, 8))
    for left, first in ((-1, 0), (3, 0), (2, 2), (0, 5), (-1, 7)):
        spec = {"window_left": left, "window_right": 0, "n_global": first}
        o, lse = oracle.attention_fwd_masked(q[None], k[None], v[None], 0.3, spec)
        got, got_lse, _ = oracle.decode_window(q[:, -3:], k, v, 0.3, left, first)
        assert np.allclose(got, o[0][:, -3:]) and np.allclose(got_lse, lse[0][:, -3:])


def test_oracle_ignores_hidden_keys_and_empty_rows():
    q, k, v = np.ones((1, 3, 4)), np.full((1, 2, 4), 0.5), np.arange(8.0).reshape(1, 2, 4)
    o, lse, _ = oracle.decode_window(q, k, v, 1.0)
    assert np.all(o[0, 0] == 0) and lse[0, 0] == -np.inf          # position -1
    assert np.allclose(o[0, 1], v[0, 0]) and np.allclose(o[0, 2], v.mean(1))
    k2, v2 = k.copy(), v.copy()
    k2[0, 1], v2[0, 1] = np.nan, np.inf
    o2, lse2, _ = oracle.decode_window(q, k2, v2, 1.0)
    assert np.array_equal(o2[0, :2], o[0, :2]) and np.array_equal(lse2[0, :2], lse[0, :2])


# ------------------------------------------------------------------ refusals

P = 1 << 32


@pytest.fixture(scope="module")
def lib():
    import __graft_entry__
    __graft_entry__.build()
    import online_softmax_tiled_gb300 as ost
    return ost.lib()


def _call(lib, four=False, q=P, k=2 * P, ks=3 * P, v=4 * P, vs=5 * P, table=6 * P, lens=7 * P,
          o=8 * P, lse=9 * P, B=2, Hq=8, Hkv=2, T=2, pages=9, page=16, mp=4, d=64, scale=0.1, left=5,
          first=4, ws=10 * P, nb=1 << 30):
    pools = (k, ks, v, vs) if four else (k, v)
    f = lib.attn_decode_cache4 if four else lib.attn_decode_window
    return f(q, *pools, table, lens, o, lse, B, Hq, Hkv, T, pages, page, mp, d, scale, left, first,
             ws, nb, None)


NAN, INF = float("nan"), float("inf")


@pytest.mark.parametrize("four", [False, True])
@pytest.mark.parametrize("kwargs,expected", [
    (dict(B=0), INVALID), (dict(Hq=0), INVALID), (dict(Hkv=0), INVALID), (dict(Hq=7), INVALID),
    (dict(T=0), INVALID), (dict(T=-1), INVALID), (dict(pages=0), INVALID), (dict(page=0), INVALID),
    (dict(mp=0), INVALID), (dict(d=0), INVALID), (dict(first=-1), INVALID),
    (dict(q=None), INVALID), (dict(k=None), INVALID), (dict(v=None), INVALID),
    (dict(table=None), INVALID), (dict(lens=None), INVALID), (dict(o=None), INVALID),
    (dict(scale=NAN), INVALID), (dict(scale=0.0), INVALID), (dict(scale=-1.0), INVALID),
    (dict(scale=INF), INVALID),
    (dict(d=96), UNSUPPORTED), (dict(d=256), UNSUPPORTED), (dict(B=65536), UNSUPPORTED),
    (dict(T=1 << 15), UNSUPPORTED), (dict(page=1 << 15, mp=(1 << 15) + 1), UNSUPPORTED),
    (dict(pages=1 << 27), UNSUPPORTED), (dict(B=60000, mp=1 << 18), UNSUPPORTED),
    (dict(q=P + 8), MISALIGNED), (dict(k=2 * P + 8), MISALIGNED), (dict(v=4 * P + 4), MISALIGNED),
    (dict(o=8 * P + 2), MISALIGNED), (dict(table=6 * P + 2), MISALIGNED),
    (dict(lens=7 * P + 1), MISALIGNED), (dict(lse=9 * P + 2), MISALIGNED),
])
def test_refusals(lib, four, kwargs, expected):
    assert _call(lib, four, **kwargs) == expected


@pytest.mark.parametrize("kwargs", [dict(ks=None), dict(vs=None)])
def test_refusals_of_absent_scales(lib, kwargs):
    assert _call(lib, True, **kwargs) == INVALID


@pytest.mark.parametrize("four", [False, True])
@pytest.mark.parametrize("kwargs,expected", [
    (dict(ws=None, nb=0), WORKSPACE), (dict(ws=10 * P + 16), MISALIGNED), (dict(o=P), INVALID),
    (dict(o=2 * P), INVALID), (dict(o=4 * P + 16), INVALID), (dict(lse=4 * P), INVALID),
    (dict(o=6 * P), INVALID), (dict(lse=7 * P), INVALID), (dict(lse=8 * P + 4), INVALID),
    (dict(ws=2 * P), INVALID), (dict(ws=8 * P), INVALID), (dict(ws=9 * P), INVALID),
    (dict(ws=P - (1 << 30) + 256), INVALID), (dict(ws=7 * P), INVALID),
])
def test_refusals_of_workspaces_and_overlaps(lib, four, kwargs, expected):
    assert _call(lib, four, **kwargs) == expected


def test_outputs_next_to_inputs_are_not_refused(lib):
    if torch.cuda.is_available():
        pytest.skip("made-up addresses: nothing may launch")
    for four in (False, True):
        size = 2 * 8 * 2 * 64 * 2                       # bytes of q
        for kwargs in (dict(), dict(o=P + size), dict(o=P - size), dict(lse=None),
                       dict(left=-5), dict(left=2 ** 31 - 1, first=2 ** 31 - 1)):
            assert _call(lib, four, **kwargs) == -5     # no device to run on


def test_workspace_sizes_of_refused_sizes(lib):
    f = lib.attn_decode_window_workspace_size
    assert f(0, 8, 2, 1, 64) == 0 and f(2, 7, 2, 1, 64) == 0 and f(2, 8, 2, 1, 96) == 0
    assert f(2, 8, 2, 0, 64) == 0 and f(70000, 8, 2, 1, 64) == 0


# ------------------------------------------------------------------ GPU


def _ints(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


class Cache:
    """Pools of B requests' keys in shuffled pages, in bf16 or 4 bits; pages that
    no token sees are absent from the table (-1), and all rows that no token sees
    hold NaN (4 bits: any codes and NaN scales)."""

    def __init__(self, four, lens, Hkv, d, page, T, left, first, seed, gain=1.0):
        self.four, self.lens, self.page, self.d = four, lens, page, d
        width = max([1] + [-(-n // page) for n in lens])
        g = torch.Generator().manual_seed(seed)
        table = torch.full((len(lens), width), -1)
        self.rows, need = [], 0
        for b, n in enumerate(lens):
            lo = 0 if left < 0 else max(0, n - T - left)
            seen = [j for j in range(n) if j < first or j >= lo]
            self.rows.append(torch.tensor(seen, dtype=torch.long))
            pages = sorted({j // page for j in seen})
            table[b, pages] = need + torch.arange(len(pages))
            need += len(pages)
        total = need + 2
        order = torch.randperm(total, generator=g)
        self.table = torch.where(table >= 0, order[table.clamp(min=0)], -1).to(torch.int32)
        shape = (total, Hkv, page, d)
        live = torch.zeros(total, page, dtype=torch.bool)
        for b, j in enumerate(self.rows):
            live[self.table[b, j // page].long(), j % page] = True
        dead = ~live[:, None, :, None]
        if four:
            self.pools = []
            for i in range(2):
                c = torch.randint(0, 256, (*shape[:3], d // 2), generator=g).to(torch.uint8)
                s = torch.rand(*shape[:3], d // 32, generator=g) * 0.4 + 0.1
                if gain != 1.0:
                    s = s * gain ** (torch.rand(*shape[:3], 1, generator=g) - 0.5)
                self.pools += [c, s.to(BF).masked_fill(dead, float("nan"))]
        else:
            self.pools = [random_like_shape(shape, BF, seed + 1 + i).masked_fill(dead, float("nan"))
                          for i in range(2)]

    def to(self, dev):
        return [x.to(dev) for x in self.pools], self.table.to(dev), _ints(self.lens)

    def values(self, which):
        """The whole pool as float64 values."""
        if not self.four:
            return to_f64(self.pools[which])
        codes, scales = self.pools[2 * which:2 * which + 2]
        return oracle.values4(oracle.unpack4(codes.numpy()), to_f64(scales))

    def of_request(self, which, b, pool):
        """[Hkv, n, d]; rows that are nowhere are NaN."""
        out = np.full((pool.shape[1], self.lens[b], self.d), np.nan)
        j = self.rows[b]
        at = self.table[b, j // self.page].long().numpy()
        out[:, j.numpy()] = pool[at, :, (j % self.page).numpy()].transpose(1, 0, 2)
        return out


def _check(ost, four, lens, Hq, Hkv, T, d, page, left, first, seed=0, scale=None, cache=None,
           q=None, gain=1.0, extra=0.0):
    scale = d ** -0.5 if scale is None else scale
    c = Cache(four, lens, Hkv, d, page, T, left, first, seed, gain) if cache is None else cache
    B = len(lens)
    q = random_like_shape((B, Hq, T, d), BF, seed + 7) if q is None else q
    pools, table, n = c.to(DEV)
    f = ost.decode_cache4 if four else ost.decode_window
    o, lse = f(q.to(DEV), *pools, table, n, window_left=left, n_global=first, scale=scale)
    assert ost.attn_sync_status() == 0
    kv = [c.values(i) for i in range(2)]
    for b in range(B):
        k, v = (c.of_request(i, b, kv[i]) for i in range(2))
        ro, rl, spread = oracle.decode_window(to_f64(q[b]), k, v, scale, left, first)
        go, gl = to_f64(o[b]), to_f64(lse[b])
        none = np.isneginf(rl)
        assert np.array_equal(np.isneginf(gl), none), (b, lens[b])
        assert np.all(go[none] == 0)
        long = len(c.rows[b]) * 2.0 ** -24
        with np.errstate(invalid="ignore"):
            bad = np.abs(gl - rl) > 2.0 ** -11 + long
        assert not bad[~none].any(), (b, lens[b], np.abs(gl - rl)[~none].max())
        tol = 2.0 ** -8 * np.abs(ro) + ((2.0 ** -9.4 if four else 2.0 ** -10) + 2 * long) * spread
        err = np.abs(go - ro)
        assert np.all(err <= tol + extra), (b, lens[b], np.max(err - tol))
    return o, lse


CASES = [
    # lens, Hq, Hkv, T, d, page, window_left, n_global
    ([1, 2, 15, 16, 17, 63, 64, 65, 300], 8, 2, 1, 128, 16, -1, 0),
    ([0, 1, 5, 0, 129], 4, 4, 1, 64, 16, -1, 0),
    ([1000, 40, 700], 8, 1, 1, 128, 64, 99, 4),
    ([500, 3, 20], 16, 2, 1, 64, 24, 0, 0),
    ([500, 3, 20], 4, 2, 1, 128, 7, 30, 20),
    ([100, 200], 2, 1, 1, 128, 300, 63, 1),
    ([77, 33], 3, 1, 1, 64, 1, 40, 3),
    ([400, 2, 0, 5, 97], 4, 2, 4, 128, 16, -1, 0),           # 8 query rows a KV head
    ([400, 2, 0, 5, 97], 6, 2, 3, 128, 16, 50, 4),           # 9: two blocks of 8 in one
    ([300, 16, 31], 8, 2, 4, 64, 48, 10, 0),
    ([300, 150], 16, 1, 4, 128, 16, 100, 18),                # 64 query rows: four blocks of 16
    ([90, 17], 5, 1, 5, 64, 16, 3, 2),                       # 25
    ([260], 1, 1, 33, 128, 16, 20, 4),                       # a chunk of a prompt
    ([30, 8], 2, 2, 12, 64, 16, 5, 100),                     # first tokens past the end
    ([64, 80], 4, 1, 2, 128, 32, 1000000, 0),                # a window wider than the cache
]


@pytest.mark.gpu
@pytest.mark.parametrize("four", [False, True])
@pytest.mark.parametrize("case", CASES)
def test_parity(ost, four, case):
    _check(ost, four, *case, seed=3)


@pytest.mark.gpu
@pytest.mark.parametrize("four", [False, True])
@pytest.mark.parametrize("seed", range(6))
def test_parity_of_drawn_sizes(ost, four, seed):
    rng = np.random.default_rng(100 + seed)
    Hkv = int(rng.integers(1, 5))
    G, T = int(rng.integers(1, 9)), int(rng.choice([1, 1, 2, 3, 7]))
    lens = [int(x) for x in rng.integers(0, 900, int(rng.integers(1, 12)))]
    _check(ost, four, lens, Hkv * G, Hkv, T, int(rng.choice([64, 128])),
           int(rng.choice([1, 5, 16, 40, 128])), int(rng.choice([-1, 0, 33, 250])),
           int(rng.choice([0, 0, 4, 37])), seed=200 + seed)


@pytest.mark.gpu
@pytest.mark.parametrize("four", [False, True])
@pytest.mark.parametrize("lens,Hq,Hkv,T,left,first", [
    ([20000], 4, 1, 1, -1, 0),                  # one request over all CTAs
    ([9000, 1, 3500, 0, 12000], 16, 2, 2, -1, 0),
    ([30000, 800], 8, 2, 1, 11000, 4),
    ([1 + (i * 37) % 90 for i in range(700)], 2, 1, 1, -1, 0),   # more requests than threads
    ([0] * 300 + [400] + [0] * 50, 4, 2, 1, 100, 2),
    ([129 * (i % 3) for i in range(200)], 8, 8, 1, -1, 0),
])
def test_shares_of_many_and_of_long_requests(ost, four, lens, Hq, Hkv, T, left, first):
    _check(ost, four, lens, Hq, Hkv, T, 64, 64, left, first, seed=5)


@pytest.mark.gpu
@pytest.mark.parametrize("four", [False, True])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("page", [32, 24])
@pytest.mark.parametrize("Hq,T", [(6, 1), (8, 2), (6, 4), (4, 20)])   # 3, 8, 12, 40 rows a KV head
@pytest.mark.parametrize("left", [-1, 2500])
def test_shares_at_every_number_of_rows(ost, four, d, page, Hq, T, left):
    _check(ost, four, [4000, 1, 900, 0, 3977], Hq, 2, T, d, page, left, 5, seed=6)


@pytest.mark.gpu
@pytest.mark.parametrize("four", [False, True])
@pytest.mark.parametrize("d", [64, 128])
def test_peaked_rows_and_moving_references(ost, four, d):
    """Scores that rise along the keys by far more than the reference lets pass."""
    lens, Hkv, Hq = [600], 1, 2
    c = Cache(four, lens, Hkv, d, 16, 1, -1, 0, 9)
    at, j = c.table[0], torch.arange(600)
    if four:
        ramp = (0.05 + j / 600).to(BF)
        c.pools[1][at[j // 16].long(), 0, j % 16] = ramp[:, None].expand(-1, d // 32)
    else:
        c.pools[0][at[j // 16].long(), 0, j % 16] *= (j / 60)[:, None].to(BF)
    q = random_like_shape((1, Hq, 1, d), BF, 8) * 2
    kv = c.of_request(0, 0, c.values(0))
    big = np.max(d ** -0.5 * np.abs(to_f64(q[0]) @ kv[0].T))
    assert big > 12                  # the reference lets 8 binary orders pass, 5.5
    # scores are off by (d + 4) u Σ|q k| scale, here up to
    size = np.max(d ** -0.5 * np.abs(to_f64(q[0])) @ np.abs(kv[0].T))
    extra = (d + 4) * 2.0 ** -24 * size * 2 * 6.0
    pools, table, n = c.to(DEV)
    f = ost.decode_cache4 if four else ost.decode_window
    o, lse = f(q.to(DEV), *pools, table, n)
    v = c.of_request(1, 0, c.values(1))
    ro, rl, spread = oracle.decode_window(to_f64(q[0]), kv, v, d ** -0.5)
    assert np.max(np.abs(to_f64(lse[0]) - rl)) <= (d + 4) * 2.0 ** -24 * size + 2.0 ** -11
    assert np.all(np.abs(to_f64(o[0]) - ro) <= 2.0 ** -8 * np.abs(ro) + 2.0 ** -9.4 * spread + extra)


@pytest.mark.gpu
@pytest.mark.parametrize("d", [64, 128])
def test_scales_of_many_magnitudes(ost, d):
    """V scales over 2^30: the power of two that P is taken with follows the
    largest, what falls below 2^-24 of it in float16 is lost: 2^-24 / 64 of the
    largest scale per key and code (6), at most."""
    lens = [700, 90]
    for seed, gain in ((1, 2.0 ** 30), (2, 2.0 ** 12)):
        c = Cache(True, lens, 2, d, 16, 1, -1, 0, seed)
        g = torch.Generator().manual_seed(seed)
        s = c.pools[3]
        c.pools[3] = (s.float() * gain ** (torch.rand(s.shape[:3], generator=g)[..., None] - 0.5)
                      ).to(BF)
        top = float(torch.nan_to_num(c.pools[3].float(), nan=0.0).max())
        _check(ost, True, lens, 8, 2, 1, d, 16, -1, 0, cache=c,
               extra=700 * 2.0 ** -24 / 64 * 6 * top / 100)


@pytest.mark.gpu
@pytest.mark.parametrize("four", [False, True])
@pytest.mark.parametrize("T,left,first", [(4, -1, 0), (4, 20, 3), (3, 1, 0)])
def test_keys_that_only_some_tokens_see_may_hold_anything(ost, four, T, left, first):
    """NaN and infinities in keys and values that a drafted token sees leave the
    tokens before it (and behind its window) as they are."""
    lens, Hq, Hkv, d, page = [50, 97], 4, 2, 128, 16
    c = Cache(four, lens, Hkv, d, page, T, left, first, 31)
    q = random_like_shape((2, Hq, T, d), BF, 32)
    want = _check(ost, four, lens, Hq, Hkv, T, d, page, left, first, cache=c, q=q)
    at = {}
    for b, n in enumerate(lens):                    # the last token's own key
        at[b] = [n - 1]
        if left >= 0 and n - T - left >= first:     # and the first key of the first token's window
            at[b].append(n - T - left)
    for what in (float("nan"), float("inf")):
        bad = [p.clone() for p in c.pools]
        for b in at:
            for j in at[b]:
                pg, slot = int(c.table[b, j // page]), j % page
                for x in (bad[1::2] if four else bad):
                    x[pg, :, slot] = what
        pools = [x.to(DEV) for x in bad]
        f = ost.decode_cache4 if four else ost.decode_window
        o, lse = f(q.to(DEV), *pools, c.table.to(DEV), _ints(lens), window_left=left,
                   n_global=first)
        for b, n in enumerate(lens):
            for i in range(T):
                p = n - T + i
                hit = any(j <= p and (left < 0 or j >= p - left) for j in at[b])
                if hit:
                    assert not torch.isfinite(o[b, :, i]).any() or what == float("inf")
                else:
                    # (bf16: the same products in another order)
                    tol = 2.0 ** -7 * want[0][b, :, i].abs().float() + 2.0 ** -10
                    assert torch.all((o[b, :, i] - want[0][b, :, i]).abs().float() <= tol), (b, i)
                    assert torch.allclose(lse[b, :, i], want[1][b, :, i], atol=2.0 ** -11)


@pytest.mark.gpu
def test_a_bad_group_of_v_spoils_its_elements_alone(ost):
    lens, d = [40], 128
    c = Cache(True, lens, 1, d, 16, 1, -1, 0, 41)
    q = random_like_shape((1, 4, 1, d), BF, 42)
    want, lse0 = _check(ost, True, lens, 4, 1, 1, d, 16, -1, 0, cache=c, q=q)
    for what in (float("nan"), float("inf")):
        pools = [p.clone() for p in c.pools]
        pools[3][int(c.table[0, 1]), 0, 3, 2] = what
        o, lse = ost.decode_cache4(q.to(DEV), *[p.to(DEV) for p in pools], c.table.to(DEV),
                                   _ints(lens))
        assert torch.equal(lse, lse0)
        assert not torch.isfinite(o[..., 64:96]).any() or what == float("inf")
        keep = torch.ones(d, dtype=torch.bool, device=DEV)
        keep[64:96] = False
        tol = 2.0 ** -7 * want.abs().float() + 2.0 ** -10
        assert torch.all(((o - want).abs().float() <= tol)[..., keep])


@pytest.mark.gpu
@pytest.mark.parametrize("four", [False, True])
def test_bad_lengths_and_pages_are_flagged_not_read(ost, four):
    lens, d, page = [40, 40, 40], 64, 16
    c = Cache(four, lens, 2, d, page, 1, -1, 0, 51)
    q = random_like_shape((3, 4, 1, d), BF, 52).to(DEV)
    pools, table, n = c.to(DEV)
    f = ost.decode_cache4 if four else ost.decode_window
    want = f(q, *pools, table, n)
    for bad in (-1, 49):
        o, lse = f(q, *pools, table, _ints([40, bad, 40]))
        assert ost.attn_sync_status() == -7
        assert torch.all(o[1] == 0) and torch.all(torch.isneginf(lse[1]))
        assert torch.equal(o[0], want[0][0]) and torch.equal(lse[2], want[1][2])
    kv = [c.of_request(i, 1, c.values(i)) for i in range(2)]
    for bad in (-1, -2, pools[0].shape[0], 2 ** 31 - 1):
        t = table.clone()
        t[1, 1] = bad                               # keys 16 .. 31 of request 1
        o, lse = f(q, *pools, t, n)
        assert ost.attn_sync_status() == -7
        assert torch.equal(o[0], want[0][0]) and torch.equal(o[2], want[0][2])
        keep = np.r_[0:16, 32:40]
        ro, rl, spread = oracle.decode_window(to_f64(q[1]), kv[0][:, keep], kv[1][:, keep], d ** -0.5)
        assert np.max(np.abs(to_f64(lse[1]) - rl)) <= 2.0 ** -11
        assert np.all(np.abs(to_f64(o[1]) - ro) <= 2.0 ** -8 * np.abs(ro) + 2.0 ** -9.4 * spread)
    # a page that no token sees is not looked at
    t = table.clone()
    t[:, 0] = 2 ** 31 - 1
    f(q, *pools, t, n, window_left=20)
    assert ost.attn_sync_status() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("four", [False, True])
@pytest.mark.parametrize("d,page,T", [(64, 16, 1), (128, 64, 4), (128, 24, 1)])
def test_bad_pages_are_not_seen_whatever_page_0_holds(ost, four, d, page, T):
    lens = [3 * page, 2 * page + 5]
    c = Cache(four, lens, 2, d, page, T, -1, 0, 61)
    c.pools = [torch.cat([torch.full_like(x[:1], float("nan") if x.is_floating_point() else 255), x])
               for x in c.pools]
    c.table = torch.where(c.table >= 0, c.table + 1, c.table).to(torch.int32)
    q = random_like_shape((2, 4, T, d), BF, 62)
    pools, table, n = c.to(DEV)
    table[:, 1] = -1
    f = ost.decode_cache4 if four else ost.decode_window
    o, lse = f(q.to(DEV), *pools, table, n)
    assert ost.attn_sync_status() == -7
    for b, length in enumerate(lens):
        k, v = (c.of_request(i, b, c.values(i)) for i in range(2))
        keep = np.r_[0:page, 2 * page:length]
        # (positions stay: every token sees the keys that are left, but those behind it)
        for i in range(T):
            seen = keep[keep <= length - T + i]
            ro, rl, spread = oracle.decode_window(to_f64(q[b, :, i:i + 1]), k[:, seen], v[:, seen],
                                                  d ** -0.5)
            assert np.max(np.abs(to_f64(lse[b, :, i]) - rl[:, 0])) <= 2.0 ** -11
            assert np.all(np.abs(to_f64(o[b, :, i]) - ro[:, 0])
                          <= 2.0 ** -8 * np.abs(ro[:, 0]) + 2.0 ** -9.4 * spread[:, 0])


@pytest.mark.gpu
def test_agrees_with_paged_decode(ost):
    lens, Hq, Hkv, d, page = [700, 1, 33, 2000], 8, 2, 128, 16
    c = Cache(False, lens, Hkv, d, page, 1, -1, 0, 61)
    q = random_like_shape((4, Hq, d), BF, 62).to(DEV)
    pools, table, n = c.to(DEV)
    o, lse = ost.decode_window(q, *pools, table, n)
    assert o.shape == (4, Hq, d) and lse.shape == (4, Hq)
    o2, lse2 = ost.decode_paged(q, *pools, table, n, 4)
    # each within its own tolerance of the same sums
    assert torch.all((o - o2).abs().float() <= 2.0 ** -7 * o.abs().float() + 2.0 ** -9)
    assert torch.allclose(lse, lse2, atol=2.0 ** -10)


@pytest.mark.gpu
@pytest.mark.parametrize("four", [False, True])
def test_offsets_past_32_bits(ost, four):
    """Keys in the last pages of pools of more than 2^32 bytes."""
    d, Hkv, page = 128, 2, 64
    row = d // 2 if four else 2 * d
    total = (1 << 32) // (Hkv * page * row) + 16
    lens = [300, 500]
    c = Cache(four, lens, Hkv, d, page, 2, 250, 4, 71)
    small = c.pools[0].shape[0]
    q = random_like_shape((2, 8, 2, d), BF, 72)
    want = _check(ost, four, lens, 8, Hkv, 2, d, page, 250, 4, cache=c, q=q)
    big = []
    for p in c.pools:
        x = torch.empty((total, *p.shape[1:]), dtype=p.dtype, device=DEV)
        x[-small:] = p.to(DEV)
        big.append(x)
    table = torch.where(c.table >= 0, c.table + (total - small), c.table).to(DEV)
    f = ost.decode_cache4 if four else ost.decode_window
    got = f(q.to(DEV), *big, table, _ints(lens), window_left=250, n_global=4)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.gpu
@pytest.mark.parametrize("four", [False, True])
def test_streams_graphs_workspaces_and_calls_at_once(ost, four):
    """The same bits on another stream, from a poisoned workspace, from two calls at
    once with workspaces of their own, and from two captured graphs that share one,
    replayed on new lengths."""
    B, Hq, Hkv, T, d, page, cap = 5, 8, 2, 2, 128, 16, 800
    f = ost.decode_cache4 if four else ost.decode_window
    raw = ost.attn_decode_cache4 if four else ost.attn_decode_window
    c = Cache(four, [cap] * B, Hkv, d, page, T, -1, 0, 81)
    pools, table, n = c.to(DEV)
    qs = [random_like_shape((B, Hq, T, d), BF, 82 + i).to(DEV) for i in range(2)]
    lens = [_ints([cap, 3, 0, 511, 640]), _ints([1, cap, 77, 300, 2])]
    kw = dict(window_left=200, n_global=4)
    want = {(i, j): f(qs[i], *pools, table, lens[j], **kw) for i in range(2) for j in range(2)}
    nb = ost.attn_decode_window_workspace_size(B, Hq, Hkv, T, d)
    ws = [torch.full((nb,), 0xff, dtype=torch.uint8, device=DEV) for _ in range(2)]

    def same(got, i, j):
        return torch.equal(got[0], want[i, j][0]) and torch.equal(got[1], want[i, j][1])
    for _ in range(3):
        assert same(f(qs[0], *pools, table, lens[0], workspace=ws[0], **kw), 0, 0)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for _ in range(5):
        a = f(qs[0], *pools, table, lens[0], workspace=ws[0], **kw)
        b = f(qs[1], *pools, table, lens[1], workspace=ws[1], stream=side, **kw)
        d_ = f(qs[1], *pools, table, lens[0], stream=side, **kw)
    torch.cuda.synchronize()
    assert same(a, 0, 0) and same(b, 1, 1) and same(d_, 1, 0)
    graphs, outs = [], []
    held = [t.clone() for t in lens]
    for i in range(2):
        o, lse = torch.empty_like(qs[i]), torch.empty(B, Hq, T, device=DEV)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            raw(qs[i], *pools, table, held[i], o, lse, d ** -0.5, 200, 4, ws[0])
        graphs.append(graph)
        outs.append((o, lse))
    for j in (1, 0, 1):
        for i in range(2):
            held[i].copy_(lens[j])
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        assert same(outs[0], 0, j) and same(outs[1], 1, j)


@pytest.mark.gpu
def test_binding_refusals(ost):
    c = Cache(False, [40, 9], 2, 64, 16, 1, -1, 0, 91)
    (k, v), table, n = c.to(DEV)
    q = random_like_shape((2, 4, 64), BF, 92).to(DEV)
    for bad in (dict(q=q.float()), dict(q=q[:1]), dict(q=q.cpu()), dict(k_pages=k[:, :1]),
                dict(k_pages=k.transpose(0, 1)), dict(v_pages=v.float()), dict(v_pages=v[:2]),
                dict(block_table=table[:1]), dict(block_table=table.long()),
                dict(seq_lens=n[:1]), dict(seq_lens=n.float()),
                dict(workspace=torch.zeros(2, 256, device=DEV).t())):
        with pytest.raises((ValueError, TypeError)):
            ost.decode_window(**{**dict(q=q, k_pages=k, v_pages=v, block_table=table, seq_lens=n),
                                 **bad})
    for bad in (dict(scale=-1.0), dict(n_global=-1), dict(workspace=torch.zeros(256, device=DEV))):
        with pytest.raises(ost.AttnError):
            ost.decode_window(q, k, v, table, n, **bad)
    kc, ks = torch.zeros(*k.shape[:3], 32, dtype=torch.uint8, device=DEV), k[..., :2].contiguous()
    for bad in ((kc, ks, kc, ks[..., :1].contiguous()), (kc, ks.float(), kc, ks.float()),
                (kc.to(torch.int8), ks, kc, ks), (kc[..., :16].contiguous(), ks, kc, ks)):
        with pytest.raises((ValueError, TypeError)):
            ost.decode_cache4(q, *bad, table, n)
