"""Decode of several tokens over paged caches: what one token sees and another
does not leaves the other alone, in value and in time.

Tolerances as in test_decode_window.py: 2^-8 of the result and 2^-9.4 (4 bits) or
2^-10 (bf16) of the row's weighted mean of |v|. In 4 bits a probability times
its scale s enters the product in float16 next to the row's largest scale S at
2^6 and more: where s is far smaller it is off by half a step of the smallest
float16 values, 2^-25 · S / 2^6, which a code carries at most 6 times into the sum
over n keys, divided by Σ p >= 1: n · 6 · 2^-31 · S.
"""

import numpy as np
import pytest
import torch

import oracle
from test_decode_window import BF, DEV, Cache, _ints
from workloads import random_like_shape, to_f64


def _pool_row(c, b, j):
    return int(c.table[b, j // c.page]), j % c.page


@pytest.mark.gpu
@pytest.mark.parametrize("d,page,Hq,T", [(128, 16, 2, 4), (64, 24, 2, 4), (128, 64, 4, 4),
                                         (64, 16, 8, 4), (128, 24, 4, 7)])
@pytest.mark.parametrize("lens,left,first", [([97, 32], -1, 0), ([97, 400], 60, 3),
                                             ([3000, 97], -1, 0), ([6000, 40], 5000, 3)])
@pytest.mark.parametrize("power", [30, 80, -40])
def test_scales_of_keys_that_only_some_tokens_see(ost, d, page, Hq, T, lens, left, first, power):
    """4 bits: a finite scale of V, 2^power, at the last token's own key and at the
    first key of the first token's window. (2^-40: the largest there is for nobody.)"""
    Hkv = 2
    c = Cache(True, lens, Hkv, d, page, T, left, first, 131)
    q = random_like_shape((len(lens), Hq, T, d), BF, 132)
    for b, n in enumerate(lens):
        for j in [n - 1] + ([n - T - left] if left >= 0 and n - T - left >= first else []):
            pg, slot = _pool_row(c, b, j)
            c.pools[3][pg, :, slot] = 2.0 ** power
    pools, table, n = c.to(DEV)
    o, lse = ost.decode_cache4(q.to(DEV), *pools, table, n, window_left=left, n_global=first)
    assert ost.attn_sync_status() == 0
    kv = [c.values(i) for i in range(2)]
    scales = to_f64(c.pools[3])
    for b, n in enumerate(lens):
        k, v = (c.of_request(i, b, kv[i]) for i in range(2))
        ro, rl, spread = oracle.decode_window(to_f64(q[b]), k, v, d ** -0.5, left, first)
        assert np.max(np.abs(to_f64(lse[b]) - rl)) <= 2.0 ** -11 + n * 2.0 ** -24
        for i in range(T):
            p = n - T + i
            seen = [j for j in range(n) if j < first or (j <= p and (left < 0 or j >= p - left))]
            top = max(scales[_pool_row(c, b, j)[0], :, j % page].max() for j in seen)
            tol = (2.0 ** -8 * np.abs(ro[:, i]) + (2.0 ** -9.4 + n * 2.0 ** -23) * spread[:, i] +
                   n * 6 * 2.0 ** -31 * top)
            err = np.abs(to_f64(o[b, :, i]) - ro[:, i])
            assert np.all(err <= tol), (b, i, np.max(err / tol))


@pytest.mark.gpu
@pytest.mark.parametrize("d,page,Hq,T", [(128, 16, 8, 1), (64, 24, 16, 1), (128, 64, 8, 4),
                                         (64, 16, 12, 3)])
@pytest.mark.parametrize("lens", [[97, 300], [5000, 33]])
def test_infinite_values_that_a_token_sees(ost, d, page, Hq, T, lens):
    """bf16: an infinite element of V is infinite in O for the tokens that see it,
    NaN next to the other infinity; other tokens and elements stay."""
    inf = float("inf")
    c = Cache(False, lens, 2, d, page, T, -1, 0, 141)
    q = random_like_shape((len(lens), Hq, T, d), BF, 142)
    for b, n in enumerate(lens):
        for e, j, x in ((3, n // 2, inf), (8, n // 3, -inf), (20, n - 1, inf), (21, n - 1, -inf),
                        (40, n // 2, inf), (40, n // 2 + 1, -inf), (50, 7, inf), (50, n - 2, inf)):
            pg, slot = _pool_row(c, b, j)
            c.pools[1][pg, :, slot, e] = x
    pools, table, n = c.to(DEV)
    o, lse = ost.decode_window(q.to(DEV), *pools, table, n)
    assert ost.attn_sync_status() == 0
    kv = [c.values(i) for i in range(2)]
    for b, n in enumerate(lens):
        k, v = (c.of_request(i, b, kv[i]) for i in range(2))
        with np.errstate(invalid="ignore"):
            ro, rl, spread = oracle.decode_window(to_f64(q[b]), k, v, d ** -0.5)
            assert np.max(np.abs(to_f64(lse[b]) - rl)) <= 2.0 ** -11 + n * 2.0 ** -24
            got, finite = to_f64(o[b]), np.isfinite(ro)
            assert np.array_equal(np.isnan(got), np.isnan(ro)), b
            assert np.array_equal(got[~finite & ~np.isnan(ro)], ro[~finite & ~np.isnan(ro)]), b
            tol = 2.0 ** -8 * np.abs(ro) + (2.0 ** -10 + n * 2.0 ** -23) * spread
            assert np.all(np.abs(got[finite] - ro[finite]) <= tol[finite]), b


@pytest.mark.gpu
@pytest.mark.parametrize("d,T", [(128, 1), (64, 4)])
def test_infinite_scales_of_v_that_a_token_sees(ost, d, T):
    """4 bits: the elements of a group whose scale is infinite are infinities of their
    codes' signs, NaN where a code is 0."""
    lens, page = [97, 300], 16
    c = Cache(True, lens, 2, d, page, T, -1, 0, 151)
    q = random_like_shape((2, 4, T, d), BF, 152)
    for b, n in enumerate(lens):
        for group, j in ((0, n // 2), (1, n - 1)):
            pg, slot = _pool_row(c, b, j)
            c.pools[3][pg, :, slot, group] = float("inf")
    pools, table, n = c.to(DEV)
    o, lse = ost.decode_cache4(q.to(DEV), *pools, table, n)
    with np.errstate(invalid="ignore"):
        kv = [c.values(i) for i in range(2)]
        for b, n in enumerate(lens):
            k, v = (c.of_request(i, b, kv[i]) for i in range(2))
            ro, rl, spread = oracle.decode_window(to_f64(q[b]), k, v, d ** -0.5)
            assert np.max(np.abs(to_f64(lse[b]) - rl)) <= 2.0 ** -11
            got, finite = to_f64(o[b]), np.isfinite(ro)
            assert (~finite).any() and finite.any()
            assert np.array_equal(np.isnan(got), np.isnan(ro)), b
            assert np.array_equal(got[~finite & ~np.isnan(ro)], ro[~finite & ~np.isnan(ro)]), b
            tol = 2.0 ** -8 * np.abs(ro) + 2.0 ** -9.4 * spread
            assert np.all(np.abs(got[finite] - ro[finite]) <= tol[finite]), b


@pytest.mark.gpu
@pytest.mark.parametrize("Hq,T,d,page,left,first", [(1, 40, 128, 16, -1, 0), (3, 20, 64, 16, 25, 2),
                                                   (3, 20, 128, 24, -1, 0), (5, 7, 64, 48, 9, 0),
                                                   (2, 33, 64, 24, 40, 20)])
def test_values_that_are_not_finite_among_many_tokens(ost, Hq, T, d, page, left, first):
    """bf16: blocks of 16 query rows that hold some of the tokens, or tokens of two
    heads; NaN in V at keys that some of the tokens see."""
    lens = [max(T, 30) + 45, T]
    c = Cache(False, lens, 1, d, page, T, left, first, 161)
    q = random_like_shape((2, Hq, T, d), BF, 162)
    for b, n in enumerate(lens):
        for e, j in ((1, n - 1), (9, n - T // 2), (33, n - T + 1), (60, max(0, n - T - left + 3))):
            pg, slot = _pool_row(c, b, j)
            c.pools[1][pg, :, slot, e] = float("nan") if e != 9 else float("-inf")
    pools, table, n = c.to(DEV)
    o, lse = ost.decode_window(q.to(DEV), *pools, table, n, window_left=left, n_global=first)
    assert ost.attn_sync_status() == 0
    kv = [c.values(i) for i in range(2)]
    for b, n in enumerate(lens):
        k, v = (c.of_request(i, b, kv[i]) for i in range(2))
        with np.errstate(invalid="ignore"):
            ro, rl, spread = oracle.decode_window(to_f64(q[b]), k, v, d ** -0.5, left, first)
        got, finite = to_f64(o[b]), np.isfinite(ro)
        assert (~finite).any() and np.array_equal(np.isnan(got), np.isnan(ro)), b
        assert np.array_equal(got[np.isinf(ro)], ro[np.isinf(ro)]), b
        tol = 2.0 ** -8 * np.abs(ro) + 2.0 ** -10 * spread
        assert np.all(np.abs(got[finite] - ro[finite]) <= tol[finite]), b
        assert np.max(np.abs(to_f64(lse[b]) - rl)) <= 2.0 ** -11


@pytest.mark.gpu
@pytest.mark.parametrize("what", ["behind the last key", "at the last key"])
def test_what_rows_hold_does_not_change_the_time(ost, what):
    """A chunk of 2040 tokens: NaN behind the last key of its last page, or in the
    last token's own value, against a page without (one pass per token of the
    request over the tile took 30 times as long)."""
    T, d, page = 2040, 128, 16
    c = Cache(False, [T], 1, d, page, T, -1, 0, 171)
    q = random_like_shape((1, 1, T, d), BF, 172).to(DEV)
    pools, table, n = c.to(DEV)
    last = pools[1][int(c.table[0, -1])]
    clean, spoilt = pools[1].clone(), pools[1].clone()
    clean[int(c.table[0, -1]), :, T % page:] = 0
    if what == "at the last key":
        spoilt.copy_(clean)
        spoilt[int(c.table[0, -1]), :, T % page - 1] = float("nan")
    assert not torch.isfinite(last[:, T % page:]).any()
    times = []
    for v in (clean, spoilt, clean, spoilt):
        ost.decode_window(q, pools[0], v, table, n)
        a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
        a.record()
        for _ in range(10):
            o, _ = ost.decode_window(q, pools[0], v, table, n)
        b.record()
        torch.cuda.synchronize()
        times.append(a.elapsed_time(b))
        assert torch.isfinite(o[:, :, :-1]).all()
    # (the passes over the last tile of a block are 17 instead of one, of its 128 tiles)
    assert min(times[1::2]) < 2 * min(times[::2]), times


@pytest.mark.gpu
@pytest.mark.parametrize("d,Hq,T", [(128, 4, 1), (128, 16, 1), (64, 4, 4), (64, 16, 1)])
def test_largest_scales_of_k(ost, d, Hq, T):
    """4 bits: sums of a row are of queries below 2^9 times codes up to 6, scaled: 128 · 6 ·
    2^9 · 2^109 < 2^128 where all elements are as large as can be. One key has
    them, the others are smaller by 2^8: it takes all of the probability."""
    lens, page = [97, 300], 16
    c = Cache(True, lens, 1, d, page, T, -1, 0, 181)
    q = torch.full((2, Hq, T, d), 2.0 ** -100 * (2 - 2.0 ** -7), dtype=BF)
    for b in range(2):
        for j in range(lens[b]):
            pg, slot = _pool_row(c, b, j)
            c.pools[0][pg, :, slot] = 0x77 if j == 20 else 0x55
            c.pools[1][pg, :, slot] = 2.0 ** 109 * (1 - 2.0 ** -8) if j == 20 else 2.0 ** 101
    pools, table, n = c.to(DEV)
    o, lse = ost.decode_cache4(q.to(DEV), *pools, table, n)
    assert torch.isfinite(lse).all()
    kv = [c.values(i) for i in range(2)]
    for b in range(2):
        k, v = (c.of_request(i, b, kv[i]) for i in range(2))
        ro, rl, spread = oracle.decode_window(to_f64(q[b]), k, v, d ** -0.5)
        assert np.all(rl > 2.0 ** 14)
        assert np.all(np.abs(to_f64(lse[b]) - rl) <= (d + 8) * 2.0 ** -24 * rl)
        # (a probability of 1 in float16 times its scale: exact; one rounding of the result)
        assert np.all(np.abs(to_f64(o[b]) - ro) <= 2.0 ** -8 * np.abs(ro) + 2.0 ** -9.4 * spread)
