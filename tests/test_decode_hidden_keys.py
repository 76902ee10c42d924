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
            assert np.all(np.abs(got - ro)[finite] <= tol[finite]), b


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
            assert np.all(np.abs(got - ro)[finite] <= tol[finite]), b
