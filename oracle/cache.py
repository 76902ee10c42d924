"""Float64 reference for the operators around the KV cache.

TEST INFRASTRUCTURE ONLY (see the package docstring). Sources:

* KV-compression post (shreyansh26.github.io feed): cached keys carry their
  rotary position (learned compaction un-rotates them first); eviction
  policies keep the first tokens (attention sinks), a recent window and the
  keys with the highest attention weight, summed over the query heads of a KV
  head (the grouped heads of the SnapKV code).
* ML notes (haolingpu.github.io), KV-cache Q&A: requests that share a prefix
  share its cache blocks.

Readings where the pages are silent: a pair is turned by p·w (counter-
clockwise in the (a, b) plane); ties between scores go to the lowest index; a
NaN score ranks as -inf. Every function is pinned on the CPU by the tests of
its operator: ``tests/test_rope.py``, ``tests/test_decode_shared.py``,
``tests/test_key_weights.py`` and ``tests/test_evict.py``.
"""

from __future__ import annotations

import numpy as np

from .attention import NEG_INF, gather_paged, logsumexp_rows, softmax_rows


def _inverse_two_pi(bits: int) -> int:
    """floor(2^bits / (2π)), π by Machin's formula in integers."""
    unity = 1 << (bits + 32)

    def arctan_inv(x: int) -> int:
        total = term = unity // x
        n, sign = 3, -1
        while term:
            term //= x * x
            total += sign * (term // n)
            n, sign = n + 2, -sign
        return total

    pi = 4 * (4 * arctan_inv(5) - arctan_inv(239))
    return (unity << bits) // (2 * pi)


_BITS = 1300                      # covers every finite float64 frequency below 2^100
_INV_2PI = _inverse_two_pi(_BITS)


def rope_angles(positions: np.ndarray, inv_freq: np.ndarray) -> np.ndarray:
    """p·w modulo one turn, in (-π, π], from exact integers: positions [B, N]
    int, inv_freq [F] float64 -> [B, N, F] float64."""
    pos = np.asarray(positions)
    out = np.empty(pos.shape + (len(inv_freq),))
    one = 1 << _BITS
    for f, w in enumerate(inv_freq):
        num, den = float(w).as_integer_ratio()          # den is a power of two
        step = num * _INV_2PI // den                    # turns per position, fixed point
        for at, p in np.ndenumerate(pos):
            t = (int(p) * step) % one
            if t > one // 2:
                t -= one
            out[at + (f,)] = 2 * np.pi * (t >> (_BITS - 80)) * 2.0 ** -80
    return out


def rope(x: np.ndarray, positions: np.ndarray, inv_freq: np.ndarray, interleaved: bool = False,
         magnitude: float = 1.0, inverse: bool = False) -> np.ndarray:
    """Rotary positions of x [B, H, N, d]; positions [B, N]."""
    r = 2 * len(inv_freq)
    ang = rope_angles(positions, inv_freq)[:, None]     # [B, 1, N, r/2]
    c = magnitude * np.cos(ang)
    s = magnitude * np.sin(-ang if inverse else ang)
    a_at = np.arange(0, r, 2) if interleaved else np.arange(r // 2)
    b_at = a_at + 1 if interleaved else a_at + r // 2
    y = np.array(x, dtype=np.float64)
    y[..., a_at] = x[..., a_at] * c - x[..., b_at] * s
    y[..., b_at] = x[..., b_at] * c + x[..., a_at] * s
    return y


def decode_shared(q, k_prefix, v_prefix, prefix_table, prefix_lens, prefix_start, k_pages,
                  v_pages, block_table, seq_lens, scale):
    """One query token per request over its prefix's keys followed by its
    own: requests prefix_start[p] .. prefix_start[p + 1] - 1 share prefix p,
    requests outside have none. Pages [n, Hkv, page_size, d]."""
    B, Hq, d = q.shape
    Hkv = k_pages.shape[1]
    o, lse = np.zeros((B, Hq, d)), np.full((B, Hq), NEG_INF)
    for b in range(B):
        k = [gather_paged(k_pages, block_table[b], int(seq_lens[b]), k_pages.shape[2])]
        v = [gather_paged(v_pages, block_table[b], int(seq_lens[b]), v_pages.shape[2])]
        for p in range(len(prefix_lens)):
            if prefix_start[p] <= b < prefix_start[p + 1]:
                n = int(prefix_lens[p])
                k.insert(0, gather_paged(k_prefix, prefix_table[p], n, k_prefix.shape[2]))
                v.insert(0, gather_paged(v_prefix, prefix_table[p], n, v_prefix.shape[2]))
        k, v = np.concatenate(k, 1), np.concatenate(v, 1)
        if k.shape[1] == 0:
            continue
        for h in range(Hq):
            g = h // (Hq // Hkv)
            sc = scale * (k[g] @ q[b, h])
            o[b, h] = softmax_rows(sc[None, :])[0] @ v[g]
            lse[b, h] = logsumexp_rows(sc[None, :])[0]
    return o, lse


def key_weights(q, k, lse, scale, causal=True):
    """Attention weight each key received: q [Hq, T, d] are the last T of the
    n positions of k [Hkv, n, d] (key j visible to query i iff
    j <= n - T + i), lse [Hq, T]; summed over queries and the heads of a KV
    head: [Hkv, n]. A query with lse = -inf gives nothing."""
    Hq, T, _ = q.shape
    Hkv, n, _ = k.shape
    out = np.zeros((Hkv, n))
    for h in range(Hq):
        g = h // (Hq // Hkv)
        for i in range(T):
            last = min(n, n - T + i + 1) if causal else n
            if last <= 0 or lse[h, i] == NEG_INF:
                continue
            out[g, :last] += np.exp(scale * (k[g, :last] @ q[h, i]) - lse[h, i])
    return out


def evict(scores, n_keep, n_sink=0, n_recent=0):
    """Indices kept, in order, of the n scores of one KV head: all when
    n <= n_keep, else the first n_sink, the last n_recent and the best of the
    others (higher score first, then lower index; NaN ranks as -inf)."""
    n = len(scores)
    if n <= n_keep:
        return np.arange(n)
    middle = range(n_sink, n - n_recent)
    rank = sorted(middle, key=lambda j: (np.inf if np.isnan(scores[j]) else -scores[j], j))
    best = rank[:n_keep - n_sink - n_recent]
    return np.array(sorted([*range(n_sink), *best, *range(n - n_recent, n)]), dtype=np.int64)

