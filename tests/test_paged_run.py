"""The paged-cache operators together, as a serving loop uses them: prompts of
uneven lengths are appended in chunks (rotated, in bf16 or in 4 bits), each chunk
attends to what is cached so far, then tokens are drafted, several a step, decoded
under a window with first tokens that stay visible, and those that are not accepted
are taken back by the lengths alone. Every step is checked against the float64
oracle fed with the tensors that step read.

Tolerances are those of the calls' own tests (test_decode_window.py: 2^-10 of the
weighted mean of |v|, in 4 bits 2^-9.4, and half a step of the bf16 result;
attn_fwd_masked: 1e-2 of the largest output).
"""

import numpy as np
import pytest
import torch

import oracle
from workloads import random_like_shape, to_f64

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF = torch.bfloat16


def _ints(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


class Pools:
    """Pages for B requests in shuffled order; in 4 bits codes and scales."""

    def __init__(self, four, B, Hkv, d, page, width, seed):
        self.four = four
        g = torch.Generator().manual_seed(seed)
        total = B * width + 3
        self.table = torch.randperm(total, generator=g)[:B * width].view(B, width) \
            .to(torch.int32).to(DEV)
        row = (total, Hkv, page)
        if four:
            self.parts = [torch.full((*row, n), x, dtype=t, device=DEV) for _ in range(2)
                          for n, x, t in ((d // 2, 255, torch.uint8), (d // 32, float("nan"), BF))]
        else:
            self.parts = [torch.full((*row, d), float("nan"), dtype=BF, device=DEV)
                          for _ in range(2)]

    def rows(self, b, n):
        """Keys and values of request b's first n rows, float64 [Hkv, n, d]."""
        out = []
        pages = self.table[b].long()
        for i in range(2):
            if self.four:
                codes, scales = (p[pages].cpu() for p in self.parts[2 * i:2 * i + 2])
                x = oracle.values4(oracle.unpack4(codes.numpy()), to_f64(scales))
            else:
                x = to_f64(self.parts[i][pages].cpu())
            out.append(x.transpose(1, 0, 2, 3).reshape(x.shape[1], -1, x.shape[-1])[:, :n])
        return out


@pytest.mark.parametrize("four", [False, True])
@pytest.mark.parametrize("d,Hq,Hkv,page", [(128, 8, 2, 16), (64, 6, 2, 24), (128, 4, 1, 64)])
def test_serving_loop(ost, four, d, Hq, Hkv, page):
    B, chunk, left, first, T, width = 4, 70, 100, 4, 3, -(-260 // page)
    scale, w = d ** -0.5, ost.rope_frequencies(d, device=DEV)
    cache = Pools(four, B, Hkv, d, page, width, 1)
    append = ost.cache_append4 if four else ost.cache_append
    decode = ost.decode_cache4 if four else ost.decode_window
    slack = 2.0 ** -9.4 if four else 2.0 ** -10

    def check(q, o, lse, lens):
        for b, n in enumerate(lens):
            k, v = cache.rows(b, n)
            ro, rl, spread = oracle.decode_window(to_f64(q[b]), k, v, scale, left, first)
            assert np.all(np.abs(to_f64(o[b]) - ro) <= 2.0 ** -8 * np.abs(ro) + slack * spread)
            seen = np.isfinite(rl)
            assert np.array_equal(np.isfinite(to_f64(lse[b])), seen)
            assert np.all(np.abs(to_f64(lse[b]) - rl)[seen] <= 2.0 ** -11)

    # prompts, in chunks; a request whose prompt ends sooner is padded
    prompt, lens = [150, 70, 1, 203], np.zeros(B, int)
    while lens.max() < max(prompt):
        new = np.minimum(np.array(prompt) - lens, chunk)
        lens += new
        x = random_like_shape((B, chunk, Hq + 2 * Hkv, d), BF, 10 + int(lens.sum())).to(DEV)
        q0, k0, v0 = (t.transpose(1, 2) for t in x.split([Hq, Hkv, Hkv], dim=2))
        q = append(q0, k0, v0, *cache.parts, cache.table, _ints(lens.tolist()), w,
                   new_lens=_ints(new.tolist()))
        for b in range(B):
            if new[b] == 0:
                continue
            # the queries, turned by their positions
            pos = np.arange(lens[b] - new[b], lens[b])
            assert torch.equal(q[b, :, :new[b]], ost.rope(
                q0[b:b + 1, :, :new[b]], None, _ints([pos.tolist()]), w)[0][0])
            # the chunk over all that is cached
            if four:
                kb, vb = ost.cache_read4(*cache.parts, cache.table[b:b + 1].contiguous(),
                                         _ints([int(lens[b])]), length=int(lens[b]))
                k64, v64 = cache.rows(b, lens[b])
                assert np.all(np.abs(to_f64(kb[0]) - k64) <= 2.0 ** -8 * np.abs(k64))
                assert np.all(np.abs(to_f64(vb[0]) - v64) <= 2.0 ** -8 * np.abs(v64))
            else:
                kb, vb = (torch.from_numpy(t).to(BF).to(DEV)[None] for t in cache.rows(b, lens[b]))
            if new[b] < 2:
                continue
            qb = q[b:b + 1, :, :new[b]].contiguous()
            o = torch.empty_like(qb)
            lse = torch.empty(qb.shape[:3], device=DEV)
            end = torch.from_numpy(pos + 1).to(torch.int32).to(DEV)
            begin = torch.zeros_like(end)
            mask = ost.make_mask(row_kv_start=begin, row_kv_end=end)
            ost.attn_fwd_masked(qb, kb, vb, o, lse, scale, mask)
            ro, _, _ = oracle.decode_window(to_f64(qb[0]), to_f64(kb[0]), to_f64(vb[0]), scale)
            assert np.max(np.abs(to_f64(o[0]) - ro)) <= 1e-2 * np.max(np.abs(ro))
        # the same chunk by the decode call, under the window
        full = [b for b in range(B) if new[b] == chunk]
        if full:
            qc = q[full].contiguous()
            oc, lc = decode(qc, *cache.parts, cache.table[full].contiguous(),
                            _ints(lens[full].tolist()), left, first)
            for i, b in enumerate(full):
                k, v = cache.rows(b, lens[b])
                ro, rl, spread = oracle.decode_window(to_f64(qc[i]), k, v, scale, left, first)
                assert np.all(np.abs(to_f64(oc[i]) - ro)
                              <= 2.0 ** -8 * np.abs(ro) + slack * spread)

    # drafts of T tokens, of which 1 .. T stay; the third request stops after two steps
    rng = np.random.default_rng(5)
    for step in range(8):
        new = np.array([T, T, T if step < 2 else 0, T])
        lens = lens + new
        x = random_like_shape((B, T, Hq + 2 * Hkv, d), BF, 100 + step).to(DEV)
        q0, k0, v0 = (t.transpose(1, 2) for t in x.split([Hq, Hkv, Hkv], dim=2))
        n = _ints(lens.tolist())
        out = torch.zeros(B, Hq, T, d, dtype=BF, device=DEV)
        q = append(q0, k0, v0, *cache.parts, cache.table, n, w, new_lens=_ints(new.tolist()),
                   out=out)
        o, lse = decode(q, *cache.parts, cache.table, n, left, first)
        check(q, o, lse, lens)
        lens = lens - np.where(new > 0, rng.integers(0, T, B), 0)
    # one token without a token axis
    lens = lens + 1
    n = _ints(lens.tolist())
    x = random_like_shape((B, Hq + 2 * Hkv, d), BF, 200).to(DEV)
    q = append(x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:], *cache.parts, cache.table, n, w)
    o, lse = decode(q, *cache.parts, cache.table, n, left, first)
    check(q[:, :, None], o[:, :, None], lse[:, :, None], lens)
    assert ost.attn_sync_status() == 0


@pytest.mark.parametrize("four", [False, True])
@pytest.mark.parametrize("B,left", [(3, 60), (40, 500)])        # clusters; shares and a join
def test_library_calls_alone_hand_over_rows_and_queries(ost, four, B, left):
    """Rows and queries that one call writes and the next reads, with no other kernel
    between them: the same results as with the device idle between calls, also from
    a captured graph."""
    Hq, Hkv, d, page, width, T, steps = 8, 2, 128, 16, 40, 2, 12
    w = ost.rope_frequencies(d, device=DEV)
    x = [random_like_shape((B, T, Hq + 2 * Hkv, d), BF, 300 + i).to(DEV) for i in range(steps)]
    lens = [_ints([(531 * b) % 600 + T * (i + 1) for b in range(B)]) for i in range(steps)]
    start = random_like_shape((B, Hkv, 640, d), BF, 400).to(DEV)
    nb = ost.attn_decode_window_workspace_size(B, Hq, Hkv, T, d)
    ws = torch.empty(nb, dtype=torch.uint8, device=DEV)
    append = ost.attn_cache_append4 if four else ost.attn_cache_append
    decode = ost.attn_decode_cache4 if four else ost.attn_decode_window
    full = _ints([640] * B)

    def run(idle, graph=None):
        cache = Pools(four, B, Hkv, d, page, width, 7)
        append(None, start, start, *cache.parts, cache.table, full, None, w)
        q = torch.zeros(B, Hq, T, d, dtype=BF, device=DEV)
        outs = [(torch.zeros_like(q), torch.zeros(B, Hq, T, device=DEV)) for _ in range(steps)]
        back = [torch.zeros(B, Hkv, 640, d, dtype=BF, device=DEV) for _ in range(2)]
        torch.cuda.synchronize()
        after = torch.cuda.synchronize if idle else (lambda: None)

        def calls():
            for (o, lse), xi, n in zip(outs, x, lens):
                q0, k0, v0 = (t.transpose(1, 2) for t in xi.split([Hq, Hkv, Hkv], dim=2))
                append(q0, k0, v0, *cache.parts, cache.table, n, q, w)
                after()
                decode(q, *cache.parts, cache.table, n, o, lse, d ** -0.5, left, 4, ws)
                after()
            if four:
                ost.attn_cache_read4(*cache.parts, cache.table, lens[-1], *back)
        if graph is None:
            calls()
        else:
            with torch.cuda.graph(graph):
                calls()
            graph.replay()
        torch.cuda.synchronize()
        return [t for o in outs for t in o] + back + [p.view(torch.uint8) for p in cache.parts]
    want = run(True)
    for _ in range(4):
        assert all(torch.equal(a, b) for a, b in zip(want, run(False)))
    assert all(torch.equal(a, b) for a, b in zip(want, run(False, torch.cuda.CUDAGraph())))
    assert ost.attn_sync_status() == 0


@pytest.mark.parametrize("four", [False, True])
def test_allocating_calls_captured_and_replayed(ost, four):
    """Each call allocates its outputs and workspace inside a captured graph; two
    graphs from one pool, replayed in turn on new inputs, give what the same calls
    give outside."""
    B, Hq, Hkv, d, page, width, T = 6, 8, 4, 64, 32, 20, 2
    w = ost.rope_frequencies(d, device=DEV)
    cache = Pools(four, B, Hkv, d, page, width, 11)
    append = ost.cache_append4 if four else ost.cache_append
    decode = ost.decode_cache4 if four else ost.decode_window
    start = random_like_shape((B, Hkv, 640, d), BF, 500).to(DEV)
    append(None, start, start, *cache.parts, cache.table, _ints([640] * B), w)

    def inputs(seed):
        g = torch.Generator().manual_seed(seed)
        return [random_like_shape((B, Hq, T, d), BF, seed).to(DEV),
                random_like_shape((B, Hkv, T, d), BF, seed + 1).to(DEV),
                random_like_shape((B, Hkv, T, d), BF, seed + 2).to(DEV),
                torch.randint(T, 641, (B,), generator=g).to(torch.int32).to(DEV)]

    def calls(q, k, v, n):
        qr = append(q, k, v, *cache.parts, cache.table, n, w)
        o, lse = decode(qr, *cache.parts, cache.table, n, 300, 4)
        more = ost.cache_read4(*cache.parts, cache.table, n) if four else ()
        return (qr, o, lse, *more)
    x = inputs(510)
    calls(*x)
    torch.cuda.synchronize()
    graphs, outs, pool = [], [], None
    for _ in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, pool=pool):
            outs.append(calls(*x))
        pool = graph.pool()
        graphs.append(graph)
    for seed in (520, 540, 560):
        for a, b in zip(x, inputs(seed)):
            a.copy_(b)
        want = calls(*x)
        for graph, got in zip(graphs, outs):
            for t in got:
                t.view(torch.uint8).fill_(0xff)
            graph.replay()
            torch.cuda.synchronize()
            assert all(torch.equal(p, r) for p, r in zip(got, want))
