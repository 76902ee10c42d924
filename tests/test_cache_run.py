"""The cache operators together, as a serving loop uses them: prompts behind a
shared prefix are rotated and cached, decode steps read prefix and own keys
and add up the weight each own key received, the caches are cut to the keys
that received most, and decoding goes on over what is left. Every step is
checked against the float64 oracle fed with the tensors that step read.
"""

import numpy as np
import pytest
import torch

import oracle
from workloads import random_like_shape, to_f64

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def _close(got, ref, tol=1e-2):
    err, mx = np.max(np.abs(to_f64(got) - ref)), np.max(np.abs(ref))
    assert err <= tol * mx, (err, mx)


@pytest.mark.parametrize("d,Hq,Hkv", [(128, 8, 2), (64, 4, 4)])
def test_serving_loop(ost, d, Hq, Hkv):
    B, P, N, steps, cap, keep = 6, 300, 90, 5, 128, 40
    scale, w = d ** -0.5, ost.rope_frequencies(d, device=DEV)
    bf = torch.bfloat16

    def rotated_ref(x, pos):
        return oracle.rope(to_f64(x), pos.cpu().numpy(), w.cpu().numpy())

    # the shared prefix: rotated once, one page of P keys
    kp0 = random_like_shape((1, Hkv, P, d), bf, 1).to(DEV)
    vp = random_like_shape((1, Hkv, P, d), bf, 2).to(DEV)
    ppos = torch.arange(P, dtype=torch.int32, device=DEV)[None]
    kp, _ = ost.rope(kp0, None, ppos, w)
    _close(kp, rotated_ref(kp0, ppos), 2 ** -8 * 1.01)

    # each request's own prompt, at the positions behind the prefix, into caches of `cap` keys
    k = torch.zeros(B, Hkv, cap, d, dtype=bf, device=DEV)
    v = torch.zeros(B, Hkv, cap, d, dtype=bf, device=DEV)
    qkv = random_like_shape((B, N, Hq + 2 * Hkv, d), bf, 3).to(DEV)
    pos = (P + torch.arange(N, dtype=torch.int32, device=DEV)).expand(B, N).contiguous()
    q0, k0 = qkv[:, :, :Hq].transpose(1, 2), qkv[:, :, Hq:Hq + Hkv].transpose(1, 2)
    q = torch.empty(B, Hq, N, d, dtype=bf, device=DEV)
    ost.rope(q0, k0, pos, w, out=(q, k[:, :, :N]))
    v[:, :, :N] = qkv[:, :, Hq + Hkv:].transpose(1, 2)
    _close(k[:, :, :N], rotated_ref(k0, pos), 2 ** -8 * 1.01)
    assert torch.all(k[:, :, N:] == 0)

    # weights of the prompt's last 16 tokens over the own keys
    _, lse = ost.forward(q, k[:, :, :N].contiguous(), v[:, :, :N].contiguous(), causal=True)
    lens = torch.full((B,), N, dtype=torch.int32, device=DEV)
    score = torch.zeros(B, Hkv, cap, device=DEV)
    qw, lw = q[:, :, -16:].contiguous(), lse[:, :, -16:].contiguous()
    ost.key_weights(qw, k, lw, out=score, seq_lens=lens)
    ref = np.stack([oracle.key_weights(to_f64(qw[b]), to_f64(k[b, :, :N]), to_f64(lw[b]), scale)
                    for b in range(B)])
    _close(score[:, :, :N], ref, 1e-3)

    table = torch.arange(B, dtype=torch.int32, device=DEV)[:, None].contiguous()
    ptable = torch.zeros(1, 1, dtype=torch.int32, device=DEV)
    plen = torch.tensor([P], dtype=torch.int32, device=DEV)
    pstart = torch.tensor([0, B], dtype=torch.int32, device=DEV)

    def step(k, v, score, lens, cap, seed, at):
        """One token: rotate, append, decode, accumulate; returns the score reference."""
        x = random_like_shape((B, Hq + 2 * Hkv, d), bf, seed).to(DEV)
        p = torch.full((B,), at, dtype=torch.int32, device=DEV)
        qt, kt = ost.rope(x[:, :Hq], x[:, Hq:Hq + Hkv], p, w)
        rows = torch.arange(B, device=DEV)
        k[rows, :, lens.long()] = kt
        v[rows, :, lens.long()] = x[:, Hq + Hkv:]
        lens += 1
        o, lse = ost.decode_shared(qt, kp, vp, ptable, plen, pstart, k, v, table, lens)
        pages = [to_f64(t) for t in (kp, vp)], [to_f64(t) for t in (k, v)]
        o_ref, lse_ref = oracle.decode_shared(
            to_f64(qt), *pages[0], np.zeros((1, 1), int), np.array([P]), np.array([0, B]),
            *pages[1], np.arange(B)[:, None], lens.cpu().numpy(), scale)
        _close(o, o_ref)
        assert np.max(np.abs(to_f64(lse) - lse_ref)) <= 1e-3
        before = to_f64(score)
        ost.key_weights(qt, k, lse, prev=score, out=score, seq_lens=lens, block_table=table)
        for b in range(B):
            n = int(lens[b])
            ref = before[b, :, :n] + oracle.key_weights(
                to_f64(qt[b, :, None]), pages[1][0][b, :, :n], to_f64(lse[b, :, None]), scale)
            assert np.max(np.abs(to_f64(score[b, :, :n]) - ref)) <= 1e-3 * np.max(ref)
            assert np.array_equal(to_f64(score[b, :, n:]), before[b, :, n:])

    for i in range(steps):
        step(k, v, score, lens, cap, 10 + i, P + N + i)

    # cut to `keep` keys in caches with room to grow, then go on
    room = keep + steps
    out = (torch.zeros(B, Hkv, room, d, dtype=bf, device=DEV),
           torch.zeros(B, Hkv, room, d, dtype=bf, device=DEV),
           torch.zeros(B, Hkv, room, device=DEV),
           torch.empty(B, Hkv, keep, dtype=torch.int32, device=DEV),
           torch.empty(B, dtype=torch.int32, device=DEV))
    ost.evict(k, v, score, keep, n_sink=2, n_recent=8, seq_lens=lens, block_table=table, out=out)
    k2, v2, score2, kept, lens2 = out
    assert torch.all(lens2 == keep)
    for b in range(B):
        for h in range(Hkv):
            at = oracle.evict(to_f64(score[b, h, :N + steps]), keep, 2, 8)
            assert np.array_equal(kept[b, h].cpu().numpy(), at)
            assert torch.equal(k2[b, h, :keep], k[b, h, at]) and \
                torch.equal(v2[b, h, :keep], v[b, h, at]) and \
                torch.equal(score2[b, h, :keep], score[b, h, at])
    for i in range(steps):
        step(k2, v2, score2, lens2, room, 50 + i, P + N + steps + i)
    assert ost.attn_sync_status() == 0


def test_library_calls_alone_hand_over_queries_and_lengths(ost):
    """Queries, lengths and caches that one call rewrites in place and the next
    reads, with no other kernel of any kind between them: the same results as
    with the device idle between calls."""
    B, Hq, Hkv, d, L, P, T, keep = 12, 8, 2, 128, 200, 900, 80, 48
    bf, steps = torch.bfloat16, 8
    w = ost.rope_frequencies(d, device=DEV)
    q0 = random_like_shape((B, Hq, d), bf, 1).to(DEV)
    pos = [torch.full((B, 1), 1000 * i, dtype=torch.int32, device=DEV) for i in range(steps)]
    lens = [torch.tensor([(37 * i + 11 * b) % 60 for b in range(B)], dtype=torch.int32, device=DEV)
            for i in range(steps)]
    k, v = (random_like_shape((B, Hkv, L, d), bf, s).to(DEV) for s in (2, 3))
    kp, vp = (random_like_shape((1, Hkv, P, d), bf, s).to(DEV) for s in (4, 5))
    scores = [random_like_shape((B, Hkv, L), torch.float32, 6 + i).to(DEV) for i in range(steps)]
    qt = random_like_shape((B, Hq, T, d), bf, 30).to(DEV)
    lt = torch.full((B, Hq, T), 7.0, device=DEV)
    prefix = [torch.zeros(1, 1, dtype=torch.int32, device=DEV),
              torch.tensor([P], dtype=torch.int32, device=DEV),
              torch.tensor([0, B], dtype=torch.int32, device=DEV)]
    table = torch.arange(B, dtype=torch.int32, device=DEV)[:, None].contiguous()
    n1 = ost.attn_decode_shared_workspace_size(q0, kp, prefix[0], k[:, :, :keep], table)
    n2 = ost.attn_key_weights_workspace_size(B, Hq, Hkv, T, keep, keep)
    assert n2 > 0                                   # more rows than are kept: sums are joined
    ws1, ws2 = (torch.empty(n, dtype=torch.uint8, device=DEV) for n in (n1, n2))

    def run(idle):
        z = lambda *s, t=torch.float32: torch.zeros(*s, dtype=t, device=DEV)  # noqa: E731
        q, ko, vo = z(B, Hq, d, t=bf), z(B, Hkv, keep, d, t=bf), z(B, Hkv, keep, d, t=bf)
        so, kept, new = z(B, Hkv, keep), z(B, Hkv, keep, t=torch.int32), z(B, t=torch.int32)
        outs = [(z(B, Hq, d, t=bf), z(B, Hq), z(B, Hkv, keep), z(B, Hkv, 20, d, t=bf),
                 z(B, Hkv, 20, d, t=bf), z(B, Hkv, 20, t=torch.int32), z(B, t=torch.int32))
                for _ in range(steps)]
        torch.cuda.synchronize()
        after = torch.cuda.synchronize if idle else (lambda: None)
        for i, (o, lse, sums, k2, v2, kept2, new2) in enumerate(outs):
            ost.attn_cache_evict(k, v, scores[i], ko, vo, so, kept, new, 2, 3, seq_lens=lens[i])
            after()
            ost.attn_rope(q0, None, q, None, pos[i], w)
            after()
            ost.attn_decode_shared(q, kp, vp, *prefix, ko, vo, table, new, o, lse, d ** -0.5, 0, 0,
                                   ws1)
            after()
            ost.attn_key_weights(qt, ko, lt, None, sums, d ** -0.5, seq_lens=new, workspace=ws2)
            after()
            ost.attn_cache_evict(ko, vo, sums, k2, v2, None, kept2, new2, 1, 1, seq_lens=new)
            after()
            ost.attn_rope(q0, None, q, None, pos[-1 - i], w)
            after()
        torch.cuda.synchronize()
        return outs
    want = run(True)
    for _ in range(5):
        for a, b in zip(want, run(False)):
            assert all(torch.equal(x, y) for x, y in zip(a, b))


def test_allocating_calls_captured_and_replayed(ost):
    """Each call allocates its outputs and workspace inside a captured graph; two
    graphs from one pool, replayed in turn on new inputs, give what the same
    calls give outside."""
    B, Hq, Hkv, d, L, P, T, keep = 6, 16, 2, 128, 300, 700, 40, 64
    bf = torch.bfloat16
    w = ost.rope_frequencies(d, device=DEV)
    table = torch.arange(B, dtype=torch.int32, device=DEV)[:, None].contiguous()
    prefix = [torch.zeros(1, 1, dtype=torch.int32, device=DEV),
              torch.tensor([P], dtype=torch.int32, device=DEV),
              torch.tensor([0, B], dtype=torch.int32, device=DEV)]
    kp, vp = (random_like_shape((1, Hkv, P, d), bf, s).to(DEV) for s in (1, 2))

    def inputs(seed):
        x = [random_like_shape(s, bf, seed + i) for i, s in
             enumerate([(B, Hq, d), (B, Hkv, L, d), (B, Hkv, L, d), (B, Hq, T, d)])]
        g = torch.Generator().manual_seed(seed)
        return [t.to(DEV) for t in x] + [
            torch.randint(0, L + 1, (B,), generator=g).to(torch.int32).to(DEV),
            torch.randint(0, 5000, (B,), generator=g).to(torch.int32).to(DEV),
            torch.full((B, Hq, T), 6.0).to(DEV)]

    def calls(q, k, v, qt, lens, pos, lt):
        qr, _ = ost.rope(q, None, pos, w)
        o, lse = ost.decode_shared(qr, kp, vp, *prefix, k, v, table, lens)
        score = ost.key_weights(qt, k, lt, seq_lens=lens)             # joined sums
        score = ost.key_weights(qr, k, lse, prev=score, out=score, seq_lens=lens)
        return (qr, o, lse, score, *ost.evict(k, v, score, keep, 2, 5, seq_lens=lens))
    x = inputs(10)
    calls(*x)
    torch.cuda.synchronize()
    graphs, outs, pool = [], [], None
    for _ in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, pool=pool):
            outs.append(calls(*x))
        pool = graph.pool()
        graphs.append(graph)
    for seed in (20, 40, 60):
        for a, b in zip(x, inputs(seed)):
            a.copy_(b)
        want = calls(*x)
        for graph, got in zip(graphs, outs):
            for t in got:
                t.view(torch.uint8).fill_(0xff)        # (zeroed again by the graph itself)
            graph.replay()
            torch.cuda.synchronize()
            assert all(torch.equal(p, r) for p, r in zip(got, want))
