"""Appending to paged caches, in their own type and in 4 bits, and reading 4
bits back: the oracle's pins, refusals on the CPU, the GPU kernels against
attn_rope (bit for bit), the float64 oracle and exact integer arithmetic.

Tolerances. Rotated keys equal attn_rope's, whose own tolerance against the
oracle is 2^-20 (|x_a| + |x_b|) plus half a step of the type (tests/test_rope.py).
A 4-bit element is off by at most its scale, half the widest step between codes:
while the scale is a normal bf16 number, the largest element over the scale is at
most 6 (1 + 2^-8) (1 + 2^-23), and 6 stands in for it. Read back, a value is code *
scale rounded to bf16 once: equal.
"""

import numpy as np
import pytest
import torch

import oracle
from workloads import random_like_shape, to_f64

DEV = "cuda:0"
INVALID, UNSUPPORTED, MISALIGNED = -1, -2, -3
BF, F32 = torch.bfloat16, torch.float32


# ------------------------------------------------------------------ oracle


def test_oracle_bf16_rounding_is_torchs():
    x = np.concatenate([np.random.default_rng(0).standard_normal(500),
                        [0.0, 1.0, 1 + 2.0 ** -8, 1 + 3 * 2.0 ** -8, 1e-40, 3e38, 2.0 ** -130]])
    x = x.astype(np.float32)
    want = torch.from_numpy(x).to(BF).double().numpy()
    assert np.array_equal(oracle.round_bf16(x), want)


def test_oracle_codes_are_nearest_and_ties_even():
    x = np.zeros(32)
    x[:16] = [6, -6, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5, -5, 0.24, 5.01, -0.26, -3.4, 0, 2]
    codes, scale = oracle.quantise4(x)
    assert scale == [1.0]
    assert np.array_equal(oracle.values4(codes, scale)[:16],
                          [6, -6, 0, 1, 1, 2, 2, 4, 4, -4, 0, 6, -0.5, -3, 0, 2])
    codes, scale = oracle.quantise4(np.zeros((3, 64)))
    assert not codes.any() and not scale.any()
    x = np.random.default_rng(1).standard_normal((50, 64)) * 10.0 ** np.arange(-25, 25)[:, None]
    codes, scale = oracle.quantise4(x)
    assert np.all(np.abs(oracle.values4(codes, scale) - x) <= np.repeat(scale, 32, -1))


@pytest.mark.parametrize("d", [64, 128])
def test_oracle_layout_holds_every_element_once(d):
    packed = np.random.default_rng(2).integers(0, 256, (3, d // 2))
    codes = oracle.unpack4(packed)
    assert np.array_equal(np.sort(codes, -1),
                          np.sort(np.concatenate([packed % 16, packed // 16], -1), -1))
    # the bytes of one g hold four adjacent elements of each group
    for g in range(8):
        at = packed[0, d // 16 * g:d // 16 * (g + 1)]
        want = [codes[0, 32 * c + 4 * g + i] for c in range(d // 32) for i in range(4)]
        assert np.array_equal(np.stack([at % 16, at // 16], -1).ravel(), want)


# ------------------------------------------------------------------ refusals

P = 1 << 32


@pytest.fixture(scope="module")
def lib():
    import __graft_entry__
    __graft_entry__.build()
    import online_softmax_tiled_gb300 as ost
    return ost.lib()


def _call(lib, four=False, q=P, qs=None, qo=2 * P, qos=None, k=3 * P, ks=None, v=4 * P, vs=None,
          kp=5 * P, vp=6 * P, ksc=7 * P, vsc=8 * P, table=9 * P, lens=10 * P, new=11 * P, pos=12 * P,
          pstride=4, w=13 * P, B=2, Hq=4, Hkv=2, N=4, d=64, rot=64, inter=0, mag=1.0, pages=9,
          page=16, mp=4, dt=1):
    from online_softmax_tiled_gb300 import AttnStrides
    st = [None if s is None else AttnStrides(*s) for s in (qs, qos, ks, vs)]
    pools = (kp, ksc, vp, vsc) if four else (kp, vp)
    f = lib.attn_cache_append4 if four else lib.attn_cache_append
    import ctypes
    r = [None if s is None else ctypes.addressof(s) for s in st]
    return f(q, r[0], qo, r[1], k, r[2], v, r[3], *pools, table, lens, new, pos, pstride, w, B, Hq,
             Hkv, N, d, rot, inter, mag, pages, page, mp, dt, None)


NAN, INF = float("nan"), float("inf")


@pytest.mark.parametrize("four", [False, True])
@pytest.mark.parametrize("kwargs,expected", [
    (dict(B=0), INVALID), (dict(Hq=-1), INVALID), (dict(Hkv=0), INVALID), (dict(N=0), INVALID),
    (dict(d=0), INVALID), (dict(pages=0), INVALID), (dict(page=0), INVALID), (dict(mp=0), INVALID),
    (dict(q=None), INVALID), (dict(qo=None), INVALID), (dict(k=None), INVALID),
    (dict(v=None), INVALID), (dict(kp=None), INVALID), (dict(vp=None), INVALID),
    (dict(table=None), INVALID), (dict(lens=None), INVALID), (dict(w=None), INVALID),
    (dict(dt=2), INVALID), (dict(rot=63), INVALID), (dict(rot=66), INVALID),
    (dict(rot=-2), INVALID), (dict(inter=2), INVALID), (dict(mag=NAN), INVALID),
    (dict(mag=INF), INVALID), (dict(pstride=-1), INVALID), (dict(qs=(-1, 1, 1)), INVALID),
    (dict(ks=(1, -1, 1)), INVALID), (dict(vs=(1, 1, -1)), INVALID),
    (dict(qos=(0, 256, 64)), INVALID),                        # rows on top of each other
    (dict(qo=P, qos=(1024, 256, 64), qs=(1024, 64, 256)), INVALID),
    (dict(qo=3 * P), INVALID), (dict(qo=4 * P + 8), INVALID), (dict(qo=5 * P), INVALID),
    (dict(kp=3 * P), INVALID), (dict(kp=4 * P), INVALID), (dict(vp=5 * P), INVALID),
    (dict(kp=9 * P), INVALID), (dict(kp=10 * P), INVALID), (dict(vp=11 * P), INVALID),
    (dict(vp=12 * P), INVALID), (dict(vp=13 * P), INVALID), (dict(kp=P), INVALID),
    (dict(qo=9 * P), INVALID), (dict(qo=13 * P), INVALID),
    (dict(d=96, rot=32), UNSUPPORTED), (dict(d=256), UNSUPPORTED),
    (dict(B=1 << 16, N=1 << 15), UNSUPPORTED), (dict(Hq=4 * 65535), UNSUPPORTED),
    (dict(page=1 << 15, mp=(1 << 15) + 1), UNSUPPORTED), (dict(pages=1 << 27), UNSUPPORTED),
    (dict(q=P + 1), MISALIGNED), (dict(k=3 * P + 1), MISALIGNED), (dict(v=4 * P + 1), MISALIGNED),
    (dict(q=P + 2, dt=0), MISALIGNED), (dict(kp=5 * P + 8), MISALIGNED),
    (dict(vp=6 * P + 4), MISALIGNED), (dict(table=9 * P + 2), MISALIGNED),
    (dict(lens=10 * P + 1), MISALIGNED), (dict(new=11 * P + 2), MISALIGNED),
    (dict(pos=12 * P + 2), MISALIGNED), (dict(w=13 * P + 4), MISALIGNED),
])
def test_refusals(lib, four, kwargs, expected):
    assert _call(lib, four, **kwargs) == expected


@pytest.mark.parametrize("kwargs,expected", [
    (dict(ksc=None), INVALID), (dict(vsc=None), INVALID), (dict(ksc=5 * P), INVALID),
    (dict(vsc=7 * P), INVALID), (dict(vsc=3 * P), INVALID), (dict(qo=8 * P), INVALID),
    (dict(ksc=7 * P + 8), MISALIGNED),
])
def test_refusals_of_scales(lib, kwargs, expected):
    assert _call(lib, True, **kwargs) == expected


def test_absent_arguments_are_not_refused(lib):
    if torch.cuda.is_available():
        pytest.skip("made-up addresses: nothing may launch")
    for four in (False, True):
        for kwargs in (dict(), dict(new=None), dict(pos=None), dict(w=None, rot=0),
                       dict(q=None, qo=None, Hq=0), dict(Hq=3), dict(qo=P)):
            assert _call(lib, four, **kwargs) not in (INVALID, UNSUPPORTED, MISALIGNED), kwargs


def _read(lib, kc=P, ks=2 * P, vc=3 * P, vs=4 * P, table=5 * P, lens=6 * P, ko=7 * P, vo=8 * P, B=2,
          Hkv=2, L=50, pages=9, page=16, mp=4, d=64):
    return lib.attn_cache_read4(kc, ks, vc, vs, table, lens, ko, vo, B, Hkv, L, pages, page, mp, d,
                                None)


@pytest.mark.parametrize("kwargs,expected", [
    (dict(kc=None), INVALID), (dict(ks=None), INVALID), (dict(vc=None), INVALID),
    (dict(vs=None), INVALID), (dict(table=None), INVALID), (dict(lens=None), INVALID),
    (dict(ko=None), INVALID), (dict(vo=None), INVALID), (dict(B=0), INVALID),
    (dict(Hkv=0), INVALID), (dict(L=0), INVALID), (dict(pages=0), INVALID), (dict(page=0), INVALID),
    (dict(mp=0), INVALID), (dict(ko=P), INVALID), (dict(vo=2 * P), INVALID),
    (dict(vo=7 * P), INVALID), (dict(ko=5 * P), INVALID), (dict(ko=6 * P), INVALID),
    (dict(d=32), UNSUPPORTED), (dict(B=300, Hkv=300), UNSUPPORTED),
    (dict(pages=1 << 27), UNSUPPORTED), (dict(kc=P + 8), MISALIGNED), (dict(vs=4 * P + 2), MISALIGNED),
    (dict(ko=7 * P + 8), MISALIGNED), (dict(table=5 * P + 2), MISALIGNED),
])
def test_read_refusals(lib, kwargs, expected):
    assert _read(lib, **kwargs) == expected


# ------------------------------------------------------------------ GPU


def _ints(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def _pool(shape, dtype, seed):
    if dtype == torch.uint8:
        g = torch.Generator().manual_seed(seed)
        return torch.randint(0, 256, shape, generator=g).to(torch.uint8).to(DEV)
    return random_like_shape(shape, dtype, seed).to(DEV)


def _bytes(t):
    return t.contiguous().view(torch.uint8)


def _paged(B, lens, page, seed, spare=2):
    """A table of pages in random order, -1 past each request's, and the pool's size."""
    n = [-(-max(0, x) // page) for x in lens]
    width, total = max([1, *n]), sum(n) + spare
    g = torch.Generator().manual_seed(seed)
    order, table, at = torch.randperm(total, generator=g), torch.full((B, width), -1), 0
    for b in range(B):
        table[b, :n[b]] = order[at:at + n[b]]
        at += n[b]
    return table.to(torch.int32).to(DEV), total


def _heads_view(x, fused, shift):
    """x [B, H, N, d], or views of it: out of [B, N, H, d], starting `shift`
    elements off a multiple of 16 bytes."""
    if not fused:
        return x
    B, H, N, d = x.shape
    flat = torch.zeros(B * N * H * d + shift, dtype=x.dtype, device=x.device)
    y = flat[shift:].view(B, N, H, d)
    y.copy_(x.transpose(1, 2))
    return y.transpose(1, 2)


CASES = [
    # B, Hq, Hkv, N, d, rot, interleaved, dtype, page, old keys, new (None: N), fused, shift
    (3, 4, 2, 1, 128, 128, False, BF, 16, [0, 15, 200], None, True, 0),
    (2, 8, 8, 33, 128, 128, True, BF, 16, [0, 7], [33, 12], True, 0),
    (2, 3, 1, 40, 64, 32, False, BF, 24, [5, 0], [0, 40], False, 0),
    (3, 1, 3, 9, 128, 64, True, F32, 7, [3, 0, 90], [9, 1, 5], False, 0),
    (2, 5, 2, 17, 64, 64, False, F32, 64, [64, 63], None, True, 0),
    (2, 2, 2, 5, 64, 22, False, BF, 16, [1, 2], None, False, 0),     # rows piece by piece
    (2, 2, 2, 5, 128, 20, True, BF, 16, [1, 2], [3, 5], True, 1),
    (1, 6, 2, 70, 128, 126, False, F32, 1, [0], None, True, 3),
    (2, 2, 1, 6, 128, 0, False, BF, 16, [9, 30], None, False, 0),    # no rotation
    (1, 33, 7, 300, 64, 64, False, BF, 48, [11], None, True, 0),
    (5, 0, 4, 3, 128, 128, False, BF, 16, [0, 1, 2, 3, 4], [3, 0, 1, 2, 3], False, 0),
]
# as many tokens as fill the SMs without warps that share theirs, in 4 bits 8 and 16
# heads a thread
LARGE = [
    (2, 44, 2, 3400, 128, 128, False, BF, 16, [5, 0], [3400, 3111], True, 0),
    (1, 44, 2, 3300, 128, 64, True, BF, 48, [700], None, True, 0),
    (4, 44, 2, 3300, 64, 64, False, BF, 16, [0, 1, 2, 3], [3300, 0, 17, 3300], True, 0),
    (2, 45, 3, 3300, 64, 32, True, F32, 24, [9, 100], None, False, 0),
    (2, 43, 2, 1700, 128, 128, False, F32, 16, [0, 30], None, True, 0),
]


def _setup(case, seed):
    B, Hq, Hkv, N, d, rot, inter, dt, page, old, new, fused, shift = case
    new_l = [N] * B if new is None else new
    lens = [o + m for o, m in zip(old, new_l)]
    q, k, v = (_heads_view(random_like_shape((B, H, N, d), dt, seed + i).to(DEV), fused, shift)
               if H else None for i, H in enumerate((Hq, Hkv, Hkv)))
    table, total = _paged(B, lens, page, seed)
    w = None if rot == 0 else (10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)).to(DEV)
    row = [[lens[b] - new_l[b] + i for i in range(N)] for b in range(B)]
    return q, k, v, table, total, w, lens, new_l, row


def _turn(ost, x, pos, w, inter, mag):
    if x is None or w is None:
        return x
    return ost.rope(x.contiguous(), None, pos, w, interleaved=inter, magnitude=mag)[0]


@pytest.mark.gpu
@pytest.mark.parametrize("given", [False, True])
@pytest.mark.parametrize("case", CASES + LARGE)
def test_rows_are_those_of_rope(ost, case, given):
    """Keys bit for bit attn_rope's, values as they are, everything else untouched."""
    B, Hq, Hkv, N, d, rot, inter, dt, page, old, new, fused, shift = case
    q, k, v, table, total, w, lens, new_l, row = _setup(case, 1)
    pos = _ints(row) + (_ints([[1000 * b - 70] for b in range(B)]) if given else 0)
    mag = 1.25 if given else 1.0
    kp, vp = (_pool((total, Hkv, page, d), dt, s) for s in (5, 6))
    kp0, vp0 = kp.clone(), vp.clone()
    out = None if q is None else torch.full((B, Hq, N, d), 7.0, dtype=dt, device=DEV)
    got = ost.cache_append(q, k, v, kp, vp, table, _ints(lens), inv_freq=w,
                           positions=pos if given else None,
                           new_lens=None if new is None else _ints(new), interleaved=inter,
                           magnitude=mag, out=out)
    qr, kr = (_turn(ost, x, pos, w, inter, mag) for x in (q, k))
    tb = table.cpu()
    for b in range(B):
        m = new_l[b]
        if q is not None:
            assert got is out
            assert torch.equal(_bytes(out[b, :, :m]), _bytes(qr[b, :, :m]))
            assert torch.all(out[b, :, m:] == 7.0)
        for i in range(m):
            at, slot = int(tb[b, row[b][i] // page]), row[b][i] % page
            kp0[at, :, slot] = kr[b, :, i]
            vp0[at, :, slot] = v[b, :, i]
    assert torch.equal(_bytes(kp), _bytes(kp0)) and torch.equal(_bytes(vp), _bytes(vp0))


@pytest.mark.gpu
@pytest.mark.parametrize("case", CASES + LARGE)
def test_rows_in_four_bits(ost, case):
    """Scales and codes equal those worked out from attn_rope's float32 keys in
    float32 divisions; what they stand for is as near as 4 bits allow, and is read
    back exactly; everything else untouched."""
    B, Hq, Hkv, N, d, rot, inter, dt, page, old, new, fused, shift = case
    q, k, v, table, total, w, lens, new_l, row = _setup(case, 11)
    shapes = [((total, Hkv, page, d // 2), torch.uint8), ((total, Hkv, page, d // 32), BF)] * 2
    pools = [_pool(s, t, 15 + i) for i, (s, t) in enumerate(shapes)]
    want = [x.clone() for x in pools]
    out = None if q is None else torch.full((B, Hq, N, d), 7.0, dtype=dt, device=DEV)
    ost.cache_append4(q, k, v, *pools, table, _ints(lens), inv_freq=w,
                      new_lens=None if new is None else _ints(new), interleaved=inter, out=out)
    pos = _ints(row)
    qr, kr = (_turn(ost, x, pos, w, inter, 1.0) for x in (q, None if k is None else k.float()))
    tb = table.cpu()
    exact = []
    for which, x in ((0, kr.float()), (2, v.float())):
        g = x.contiguous().cpu().unflatten(-1, (-1, 32))
        scale = (g.abs().amax(-1) / 6.0).to(BF)
        y = (g / scale.float()[..., None]).double().numpy()
        near = np.abs(np.abs(y)[..., None] - oracle.LEVELS)
        pick = np.argmin(np.where(near == near.min(-1, keepdims=True), np.arange(8) % 2, 2), -1)
        codes = (pick + 8 * np.signbit(y)).reshape(*x.shape)
        val = oracle.values4(codes, scale.double().numpy())
        assert np.all(np.abs(val - x.double().cpu().numpy()) <=
                      np.repeat(scale.double().numpy(), 32, -1))
        exact.append((codes, scale.double().numpy()))
        packed = np.zeros((*x.shape[:-1], d // 2), dtype=np.uint8)
        for e in range(d):
            c, r = e // 32, e % 32
            packed[..., d // 16 * (r // 4) + 2 * c + r % 4 // 2] |= (
                codes[..., e] << (4 * (e % 2))).astype(np.uint8)
        packed = torch.from_numpy(packed).to(DEV)
        for b in range(B):
            for i in range(new_l[b]):
                at, slot = int(tb[b, row[b][i] // page]), row[b][i] % page
                want[which][at, :, slot] = packed[b, :, i]
                want[which + 1][at, :, slot] = scale[b, :, i].to(DEV)
    for got, ref in zip(pools, want):
        assert torch.equal(_bytes(got), _bytes(ref))
    if q is not None:
        for b in range(B):
            assert torch.equal(_bytes(out[b, :, :new_l[b]]), _bytes(qr[b, :, :new_l[b]]))
    L = max(lens) + 3
    back = [torch.full((B, Hkv, L, d), 9.0, dtype=BF, device=DEV) for _ in range(2)]
    assert ost.cache_read4(*pools, table, _ints(lens), out=tuple(back))[0] is back[0]
    for b in range(B):
        for which, (x, (codes, scale)) in enumerate(zip(back, exact)):
            o, n = row[b][0], lens[b]
            val = oracle.round_bf16(oracle.values4(codes[b], scale[b]))
            assert np.array_equal(to_f64(x[b, :, o:n]), val[:, :n - o])
            assert torch.all(x[b, :, n:] == 9.0)
            if o:
                j = np.arange(o)
                at = tb[b].numpy()[j // page]
                c, s = (to_f64(p) if p.dtype == BF else p.cpu().numpy()
                        for p in pools[2 * which:2 * which + 2])
                val = oracle.values4(oracle.unpack4(c[at, :, j % page]), s[at, :, j % page])
                assert np.array_equal(to_f64(x[b, :, :o]),
                                      oracle.round_bf16(val).transpose(1, 0, 2))


@pytest.mark.gpu
@pytest.mark.parametrize("d", [64, 128])
def test_every_border_between_codes(ost, d):
    """Values on, just below and just above every border, groups of zeros, tiny
    and huge groups: equal to the float64 oracle where the quotient is exact."""
    eps = 2.0 ** -7
    marks = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0])
    vals = np.concatenate([marks, marks * (1 - eps), marks * (1 + eps), [0.0, -0.0, 6.0]])
    group = np.concatenate([vals, -vals[:8]])[:32]
    group[31] = 6.0
    rows = [group * s for s in (1.0, 2.0 ** -100, 2.0 ** 100, 0.5, 2.0 ** -126)]
    rows += [np.zeros(32), np.full(32, 3.0), -np.arange(32.0)]
    x = np.stack([np.concatenate([rows[(i + c) % len(rows)] for c in range(d // 32)])
                  for i in range(16)])
    v = torch.from_numpy(x).to(F32).view(1, 1, 16, d).to(DEV)
    pools = [_pool((1, 1, 16, d // 2), torch.uint8, 1), _pool((1, 1, 16, d // 32), BF, 2)] + \
        [_pool((1, 1, 16, d // 2), torch.uint8, 3), _pool((1, 1, 16, d // 32), BF, 4)]
    ost.cache_append4(None, v, v, *pools, _ints([[0]]), _ints([16]))
    for c, s in (pools[:2], pools[2:]):
        codes, scale = oracle.quantise4(to_f64(v)[0, 0])
        assert np.array_equal(to_f64(s)[0, 0], scale)
        got = oracle.unpack4(c.cpu().numpy()[0, 0])
        assert np.array_equal(oracle.values4(got, scale), oracle.values4(codes, scale))


@pytest.mark.gpu
def test_quotients_are_those_of_ieee_divisions(ost):
    """Every significand of a scale, at several exponents, with elements within two
    float32 steps of every border times the scale: the codes of the float32 quotients,
    correctly rounded (numpy's)."""
    marks = np.float32([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0])
    levels = np.array(oracle.LEVELS)
    rows, scales = [], []
    for e in (-89, -30, 0, 3, 88):
        for m in range(128):
            s = np.float32((1 + m / 128) * 2.0 ** e)
            y = marks * s
            near = np.concatenate([y] + [y := np.nextafter(y, np.float32(np.inf) * d)
                                         for d in (1, 1, -1, -1, -1, -1)])[7:]
            near = np.concatenate([near, y]).astype(np.float32)          # 42 and 7
            for at in (near[:31], np.concatenate([near[31:], -near[:13]])):
                rows.append(np.concatenate([at[:31], [6 * s]]).astype(np.float32))
                scales.append(s)
    x, s = np.stack(rows), np.float32(scales)
    x = x[:x.shape[0] // 4 * 4].reshape(1, 1, -1, 128)
    s = s[:x.shape[2] * 4].reshape(-1, 4)
    v = torch.from_numpy(x).to(DEV)
    n = x.shape[2]
    pools = [t for i in range(2) for t in (_pool((1, 1, n, 64), torch.uint8, i),
                                           _pool((1, 1, n, 4), BF, 9 + i))]
    ost.cache_append4(None, v, v, *pools, _ints([[0]]), _ints([n]))
    q = x[0, 0] / np.repeat(s, 32, -1)
    assert q.dtype == np.float32
    mids = (levels[1:] + levels[:-1]) / 2
    a = np.abs(q).astype(np.float64)
    at = np.searchsorted(mids, a, side="left")                    # ties to the lower code,
    at += (at < 7) & (a == mids[np.minimum(at, 6)]) & (at % 2 == 1)   # or the even one above
    want = np.sign(q) * levels[at] * np.repeat(s.astype(np.float64), 32, -1)
    for c, sc in (pools[:2], pools[2:]):
        assert np.array_equal(to_f64(sc)[0, 0], s)
        got = oracle.values4(oracle.unpack4(c.cpu().numpy()[0, 0]), to_f64(sc)[0, 0])
        assert np.array_equal(got, want)


@pytest.mark.gpu
def test_values_that_are_not_finite_spoil_their_group_alone(ost):
    v = random_like_shape((1, 1, 4, 128), BF, 3).to(DEV)
    v[0, 0, 0, 5], v[0, 0, 1, 40], v[0, 0, 2, 127] = float("nan"), float("inf"), -float("inf")
    pools = [t for i in range(2) for t in (_pool((1, 1, 16, 64), torch.uint8, i),
                                           _pool((1, 1, 16, 4), BF, 9 + i))]
    ost.cache_append4(None, v, v, *pools, _ints([[0]]), _ints([4]))
    back = ost.cache_read4(*pools, _ints([[0]]), _ints([4]), length=4)[0][0, 0]
    bad = torch.isnan(back).view(4, 4, 32)
    want = torch.zeros(4, 4, dtype=torch.bool, device=DEV)
    want[0, 0] = want[1, 1] = want[2, 3] = True
    assert torch.equal(bad.all(-1), want) and torch.equal(bad.any(-1), want)


@pytest.mark.gpu
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("dt,H,N", [(BF, 9, 37), (F32, 6, 50)])
def test_queries_turned_in_place(ost, dt, H, N, inter):
    q, k, v = (random_like_shape((2, h, N, 128), dt, 4 + h).to(DEV) for h in (H, 2, 2))
    w, table = ost.rope_frequencies(128, device=DEV), _ints([[0, 1, 2, 3], [4, 5, 6, 7]])
    kp, vp = (torch.zeros(8, 2, 16, 128, dtype=dt, device=DEV) for _ in range(2))
    want = ost.cache_append(q, k, v, kp, vp, table, _ints([N, N]), inv_freq=w, interleaved=inter)
    assert ost.cache_append(q, k, v, kp, vp, table, _ints([N, N]), inv_freq=w, interleaved=inter,
                            out=q) is q
    assert torch.equal(q, want)


@pytest.mark.gpu
def test_one_token_form_and_position_shapes(ost):
    B, w = 4, ost.rope_frequencies(64, device=DEV)
    x = random_like_shape((B, 8, 64), BF, 5).to(DEV)
    q, k, v = x[:, :4], x[:, 4:6], x[:, 6:]
    table = _ints([[i] for i in range(B)])
    res = []
    for pos in (_ints([3, 3, 3, 3]), _ints([[3]] * 4), _ints([3]), None):
        kp, vp = (torch.zeros(B, 2, 16, 64, dtype=BF, device=DEV) for _ in range(2))
        o = ost.cache_append(q, k, v, kp, vp, table, _ints([4] * B), inv_freq=w, positions=pos)
        assert o.shape == (B, 4, 64)
        res.append((o, kp, vp))
    for r in res[1:]:
        assert all(torch.equal(a, b) for a, b in zip(res[0], r))
    assert torch.equal(res[0][1][:, :, 3], ost.rope(k, None, _ints([3]), w)[0])


@pytest.mark.gpu
@pytest.mark.parametrize("four", [False, True])
def test_bad_lengths_and_pages_are_flagged_not_written(ost, four):
    B, N, page, d = 4, 3, 16, 64
    q, k, v = (random_like_shape((B, h, N, d), BF, 6 + h).to(DEV) for h in (2, 1, 1))
    w = ost.rope_frequencies(d, device=DEV)
    shapes = [((6, 1, page, d // 2), torch.uint8), ((6, 1, page, 2), BF)] * 2 if four else \
        [((6, 1, page, d), BF)] * 2
    pools = [_pool(s, t, i) for i, (s, t) in enumerate(shapes)]
    f = ost.cache_append4 if four else ost.cache_append

    def run(lens, new, table):
        work, out = [p.clone() for p in pools], torch.full_like(q, 7.0)
        f(q, k, v, *work, table, _ints(lens), inv_freq=w, new_lens=_ints(new), out=out)
        return work, out, ost.attn_sync_status()
    table = _ints([[0, 1], [2, 3], [4, 5], [0, 1]])
    for lens, new in (([33, -1, 2, 3], [3, 3, 3, 0]), ([3, 3, 3, 3], [4, -1, 0, 0])):
        work, out, status = run(lens, new, table)
        assert status == -7
        assert torch.all(out[1] == 7.0) and torch.all(out[0] == 7.0)
        assert torch.equal(work[0][:4].view(torch.uint8), pools[0][:4].view(torch.uint8))
    work, out, status = run([16, 17, 18, 0], [3, 3, 3, 0], _ints([[0, -1], [6, 2], [3, -5], [0, 0]]))
    assert status == -7                     # pages 6 and -5; -1 is of no new token
    want, _, _ = run([16, 17, 18, 0], [3, 0, 0, 0], table)
    last = _ints([[0, 0], [0, 2], [3, 0], [0, 0]])
    ok, _, status = run([16, 17, 18, 0], [3, 0, 0, 0], last)
    assert status == 0
    assert torch.all(out[1] != 7.0) and torch.all(out[3] == 7.0)     # queries are turned all the same
    assert torch.equal(work[0][0].view(torch.uint8), ok[0][0].view(torch.uint8))
    assert not torch.equal(work[0][2].view(torch.uint8), pools[0][2].view(torch.uint8))
    assert torch.equal(work[0][4:].view(torch.uint8), pools[0][4:].view(torch.uint8))
    if four:
        out = tuple(torch.full((4, 1, 20, d), 3.0, dtype=BF, device=DEV) for _ in range(2))
        ost.cache_read4(*pools, _ints([[0, 1], [2, 9], [0, 0], [1, 1]]), _ints([21, 18, -2, 5]),
                        out=out)
        assert ost.attn_sync_status() == -7
        assert torch.all(out[0][0] == 3.0) and torch.all(out[0][2] == 3.0)
        assert torch.all(out[0][1, :, 16:] == 3.0) and torch.all(out[0][3, :, 5:] == 3.0)
        assert not torch.any(out[0][1, :, :16] == 3.0)


@pytest.mark.gpu
@pytest.mark.parametrize("four", [False, True])
def test_offsets_past_32_bits(ost, four):
    """The last pages of pools of more than 2^32 bytes."""
    d, Hkv, page = 128, 2, 64
    row = d // 2 if four else 2 * d
    total = (1 << 32) // (Hkv * page * row) + 8
    shapes = [((total, Hkv, page, d // 2), torch.uint8), ((total, Hkv, page, d // 32), BF)] * 2 \
        if four else [((total, Hkv, page, d), BF)] * 2
    pools = [torch.zeros(s, dtype=t, device=DEV) for s, t in shapes]
    small = [torch.zeros((4, *s[1:]), dtype=t, device=DEV) for s, t in shapes]
    k, v = (random_like_shape((1, Hkv, 200, d), BF, s).to(DEV) for s in (1, 2))
    f = ost.cache_append4 if four else ost.cache_append
    f(None, k, v, *pools, _ints([[total - 1 - i for i in range(4)]]), _ints([200]))
    f(None, k, v, *small, _ints([[3 - i for i in range(4)]]), _ints([200]))
    for x, y in zip(pools, small):
        assert torch.equal(x[-4:].view(torch.uint8), y.view(torch.uint8))
        assert int(torch.count_nonzero(x[:-4])) == 0
    if four:
        a = ost.cache_read4(*pools, _ints([[total - 1 - i for i in range(4)]]), _ints([200]))
        b = ost.cache_read4(*small, _ints([[3 - i for i in range(4)]]), _ints([200]))
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.mark.gpu
@pytest.mark.parametrize("four", [False, True])
def test_streams_and_graphs(ost, four):
    """On another stream, and captured, replayed on new inputs and lengths."""
    B, N, d, page = 3, 2, 128, 16
    w = ost.rope_frequencies(d, device=DEV)
    table = torch.arange(3 * B, dtype=torch.int32, device=DEV).view(B, 3)
    shapes = [((9, 2, page, d // 2), torch.uint8), ((9, 2, page, d // 32), BF)] * 2 if four else \
        [((9, 2, page, d), BF)] * 2
    f = ost.cache_append4 if four else ost.cache_append

    def fresh():
        return [torch.zeros(s, dtype=t, device=DEV) for s, t in shapes]

    def inputs(seed):
        return [random_like_shape((B, h, N, d), BF, seed + h).to(DEV) for h in (4, 2)] + \
            [random_like_shape((B, 2, N, d), BF, seed + 9).to(DEV), _ints([2 + seed, 40, 30 - seed])]

    def call(x, pools, **kw):
        out = [f(*x[:3], *pools, table, x[3], inv_freq=w, **kw)]
        if four:
            out += ost.cache_read4(*pools, table, x[3], **kw)
        return out
    x, pools = inputs(3), fresh()
    want = call(x, pools) + pools
    side, pools2 = torch.cuda.Stream(), fresh()
    side.wait_stream(torch.cuda.current_stream())
    got = call(x, pools2, stream=side) + pools2
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    graph, pools3 = torch.cuda.CUDAGraph(), fresh()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        out = call(x, pools3)
    for seed in (5, 8):
        for a, b in zip(x, inputs(seed)):
            a.copy_(b)
        for p in pools3:
            p.zero_()
        graph.replay()
        pools4 = fresh()
        want = call(x, pools4) + pools4
        assert all(torch.equal(a, b) for a, b in zip(out + pools3, want))


@pytest.mark.gpu
def test_binding_refusals(ost):
    q, k, v = (random_like_shape((2, h, 3, 64), BF, h).to(DEV) for h in (4, 2, 2))
    kp, vp = (torch.zeros(4, 2, 16, 64, dtype=BF, device=DEV) for _ in range(2))
    kc, ks = torch.zeros(4, 2, 16, 32, dtype=torch.uint8, device=DEV), kp[..., :2].contiguous()
    vc, vs = kc.clone(), ks.clone()
    base = dict(q=q, k=k, v=v, block_table=_ints([[0], [1]]), seq_lens=_ints([3, 3]),
                inv_freq=ost.rope_frequencies(64, device=DEV))
    rows, four = dict(k_pages=kp, v_pages=vp), dict(k_codes=kc, k_scales=ks, v_codes=vc, v_scales=vs)
    for bad in (dict(k=k.float()), dict(v=v[:, :1]), dict(q=q[:1]), dict(q=q.cpu()),
                dict(block_table=_ints([[0]])), dict(seq_lens=torch.tensor([3, 3], device=DEV)),
                dict(positions=_ints([[1, 2]])), dict(new_lens=_ints([1])),
                dict(inv_freq=base["inv_freq"].float()), dict(out=q[:, :2]),
                dict(k=k.transpose(2, 3)), dict(q=None, out=q)):
        for f, pools in ((ost.cache_append, rows), (ost.cache_append4, four)):
            with pytest.raises((ValueError, TypeError)):
                f(**{**base, **pools, **bad})
    for bad in (dict(k_pages=kp[:, :1].contiguous()), dict(v_pages=vp.float()),
                dict(v_pages=vp[:3])):
        with pytest.raises((ValueError, TypeError)):
            ost.cache_append(**{**base, **rows, **bad})
    for bad in (dict(k_codes=kc.to(torch.int8)), dict(k_scales=ks.float()),
                dict(v_scales=vs[..., :1].contiguous()), dict(v_codes=vc[:3])):
        with pytest.raises((ValueError, TypeError)):
            ost.cache_append4(**{**base, **four, **bad})
    with pytest.raises(ost.AttnError):
        ost.cache_append(**{**base, **rows, "k_pages": vp})        # one pool for both
    with pytest.raises((ValueError, TypeError)):
        ost.cache_read4(kc, ks, vc, vs, _ints([[0], [1]]), _ints([3, 3]), out=(k, v.float()))
    assert not kp.any() and not vp.any() and not kc.any() and not ks.any()
