"""Rotary positions: the oracle's own pins, refusals on the CPU, and the GPU
kernel against the float64 oracle.

Tolerance of the kernel, per element, from its roundings (u = 2^-24): the
angle is rounded once (relative u, so at most π·u absolute), sincospi is
within 2 ulp, each output takes two products and a sum: in all below
2^-20 · m (|x_a| + |x_b|); bf16 outputs add half a step, 2^-8 of the value
(float32: 2^-24). Copied elements are equal.
"""

import ctypes
import math

import numpy as np
import pytest
import torch

import oracle
from workloads import random_like_shape, to_f64

DEV = "cuda:0"
INVALID, UNSUPPORTED, MISALIGNED = -1, -2, -3


# ------------------------------------------------------------------ oracle


def test_oracle_angles_match_float64_at_near_positions():
    w = 10000.0 ** (-np.arange(16) / 16)
    pos = np.array([[0, 1, -1, 7, 1000]])
    ang = oracle.rope_angles(pos, w)
    want = pos[..., None] * w
    assert np.max(np.abs(np.exp(1j * ang) - np.exp(1j * want))) < 1e-12


def test_oracle_rotation_is_orthogonal_and_inverts():
    rng = np.random.default_rng(0)
    x = rng.standard_normal((2, 3, 5, 16))
    pos = rng.integers(-50, 5000, (2, 5))
    w = 100.0 ** (-np.arange(6) / 6)
    for inter in (False, True):
        y = oracle.rope(x, pos, w, inter)
        assert np.allclose(np.sum(x ** 2, -1), np.sum(y ** 2, -1))
        assert np.allclose(oracle.rope(y, pos, w, inter, inverse=True), x)
        assert np.array_equal(y[..., 12:], x[..., 12:])


def test_oracle_scores_depend_on_distance_only():
    rng = np.random.default_rng(1)
    q, k = rng.standard_normal((2, 1, 1, 1, 8))
    w = np.array([1.0, 0.3, 0.01, 1e-4])

    def score(i, j):
        return float(np.sum(oracle.rope(q, np.array([[i]]), w) *
                            oracle.rope(k, np.array([[j]]), w)))
    assert math.isclose(score(10, 3), score(100010, 100003), rel_tol=1e-9)


def test_oracle_gradient_by_differences():
    """The inverse call on dy is the derivative of sum(dy · rope(x))."""
    rng = np.random.default_rng(2)
    x, dy = rng.standard_normal((2, 1, 2, 3, 8))
    pos, w, m = np.array([[4, 9, 100]]), np.array([1.0, 0.2, 0.05]), 1.3
    for inter in (False, True):
        dx = oracle.rope(dy, pos, w, inter, m, inverse=True)
        for at in np.ndindex(x.shape):
            e = np.zeros_like(x)
            e[at] = 1e-4
            num = np.sum(dy * (oracle.rope(x + e, pos, w, inter, m) -
                               oracle.rope(x - e, pos, w, inter, m))) / 2e-4
            # copied elements: the magnitude does not apply
            assert abs(num - dx[at]) < 1e-6


def test_frequencies():
    import online_softmax_tiled_gb300 as ost
    f = ost.rope_frequencies(8)
    assert torch.allclose(f, torch.tensor([1.0, 0.1, 0.01, 0.001], dtype=torch.float64))
    assert torch.allclose(ost.rope_frequencies(8, scaling="linear", factor=4.0), f / 4)
    b = ost.rope_frequencies(8, scaling="base", factor=4.0)
    assert b[0] == 1.0 and math.isclose(float(b[-1]), float(f[-1]) / 4, rel_tol=1e-12)
    r = ost.rope_frequencies(64, scaling="ramp", factor=8.0, original_length=4096)
    g = ost.rope_frequencies(64)
    turns = 4096 * g / (2 * math.pi)
    assert torch.equal(r[turns > 32], g[turns > 32])
    assert torch.allclose(r[turns < 1], g[turns < 1] / 8)
    mid = (turns > 1) & (turns < 32)
    assert mid.any() and torch.all((r[mid] < g[mid]) & (r[mid] > g[mid] / 8))
    for bad in (dict(rot_dim=7), dict(rot_dim=8, scaling="other"), dict(rot_dim=2, scaling="base"),
                dict(rot_dim=8, scaling="ramp"), dict(rot_dim=8, factor=0.0)):
        with pytest.raises(ValueError):
            ost.rope_frequencies(**bad)


# ------------------------------------------------------------------ refusals

P = 1 << 20  # an aligned stand-in address; never dereferenced on these paths


@pytest.fixture(scope="module")
def lib():
    import __graft_entry__
    __graft_entry__.build()
    import online_softmax_tiled_gb300 as ost
    return ost.lib()


def _call(lib, q=P, qs=None, qo=P, qos=None, k=P, ks=None, ko=P, kos=None, pos=P, pstride=4, w=P,
          B=2, Hq=4, Hkv=2, N=4, d=64, rot=64, inter=0, mag=1.0, inv=0, dt=1):
    from online_softmax_tiled_gb300 import AttnStrides
    st = [None if s is None else ctypes.byref(AttnStrides(*s)) for s in (qs, qos, ks, kos)]
    return lib.attn_rope(q, st[0], qo, st[1], k, st[2], ko, st[3], pos, pstride, w, B, Hq, Hkv, N,
                         d, rot, inter, mag, inv, dt, None)


@pytest.mark.parametrize("kwargs,expected", [
    (dict(B=0), INVALID), (dict(Hq=0), INVALID), (dict(Hkv=-1), INVALID), (dict(N=0), INVALID),
    (dict(q=None), INVALID), (dict(qo=None), INVALID), (dict(k=None), INVALID),
    (dict(ko=None), INVALID), (dict(pos=None), INVALID), (dict(w=None), INVALID),
    (dict(dt=2), INVALID), (dict(rot=63), INVALID), (dict(rot=0), INVALID),
    (dict(rot=66), INVALID), (dict(inter=2), INVALID), (dict(inv=-1), INVALID),
    (dict(mag=float("nan")), INVALID), (dict(mag=float("inf")), INVALID),
    (dict(pstride=-1), INVALID), (dict(d=65, rot=64), UNSUPPORTED), (dict(d=514), UNSUPPORTED),
    (dict(B=1 << 16, N=1 << 15), UNSUPPORTED), (dict(Hq=300000), UNSUPPORTED),
    (dict(q=P + 1), MISALIGNED), (dict(pos=P + 2), MISALIGNED), (dict(w=P + 4), MISALIGNED),
    (dict(dt=0, ko=P + 2), MISALIGNED),
    (dict(qs=(-64, 64, 64)), INVALID),                       # negative input stride
    (dict(qo=2 * P, qos=(64, 64, 64)), INVALID),             # output rows on top of each other
    (dict(qo=2 * P, qos=(4 * 256, 128, 64)), INVALID),       # heads step into each other's tokens
    (dict(qs=(2048, 256, 64)), INVALID),                     # in place with other strides
])
def test_refusals(lib, kwargs, expected):
    assert _call(lib, **kwargs) == expected


# ------------------------------------------------------------------ GPU


def _freq(rot, base=10000.0):
    return base ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)


def _check(got, x, pos, w, inter, m, inverse, where=""):
    """Element-wise bound of the module docstring."""
    x64, got = to_f64(x), got.detach()
    ref = oracle.rope(x64, pos.cpu().numpy(), w.cpu().numpy(), inter, m, inverse)
    swap = np.abs(x64)
    r = 2 * len(w)
    a_at = np.arange(0, r, 2) if inter else np.arange(r // 2)
    b_at = a_at + 1 if inter else a_at + r // 2
    both = np.zeros_like(ref)
    both[..., a_at] = both[..., b_at] = swap[..., a_at] + swap[..., b_at]
    half = torch.finfo(got.dtype).eps / 2
    err = np.abs(to_f64(got) - ref)
    assert np.all(err <= half * np.abs(ref) + 2.0 ** -20 * m * both), (where, err.max())
    assert torch.equal(got[..., r:], x[..., r:])


CASES = [  # B, Hq, Hkv, N, d, rot, interleaved, dtype
    (64, 32, 8, 1, 128, 128, False, torch.bfloat16),
    (2, 4, 2, 33, 128, 128, False, torch.bfloat16),
    (1, 3, 1, 257, 64, 64, True, torch.bfloat16),
    (3, 5, 5, 17, 128, 64, False, torch.bfloat16),
    (2, 2, 1, 19, 64, 16, True, torch.float32),
    (1, 9, 3, 100, 128, 96, False, torch.float32),
    (2, 3, 1, 11, 64, 24, False, torch.bfloat16),     # 12 pairs: element by element
    (1, 2, 2, 7, 10, 6, True, torch.float32),         # a head of ten
    (1, 1, 0, 5, 512, 512, False, torch.bfloat16),    # the widest head, q alone
    (1, 1, 0, 3, 510, 2, True, torch.bfloat16),       # one pair of the widest odd row
    (1, 20, 20, 1024, 128, 128, False, torch.bfloat16),  # several heads a thread
]


@pytest.mark.gpu
@pytest.mark.parametrize("B,Hq,Hkv,N,d,rot,inter,dt", CASES)
@pytest.mark.parametrize("inverse", [False, True])
def test_parity(ost, B, Hq, Hkv, N, d, rot, inter, dt, inverse):
    g = torch.Generator().manual_seed(B * 1000 + N)
    q = random_like_shape((B, Hq, N, d), dt, 1).to(DEV)
    k = random_like_shape((B, Hkv, N, d), dt, 2).to(DEV) if Hkv else None
    pos = (torch.randint(-1000, 200000, (B, 1), generator=g) + torch.arange(N)).to(torch.int32)
    w, m = _freq(rot), 1.25
    yq, yk = ost.rope(q, k, pos.to(DEV), w.to(DEV), interleaved=inter, magnitude=m,
                      inverse=inverse)
    _check(yq, q, pos, w, inter, m, inverse, "q")
    if Hkv:
        _check(yk, k, pos, w, inter, m, inverse, "k")
    else:
        assert yk is None


@pytest.mark.gpu
def test_far_positions_keep_their_angle(ost):
    """The ends of the 32-bit range, and frequencies from one radian (and a
    few turns) a position to next to nothing, zero and negative among them."""
    pos = torch.tensor([[2 ** 31 - 1, -2 ** 31, 2 ** 31 - 2, 0, 1, -1, 2 ** 24 + 1, 10 ** 9]],
                       dtype=torch.int32)
    w = torch.tensor([1.0, 0.9999999, 1e-3, 1e-9, 0.0, -0.37, 19.7, 1e-300, 3.9, 2 * math.pi,
                      1e-19, 2.5e-17, 1023.0, 4.0, 2.0, 0.5], dtype=torch.float64)
    x = random_like_shape((1, 2, 8, 32), torch.float32, 3).to(DEV)
    y, _ = ost.rope(x, None, pos.to(DEV), w.to(DEV))
    _check(y, x, pos, w, False, 1.0, False)


@pytest.mark.gpu
def test_frequencies_that_are_not_finite_give_nan(ost):
    w = torch.tensor([1.0, math.nan, math.inf, 0.1], dtype=torch.float64)
    x = random_like_shape((1, 1, 2, 16), torch.float32, 4).to(DEV)
    pos = torch.tensor([[3, 5]], dtype=torch.int32, device=DEV)
    y = ost.rope(x, None, pos, w.to(DEV))[0]
    bad = torch.zeros(16, dtype=torch.bool)
    bad[[1, 2, 5, 6]] = True
    assert torch.equal(y[0, 0].isnan().cpu(), bad.expand(2, 16))


@pytest.mark.gpu
@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("shift", [0, 1])
def test_views_of_a_fused_projection(ost, dt, shift):
    """q and k as strided views of [B, N, Hq + 2 Hkv, d], from an address that
    is (shift 0) or is not a multiple of 16 bytes, into strided outputs, and
    in place; v and everything around stay as they were."""
    B, N, Hq, Hkv, d = 2, 21, 4, 2, 64
    buf = random_like_shape((B * N * (Hq + 2 * Hkv) * d + 1,), dt, 5).to(DEV)
    qkv = buf[shift:buf.numel() - 1 + shift].view(B, N, Hq + 2 * Hkv, d)
    q, k = qkv[:, :, :Hq].transpose(1, 2), qkv[:, :, Hq:Hq + Hkv].transpose(1, 2)
    pos = torch.arange(N, dtype=torch.int32) * 3
    w = _freq(d)
    yq, yk = ost.rope(q, k, pos.to(DEV), w.to(DEV))
    _check(yq, q, pos.expand(B, N), w, False, 1.0, False)
    _check(yk, k, pos.expand(B, N), w, False, 1.0, False)
    assert yq.is_contiguous() and yk.is_contiguous()
    # a strided output: the [B, N, H, d] order
    zq = torch.full((B, N, Hq, d), 7.0, dtype=dt, device=DEV)
    zk = torch.full((B, N, Hkv, d), 7.0, dtype=dt, device=DEV)
    ost.rope(q, k, pos.to(DEV), w.to(DEV), out=(zq.transpose(1, 2), zk.transpose(1, 2)))
    assert torch.equal(zq.transpose(1, 2), yq) and torch.equal(zk.transpose(1, 2), yk)
    # in place
    before = buf.clone()
    ost.rope(q, k, pos.to(DEV), w.to(DEV), out=(q, k))
    assert torch.equal(q, yq) and torch.equal(k, yk)
    mask = torch.ones_like(buf, dtype=torch.bool)
    mask[shift:buf.numel() - 1 + shift].view(qkv.shape)[:, :, :Hq + Hkv] = False
    assert torch.equal(buf[mask], before[mask])


@pytest.mark.gpu
def test_broadcast_input_and_one_token_form(ost):
    """A head-broadcast input (stride 0), and [B, H, d] with positions [B]."""
    w = _freq(128)
    x = random_like_shape((2, 1, 5, 128), torch.bfloat16, 6).to(DEV).expand(2, 4, 5, 128)
    pos = torch.arange(10, dtype=torch.int32).view(2, 5)
    y, _ = ost.rope(x, None, pos.to(DEV), w.to(DEV))
    _check(y, x, pos, w, False, 1.0, False)
    q = random_like_shape((6, 4, 128), torch.bfloat16, 7).to(DEV)
    p = torch.tensor([0, 5, 11, 70000, 3, 9], dtype=torch.int32)
    z, _ = ost.rope(q, None, p.to(DEV), w.to(DEV))
    _check(z[:, :, None], q[:, :, None], p[:, None], w, False, 1.0, False)


@pytest.mark.gpu
def test_gradient_through_attention(ost):
    """Rotation, causal attention and the whole backward pass in float32
    against central differences of the float64 oracle."""
    B, H, Hkv, N, d = 1, 2, 1, 6, 64
    q = random_like_shape((B, H, N, d), torch.float32, 8)
    k, v = (random_like_shape((B, Hkv, N, d), torch.float32, s) for s in (9, 10))
    do = random_like_shape((B, H, N, d), torch.float32, 11)
    pos, w = torch.arange(N, dtype=torch.int32)[None] * 50, _freq(d // 2)
    x = [t.to(DEV) for t in (q, k, v, do)]
    qr, kr = ost.rope(x[0], x[1], pos.to(DEV), w.to(DEV), interleaved=True)
    o, lse = ost.forward(qr, kr, x[2], causal=True)
    dqr, dkr, _ = ost.backward(qr, kr, x[2], o, x[3], lse, causal=True)
    dq, dk = ost.rope(dqr, dkr, pos.to(DEV), w.to(DEV), interleaved=True, inverse=True)

    def loss(q64, k64):
        qq, kk = (oracle.rope(t, pos.numpy(), w.numpy(), True) for t in (q64, k64))
        return float(np.sum(do.double().numpy() * oracle.attention_fwd(
            qq, kk, v.double().numpy(), d ** -0.5, True)[0]))
    rng = np.random.default_rng(0)
    for got, which in ((dq, 0), (dk, 1)):
        base = [q.double().numpy(), k.double().numpy()]
        for _ in range(12):
            e = rng.standard_normal(base[which].shape) * 1e-5
            hi = [t + e if i == which else t for i, t in enumerate(base)]
            lo = [t - e if i == which else t for i, t in enumerate(base)]
            num = (loss(*hi) - loss(*lo)) / 2
            ana = float(np.sum(to_f64(got) * e))
            # float32 gradients: 1e-5 of the direction's full weight
            assert abs(num - ana) <= 1e-5 * np.sum(np.abs(to_f64(got) * e)) + 1e-12


@pytest.mark.gpu
def test_offsets_past_32_bits(ost):
    """Rows past 2^32 bytes (2^31 elements) turn like the same rows alone."""
    N, Hq, Hkv, d = 460000, 32, 5, 128
    x = torch.zeros(1, N, Hq + Hkv, d, dtype=torch.bfloat16, device=DEV)
    x[0, -64:] = random_like_shape((64, Hq + Hkv, d), torch.bfloat16, 1).to(DEV)
    q, k = (y.transpose(1, 2) for y in (x[:, :, :Hq], x[:, :, Hq:]))
    pos = torch.arange(N, dtype=torch.int32, device=DEV)
    f = ost.rope_frequencies(d, device=DEV)
    want = ost.rope(q[:, :, -64:], k[:, :, -64:], pos[-64:].contiguous(), f)
    got = ost.rope(q, k, pos, f, out=(q, k))
    torch.cuda.synchronize()
    assert torch.equal(got[0][:, :, -64:], want[0]) and torch.equal(got[1][:, :, -64:], want[1])
    assert not bool(x[0, :-64].any())


@pytest.mark.gpu
def test_stream_graph_and_binding_refusals(ost):
    w = _freq(64).to(DEV)
    x = random_like_shape((2, 4, 9, 64), torch.bfloat16, 12).to(DEV)
    pos = torch.arange(18, dtype=torch.int32, device=DEV).view(2, 9)
    want, _ = ost.rope(x, None, pos, w)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got, _ = ost.rope(x, None, pos, w, stream=side)
    side.synchronize()
    assert torch.equal(got, want)
    out = torch.empty_like(x)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ost.rope(x, None, pos, w, out=(out, None))
    x.copy_(x.flip(2))
    pos.copy_(pos.flip(1))
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want.flip(2))
    for bad in (dict(positions=pos.long()), dict(inv_freq=w.float()), dict(positions=pos[:, :4]),
                dict(k=x[:, :2, :4]), dict(k=x.float()), dict(q=x.transpose(2, 3)),
                dict(q=x.cpu())):
        args = {"q": x, "k": None, "positions": pos, "inv_freq": w, **bad}
        with pytest.raises((ValueError, TypeError)):
            ost.rope(**args)


@pytest.mark.gpu
def test_position_shapes(ost):
    """[B, N], [N] or [1, N]; for one token also [B] or [1]. Other shapes of
    the same size are refused, not read in another order."""
    w = _freq(64).to(DEV)
    x = random_like_shape((3, 2, 5, 64), torch.bfloat16, 13).to(DEV)
    pos = torch.arange(2, 7, dtype=torch.int32, device=DEV)
    want = ost.rope(x, None, pos.expand(3, 5).contiguous(), w)[0]
    assert torch.equal(ost.rope(x, None, pos, w)[0], want)
    assert torch.equal(ost.rope(x, None, pos[None], w)[0], want)
    one = ost.rope(x[:, :, 0], None, pos[:1], w)[0]
    assert torch.equal(ost.rope(x[:, :, 0], None, pos[:1].expand(3).contiguous(), w)[0], one)
    all_of = torch.arange(15, dtype=torch.int32, device=DEV)
    for bad in (all_of, all_of.view(5, 3), all_of.view(3, 5, 1), all_of[:3], all_of[:5].view(5, 1),
                all_of[0]):
        with pytest.raises(ValueError):
            ost.rope(x, None, bad, w)


@pytest.mark.gpu
def test_far_positions_of_large_frequencies(ost):
    """The bound of the module docstring up to 2^64 radians a position (the
    fixed-point angle is off by 2^-32 turns at most, 2^-28 radians, well
    inside it); from there on NaN, not a wrong angle."""
    pos = torch.tensor([[2 ** 31 - 1, -2 ** 31, 2 ** 30 + 12345, 0, 1, -1, 3, 10 ** 9]],
                       dtype=torch.int32)
    w = torch.tensor([1e6, -1e10, 1e4, 8.1, 1e15, 2.0 ** 63, 1.8e19, math.nextafter(2.0 ** 64, 0),
                      2.0 ** 64, -1e20, 2.0 ** 65, 1e300, -2.0 ** 40, 1.2345e12, 4.4e18, 100.0],
                     dtype=torch.float64)
    for dt, inter in ((torch.float32, False), (torch.bfloat16, True)):
        x = random_like_shape((1, 2, 8, 32), dt, 3).to(DEV)
        y, _ = ost.rope(x, None, pos.to(DEV), w.to(DEV), inter)
        pairs = y.view(1, 2, 8, 16, 2) if inter else y.view(1, 2, 8, 2, 16).transpose(3, 4)
        bad = w.abs() >= 2.0 ** 64
        assert bad.sum() == 4 and bool(pairs[..., bad, :].isnan().all())
        good = torch.where(bad, torch.tensor(0.0, dtype=torch.float64), w)
        xz = x.clone()
        (xz.view(1, 2, 8, 16, 2) if inter else xz.view(1, 2, 8, 2, 16).transpose(3, 4)
         )[..., bad, :] = 0
        pairs[..., bad, :] = 0                       # (a frequency of zero leaves zeros)
        _check(y, xz, pos, good, inter, 1.0, False)


def _rows_of(base, strides, B, H, N, d):
    """Bytes of the float32 rows of a [B, H, N, d] tensor."""
    return {base + 4 * (b * strides[0] + h * strides[1] + n * strides[2]) + i
            for b in range(B) for h in range(H) for n in range(N) for i in range(4 * d)}


def test_outputs_on_top_of_inputs_or_each_other_are_refused(lib):
    """Exactly the calls whose outputs share a byte with an input (but for one
    turned in place) or with each other, among 3000 random layouts in one small
    range of addresses, and some by hand."""
    if torch.cuda.is_available():
        pytest.skip("made-up addresses: nothing may launch")
    rng = np.random.default_rng(5)
    seen = [0, 0]
    for _ in range(3000):
        B, Hq, Hkv, N, d = (int(x) for x in rng.integers([1, 1, 1, 1, 1], [3, 4, 3, 4, 3]))
        d *= 2

        def layout(H):
            if rng.random() < 0.5:                  # heads of a fused projection
                per = H + int(rng.integers(0, 4))
                return [N * per * d, d, per * d]
            gap = int(rng.integers(0, 3)) * d
            return [H * (N * d + gap), N * d + gap, d]
        at = [P + 4 * int(rng.integers(0, 60)) for _ in range(4)]
        st = [layout(H) for H in (Hq, Hq, Hkv, Hkv)]
        for i in (0, 2):                            # in place
            if rng.random() < 0.5:
                at[i + 1], st[i + 1] = at[i], st[i]
        rows = [_rows_of(a, s, B, H, N, d) for a, s, H in zip(at, st, (Hq, Hq, Hkv, Hkv))]
        meet = bool(rows[1] & rows[3]) or bool(rows[1] & rows[2]) or bool(rows[3] & rows[0])
        for i in (0, 2):
            # (strides of extents of one do not matter)
            same = at[i] == at[i + 1] and rows[i] == rows[i + 1]
            meet |= not same and bool(rows[i] & rows[i + 1])
        got = _call(lib, q=at[0], qs=st[0], qo=at[1], qos=st[1], k=at[2], ks=st[2], ko=at[3],
                    kos=st[3], pos=1 << 30, w=1 << 31, pstride=N, B=B, Hq=Hq, Hkv=Hkv, N=N, d=d,
                    rot=d, dt=0)
        assert (got == INVALID) == meet, (B, Hq, Hkv, N, d, at, st)
        seen[meet] += 1
    assert min(seen) > 300
    far = 1 << 30
    size = 2 * 4 * 4 * 64 * 2                       # bytes of q
    free = dict(qo=far, k=2 * far, ko=3 * far, pos=4 * far, w=5 * far)
    assert _call(lib, **free) != INVALID
    for bad in (dict(qo=P + 128), dict(qo=P + size - 16), dict(ko=far), dict(ko=P), dict(qo=2 * far),
                dict(qo=2 * far, ko=P), dict(pos=far + size - 4), dict(w=3 * far + 8),
                dict(pos=far - 4)):
        assert _call(lib, **{**free, **bad}) == INVALID, bad
    assert _call(lib, **{**free, "qo": P, "ko": 2 * far}) != INVALID


@pytest.mark.gpu
def test_binding_refuses_swapped_and_shifted_outputs(ost):
    w, pos = _freq(64).to(DEV), torch.arange(9, dtype=torch.int32, device=DEV)
    buf = random_like_shape((3, 2, 4, 10, 64), torch.float32, 14).to(DEV)
    q, k = buf[0, :, :, :9], buf[1, :, :, :9]
    before = buf.clone()
    for out in ((k, q), (buf[0, :, :, 1:], buf[2, :, :, :9]), (buf[2, :, :, :9], buf[2, :, :, 1:]),
                (buf[2, :, :, :9], buf[2, :, :, :9]), (k, buf[2, :, :, :9])):
        with pytest.raises(ost.AttnError):
            ost.rope(q, k, pos, w, out=out)
    with pytest.raises(ost.AttnError):
        ost.rope(q, q, pos, w, out=(q, k))          # turned in place and read as k
    torch.cuda.synchronize()
    assert torch.equal(buf, before)
    want = ost.rope(q, k, pos, w)
    ost.rope(q, k, pos, w, out=(q, k))
    assert torch.equal(q, want[0]) and torch.equal(k, want[1])
    assert torch.equal(buf[2], before[2]) and torch.equal(buf[:2, :, :, 9], before[:2, :, :, 9])
