"""Token rows: the residual's addition with RMSNorm (bf16 and 8-bit output), its
backward, and rows in 8 bits, against their definitions in float64.

Tolerances, from the arithmetic (u = 2^-24, one fp32 rounding):
* h is the exact sum rounded once to bf16 (the fp32 sum of two bf16 values
  rounded again gives the same): equal bits.
* r: a lane adds at most 32 squares, then at most 10 levels join the lanes; the
  mean and eps round once, the root once, and the root halves the error of its
  argument: 43 u / 2 + u < 2^-19 relative.
* y = bf16(g h r): half a bf16 step (2^-8 relative at most) and r's error with two
  products, below 2^-18.
* the scale s: as r with the products and a division, 2^-18.  y8: the quotient
  z / s within 2^-17 of the exact one, then half an e4m3 step: 2^-4 relative, or
  2^-10 among the subnormals.
* dx: half a bf16 step and, for u n summed like the squares, 64 u of the terms'
  magnitudes.  dg: a fixed tree over the rows, at most 128 roundings on any
  path at these sizes: 128 u of the terms' magnitudes.
"""
import numpy as np
import pytest
import torch

from joint_attention_gb300 import STATUS_CODE
import joint_attention_gb300 as pkg
from joint_attention_gb300.build import build

U = 2.0 ** -24
EPS = 1e-6
FLOOR = 2.0 ** -80
FLOOR_SCALE = float(np.float32(FLOOR / 448))  # the scale of a row of zeros
gpu = pytest.mark.gpu


@pytest.fixture(scope="module")
def lib():
    build()
    return pkg.load_library()


@pytest.fixture(scope="module")
def ja(lib):
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    return pkg


def randn(shape, seed, scale=1.0, dtype=torch.bfloat16):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(shape, generator=g, device="cuda") * scale).to(dtype)


def gains(C, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.rand(C, generator=g, device="cuda") + 0.5


def norm64(x, res, g, eps=EPS):
    """h (bf16), r and z in float64."""
    h = x if res is None else (x.double() + res.double()).to(torch.bfloat16)
    h64 = h.double()
    r = 1.0 / torch.sqrt((h64 * h64).mean(-1) + eps)
    return h, r, h64 * r[..., None] * g.double()


def check_norm(y, h, r, x, res, g, eps=EPS):
    h0, r0, z0 = norm64(x, res, g, eps)
    assert torch.equal(h.view(torch.int16), h0.view(torch.int16))
    assert ((r.double() - r0).abs() <= 2.0 ** -19 * r0).all()
    assert ((y.double() - z0).abs() <= z0.abs() * (2.0 ** -8 + 2.0 ** -18) + 1e-38).all()


def check_e4m3(q, s, z0):
    """q (e4m3) and s against the float64 values z0."""
    s0 = z0.abs().amax(-1).clamp_min(FLOOR) / 448
    assert ((s.double() - s0).abs() <= 2.0 ** -18 * s0).all()
    v = z0 / s0[..., None]
    off = (q.float().double() - v).abs()
    assert (off <= v.abs() * (2.0 ** -4 + 2.0 ** -17) + 2.0 ** -10).all()
    # not merely within a step: nearly all are the nearest e4m3 value
    near = v.to(torch.float8_e4m3fn).float() == q.float()
    assert (~near).double().mean() <= 1e-3 + 3.0 / q.numel()


def check_quant(x8, s, x):
    """Bit for bit: both quotients are of values exact in fp32 and round once (float64 quotients of
    such values round to fp32 as the exact ones do).  Midpoints of e4m3 are common here."""
    m = x.double().abs().amax(-1)
    assert torch.equal(s, (m / 448).float())
    want = (448 * x.double() / m[:, None]).float().to(torch.float8_e4m3fn)
    assert torch.equal(x8.view(torch.uint8), want.view(torch.uint8))


SIZES = [(1, 8), (1, 768), (7, 200), (333, 776), (5, 1024), (3, 1032), (100, 1096), (9, 2048), (6, 4096),
         (2, 16384), (2305, 768)]


@gpu
@pytest.mark.parametrize("T,C", SIZES)
@pytest.mark.parametrize("with_res", [False, True])
def test_add_norm(ja, T, C, with_res):
    x, g = randn((T, C), 1), gains(C, 2)
    res = randn((T, C), 3, 4.0) if with_res else None
    y, h, r = ja.add_norm(x, g, res)
    check_norm(y, h, r, x, res, g)
    y8, s, h8, r8 = ja.add_norm_fp8(x, g, res)
    assert torch.equal(h8.view(torch.int16), h.view(torch.int16)) and torch.equal(r8, r)
    check_e4m3(y8, s, norm64(x, res, g)[2])


@gpu
@pytest.mark.parametrize("T,C", SIZES)
def test_quant_rows(ja, T, C):
    x = randn((T, C), 5, 0.03)
    x8, s = ja.quant_rows(x)
    check_quant(x8, s, x)


def bwd64(dy, dh, h, r, g):
    dy, h, g, r = dy.double(), h.double(), g.double(), r.double()[..., None]
    n, u = h * r, dy * g
    m = (u * n).mean(-1, keepdim=True)
    dh = 0.0 if dh is None else dh.double()
    mag = (u * n).abs().mean(-1, keepdim=True)
    dx = dh + r * (u - n * m)
    dx_mag = (dh.abs() if isinstance(dh, torch.Tensor) else 0.0) + r * (u.abs() + n.abs() * mag)
    return dx, dx_mag, (dy * n).sum(0), (dy * n).abs().sum(0)


def e4m3_of(q):
    """The e4m3 value nearest to q (float64, at most 448 in magnitude; ties to even), as float64."""
    step = torch.exp2(torch.floor(torch.log2(q.abs().clamp_min(2.0 ** -6))) - 3)
    return torch.round(q / step) * step


@gpu
@pytest.mark.parametrize("T,C", [(20000, 768), (4000, 2048), (3001, 1096), (500, 16384), (7000, 8)])
@pytest.mark.parametrize("g_bits", [24, 3])
def test_norm_rows_are_the_nearest_e4m3_values(ja, T, C, g_bits):
    """448 z / max |z| does not depend on r: with the exact products h g (32 bits) in float64 the quotient is off by
    2^-53; it is rounded to fp32 and then to e4m3, which that decides alike unless it lies within 2^-53 of the
    midpoint of two fp32 values next to a midpoint of e4m3 (one in 2^48).  With gains of 3 bits many are midpoints
    of e4m3."""
    x, res, g = randn((T, C), 55), randn((T, C), 56, 2.0), gains(C, 57)
    if g_bits < 24:
        g = torch.round(g * 4) / 4
        x[:, 0], res[:, 0] = 14.0, 0.0
        g[0] = 2.0  # the row's maximum 28 = 448 / 16 (or a few larger ones): quotients are z times a power of two
    y8, s, h, r = ja.add_norm_fp8(x, g, res)
    z = h.double() * g.double()
    want = e4m3_of((448 * z / z.abs().amax(-1, keepdim=True)).float().double())
    assert torch.equal(y8.float().double(), want)


@gpu
@pytest.mark.parametrize("T,C", SIZES + [(5000, 256), (1217, 2048)])
@pytest.mark.parametrize("with_dh", [False, True])
def test_add_norm_backward(ja, T, C, with_dh):
    h, g, dy = randn((T, C), 7, 3.0), gains(C, 8), randn((T, C), 9)
    dh = randn((T, C), 10) if with_dh else None
    _, _, r = ja.add_norm(h, g)
    dx, dg = ja.add_norm_backward(dy, h, r, g, dh)
    dx0, mag, dg0, dg_mag = bwd64(dy, dh, h, r, g)
    assert ((dx.double() - dx0).abs() <= dx0.abs() * 2.0 ** -8 + 64 * U * mag + 1e-38).all()
    assert ((dg.double() - dg0).abs() <= 128 * U * dg_mag + 1e-38).all()
    again = ja.add_norm_backward(dy, h, r, g, dh)
    assert torch.equal(dx.view(torch.int16), again[0].view(torch.int16)) and torch.equal(dg, again[1])


@gpu
def test_add_norm_backward_is_the_gradient_by_differences(ja):
    """<dx, v> and <dg, w> against central differences of L = sum(dy y) + sum(dh h) in float64, where
    neither h nor y is rounded: dx differs by its bf16 rounding alone."""
    T, C = 13, 328
    x, res, g = randn((T, C), 11), randn((T, C), 12, 2.0), gains(C, 13)
    dy, dh = randn((T, C), 14), randn((T, C), 15)
    h = (x.double() + res.double()).to(torch.bfloat16)
    _, _, r = ja.add_norm(h, g)
    dx, dg = ja.add_norm_backward(dy, h, r, g, dh)

    def loss(t, gain):
        rr = 1.0 / torch.sqrt((t * t).mean(-1, keepdim=True) + EPS)
        return (dy.double() * t * rr * gain).sum() + (dh.double() * t).sum()

    for k in range(4):
        v, w, e = randn((T, C), 20 + k, dtype=torch.float64), randn((C,), 30 + k, dtype=torch.float64), 1e-5
        t, gain = h.double(), g.double()
        by_x = (loss(t + e * v, gain) - loss(t - e * v, gain)) / (2 * e)
        by_g = (loss(t, gain + e * w) - loss(t, gain - e * w)) / (2 * e)
        # each dx is off by at most 2^-8 of itself (and fp32 terms), with signs of their own
        tol = (2.0 ** -7 * dx.double() * v).norm() * 4
        assert abs((dx.double() * v).sum() - by_x) <= tol + 1e-4
        assert abs((dg.double() * w).sum() - by_g) <= 128 * U * (dg.double() * w).abs().sum() * 8 + 1e-4


@gpu
@pytest.mark.parametrize("C", [768, 2048])
def test_in_place_forms_give_the_same_bits(ja, C):
    T = 301
    x, res, g = randn((T, C), 40), randn((T, C), 41, 2.0), gains(C, 42)
    y, h, r = ja.add_norm(x, g, res)
    y2, stream = torch.empty_like(y), res.clone()
    ja.jattn_add_norm(x, stream, g, T, C, EPS, stream, y2, None)
    assert torch.equal(y2, y) and torch.equal(stream, h)
    dy, dh = randn((T, C), 43), randn((T, C), 44)
    dx, dg = ja.add_norm_backward(dy, h, r, g, dh)
    buf, dg2 = dh.clone(), torch.empty_like(dg)
    work = torch.full((ja.jattn_add_norm_bwd_bytes(T, C),), 0xFF, dtype=torch.uint8, device="cuda")
    ja.jattn_add_norm_bwd(dy, buf, h, r, g, T, C, buf, dg2, work)
    assert torch.equal(buf, dx) and torch.equal(dg2, dg)


@gpu
@pytest.mark.parametrize("C", [776, 2048])
def test_rows_of_zeros_infinities_and_nan(ja, C):
    T = 12
    x, g = randn((T, C), 50), gains(C, 51)
    x[1] = 0.0
    x[3, 5] = float("nan")
    x[5, 7] = float("inf")
    x[7] = torch.finfo(torch.bfloat16).min  # squares pass the fp32 range: r = 0
    x[9] = 1e-38
    y, _, r = ja.add_norm(x, g)
    y8, s, _, _ = ja.add_norm_fp8(x, g)
    fine = [0, 1, 2, 4, 6, 8, 9, 10, 11]
    check_norm(y[fine], x[fine], r[fine], x[fine], None, g)
    check_e4m3(y8[fine], s[fine], norm64(x[fine], None, g)[2])
    assert not y[1].any() and not y8[1].float().any() and s[1].item() == FLOOR_SCALE
    assert y[3].isnan().all() and y8[3].float().isnan().all()
    assert y[5].isnan().sum() == 1 and not y[5].nan_to_num(0.0).any()  # inf * 0 is NaN, the others are 0
    assert r[7] == 0 and not y[7].any() and not y8[7].float().any()
    x8, s = ja.quant_rows(x)
    assert s[1].item() == FLOOR_SCALE and not x8[1].float().any()
    assert x8[3].float().isnan().sum() == 1 and s[3].isfinite()
    assert (x8[5].float() * s[5]).isnan().all()
    assert torch.equal(x8[7].float(), torch.full((C,), -448.0, device="cuda"))


@gpu
def test_offsets_beyond_32_bits(ja):
    C, T = 16384, (1 << 17) + 3  # 2^31 + 49152 values
    x = torch.zeros((T, C), dtype=torch.bfloat16, device="cuda")
    x[-3:] = randn((3, C), 60)
    res = torch.zeros_like(x)
    res[-2:] = randn((2, C), 61)
    g = gains(C, 62)
    y, h, r = ja.add_norm(x, g, res)
    check_norm(y[-3:], h[-3:], r[-3:], x[-3:], res[-3:], g)
    assert not y[:4].any() and not h[:4].any()
    dy = x  # any gradient: zero but for the last rows
    dx, dg = ja.add_norm_backward(dy, h, r, g)
    dx0, mag, dg0, dg_mag = bwd64(dy[-3:], None, h[-3:], r[-3:], g)
    assert ((dx[-3:].double() - dx0).abs() <= dx0.abs() * 2.0 ** -8 + 64 * U * mag + 1e-38).all()
    assert ((dg.double() - dg0).abs() <= 128 * U * dg_mag + 1e-38).all()
    del y, dx, res
    x8, s = ja.quant_rows(x)
    check_quant(x8[-3:], s[-3:], x[-3:])


@gpu
def test_on_another_stream_and_captured(ja):
    """The calls on a stream of their own, and captured into a graph that is replayed on new inputs."""
    T, C = 777, 768
    x, res, g, dy = randn((T, C), 70), randn((T, C), 71), gains(C, 72), randn((T, C), 73)
    want = ja.add_norm(x, g, res)
    want_b = ja.add_norm_backward(dy, want[1], want[2], g)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for stream in (side, side.cuda_stream):
        got = ja.add_norm(x, g, res, stream=stream)
        got_b = ja.add_norm_backward(dy, got[1], got[2], g, stream=stream)
        side.synchronize()
        for a, b in zip((*got, *got_b), (*want, *want_b)):
            assert torch.equal(a, b)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y, h, r = ja.add_norm(x, g, res)
        dx, dg = ja.add_norm_backward(dy, h, r, g)
        y8, s, _, _ = ja.add_norm_fp8(x, g, res)
    x.copy_(randn((T, C), 74))
    dy.copy_(randn((T, C), 75))
    graph.replay()
    graph.replay()
    torch.cuda.synchronize()
    want = ja.add_norm(x, g, res)
    want_b = ja.add_norm_backward(dy, want[1], want[2], g)
    want_8 = ja.add_norm_fp8(x, g, res)
    for a, b in zip((y, h, r, dx, dg, y8.view(torch.uint8), s),
                    (*want, *want_b, want_8[0].view(torch.uint8), want_8[1])):
        assert torch.equal(a, b)


@gpu
def test_profile_counts_the_token_kernels(ja):
    x, g = randn((64, 768), 80), gains(768, 81)
    ja.jattn_profile_reset()
    ja.jattn_profile_enable(True)
    y, h, r = ja.add_norm(x, g)
    ja.add_norm_backward(y, h, r, g)
    ja.quant_rows(x)
    torch.cuda.synchronize()
    ja.jattn_profile_enable(False)
    snap = ja.profile_snapshot()
    assert [snap[k][0] for k in ("add_norm", "add_norm_bwd", "add_norm_dg", "quant_rows")] == [1, 1, 1, 1]
    ja.jattn_profile_reset()


@gpu
def test_wrappers_refuse(ja):
    x, g = randn((6, 768), 90), gains(768, 91)
    with pytest.raises(ValueError):
        ja.add_norm(x[:, ::2], gains(384, 1))  # strides
    with pytest.raises(ValueError):
        ja.add_norm(x, gains(760, 1))          # another width
    with pytest.raises(ValueError):
        ja.add_norm(x, g, x[:3])               # another number of rows
    with pytest.raises(ValueError):
        ja.add_norm(x.float(), g)
    with pytest.raises(ValueError):
        ja.quant_rows(x.cpu())
    with pytest.raises(ja.JattnError):
        ja.quant_rows(randn((4, 12), 1))       # width not a multiple of 8
    with pytest.raises(ja.JattnError):
        ja.add_norm(x, g, eps=0.0)
    y, h, r = ja.add_norm(x, g)
    with pytest.raises(ValueError):
        ja.jattn_add_norm_bwd(y, None, h, r, g, 6, 768, torch.empty_like(y), torch.empty_like(g),
                              torch.empty(16, dtype=torch.uint8, device="cuda"))


# Fake, never-dereferenced device addresses: validation happens first.
A = 0x7F0000000000


def at(i):
    return A + (i << 33)


def test_token_row_validation(lib):
    code = STATUS_CODE
    base = dict(x=at(0), res=at(1), g=at(2), T=24, C=64, eps=1e-6, h=at(3), y=at(4), r=at(5))
    f = lambda **kw: lib.jattn_add_norm(*{**base, **kw}.values(), None)  # noqa: E731
    for kw in (dict(x=None), dict(g=None), dict(y=None), dict(res=None), dict(h=None), dict(T=0), dict(C=0),
               dict(T=-1), dict(eps=0.0), dict(eps=-1.0), dict(eps=float("nan")), dict(eps=float("inf"))):
        assert f(**kw) == code["JATTN_ERR_INVALID_ARG"], kw
    for kw in (dict(C=60), dict(C=16392)):
        assert f(**kw) == code["JATTN_ERR_UNSUPPORTED"], kw
    for kw in (dict(x=A + 8), dict(r=at(5) + 4)):
        assert f(**kw) == code["JATTN_ERR_MISALIGNED"], kw
    for kw in (dict(y=at(0)), dict(h=at(0)), dict(h=at(1) + 16), dict(y=at(1)), dict(r=at(3)), dict(y=at(3)),
               dict(h=at(2))):
        assert f(**kw) == code["JATTN_ERR_ALIAS"], kw
    base8 = dict(x=at(0), res=at(1), g=at(2), T=24, C=64, eps=1e-6, h=at(3), y8=at(4), s=at(5), r=at(6))
    f = lambda **kw: lib.jattn_add_norm_fp8(*{**base8, **kw}.values(), None)  # noqa: E731
    for kw in (dict(y8=None), dict(s=None), dict(res=None), dict(eps=0.0)):
        assert f(**kw) == code["JATTN_ERR_INVALID_ARG"], kw
    assert f(y8=at(0)) == code["JATTN_ERR_ALIAS"] and f(s=at(6)) == code["JATTN_ERR_ALIAS"]
    assert f(C=20) == code["JATTN_ERR_UNSUPPORTED"] and f(s=at(5) + 4) == code["JATTN_ERR_MISALIGNED"]
    baseq = dict(x=at(0), T=24, C=64, x8=at(1), s=at(2))
    f = lambda **kw: lib.jattn_quant_rows(*{**baseq, **kw}.values(), None)  # noqa: E731
    assert f(x=None) == f(x8=None) == f(s=None) == f(T=0) == code["JATTN_ERR_INVALID_ARG"]
    assert f(C=4) == code["JATTN_ERR_UNSUPPORTED"]
    assert f(x8=at(0)) == f(s=at(1)) == code["JATTN_ERR_ALIAS"]
    baseb = dict(dy=at(0), dh=at(1), h=at(2), r=at(3), g=at(4), T=24, C=64, dx=at(5), dg=at(6), work=at(7))
    f = lambda **kw: lib.jattn_add_norm_bwd(*{**baseb, **kw}.values(), None)  # noqa: E731
    for k in ("dy", "h", "r", "g", "dx", "dg", "work"):
        assert f(**{k: None}) == code["JATTN_ERR_INVALID_ARG"], k
    assert f(T=0) == code["JATTN_ERR_INVALID_ARG"] and f(C=12) == code["JATTN_ERR_UNSUPPORTED"]
    assert f(work=at(7) + 8) == code["JATTN_ERR_MISALIGNED"]
    for kw in (dict(dx=at(0)), dict(dx=at(2)), dict(dx=at(1) + 16), dict(dg=at(4)), dict(work=at(5)),
               dict(work=at(2))):
        assert f(**kw) == code["JATTN_ERR_ALIAS"], kw
    assert lib.jattn_add_norm_bwd_bytes(24, 64) > 0
    assert lib.jattn_add_norm_bwd_bytes(0, 64) == lib.jattn_add_norm_bwd_bytes(24, 60) == 0


def test_token_kernel_kinds(lib):
    names = [pkg.jattn_kernel_name(k) for k in pkg.TOKEN_KERNEL_KINDS]
    assert "unknown" not in names and len(set(names)) == len(names)
    assert pkg.jattn_kernel_name(pkg.TOKEN_KERNEL_KINDS[-1] + 1) == "unknown"
