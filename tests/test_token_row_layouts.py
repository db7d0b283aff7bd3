"""Every layout of a token row (one to sixteen warps, one to four chunks a lane) in the forward, 8-bit, quant and
backward kernels, with gains of both signs and zeros.  Tolerances: those of test_token_rows."""
import glob
import os
import re

import pytest
import torch

import joint_attention_gb300 as pkg
from joint_attention_gb300.build import CSRC, build
from test_token_rows import (FLOOR, SIZES, U, bwd64, check_e4m3, check_norm, check_quant, e4m3_of, gains, norm64,
                             randn)

gpu = pytest.mark.gpu


@pytest.fixture(scope="module")
def ja():
    build()
    pkg.load_library()
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    return pkg


# Wide and narrow rows of each layout that SIZES leaves out, with T around their rows a block.
LAYOUT_SIZES = [(9, 256), (17, 264), (8, 512), (15, 520), (5, 1536), (6, 1544), (3, 2056), (5, 3064), (2, 3080),
                (3, 4104), (2, 6144), (3, 6152), (301, 8192), (2, 8200), (3, 12288), (5, 12296), (309, 6152)]


@gpu
@pytest.mark.parametrize("T,C", LAYOUT_SIZES)
def test_every_row_layout(ja, T, C):
    """Forward, 8-bit, quant and backward kernels over every layout; gains of both signs and zeros."""
    x, res, g = randn((T, C), 101), randn((T, C), 102, 4.0), gains(C, 103)
    g[1::3] *= -1.0
    g[5::7] = 0.0
    y, h, r = ja.add_norm(x, g, res)
    check_norm(y, h, r, x, res, g)
    y8, s, h8, r8 = ja.add_norm_fp8(x, g, res)
    assert torch.equal(h8.view(torch.int16), h.view(torch.int16)) and torch.equal(r8, r)
    check_e4m3(y8, s, norm64(x, res, g)[2])
    x8, s = ja.quant_rows(x)
    check_quant(x8, s, x)
    dy, dh = randn((T, C), 104), randn((T, C), 105)
    for with_dh in (None, dh):
        dx, dg = ja.add_norm_backward(dy, h, r, g, with_dh)
        dx0, mag, dg0, dg_mag = bwd64(dy, with_dh, h, r, g)
        assert ((dx.double() - dx0).abs() <= dx0.abs() * 2.0 ** -8 + 64 * U * mag + 1e-38).all()
        assert ((dg.double() - dg0).abs() <= 128 * U * dg_mag + 1e-38).all()


@gpu
@pytest.mark.parametrize("T,C", SIZES + LAYOUT_SIZES)
@pytest.mark.parametrize("g_bits", [24, 3])
def test_norm_rows_to_e4m3_by_the_exact_quotient(ja, T, C, g_bits):
    """As test_norm_rows_are_the_nearest_e4m3_values: the exact quotient 448 z / max |z|, rounded to fp32 and then
    to e4m3, at every layout, with gains of both signs and zeros and with rows of zeros."""
    x, g = randn((T, C), 111), gains(C, 112)
    if g_bits < 24:
        g = torch.round(g * 4) / 4
        x[:, 0] = 14.0
        g[0] = -2.0
    g[1::3] *= -1.0
    g[5::7] = 0.0
    if T > 2:
        x[1] = 0.0
    y8, _, _, _ = ja.add_norm_fp8(x, g)
    z = x.double() * g.double()
    want = e4m3_of((448 * z / z.abs().amax(-1, keepdim=True).clamp_min(FLOOR)).float().double())
    assert torch.equal(y8.float().double(), want)


def test_dynamic_shared_arrays_state_their_alignment():
    """They are written by 16-byte vectors: bytes that the kernel aligns itself, or an array declared at 16 bytes (a
    narrower type's alignment would leave it to the size of the static arrays before it)."""
    found = [d for name in glob.glob(os.path.join(CSRC, "*.cu*"))
             for d in re.findall(r"extern __shared__ (.*)\[\];", open(name).read())]
    assert found
    for d in found:
        assert d == "uint8_t smem_raw" or d.startswith("__align__(16) "), d


# Fake, never-dereferenced device addresses: the refusal comes first.
A = [0x7F0000000000 + (i << 40) for i in range(10)]


@pytest.mark.parametrize("T,C", [(2 ** 32 + 24, 64), (2 ** 31, 64), (24, 2 ** 32 + 64), (24, -2 ** 32 + 64)])
def test_sizes_beyond_32_bits_are_refused(T, C):
    """The library takes 32-bit sizes: one beyond them is refused, and not cut to its low bits (24 rows of 64 here)."""
    build()
    pkg.load_library()
    for call in (lambda: pkg.jattn_quant_rows(A[0], T, C, A[1], A[2], stream=0),
                 lambda: pkg.jattn_add_norm(A[0], A[1], A[2], T, C, 1e-6, A[3], A[4], A[5], stream=0),
                 lambda: pkg.jattn_add_norm_fp8(A[0], A[1], A[2], T, C, 1e-6, A[3], A[4], A[5], A[6], stream=0),
                 lambda: pkg.jattn_add_norm_bwd(A[0], A[1], A[2], A[3], A[4], T, C, A[5], A[6], A[7], stream=0)):
        with pytest.raises(pkg.JattnError) as e:
            call()
        assert e.value.status == pkg.STATUS_CODE["JATTN_ERR_INVALID_ARG"]
    assert pkg.jattn_add_norm_bwd_bytes(T, C) == 0
