"""The QKV projection from 8-bit rows (jattn_qkv_norm_fp8) and with the batch items' low-rank
adapters (jattn_qkv_norm_lora), against their definitions in float64, and the chain from the
residual stream to the attention through them.

Tolerances, from the arithmetic:
* Y of either form accumulates K terms in fp32 (K = C, and the rank with adapters), each addition
  off by at most one ulp (2^-23) of the terms' summed magnitudes, a few fp32 products and the bias
  included (K + 8 roundings), then rounds once to bf16 (half a step, at most 2^-8 relative):
  |got - exact| <= (K + 8) 2^-23 mag + 2^-8 |exact|, mag the sum of the terms' magnitudes.
* U = scale X A^T is kept as two bf16 terms between the two products of an adapter (2^-8 of 2^-8): another
  sum_j 2^-16 |U_j B_oj|, and its own accumulation (C + 2) 2^-23 sum_j mag(U_j) |B_oj|.
* q_hat, k_hat, 1/rms: bit for bit (1/rms to 2^-21) what jattn_fwd_train keeps for the same q, k.
"""
import threading
from concurrent.futures import ThreadPoolExecutor

import numpy as np
import pytest
import torch

import oracle
from joint_attention_gb300 import STATUS_CODE
import joint_attention_gb300 as pkg
from joint_attention_gb300.build import build

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


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def randn(g, *shape, scale=1.0, dtype=torch.bfloat16):
    return (torch.randn(shape, generator=g, device="cuda") * scale).to(dtype)


def saved_parts(saved, q):
    """q_hat, k_hat, 1/rms of the q and of the k rows, as views (each part at a multiple of 256 bytes)."""
    up = lambda x: (x + 255) // 256 * 256  # noqa: E731
    n, rows = q.numel() * 2, q.numel() // q.shape[-1] * 4
    at = [0, up(n), 2 * up(n), 2 * up(n) + up(rows)]
    return ([saved[o:o + n].view(torch.bfloat16).view(q.shape) for o in at[:2]]
            + [saved[o:o + rows].view(torch.float32).view(q.shape[:-1]) for o in at[2:]])


def heads(y, H, d):
    """[B, N, 3 H d] -> q, k, v [B, H, N, d]"""
    B, N, _ = y.shape
    return y.view(B, N, 3, H, d).permute(2, 0, 3, 1, 4)


def check_y(got, exact, bound, H, d):
    """got: (q, k, v); exact, bound [B, N, 3 H d] float64 (bound: what may come before the last rounding)."""
    for t, e, b in zip(got, heads(exact, H, d), heads(bound, H, d)):
        assert t.isfinite().all()
        assert ((t.double() - e).abs() <= b + 2.0 ** -8 * e.abs() + 1e-38).all()


def check_norms(ja, q, k, v, saved, gq, gk, n_txt):
    _, _, saved0 = ja.forward_train(q, k, v, gq, gk, n_txt)
    a, b = saved_parts(saved, q), saved_parts(saved0, q)
    for i in range(2):
        assert torch.equal(a[i].view(torch.int16), b[i].view(torch.int16))
        assert ((a[2 + i] - b[2 + i]).abs() <= 2.0 ** -21 * b[2 + i]).all()


def ok(ja):
    torch.cuda.synchronize()
    assert ja.jattn_last_device_error() == 0


def rows_e4m3(x):
    m = x.float().abs().amax(-1, keepdim=True).clamp_min(2.0 ** -80)
    return (x.float() * 448 / m).to(torch.float8_e4m3fn), (m / 448).squeeze(-1).contiguous()


FP8_CASES = [
    # B, H, N_img, N_txt, d, C, bias
    (2, 4, 200, 77, 64, 256, True),    # ragged row tails in both streams
    (1, 3, 130, 5, 64, 208, False),    # partial column tile and partial K step
    (2, 2, 96, 0, 128, 128, True),     # no caption stream, d = 128
    (1, 4, 0, 40, 128, 144, True),     # caption stream only
    (1, 1, 1, 1, 64, 16, True),        # one token per stream, the narrowest width
    (33, 2, 1, 2, 64, 64, False),      # single tokens of many items
    (3, 12, 256, 77, 64, 768, True),
    (1, 16, 300, 77, 128, 2048, True),
    (3, 1, 50, 0, 64, 64, True),       # one head, one stream: an item's rows follow the last one's on in memory
    (5, 12, 1024, 77, 64, 192, True),  # more tiles than CTAs
]


def fp8_inputs(B, H, N_img, N_txt, d, C, bias, seed):
    g = gen(seed)
    t = {}
    for s, n in (("img", N_img), ("txt", N_txt)):
        t["x_" + s], t["sx_" + s] = rows_e4m3(randn(g, B, n, C))
        t["w_" + s], t["sw_" + s] = rows_e4m3(randn(g, 3 * H * d, C, scale=C ** -0.5))
        t["b_" + s] = randn(g, 3 * H * d, scale=0.1, dtype=torch.float32) if bias else None
    t["gq"], t["gk"] = (torch.rand(d, generator=g, device="cuda") + 0.5 for _ in range(2))
    return t


def fp8_call(ja, t, H, stream=None):
    return ja.qkv_norm_fp8(t["x_img"], t["sx_img"], t["w_img"], t["sw_img"], t["b_img"], t["x_txt"], t["sx_txt"],
                           t["w_txt"], t["sw_txt"], t["b_txt"], t["gq"], t["gk"], H, stream)


def fp8_exact(t):
    """Y [B, N, 3 H d] and the summed magnitudes of its terms, float64."""
    ys, mags = [], []
    for s in ("txt", "img"):
        x = t["x_" + s].double() * t["sx_" + s].double()[..., None]
        w = t["w_" + s].double() * t["sw_" + s].double()[:, None]
        b = t["b_" + s].double() if t["b_" + s] is not None else torch.zeros(len(w), dtype=torch.float64, device="cuda")
        ys.append(x @ w.t() + b)
        mags.append(x.abs() @ w.abs().t() + b.abs())
    return torch.cat(ys, 1), torch.cat(mags, 1)


@gpu
@pytest.mark.parametrize("case", FP8_CASES)
def test_qkv_norm_fp8(ja, case):
    B, H, N_img, N_txt, d, C, bias = case
    t = fp8_inputs(*case, seed=100 + C + N_img)
    q, k, v, saved = fp8_call(ja, t, H)
    ok(ja)
    y, mag = fp8_exact(t)
    check_y((q, k, v), y, (C + 8) * 2.0 ** -23 * mag, H, d)
    check_norms(ja, q, k, v, saved, t["gq"], t["gk"], N_txt)


@gpu
def test_fp8_extreme_values_and_scales(ja):
    """e4m3's largest and subnormal values, scales far apart, rows of zeros, and NaN that stays in its row."""
    B, H, N_img, N_txt, d, C = 2, 2, 40, 9, 64, 96
    t = fp8_inputs(B, H, N_img, N_txt, d, C, True, 7)
    t["x_img"][0, 0] = torch.full((C,), 448.0, device="cuda").to(torch.float8_e4m3fn)
    t["x_img"][0, 1] = torch.full((C,), 2.0 ** -9, device="cuda").to(torch.float8_e4m3fn)
    t["x_img"][0, 2] = torch.zeros(C, device="cuda").to(torch.float8_e4m3fn)
    t["sx_img"][0, 3] = 1e-30
    t["sx_img"][0, 4] = 1e20
    q, k, v, saved = fp8_call(ja, t, H)
    ok(ja)
    y, mag = fp8_exact(t)
    check_y((q, k, v), y, (C + 8) * 2.0 ** -23 * mag, H, d)
    t["sx_img"][1, 5] = float("nan")
    q2, k2, v2, _ = fp8_call(ja, t, H)
    ok(ja)
    for a, b in ((q2, q), (k2, k), (v2, v)):
        assert a[1, :, N_txt + 5].isnan().all()
        a[1, :, N_txt + 5] = b[1, :, N_txt + 5]
        assert torch.equal(a, b)


LORA_CASES = [
    # B, H, N_img, N_txt, d, C, rank, n, bias
    (2, 4, 200, 77, 64, 256, 16, 3, True),     # row tiles over two items
    (1, 3, 130, 5, 64, 200, 8, 1, False),      # half a pair of the rank, column tiles over q, k and v
    (5, 1, 1, 1, 64, 8, 24, 2, True),          # one head: all three parts in one column tile
    (140, 2, 1, 0, 64, 64, 16, 140, True),     # single tokens: 128 adapters in a row tile
    (3, 2, 96, 0, 128, 128, 128, 2, True),     # the largest rank, d = 128
    (2, 4, 40, 300, 128, 136, 40, 2, False),   # rank of two pairs and a half
    (4, 2, 128, 7, 64, 64, 112, 4, True),      # items of whole row tiles; rank beyond one product's columns
    (3, 12, 256, 77, 64, 768, 16, 4, True),
    (2, 16, 2, 77, 128, 2048, 64, 2, True),
    (70, 5, 2, 3, 64, 320, 80, 9, True),
    (3, 1, 50, 0, 64, 64, 16, 3, False),       # one head, one stream
    (5, 12, 1000, 77, 64, 192, 24, 4, True),   # more tiles than CTAs, row tiles over two items
    (3, 7, 1100, 33, 128, 72, 48, 2, True),
    (600, 8, 3, 1, 64, 64, 8, 600, True),      # 86 items in a row tile of 256
]


def lora_inputs(B, H, N_img, N_txt, d, C, rank, n, bias, seed, streams=("img", "txt")):
    g = gen(seed)
    t = {"down_img": None, "up_img": None, "down_txt": None, "up_txt": None}
    for s, N_s in (("img", N_img), ("txt", N_txt)):
        t["x_" + s] = randn(g, B, N_s, C)
        t["w_" + s] = randn(g, 3 * H * d, C, scale=C ** -0.5)
        t["b_" + s] = randn(g, 3 * H * d, scale=0.1, dtype=torch.float32) if bias else None
        if s in streams:
            t["down_" + s] = randn(g, n, 3 * rank, C, scale=C ** -0.5)
            t["up_" + s] = randn(g, n, 3 * H * d, rank, scale=rank ** -0.5)
    t["gq"], t["gk"] = (torch.rand(d, generator=g, device="cuda") + 0.5 for _ in range(2))
    t["scale"] = torch.rand(n, generator=g, device="cuda") + 0.5
    t["index"] = (torch.arange(B, device="cuda") % n).int()
    return t


def lora_call(ja, t, H, stream=None):
    return ja.qkv_norm_lora(t["x_img"], t["w_img"], t["b_img"], t["x_txt"], t["w_txt"], t["b_txt"], t["gq"], t["gk"],
                            H, t["down_img"], t["up_img"], t["down_txt"], t["up_txt"], t["scale"], t["index"], stream)


def lora_exact(t, rank):
    """Y [B, N, 3 H d], the magnitudes of its terms, and what U's rounding and accumulation may add, float64."""
    ys, mags, offs = [], [], []
    C, n = t["x_img"].shape[-1], t["scale"].numel()
    idx = t["index"].long()
    has = (idx >= 0) & (idx < n)
    at = torch.where(has, idx, 0)
    sc = torch.where(has, t["scale"][at].double(), 0.0)
    for s in ("txt", "img"):
        x, w = t["x_" + s].double(), t["w_" + s].double()
        b = t["b_" + s].double() if t["b_" + s] is not None else torch.zeros(len(w), dtype=torch.float64, device="cuda")
        y, mag = x @ w.t() + b, x.abs() @ w.abs().t() + b.abs()
        off = torch.zeros_like(y)
        if t["down_" + s] is not None:
            (B, N, _), H3 = x.shape, len(w)
            part = lambda u: u.view(B, N, 3, rank).transpose(1, 2)  # noqa: E731
            join = lambda z: z.transpose(1, 2).reshape(B, N, len(w))  # noqa: E731
            down, up = t["down_" + s][at].double(), t["up_" + s][at].double()
            up = up.view(B, 3, H3 // 3, rank).transpose(2, 3)
            u = part(x @ down.transpose(1, 2)) * sc[:, None, None, None]
            mu = part(x.abs() @ down.abs().transpose(1, 2)) * sc[:, None, None, None].abs()
            y = y + join(u @ up)
            mag = mag + join(u.abs() @ up.abs())
            off = join((2.0 ** -16 * u.abs() + (C + 2) * 2.0 ** -23 * mu) @ up.abs())
        ys.append(y), mags.append(mag), offs.append(off)
    return torch.cat(ys, 1), torch.cat(mags, 1), torch.cat(offs, 1)


def check_lora(ja, t, out, H, d, rank):
    q, k, v, saved = out
    y, mag, off = lora_exact(t, rank)
    C = t["x_img"].shape[-1]
    check_y((q, k, v), y, (C + rank + 8) * 2.0 ** -23 * mag + off, H, d)
    check_norms(ja, q, k, v, saved, t["gq"], t["gk"], t["x_txt"].shape[1])


@gpu
@pytest.mark.parametrize("case", LORA_CASES)
def test_qkv_norm_lora(ja, case):
    B, H, N_img, N_txt, d, C, rank, n, bias = case
    t = lora_inputs(*case, seed=200 + C + N_img)
    out = lora_call(ja, t, H)
    ok(ja)
    check_lora(ja, t, out, H, d, rank)
    again = lora_call(ja, t, H)
    for a, b in zip(out[:3], again[:3]):
        assert torch.equal(a, b)


@gpu
@pytest.mark.parametrize("B,H,N_img,N_txt,d", [(3, 1, 50, 0, 64), (4, 1, 0, 40, 128), (9, 1, 700, 0, 64)])
def test_qkv_norm_with_one_head_and_one_stream(ja, B, H, N_img, N_txt, d):
    """The rows of an item then follow the last one's on in memory, and a warp's 32 rows may be of two items:
    every row of q, k, v, q_hat and k_hat is written."""
    C = 64
    t = lora_inputs(B, H, N_img, N_txt, d, C, 8, 1, True, 33, streams=())
    q, k, v = (torch.full((B, H, N_img + N_txt, d), float("nan"), dtype=torch.bfloat16, device="cuda")
               for _ in range(3))
    saved = torch.full((ja.jattn_saved_bytes(B, H, N_img, N_txt, d),), 0xFF, dtype=torch.uint8, device="cuda")
    ja.jattn_qkv_norm(t["x_img"] if N_img else None, t["w_img"], t["b_img"], t["x_txt"] if N_txt else None,
                      t["w_txt"], t["b_txt"], t["gq"], t["gk"], B, H, N_img, N_txt, d, C, q, k, v, saved)
    ok(ja)
    y, mag, _ = lora_exact(t, 8)
    check_y((q, k, v), y, (C + 8) * 2.0 ** -23 * mag, H, d)
    check_norms(ja, q, k, v, saved, t["gq"], t["gk"], N_txt)


@gpu
@pytest.mark.parametrize("index", [[-1, -1, -1, -1, -1, -1], [2, 2, 2, 2, 2, 2], [0, -1, 1, 1, 3, 0],
                                   [2 ** 31 - 1, -2 ** 31, 3, 4, 2, -7]])
def test_lora_index_values(ja, index):
    """Items without an adapter (any index outside 0 .. n - 1) give jattn_qkv_norm's bits; adapters may be
    shared, in runs or apart, and the work buffer's old contents (NaN here) reach nothing."""
    B, H, N_img, N_txt, d, C, rank, n = 6, 3, 50, 21, 64, 200, 24, 4
    t = lora_inputs(B, H, N_img, N_txt, d, C, rank, n, True, 31)
    t["index"] = torch.tensor(index, dtype=torch.int32, device="cuda")
    work = torch.full((ja.jattn_qkv_norm_lora_bytes(B, H, N_img, N_txt, d, rank),), 0xFF, dtype=torch.uint8,
                      device="cuda")
    q, k, v = (torch.full((B, H, N_img + N_txt, d), float("nan"), dtype=torch.bfloat16, device="cuda")
               for _ in range(3))
    saved = torch.empty(ja.jattn_saved_bytes(B, H, N_img, N_txt, d), dtype=torch.uint8, device="cuda")
    ja.jattn_qkv_norm_lora(t["x_img"], t["w_img"], t["b_img"], t["x_txt"], t["w_txt"], t["b_txt"], t["gq"], t["gk"],
                           t["down_img"], t["up_img"], t["down_txt"], t["up_txt"], t["scale"], t["index"], n, rank,
                           B, H, N_img, N_txt, d, C, q, k, v, saved, work)
    ok(ja)
    check_lora(ja, t, (q, k, v, saved), H, d, rank)
    plain = ja.qkv_norm(t["x_img"], t["w_img"], t["b_img"], t["x_txt"], t["w_txt"], t["b_txt"], t["gq"], t["gk"], H)
    for b, a in enumerate(index):
        if not 0 <= a < n:
            for x, y in zip((q, k, v), plain):
                assert torch.equal(x[b], y[b])


@gpu
@pytest.mark.parametrize("B,H,N_img,N_txt,d", [(150, 3, 3, 1, 64), (90, 2, 1, 2, 128), (70, 16, 9, 5, 64),
                                               (40, 9, 40, 0, 128)])
def test_lora_adapters_in_turn(ja, B, H, N_img, N_txt, d):
    """Many short items that share few adapters, in turn: a tile has each adapter's rows all over it."""
    t = lora_inputs(B, H, N_img, N_txt, d, 72, 24, 7, True, 34)
    t["index"][::5] = -1
    out = lora_call(ja, t, H)
    ok(ja)
    check_lora(ja, t, out, H, d, 24)


@gpu
@pytest.mark.parametrize("streams", [(), ("img",), ("txt",)])
def test_lora_streams_without_adapters(ja, streams):
    case = (3, 2, 140, 30, 64, 128, 32, 3, True)
    t = lora_inputs(*case, seed=41, streams=streams)
    out = lora_call(ja, t, 2)
    ok(ja)
    check_lora(ja, t, out, 2, 64, 32)
    if not streams:
        plain = ja.qkv_norm(t["x_img"], t["w_img"], t["b_img"], t["x_txt"], t["w_txt"], t["b_txt"], t["gq"], t["gk"],
                            2)
        for a, b in zip(out[:3], plain[:3]):
            assert torch.equal(a, b)


@gpu
def test_lora_adapters_beyond_32_bit_offsets(ja):
    """An adapter table of more than 2^32 bytes: the last adapter's rows are its own."""
    B, H, N_img, N_txt, d, C, rank, n = 2, 4, 130, 0, 128, 2048, 128, 11000
    t = lora_inputs(B, H, N_img, N_txt, d, C, rank, 2, False, 51, streams=("img",))
    down = torch.zeros((n, 3 * rank, C), dtype=torch.bfloat16, device="cuda")  # 17 GB
    up = torch.zeros((n, 3 * H * d, rank), dtype=torch.bfloat16, device="cuda")
    down[-2:], up[-2:] = t["down_img"], t["up_img"]
    big = dict(t, down_img=down, up_img=up, scale=torch.zeros(n, device="cuda"),
               index=torch.tensor([n - 1, n - 2], dtype=torch.int32, device="cuda"))
    big["scale"][-2:] = t["scale"]
    t["index"] = torch.tensor([1, 0], dtype=torch.int32, device="cuda")
    a, b = lora_call(ja, big, H), lora_call(ja, t, H)
    ok(ja)
    for x, y in zip(a[:3], b[:3]):
        assert torch.equal(x, y)
    check_lora(ja, t, b, H, d, rank)


@gpu
@pytest.mark.parametrize("sms", [1, 5])
def test_forms_under_a_cap_on_the_ctas(ja, sms):
    """Several tiles per CTA (both accumulators, the ring's stages across tiles and adapters) give the same bits."""
    t8 = fp8_inputs(2, 4, 300, 77, 64, 272, True, 61)
    tl = lora_inputs(3, 4, 150, 77, 64, 200, 40, 3, True, 62)
    want = fp8_call(ja, t8, 4)[:3] + lora_call(ja, tl, 4)[:3]
    ja.jattn_set_sm_limit(sms)
    try:
        got = fp8_call(ja, t8, 4)[:3] + lora_call(ja, tl, 4)[:3]
        ok(ja)
    finally:
        ja.jattn_set_sm_limit(0)
    for a, b in zip(got, want):
        assert torch.equal(a, b)


@gpu
@pytest.mark.parametrize("H,d", [(5, 64), (3, 128)])
@pytest.mark.parametrize("sms", [4, 6, 11, 18, 26, 151])
def test_parts_of_the_last_tiles(ja, H, d, sms):
    """However the last tiles are shared out (whole, by two heads or by one), the same bits: tiles over the
    borders between q, k and v (H no multiple of the heads of a tile) and adapters of several items included."""
    C = 72 if d == 64 else 80
    t8 = fp8_inputs(3, H, 500, 77, d, 80, True, 63)
    tl = lora_inputs(7, H, 220, 33, d, C, 24, 3, True, 64)
    tl["index"] = torch.tensor([2, 2, 0, -1, 1, 1, 0], dtype=torch.int32, device="cuda")
    want8, want = fp8_call(ja, t8, H), lora_call(ja, tl, H)
    check_lora(ja, tl, want, H, d, 24)
    ja.jattn_set_sm_limit(sms)
    try:
        got = fp8_call(ja, t8, H)[:3] + lora_call(ja, tl, H)[:3]
        ok(ja)
    finally:
        ja.jattn_set_sm_limit(0)
    for a, b in zip(got, want8[:3] + want[:3]):
        assert torch.equal(a, b)


@gpu
@pytest.mark.parametrize("N_img", [40, 1100])
def test_outputs_at_16_byte_boundaries(ja, N_img):
    """Outputs that start at a multiple of 16 bytes, not of 32, for few and for many tokens."""
    B, H, N_txt, d, C = 2, 4, 9, 64, 128
    t = lora_inputs(B, H, N_img, N_txt, d, C, 16, 2, True, 65)
    want = lora_call(ja, t, H)
    n = want[0].numel()
    buf = torch.full((3, n + 64), float("nan"), dtype=torch.bfloat16, device="cuda")
    q, k, v = (b[8:8 + n].view(want[0].shape) for b in buf)
    assert q.data_ptr() % 32 == 16
    saved = torch.empty_like(want[3])
    work = torch.empty(ja.jattn_qkv_norm_lora_bytes(B, H, N_img, N_txt, d, 16), dtype=torch.uint8, device="cuda")
    ja.jattn_qkv_norm_lora(t["x_img"], t["w_img"], t["b_img"], t["x_txt"], t["w_txt"], t["b_txt"], t["gq"], t["gk"],
                           t["down_img"], t["up_img"], t["down_txt"], t["up_txt"], t["scale"], t["index"], 2, 16,
                           B, H, N_img, N_txt, d, C, q, k, v, saved, work)
    ok(ja)
    for a, b in zip((q, k, v), want[:3]):
        assert torch.equal(a, b)
    for a, b in zip(saved_parts(saved, q), saved_parts(want[3], q)):
        assert torch.equal(a, b)
    assert buf[:, :8].isnan().all() and buf[:, 8 + n:].isnan().all()


@gpu
def test_run_from_the_residual_stream_to_the_gradients(ja):
    """A block's attention path as a program runs it: the residual's addition and norm, the projection
    (8-bit, and with adapters), the attention, its backward, and the norm's backward; eager, and captured
    with new inputs and another choice of adapters at the replay."""
    B, H, N_img, N_txt, d, C, rank, n = 3, 4, 150, 33, 64, 256, 16, 3
    g = gen(71)
    t = lora_inputs(B, H, N_img, N_txt, d, C, rank, n, True, 72)
    w8 = {s: ja.quant_rows(t["w_" + s]) for s in ("img", "txt")}
    gain = {s: torch.rand(C, generator=g, device="cuda") + 0.5 for s in ("img", "txt")}
    branch = {s: randn(g, *t["x_" + s].shape) for s in ("img", "txt")}
    stream = {s: randn(g, *t["x_" + s].shape, scale=2.0) for s in ("img", "txt")}
    dout = randn(g, B, H, N_img + N_txt, d)

    def step():
        y, h, r = {}, {}, {}
        y8 = {}
        for s in ("img", "txt"):
            y[s], h[s], r[s] = ja.add_norm(branch[s], gain[s], stream[s])
            y8[s] = ja.add_norm_fp8(branch[s], gain[s], stream[s])[:2]
        q8, k8, v8, saved8 = ja.qkv_norm_fp8(*y8["img"], *w8["img"], t["b_img"], *y8["txt"], *w8["txt"], t["b_txt"],
                                             t["gq"], t["gk"], H)
        out8, lse8 = torch.empty_like(q8), torch.empty(q8.shape[:-1], device="cuda")
        ja.jattn_fwd_saved(v8, B, H, N_img, N_txt, d, out8, lse8, saved8)
        q, k, v, saved = ja.qkv_norm_lora(y["img"], t["w_img"], t["b_img"], y["txt"], t["w_txt"], t["b_txt"],
                                          t["gq"], t["gk"], H, t["down_img"], t["up_img"], t["down_txt"],
                                          t["up_txt"], t["scale"], t["index"])
        out, lse = torch.empty_like(q), torch.empty(q.shape[:-1], device="cuda")
        ja.jattn_fwd_saved(v, B, H, N_img, N_txt, d, out, lse, saved)
        dq, dk, dv, _, _ = ja.backward_train(q, k, v, t["gq"], t["gk"], out, lse, dout, saved, N_txt)
        # the image stream's tokens' gradient through the shared weights (the adapters are for serving)
        rows = torch.stack([dq, dk, dv])[:, :, :, N_txt:]                       # [3, B, H, N_img, d]
        dy = rows.permute(1, 3, 0, 2, 4).reshape(B, N_img, -1) @ t["w_img"]
        dx, dg = ja.add_norm_backward(dy.contiguous(), h["img"], r["img"], gain["img"])
        return q8, k8, v8, out8, q, k, v, out, dx, dg

    ja.jattn_set_deterministic(True)
    try:
        got = step()
        ok(ja)
        q8, k8, v8, out8, q, k, v, out, dx, dg = got
        for qq, kk, vv, oo in ((q8, k8, v8, out8), (q, k, v, out)):
            npf = lambda a: a.float().cpu().numpy()  # noqa: E731
            ref, _ = oracle.joint_attention_fwd(npf(qq), npf(kk), npf(vv), npf(t["gq"]), npf(t["gk"]))
            off = npf(oo).astype(np.float64) - ref
            assert np.linalg.norm(off) <= 5e-3 * np.linalg.norm(ref)
        assert dx.isfinite().all() and dg.isfinite().all() and dg.abs().max() > 0
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            kept = step()
        for s in ("img", "txt"):
            branch[s].copy_(randn(g, *branch[s].shape))
        t["index"].copy_(torch.tensor([-1, 0, 2], dtype=torch.int32))
        for _ in range(2):
            graph.replay()
        ok(ja)
        want = step()
        ok(ja)
        for a, b in zip(kept, want):
            assert torch.equal(a, b)
        assert not torch.equal(kept[4], got[4])
    finally:
        ja.jattn_set_deterministic(False)


@gpu
def test_forms_on_another_stream(ja):
    t8, tl = fp8_inputs(2, 2, 140, 9, 64, 128, True, 81), lora_inputs(2, 2, 140, 9, 64, 128, 16, 2, True, 82)
    want = fp8_call(ja, t8, 2)[:3] + lora_call(ja, tl, 2)[:3]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = fp8_call(ja, t8, 2, side)[:3] + lora_call(ja, tl, 2, side.cuda_stream)[:3]
    side.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)


@gpu
def test_adapters_of_several_ranks_in_one_graph(ja):
    """A captured call keeps what its launch needs when calls of other ranks follow, in the graph and outside."""
    ts = [lora_inputs(2, 2, 140, 9, 64, 128, rank, 2, True, 85) for rank in (128, 16, 8)]
    want = [lora_call(ja, t, 2)[:3] for t in ts]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = [lora_call(ja, t, 2)[:3] for t in ts]
    lora_call(ja, ts[2], 2)
    for t in (x for out in got for x in out):
        t.fill_(float("nan"))
    graph.replay()
    ok(ja)
    for a, b in zip(got, want):
        assert all(torch.equal(x, y) for x, y in zip(a, b))


@gpu
def test_calls_at_once(ja):
    """Host threads with a stream each: adapters of different ranks, 8-bit rows, the token rows with their
    backward, and the attention; every call gives the bits that it gives alone."""
    tl = [lora_inputs(2, 4, 200, 30, 64, 128, rank, 2, True, 86) for rank in (128, 8)]
    t8 = fp8_inputs(2, 12, 1024, 77, 64, 768, True, 87)
    g = gen(88)
    q, k, v = (randn(g, 1, 4, 333, 64) for _ in range(3))
    x, res, dy = (randn(g, 700, 768) for _ in range(3))
    gain = torch.rand(768, generator=g, device="cuda") + 0.5

    def rows(stream):
        y, h, r = ja.add_norm(x, gain, res, stream=stream)
        return y, h, *ja.add_norm_backward(dy, h, r, gain, stream=stream)

    jobs = [lambda s, t=t: lora_call(ja, t, 4, s)[:3] for t in tl]
    jobs += [lambda s: fp8_call(ja, t8, 12, s)[:3], rows, lambda s: ja.forward(q, k, v, t8["gq"], t8["gk"], 33, s)[:1]]
    want = [job(None) for job in jobs]
    ok(ja)
    start = threading.Barrier(len(jobs))

    def run(job):
        side = torch.cuda.Stream()
        start.wait()
        outs = [job(side) for _ in range(30)]
        side.synchronize()
        return outs

    with ThreadPoolExecutor(len(jobs)) as pool:
        results = list(pool.map(run, jobs))
    ok(ja)
    for outs, one in zip(results, want):
        for out in outs:
            assert all(torch.equal(a, b) for a, b in zip(out, one))


@gpu
def test_on_the_default_stream_by_its_handle(ja):
    """Stream 0 is a stream as any other, with another one current."""
    t = lora_inputs(2, 2, 140, 9, 64, 128, 16, 2, True, 89)
    want = lora_call(ja, t, 2)[:3]
    torch.cuda.synchronize()
    with torch.cuda.stream(torch.cuda.Stream()):
        got = lora_call(ja, t, 2, 0)[:3]
        torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)


@gpu
def test_wrappers_name_what_is_unsupported(ja):
    code = STATUS_CODE["JATTN_ERR_UNSUPPORTED"]
    x, gain = randn(gen(90), 4, 12), torch.ones(12, device="cuda")
    r = torch.ones(4, device="cuda")
    t8 = fp8_inputs(1, 2, 8, 0, 32, 64, False, 91)
    tl = lora_inputs(1, 2, 8, 0, 64, 64, 12, 1, False, 92)
    for call in (lambda: ja.add_norm(x, gain), lambda: ja.add_norm_backward(x, x, r, gain),
                 lambda: fp8_call(ja, t8, 2), lambda: lora_call(ja, tl, 2)):
        with pytest.raises(ja.JattnError) as e:
            call()
        assert e.value.status == code


# Fake, never-dereferenced device addresses: validation happens first.
A = 0x7F0000000000


def at(i):
    return A + (i << 33)


def test_qkv_fp8_validation(lib):
    code = STATUS_CODE
    names = ("x_img", "sx_img", "w_img", "sw_img", "b_img", "x_txt", "sx_txt", "w_txt", "sw_txt", "b_txt", "gq", "gk")
    base = {n: at(i) for i, n in enumerate(names)}
    base.update(B=2, H=3, N_img=40, N_txt=8, d=64, C=96, q=at(20), k=at(21), v=at(22), saved=at(23))
    f = lambda **kw: lib.jattn_qkv_norm_fp8(*{**base, **kw}.values(), None)  # noqa: E731
    for n in ("x_img", "sx_img", "w_img", "sw_img", "x_txt", "sx_txt", "w_txt", "sw_txt", "gq", "gk", "q", "k", "v",
              "saved"):
        assert f(**{n: None}) == code["JATTN_ERR_INVALID_ARG"], n
        assert f(**{n: base[n] + 8}) == code["JATTN_ERR_MISALIGNED"], n
    assert f(C=0) == f(B=0) == f(C=1 << 24, H=64) == code["JATTN_ERR_INVALID_ARG"]
    assert f(C=104) == f(d=32) == code["JATTN_ERR_UNSUPPORTED"]
    assert f(q=at(21)) == f(k=at(0)) == f(v=at(1)) == f(saved=at(3)) == f(q=at(8)) == code["JATTN_ERR_ALIAS"]
    # a stream without rows needs nothing (the call still fails, on d)
    assert f(N_txt=0, x_txt=None, sx_txt=None, w_txt=None, sw_txt=None, d=32) == code["JATTN_ERR_UNSUPPORTED"]


def test_qkv_lora_validation(lib):
    code = STATUS_CODE
    names = ("x_img", "w_img", "b_img", "x_txt", "w_txt", "b_txt", "gq", "gk", "down_img", "up_img", "down_txt",
             "up_txt", "scale", "index")
    base = {n: at(i) for i, n in enumerate(names)}
    base.update(n_adapters=3, rank=16, B=2, H=3, N_img=40, N_txt=8, d=64, C=96, q=at(20), k=at(21), v=at(22),
                saved=at(23), work=at(24))
    f = lambda **kw: lib.jattn_qkv_norm_lora(*{**base, **kw}.values(), None)  # noqa: E731
    for n in ("x_img", "w_img", "x_txt", "w_txt", "gq", "gk", "down_img", "up_img", "down_txt", "up_txt", "scale",
              "index", "q", "k", "v", "saved", "work"):
        assert f(**{n: None}) == code["JATTN_ERR_INVALID_ARG"], n
        assert f(**{n: base[n] + 8}) == code["JATTN_ERR_MISALIGNED"], n
    for kw in (dict(n_adapters=0), dict(n_adapters=-1), dict(rank=0), dict(rank=-8), dict(C=0), dict(H=0),
               dict(n_adapters=1 << 30)):
        assert f(**kw) == code["JATTN_ERR_INVALID_ARG"], kw
    for kw in (dict(rank=12), dict(rank=136), dict(C=100), dict(d=96)):
        assert f(**kw) == code["JATTN_ERR_UNSUPPORTED"], kw
    for kw in (dict(work=at(0)), dict(work=at(20)), dict(q=at(8)), dict(k=at(11)), dict(v=at(12)),
               dict(saved=at(13)), dict(work=at(13))):
        assert f(**kw) == code["JATTN_ERR_ALIAS"], kw
    bytes_of = lib.jattn_qkv_norm_lora_bytes
    assert bytes_of(2, 3, 40, 8, 64, 16) >= 2 * 48 * 3 * 16 * 2
    assert bytes_of(2, 3, 40, 8, 64, 12) == bytes_of(2, 3, 40, 8, 96, 16) == bytes_of(0, 3, 40, 8, 64, 16) == 0
