"""The QKV projections at the limits of their inputs and outputs: what the adapters' first product keeps, and
rows past the fp32 range.

Tolerances count the roundings that test_gpu_qkv_forms counts: each addition of a product off by at most
2^-23 of the terms' summed magnitudes, bf16 by half a step (2^-8).
"""
import pytest
import torch

import joint_attention_gb300 as pkg
from joint_attention_gb300.build import build
from test_gpu_qkv_forms import check_norms, fp8_call, fp8_inputs, lora_call, lora_inputs, ok, saved_parts

gpu = pytest.mark.gpu


@pytest.fixture(scope="module")
def ja():
    build()
    pkg.load_library()
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    return pkg


@gpu
@pytest.mark.parametrize("rank", [8, 16, 40, 128])
@pytest.mark.parametrize("H,N,d", [(2, 40, 64), (6, 1100, 64), (6, 1100, 128)])
def test_lora_first_product_is_kept_in_32_bits(ja, rank, H, N, d):
    """Y = U B^T + b with each column of B one of U's columns and b the opposite of U rounded to fp32: what is
    left is U's own error, of (C + 4) roundings of its terms' magnitudes, each at most 2^-23 (the sum, the scale, and the
    term's and the bias's addition); U kept to 2^-16 would leave up to 2^-17 of U.  All tokens of an item are alike."""
    B, C = 1, 16
    t = lora_inputs(B, H, N, 0, d, C, rank, 1, True, 303, streams=("img",))
    t["x_img"][:] = t["x_img"][:, :1].abs()
    t["down_img"].abs_()
    t["w_img"].zero_()
    u = torch.einsum("c,pjc->pj", t["x_img"][0, 0].double(), t["down_img"].double().view(3, rank, C))
    u = u * t["scale"].double()
    col = torch.arange(H * d, device="cuda") % rank
    t["up_img"].zero_()
    t["up_img"].view(3, H * d, rank)[:, torch.arange(H * d, device="cuda"), col] = 1.0
    want = u[:, col]
    t["b_img"] = -want.float().reshape(-1)
    q, k, v, _ = lora_call(ja, t, H)
    ok(ja)
    for y, w in zip((q, k, v), want.view(3, H, d)):
        off = y[0].double() - (w - w.float().double())[:, None]  # y is rounded to bf16: at most 2^-8 of itself
        assert (off.abs() <= ((C + 4) * 2.0 ** -23 * w + 2.0 ** -23 * w)[:, None] * (1 + 2.0 ** -8)).all()


@gpu
@pytest.mark.parametrize("form", ["bf16", "fp8", "lora"])
@pytest.mark.parametrize("H,N_img,d", [(2, 40, 64), (2, 40, 128), (6, 1100, 64), (6, 1100, 128)])
def test_rows_whose_squares_pass_fp32(ja, form, H, N_img, d):
    """A q or k row whose sum of squares passes the fp32 range has 1/rms 0: its q_hat and k_hat are zeros, and
    those of a row of infinities are NaN, as a training forward keeps them; other rows are as they were."""
    B, N_txt, C = 2, 9, 64
    if form == "fp8":
        t = fp8_inputs(B, H, N_img, N_txt, d, C, True, 301)
        t["sx_img"][0, 4], t["sx_img"][1, 7], t["sx_txt"][1, 3] = 1e20, float("inf"), 3e21
        q, k, v, saved = fp8_call(ja, t, H)
    else:
        t = lora_inputs(B, H, N_img, N_txt, d, C, 16, 2, True, 302)
        t["x_img"][0, 4] *= 1e20
        t["x_img"][1, 7, 0] = float("inf")  # +-inf in every column
        t["index"][1] = -1                  # (an adapter would add them to others of either sign)
        t["x_txt"][1, 3] *= 3e21
        if form == "lora":
            q, k, v, saved = lora_call(ja, t, H)
        else:
            q, k, v, saved = ja.qkv_norm(t["x_img"], t["w_img"], t["b_img"], t["x_txt"], t["w_txt"], t["b_txt"],
                                         t["gq"], t["gk"], H)
    ok(ja)
    check_norms(ja, q, k, v, saved, t["gq"], t["gk"], N_txt)
    for hat, r in zip(*(saved_parts(saved, q)[i:i + 2] for i in (0, 2))):
        for b, n in ((0, N_txt + 4), (1, 3)):
            assert not hat[b, :, n].any() and not r[b, :, n].any()
        assert hat[1, :, N_txt + 7].isnan().all()
        assert hat.isnan().sum() == H * d


@gpu
@pytest.mark.parametrize("rank", [16, 24])
@pytest.mark.parametrize("H,N", [(2, 40), (6, 1100)])
def test_lora_with_infinities_and_the_largest_values(ja, rank, H, N):
    """A token with an infinite value and positive weights is infinite, and not NaN, whatever the rank (one that is no
    multiple of 16 included); a U near the end of the fp32 range, above the largest bf16, counts as it is."""
    B, C, d = 2, 72, 64
    t = lora_inputs(B, H, N, 0, d, C, rank, 2, True, 304, streams=("img",))
    for name in ("x_img", "w_img", "down_img", "up_img"):
        t[name].abs_().clamp_min_(2.0 ** -6)
    t["x_img"][0, 5, 1] = float("inf")
    q, k, v, _ = lora_call(ja, t, H)
    ok(ja)
    for y in (q, k, v):
        assert (y[0, :, 5] == float("inf")).all()
        assert y.isfinite().sum() == y.numel() - H * d
    big = torch.finfo(torch.bfloat16).max  # 255 * 2^120
    t["w_img"].zero_(), t["b_img"].zero_(), t["up_img"].zero_(), t["down_img"].zero_(), t["x_img"].zero_()
    t["scale"][:] = 1.0
    t["x_img"][1, 7, :2] = torch.tensor([1.0, 2.0 ** 119], device="cuda")
    t["down_img"][:, :, :2] = torch.tensor([big, 1.5], device="cuda")  # U = 255.75 * 2^120
    t["up_img"][:, :, 3] = 2.0 ** -20
    q, k, v, _ = lora_call(ja, t, H)
    ok(ja)
    want = torch.tensor(255.75 * 2.0 ** 100, dtype=torch.float64).to(torch.bfloat16).item()
    for y in (q, k, v):
        assert (y[1, :, 7] == want).all()
        assert (y != 0).sum() == H * d


def misaligned(ja, form, t, B, H, N_img, N_txt, d, C, rank, n):
    """A call whose q, k, v and `saved` start at 16 mod 32 bytes, as a function of nothing, and its outputs."""
    N = N_img + N_txt
    e = B * H * N * d
    bufs = [torch.full((e + 64,), float("nan"), dtype=torch.bfloat16, device="cuda") for _ in range(3)]
    q, k, v = (b[8:8 + e].view(B, H, N, d) for b in bufs)
    keep = torch.zeros(ja.jattn_saved_bytes(B, H, N_img, N_txt, d) + 16, dtype=torch.uint8, device="cuda")
    saved = keep[16:]
    assert q.data_ptr() % 32 == saved.data_ptr() % 32 == 16
    sizes = (B, H, N_img, N_txt, d, C)
    if form == "fp8":
        call = lambda: ja.jattn_qkv_norm_fp8(  # noqa: E731
            t["x_img"], t["sx_img"], t["w_img"], t["sw_img"], t["b_img"], t["x_txt"], t["sx_txt"], t["w_txt"],
            t["sw_txt"], t["b_txt"], t["gq"], t["gk"], *sizes, q, k, v, saved)
    elif form == "lora":
        work = torch.empty(ja.jattn_qkv_norm_lora_bytes(*sizes[:5], rank), dtype=torch.uint8, device="cuda")
        call = lambda: ja.jattn_qkv_norm_lora(  # noqa: E731
            t["x_img"], t["w_img"], t["b_img"], t["x_txt"], t["w_txt"], t["b_txt"], t["gq"], t["gk"], t["down_img"],
            t["up_img"], t["down_txt"], t["up_txt"], t["scale"], t["index"], n, rank, *sizes, q, k, v, saved, work)
    else:
        call = lambda: ja.jattn_qkv_norm(  # noqa: E731
            t["x_img"], t["w_img"], t["b_img"], t["x_txt"], t["w_txt"], t["b_txt"], t["gq"], t["gk"], *sizes, q, k, v,
            saved)
    return call, (q, k, v, saved), bufs


def aligned_call(ja, form, t, H):
    if form == "fp8":
        return fp8_call(ja, t, H)
    if form == "lora":
        return lora_call(ja, t, H)
    return ja.qkv_norm(t["x_img"], t["w_img"], t["b_img"], t["x_txt"], t["w_txt"], t["b_txt"], t["gq"], t["gk"], H)


def form_inputs(form, B, H, N_img, N_txt, d, C, rank, n, seed):
    return (fp8_inputs(B, H, N_img, N_txt, d, C, True, seed) if form == "fp8"
            else lora_inputs(B, H, N_img, N_txt, d, C, rank, n, True, seed))


@gpu
@pytest.mark.parametrize("form", ["bf16", "fp8", "lora"])
@pytest.mark.parametrize("N_img,d", [(40, 64), (40, 128), (1100, 64), (1100, 128)])
def test_every_form_at_16_byte_boundaries(ja, form, N_img, d):
    """The bits of outputs at 32-byte boundaries, and nothing written beside them."""
    B, H, N_txt, C, rank, n = 3, 5, 9, 128, 24, 2
    t = form_inputs(form, B, H, N_img, N_txt, d, C, rank, n, 311)
    want = aligned_call(ja, form, t, H)
    call, got, bufs = misaligned(ja, form, t, B, H, N_img, N_txt, d, C, rank, n)
    call()
    ok(ja)
    for a, b in zip(got[:3], want[:3]):
        assert torch.equal(a, b)
    for a, b in zip(saved_parts(got[3], got[0]), saved_parts(want[3], want[0])):
        assert torch.equal(a, b)
    for b in bufs:
        assert b[:8].isnan().all() and b[8 + got[0].numel():].isnan().all()


@gpu
@pytest.mark.parametrize("form", ["bf16", "fp8", "lora"])
@pytest.mark.parametrize("B,H,N_img,d,C", [(16, 12, 1024, 64, 768), (4, 16, 2304, 128, 1024)])
def test_outputs_at_16_byte_boundaries_are_not_slow(ja, form, B, H, N_img, d, C):
    """Such a call takes the tiles of the others: at these sizes 1.03 to 1.25 times their time, where tiles of one head by
    single CTAs took 1.57 to 2.5 times.  The border is between the two, (1.25 1.57)^(1/2) = 1.4.  The best of several
    runs of each, taken in turn."""
    N_txt, rank, n = 77, 16, 4
    t = form_inputs(form, B, H, N_img, N_txt, d, C, rank, n, 312)
    odd = misaligned(ja, form, t, B, H, N_img, N_txt, d, C, rank, n)[0]

    def graph_of(call):
        g = torch.cuda.CUDAGraph()
        call()
        torch.cuda.synchronize()
        with torch.cuda.graph(g):
            for _ in range(8):
                call()
        return g

    graphs = [graph_of(odd), graph_of(lambda: aligned_call(ja, form, t, H))]
    best = [float("inf")] * 2
    for _ in range(8):
        for i, g in enumerate(graphs):
            a, b = torch.cuda.Event(True), torch.cuda.Event(True)
            g.replay()
            a.record()
            g.replay()
            b.record()
            torch.cuda.synchronize()
            best[i] = min(best[i], a.elapsed_time(b))
    assert best[0] < 1.4 * best[1], best
