"""GB300-native MM-DiT joint attention with QK-RMSNorm (forward and backward).

The compute path is libjattn.so (hand-written sm_103a CUDA kernels behind a C
ABI, declared in include/jattn.h); this package is its thin ctypes binding
plus small conveniences that allocate the output tensors with torch.
"""
from __future__ import annotations

import contextlib

from ._binding import (KERNEL_KINDS, STATUS, STATUS_CODE, JattnError, declared_symbols, jattn_bwd, jattn_fwd,
                       jattn_fwd_noalloc, jattn_fwd_varlen, jattn_bwd_varlen, jattn_selftest_wait_timeout, jattn_set_sm_limit,
                       jattn_set_deterministic, jattn_kernel_name, jattn_last_device_error, jattn_last_error_message, jattn_profile_enable, jattn_profile_read,
                       jattn_profile_reset, jattn_status_string, jattn_version, load_library, profile_snapshot,
                       jattn_saved_bytes, jattn_saved_bytes_varlen, jattn_fwd_train, jattn_bwd_train,
                       jattn_fwd_train_varlen, jattn_bwd_train_varlen, jattn_qkv_norm, jattn_fwd_saved,
                       TOKEN_KERNEL_KINDS, jattn_add_norm, jattn_add_norm_fp8, jattn_quant_rows,
                       jattn_add_norm_bwd_bytes, jattn_add_norm_bwd, jattn_qkv_norm_fp8, jattn_qkv_norm_lora,
                       jattn_qkv_norm_lora_bytes)

__all__ = ["STATUS", "STATUS_CODE", "JattnError", "declared_symbols", "jattn_bwd", "jattn_fwd",
           "jattn_last_device_error", "jattn_status_string", "jattn_version", "load_library", "forward",
           "backward", "KERNEL_KINDS", "jattn_kernel_name", "jattn_profile_enable", "jattn_profile_read",
           "jattn_profile_reset", "profile_snapshot", "jattn_last_error_message", "jattn_fwd_noalloc",
           "jattn_fwd_varlen", "jattn_bwd_varlen", "forward_varlen", "backward_varlen",
           "jattn_selftest_wait_timeout", "jattn_set_sm_limit", "jattn_set_deterministic", "jattn_saved_bytes",
           "jattn_saved_bytes_varlen", "jattn_fwd_train", "jattn_bwd_train", "jattn_fwd_train_varlen",
           "jattn_bwd_train_varlen", "forward_train", "backward_train", "jattn_qkv_norm", "jattn_fwd_saved",
           "qkv_norm", "TOKEN_KERNEL_KINDS", "jattn_add_norm", "jattn_add_norm_fp8", "jattn_quant_rows",
           "jattn_add_norm_bwd_bytes", "jattn_add_norm_bwd", "add_norm", "add_norm_fp8", "add_norm_backward",
           "quant_rows", "jattn_qkv_norm_fp8", "jattn_qkv_norm_lora", "jattn_qkv_norm_lora_bytes", "qkv_norm_fp8",
           "qkv_norm_lora"]


def forward(q, k, v, gq, gk, n_txt: int, stream=None):
    """out, lse = joint attention of [B, H, N, d] bf16 CUDA tensors (text rows first)."""
    import torch

    B, H, N, d = q.shape
    out = torch.empty_like(q)
    lse = torch.empty((B, H, N), dtype=torch.float32, device=q.device)
    jattn_fwd(q, k, v, gq, gk, B, H, N - n_txt, n_txt, d, out, lse, stream)
    return out, lse


def backward(q, k, v, gq, gk, out, lse, dout, n_txt: int, stream=None):
    """dq, dk, dv, dgq, dgk for the upstream gradient dout."""
    import torch

    B, H, N, d = q.shape
    dq, dk, dv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
    dgq = torch.empty_like(gq)
    dgk = torch.empty_like(gk)
    jattn_bwd(q, k, v, gq, gk, out, lse, dout, dq, dk, dv, dgq, dgk, B, H, N - n_txt, n_txt, d, stream)
    return dq, dk, dv, dgq, dgk


def forward_varlen(q, k, v, gq, gk, cu_seqlens, stream=None):
    """out, lse for packed sequences: q, k, v [H, T, d] bf16 CUDA tensors, sequence s in rows
    cu_seqlens[s] .. cu_seqlens[s+1]-1 of every head (cu_seqlens: host ints)."""
    import torch

    H, T, d = q.shape
    out = torch.empty_like(q)
    lse = torch.empty((H, T), dtype=torch.float32, device=q.device)
    jattn_fwd_varlen(q, k, v, gq, gk, cu_seqlens, H, d, out, lse, stream)
    return out, lse


def backward_varlen(q, k, v, gq, gk, out, lse, dout, cu_seqlens, stream=None):
    """dq, dk, dv, dgq, dgk for packed sequences (layouts as forward_varlen)."""
    import torch

    H, T, d = q.shape
    dq, dk, dv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
    dgq = torch.empty_like(gq)
    dgk = torch.empty_like(gk)
    jattn_bwd_varlen(q, k, v, gq, gk, out, lse, dout, dq, dk, dv, dgq, dgk, cu_seqlens, H, d, stream)
    return dq, dk, dv, dgq, dgk


def forward_train(q, k, v, gq, gk, n_txt: int, stream=None):
    """out, lse, saved: a training forward of [B, H, N, d] bf16 CUDA tensors that keeps the
    normalised q / k in `saved` (a uint8 CUDA tensor) for backward_train."""
    import torch

    B, H, N, d = q.shape
    out = torch.empty_like(q)
    lse = torch.empty((B, H, N), dtype=torch.float32, device=q.device)
    saved = torch.empty(jattn_saved_bytes(B, H, N - n_txt, n_txt, d), dtype=torch.uint8, device=q.device)
    jattn_fwd_train(q, k, v, gq, gk, B, H, N - n_txt, n_txt, d, out, lse, saved, stream)
    return out, lse, saved


def backward_train(q, k, v, gq, gk, out, lse, dout, saved, n_txt: int, stream=None):
    """dq, dk, dv, dgq, dgk from forward_train's outputs and `saved`."""
    import torch

    B, H, N, d = q.shape
    dq, dk, dv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
    dgq = torch.empty_like(gq)
    dgk = torch.empty_like(gk)
    jattn_bwd_train(q, k, v, gq, gk, out, lse, dout, saved, dq, dk, dv, dgq, dgk, B, H, N - n_txt, n_txt, d, stream)
    return dq, dk, dv, dgq, dgk


def qkv_norm(x_img, w_img, b_img, x_txt, w_txt, b_txt, gq, gk, H: int, stream=None):
    """q, k, v, saved: the QKV projections of the image tokens x_img [B, N_img, C] and the caption
    tokens x_txt [B, N_txt, C] (bf16 CUDA tensors; weights [3 H d, C] bf16, biases [3 H d] fp32 or
    None) into the joint [B, H, N, d] layout, with q_hat, k_hat and 1/rms in `saved` for
    jattn_fwd_saved / backward_train."""
    import torch

    B, N_img, C = x_img.shape
    N_txt = x_txt.shape[1]
    d = gq.shape[0]
    N = N_img + N_txt
    dev = x_img.device
    q = torch.empty((B, H, N, d), dtype=torch.bfloat16, device=dev)
    k, v = torch.empty_like(q), torch.empty_like(q)
    saved = torch.empty(jattn_saved_bytes(B, H, N_img, N_txt, d), dtype=torch.uint8, device=dev)
    jattn_qkv_norm(x_img, w_img, b_img, x_txt, w_txt, b_txt, gq, gk, B, H, N_img, N_txt, d, C, q, k, v, saved,
                   stream)
    return q, k, v, saved


_no_context = contextlib.nullcontext()


def _outputs_on(stream, *tensors):
    """Context in which a call's outputs are allocated: the launching stream's, so that the allocator
    orders their reuse by it.  The call runs on the current device, where its tensors must be."""
    import torch

    dev = torch.cuda.current_device()
    for t in tensors:
        if t is not None and t.get_device() != dev:
            raise ValueError(f"a tensor is on {t.device}, the current device is cuda:{dev}")
    if stream is None:
        return _no_context
    return torch.cuda.stream(torch.cuda.ExternalStream(stream) if isinstance(stream, int) else stream)


def _buffer(nbytes, device):
    """A buffer of the size that the library asks for; 0 is for sizes that the call then refuses, which
    says why only if it gets a pointer."""
    import torch

    return torch.empty(nbytes or 16, dtype=torch.uint8, device=device)


# The functions below hand the raw pointers of the outputs that they have just allocated to the
# binding: only a caller's tensors need its checks.


def add_norm(x, g, residual=None, eps: float = 1e-6, stream=None):
    """y, h, r: RMSNorm of the token rows h = x + residual (h is x without a residual) over their
    last axis with gain g [C] fp32.  x, residual, h, y [..., C] bf16; r [...] fp32, the rows' 1/rms
    for add_norm_backward."""
    import torch

    with _outputs_on(stream, x, g, residual):
        y = torch.empty_like(x)
        h = x if residual is None else torch.empty_like(x)
        r = torch.empty(x.shape[:-1], dtype=torch.float32, device=x.device)
    jattn_add_norm(x, residual, g, r.numel(), g.numel(), eps, None if residual is None else h.data_ptr(),
                   y.data_ptr(), r.data_ptr(), stream)
    return y, h, r


def add_norm_fp8(x, g, residual=None, eps: float = 1e-6, stream=None):
    """y8, scale, h, r: add_norm with 8-bit rows: y8 [..., C] float8_e4m3fn and scale [...] fp32, a row
    standing for scale * y8 (what qkv_norm_fp8 reads)."""
    import torch

    with _outputs_on(stream, x, g, residual):
        y8 = torch.empty_like(x, dtype=torch.float8_e4m3fn)
        h = x if residual is None else torch.empty_like(x)
        r = torch.empty(x.shape[:-1], dtype=torch.float32, device=x.device)
        scale = torch.empty_like(r)
    jattn_add_norm_fp8(x, residual, g, r.numel(), g.numel(), eps, None if residual is None else h.data_ptr(),
                       y8.data_ptr(), scale.data_ptr(), r.data_ptr(), stream)
    return y8, scale, h, r


def add_norm_backward(dy, h, r, g, dh=None, stream=None):
    """dx, dg from add_norm's h and r: dx is the gradient of x and of the residual alike; dh is the
    gradient of h from later uses of it (None: none)."""
    import torch

    T, C = r.numel(), g.numel()
    with _outputs_on(stream, dy, h, r, g, dh):
        dx, dg = torch.empty_like(dy), torch.empty_like(g)
        work = _buffer(jattn_add_norm_bwd_bytes(T, C), dy.device)
    jattn_add_norm_bwd(dy, dh, h, r, g, T, C, dx.data_ptr(), dg.data_ptr(), work.data_ptr(), stream)
    return dx, dg


def quant_rows(x, stream=None):
    """x8, scale: rows of the last axis in 8 bits (float8_e4m3fn), a row standing for scale * x8."""
    import torch

    with _outputs_on(stream, x):
        x8 = torch.empty_like(x, dtype=torch.float8_e4m3fn)
        scale = torch.empty(x.shape[:-1], dtype=torch.float32, device=x.device)
    jattn_quant_rows(x, scale.numel(), x.shape[-1], x8.data_ptr(), scale.data_ptr(), stream)
    return x8, scale


def _projected(x_img, x_txt, H: int, d: int):
    """q, k, v and `saved` of a projection call, and its sizes."""
    import torch

    B, N_img, C = x_img.shape
    N_txt = x_txt.shape[1]
    dev = x_img.device
    shape = (B, H, N_img + N_txt, d)
    q = torch.empty(shape, dtype=torch.bfloat16, device=dev)
    k, v = torch.empty_like(q), torch.empty_like(q)
    saved = _buffer(jattn_saved_bytes(B, H, N_img, N_txt, d), dev)
    return (q, k, v, saved), (B, H, N_img, N_txt, d, C)


def qkv_norm_fp8(x_img, sx_img, w_img, sw_img, b_img, x_txt, sx_txt, w_txt, sw_txt, b_txt, gq, gk, H: int,
                 stream=None):
    """q, k, v, saved: qkv_norm from 8-bit tokens and weights (float8_e4m3fn) with the fp32 scales of their
    rows, as add_norm_fp8 and quant_rows give them: x_* [B, N_*, C], sx_* [B, N_*], w_* [3 H d, C],
    sw_* [3 H d]."""
    with _outputs_on(stream, x_img, sx_img, w_img, sw_img, b_img, x_txt, sx_txt, w_txt, sw_txt, b_txt, gq, gk):
        out, sizes = _projected(x_img, x_txt, H, gq.shape[0])
    jattn_qkv_norm_fp8(x_img, sx_img, w_img, sw_img, b_img, x_txt, sx_txt, w_txt, sw_txt, b_txt, gq, gk, *sizes,
                       *(t.data_ptr() for t in out), stream)
    return out


def qkv_norm_lora(x_img, w_img, b_img, x_txt, w_txt, b_txt, gq, gk, H: int, down_img, up_img, down_txt, up_txt,
                  scale, index, stream=None):
    """q, k, v, saved: qkv_norm with low-rank adapters of the batch items' own: item b adds
    scale[a] (x A_a^T) B_a^T, a = index[b] (int32 on the device; outside 0 .. n - 1: none), with A in
    down_* [n, 3 rank, C] and B in up_* [n, 3 H d, rank], q, k and v each with a rank of their own
    (both None: no adapters in that stream)."""
    rank = next((u.shape[-1] for u in (up_img, up_txt) if u is not None), 8)
    with _outputs_on(stream, x_img, w_img, b_img, x_txt, w_txt, b_txt, gq, gk, down_img, up_img, down_txt, up_txt,
                     scale, index):
        out, sizes = _projected(x_img, x_txt, H, gq.shape[0])
        work = _buffer(jattn_qkv_norm_lora_bytes(*sizes[:5], rank), x_img.device)
    jattn_qkv_norm_lora(x_img, w_img, b_img, x_txt, w_txt, b_txt, gq, gk, down_img, up_img, down_txt, up_txt, scale,
                        index, scale.numel(), rank, *sizes, *(t.data_ptr() for t in out), work.data_ptr(), stream)
    return out
