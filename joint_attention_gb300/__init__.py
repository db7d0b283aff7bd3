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
                       jattn_qkv_norm_lora_bytes, jattn_layer_norm, jattn_layer_norm_bwd_bytes, jattn_layer_norm_bwd,
                       jattn_rope, jattn_rope_bwd_bytes, jattn_rope_bwd, jattn_fwd_grouped, jattn_bwd_grouped_bytes,
                       jattn_bwd_grouped)

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
           "qkv_norm_lora", "jattn_layer_norm", "jattn_layer_norm_bwd_bytes", "jattn_layer_norm_bwd", "layer_norm",
           "layer_norm_backward", "jattn_rope", "jattn_rope_bwd_bytes", "jattn_rope_bwd", "rope", "rope_backward",
           "jattn_fwd_grouped", "jattn_bwd_grouped_bytes", "jattn_bwd_grouped", "forward_grouped", "backward_grouped"]


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


def layer_norm(x, g, b=None, residual=None, eps: float = 1e-6, stream=None):
    """y, h, mean, r: LayerNorm of the token rows h = x + residual (h is x without a residual) over their
    last axis.  x, residual, h, y [..., C] bf16; gain g and bias b (or None) fp32, [C], or [items, C] for
    batch items of equally many rows each with their own; mean, r [...] fp32 for layer_norm_backward."""
    import torch

    with _outputs_on(stream, x, g, b, residual):
        y = torch.empty_like(x)
        h = x if residual is None else torch.empty_like(x)
        mean = torch.empty(x.shape[:-1], dtype=torch.float32, device=x.device)
        r = torch.empty_like(mean)
    C = g.shape[-1]
    jattn_layer_norm(x, residual, g, b, g.numel() // C, r.numel(), C, eps, None if residual is None else h.data_ptr(),
                     y.data_ptr(), mean.data_ptr(), r.data_ptr(), stream)
    return y, h, mean, r


def layer_norm_backward(dy, h, mean, r, g, dh=None, bias: bool = True, stream=None):
    """dx, dg, db from layer_norm's h, mean and r: dx is the gradient of x and of the residual alike, dg and
    db (None without bias) have g's shape; dh is the gradient of h from later uses of it (None: none)."""
    import torch

    T, C = r.numel(), g.shape[-1]
    items = g.numel() // C
    with _outputs_on(stream, dy, h, mean, r, g, dh):
        dx, dg = torch.empty_like(dy), torch.empty_like(g)
        db = torch.empty_like(g) if bias else None
        work = _buffer(jattn_layer_norm_bwd_bytes(items, T, C), dy.device)
    jattn_layer_norm_bwd(dy, dh, h, mean, r, g, items, T, C, dx.data_ptr(), dg.data_ptr(),
                         db.data_ptr() if bias else None, work.data_ptr(), stream)
    return dx, dg, db


def _rope_sizes(q, k, pos):
    """Whether the positions are each item's own, and B, Hq, Hk, N, d of [B, H, N, d] or packed [H, T, d] tensors."""
    qs, ks = q.shape, k.shape
    if len(qs) == 3 == len(ks):
        qs, ks = (1, *qs), (1, *ks)
    if len(qs) != 4 or len(ks) != 4 or (ks[0], ks[2], ks[3]) != (qs[0], qs[2], qs[3]):
        raise ValueError(f"q and k: expected [B, H, N, d] or [H, T, d] with heads of their own, got {tuple(q.shape)} "
                         f"and {tuple(k.shape)}")
    B, Hq, N, d = qs
    return pos.dim() == 3, B, Hq, ks[1], N, d


def rope(q, k, pos, freq, pairs, gq=None, gk=None, interleaved: bool = False, eps: float = 1e-6, stream=None):
    """q_rot, k_rot: rotary positions of q [B, Hq, N, d] and k [B, Hk, N, d] (or packed [H, T, d]) bf16, after
    the QK-RMSNorm with gains gq, gk [d] fp32 if they are given.  pos [N, axes], or [B, N, axes] for
    positions of each item's own, and freq [P] fp32 (radians per unit); pairs: host ints, how many of the
    P channel pairs each axis has.  Pair p is channels (2 p, 2 p + 1) if interleaved, else (p, p + P)."""
    import torch

    with _outputs_on(stream, q, k, pos, freq, gq, gk):
        q_rot, k_rot = torch.empty_like(q), torch.empty_like(k)
    per_item, B, Hq, Hk, N, d = _rope_sizes(q, k, pos)
    jattn_rope(q, k, gq, gk, pos, freq, pairs, per_item, interleaved, B, Hq, Hk, N, d, eps, q_rot.data_ptr(),
               k_rot.data_ptr(), stream)
    return q_rot, k_rot


def rope_backward(dq_rot, dk_rot, pos, freq, pairs, q=None, k=None, gq=None, gk=None, interleaved: bool = False,
                  eps: float = 1e-6, stream=None):
    """dq, dk, dgq, dgk from the gradients of rope's outputs; q, k, gq, gk as rope got them with gains, and
    None without (dgq and dgk are None then)."""
    import torch

    per_item, *sizes = _rope_sizes(dq_rot, dk_rot, pos)
    norm = gq is not None
    with _outputs_on(stream, dq_rot, dk_rot, pos, freq, q, k, gq, gk):
        dq, dk = torch.empty_like(dq_rot), torch.empty_like(dk_rot)
        dgq, dgk = (torch.empty_like(gq), torch.empty_like(gk)) if norm else (None, None)
        work = _buffer(jattn_rope_bwd_bytes(per_item, *sizes), dq_rot.device) if norm else None
    jattn_rope_bwd(dq_rot, dk_rot, q if norm else None, k if norm else None, gq, gk, pos, freq, pairs, per_item,
                   interleaved, *sizes, eps, dq.data_ptr(), dk.data_ptr(), dgq.data_ptr() if norm else None,
                   dgk.data_ptr() if norm else None, work, stream)
    return dq, dk, dgq, dgk


def _grouped_sizes(q, k, scale):
    """Hq, Hk, T, d of q [Hq, T, d] and k, and the scale (None: 1 / sqrt(d))."""
    qs, ks = q.shape, k.shape
    if len(qs) != 3 or len(ks) != 3 or qs[1] != ks[1] or qs[2] != ks[2]:
        raise ValueError(f"q and k: expected [Hq, T, d] and [Hk, T, d], got {tuple(qs)} and {tuple(ks)}")
    Hq, T, d = qs
    return (Hq, ks[0], T, d), d ** -0.5 if scale is None else scale


def forward_grouped(q, k, v, cu_seqlens, causal: bool = True, scale: float | None = None, stream=None):
    """out, lse: attention of packed sequences with grouped heads, causal or full, on q [Hq, T, d] and k, v
    [Hk, T, d] bf16 as they are (no norm); query head h reads kv head h // (Hq // Hk).  Sequence s is rows
    cu_seqlens[s] .. cu_seqlens[s+1]-1 of every head (host ints; it may be empty); rows of out and lse
    behind the last one are left as they were allocated.  scale None: 1 / sqrt(d)."""
    import torch

    (Hq, Hk, T, d), scale = _grouped_sizes(q, k, scale)
    with _outputs_on(stream, q, k, v):
        out = torch.empty_like(q)
        lse = torch.empty((Hq, T), dtype=torch.float32, device=q.device)
    jattn_fwd_grouped(q, k, v, cu_seqlens, Hq, Hk, T, d, causal, scale, out.data_ptr(), lse.data_ptr(), stream)
    return out, lse


def backward_grouped(q, k, v, out, lse, dout, cu_seqlens, causal: bool = True, scale: float | None = None,
                     stream=None):
    """dq, dk, dv from forward_grouped's out and lse for the upstream gradient dout (the same causal and
    scale)."""
    import torch

    sizes, scale = _grouped_sizes(q, k, scale)
    with _outputs_on(stream, q, k, v, out, lse, dout):
        dq, dk, dv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
        work = _buffer(jattn_bwd_grouped_bytes(cu_seqlens, *sizes), q.device)
    jattn_bwd_grouped(q, k, v, out, lse, dout, cu_seqlens, *sizes, causal, scale, dq.data_ptr(), dk.data_ptr(),
                      dv.data_ptr(), work.data_ptr(), stream)
    return dq, dk, dv
