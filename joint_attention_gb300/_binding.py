"""ctypes binding of libjattn (include/jattn.h): argument marshalling only.

Every function here forwards to the C ABI of the same name; torch tensors are
accepted for convenience and passed as raw device pointers (torch provides
device memory and streams, nothing else).  There is no fallback: if the
library is missing the import of a call fails loudly.
"""
from __future__ import annotations

import ctypes
import functools
import os
import re

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
HEADER = os.path.join(ROOT, "include", "jattn.h")
LIB_PATH = os.path.join(PKG, "libjattn.so")

STATUS = {
    0: "JATTN_OK",
    1: "JATTN_ERR_INVALID_ARG",
    2: "JATTN_ERR_UNSUPPORTED",
    3: "JATTN_ERR_MISALIGNED",
    4: "JATTN_ERR_ALIAS",
    5: "JATTN_ERR_CUDA",
    6: "JATTN_ERR_TIMEOUT",
    7: "JATTN_ERR_SCRATCH_LIMIT",
}
STATUS_CODE = {v: k for k, v in STATUS.items()}


class JattnError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        detail = jattn_last_error_message() if status == 5 else ""
        super().__init__(f"{where}: {STATUS.get(status, status)} ({jattn_status_string(status)})"
                         + (f" [{detail}]" if detail else ""))


_lib = None


def load_library(path: str | None = None, build_if_missing: bool = False) -> ctypes.CDLL:
    """Loads libjattn.so (building it first only if asked)."""
    global _lib
    if _lib is not None and path is None:
        return _lib
    p = path or LIB_PATH
    if not os.path.exists(p):
        if build_if_missing:
            from .build import build
            p = build()
        else:
            raise FileNotFoundError(f"{p} not found: run joint_attention_gb300/build.py (or __graft_entry__.build())")
    lib = ctypes.CDLL(p)
    vp, i32 = ctypes.c_void_p, ctypes.c_int
    lib.jattn_fwd.argtypes = [vp, vp, vp, vp, vp, i32, i32, i32, i32, i32, vp, vp, vp]
    lib.jattn_fwd.restype = i32
    lib.jattn_fwd_noalloc.argtypes = [vp, vp, vp, vp, vp, i32, i32, i32, i32, i32, vp, vp, vp]
    lib.jattn_fwd_noalloc.restype = i32
    lib.jattn_bwd.argtypes = [vp] * 13 + [i32] * 5 + [vp]
    lib.jattn_bwd.restype = i32
    i32p = ctypes.POINTER(ctypes.c_int)
    lib.jattn_fwd_varlen.argtypes = [vp, vp, vp, vp, vp, i32p, i32, i32, i32, vp, vp, vp]
    lib.jattn_fwd_varlen.restype = i32
    lib.jattn_bwd_varlen.argtypes = [vp] * 13 + [i32p, i32, i32, i32, vp]
    lib.jattn_bwd_varlen.restype = i32
    lib.jattn_last_device_error.argtypes = [vp]
    lib.jattn_last_device_error.restype = i32
    lib.jattn_selftest_wait_timeout.argtypes = [vp]
    lib.jattn_selftest_wait_timeout.restype = i32
    lib.jattn_status_string.argtypes = [i32]
    lib.jattn_status_string.restype = ctypes.c_char_p
    lib.jattn_version.argtypes = []
    lib.jattn_version.restype = i32
    lib.jattn_last_error_message.argtypes = []
    lib.jattn_last_error_message.restype = ctypes.c_char_p
    lib.jattn_profile_enable.argtypes = [i32]
    lib.jattn_profile_enable.restype = i32
    lib.jattn_profile_reset.argtypes = []
    lib.jattn_profile_reset.restype = i32
    lib.jattn_profile_read.argtypes = [i32, ctypes.POINTER(ctypes.c_int), ctypes.POINTER(ctypes.c_double)]
    lib.jattn_profile_read.restype = i32
    lib.jattn_set_sm_limit.argtypes = [i32]
    lib.jattn_set_sm_limit.restype = i32
    lib.jattn_set_deterministic.argtypes = [i32]
    lib.jattn_set_deterministic.restype = i32
    lib.jattn_kernel_name.argtypes = [i32]
    lib.jattn_kernel_name.restype = ctypes.c_char_p
    sz = ctypes.c_size_t
    lib.jattn_saved_bytes.argtypes = [i32] * 5
    lib.jattn_saved_bytes.restype = sz
    lib.jattn_saved_bytes_varlen.argtypes = [i32p, i32, i32, i32]
    lib.jattn_saved_bytes_varlen.restype = sz
    lib.jattn_fwd_train.argtypes = [vp] * 5 + [i32] * 5 + [vp] * 4
    lib.jattn_fwd_train.restype = i32
    lib.jattn_bwd_train.argtypes = [vp] * 14 + [i32] * 5 + [vp]
    lib.jattn_bwd_train.restype = i32
    lib.jattn_fwd_train_varlen.argtypes = [vp] * 5 + [i32p, i32, i32, i32] + [vp] * 4
    lib.jattn_fwd_train_varlen.restype = i32
    lib.jattn_bwd_train_varlen.argtypes = [vp] * 14 + [i32p, i32, i32, i32, vp]
    lib.jattn_bwd_train_varlen.restype = i32
    lib.jattn_qkv_norm.argtypes = [vp] * 8 + [i32] * 6 + [vp] * 5
    lib.jattn_qkv_norm.restype = i32
    lib.jattn_fwd_saved.argtypes = [vp] + [i32] * 5 + [vp] * 4
    lib.jattn_fwd_saved.restype = i32
    f32c = ctypes.c_float
    lib.jattn_add_norm.argtypes = [vp] * 3 + [i32, i32, f32c] + [vp] * 4
    lib.jattn_add_norm.restype = i32
    lib.jattn_add_norm_fp8.argtypes = [vp] * 3 + [i32, i32, f32c] + [vp] * 5
    lib.jattn_add_norm_fp8.restype = i32
    lib.jattn_quant_rows.argtypes = [vp, i32, i32] + [vp] * 3
    lib.jattn_quant_rows.restype = i32
    lib.jattn_add_norm_bwd_bytes.argtypes = [i32, i32]
    lib.jattn_add_norm_bwd_bytes.restype = sz
    lib.jattn_add_norm_bwd.argtypes = [vp] * 5 + [i32, i32] + [vp] * 4
    lib.jattn_add_norm_bwd.restype = i32
    lib.jattn_qkv_norm_fp8.argtypes = [vp] * 12 + [i32] * 6 + [vp] * 5
    lib.jattn_qkv_norm_fp8.restype = i32
    lib.jattn_qkv_norm_lora_bytes.argtypes = [i32] * 6
    lib.jattn_qkv_norm_lora_bytes.restype = sz
    lib.jattn_qkv_norm_lora.argtypes = [vp] * 14 + [i32] * 8 + [vp] * 6
    lib.jattn_qkv_norm_lora.restype = i32
    if path is None:
        _lib = lib
    return lib


KERNEL_KINDS = 6
TOKEN_KERNEL_KINDS = range(16, 21)  # the token-row kernels' kinds, numbered apart


def jattn_profile_enable(on: bool = True) -> int:
    return load_library().jattn_profile_enable(1 if on else 0)


def jattn_profile_reset() -> int:
    return load_library().jattn_profile_reset()


def jattn_profile_read(kind: int) -> tuple[int, float]:
    """(launches, total milliseconds) of one kernel kind since the last reset."""
    n, ms = ctypes.c_int(0), ctypes.c_double(0.0)
    rc = load_library().jattn_profile_read(int(kind), ctypes.byref(n), ctypes.byref(ms))
    if rc != 0:
        raise JattnError(rc, "jattn_profile_read")
    return n.value, ms.value


def jattn_kernel_name(kind: int) -> str:
    return load_library().jattn_kernel_name(int(kind)).decode()


def profile_snapshot() -> dict:
    """{kernel name: (launches, total ms)} for every kernel kind."""
    return {jattn_kernel_name(k): jattn_profile_read(k) for k in (*range(KERNEL_KINDS), *TOKEN_KERNEL_KINDS)}


def declared_symbols(header: str = HEADER) -> list[str]:
    """Names of the functions include/jattn.h declares."""
    text = open(header).read()
    return sorted(set(re.findall(r"^\s*(?:int|size_t|const char\*)\s+(jattn_\w+)\s*\(", text, flags=re.M)))


def _ptr(x, name: str, dtype=None, numel: int | None = None):
    """Raw pointer of a tensor (checked) or an int / None passed through."""
    if x is None or isinstance(x, int):
        return x
    try:  # the checks in one line first: a projection call has two dozen arguments
        if (x.is_cuda and x.is_contiguous() and (dtype is None or x.dtype is dtype)
                and (numel is None or x.numel() == numel)):
            return x.data_ptr()
    except AttributeError:
        pass
    import torch

    if not isinstance(x, torch.Tensor):
        raise TypeError(f"{name}: expected a torch.Tensor or an int pointer")
    if not x.is_cuda:
        raise ValueError(f"{name}: must be a CUDA tensor")
    if not x.is_contiguous():
        raise ValueError(f"{name}: must be contiguous")
    if dtype is not None and x.dtype != dtype:
        raise ValueError(f"{name}: expected {dtype}, got {x.dtype}")
    raise ValueError(f"{name}: expected {numel} elements, got {x.numel()}")


def _stream(stream):
    if stream is None:
        import torch

        raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)  # the same handle without a Stream object
        return raw(torch.cuda.current_device()) if raw else torch.cuda.current_stream().cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def jattn_fwd(q, k, v, gq, gk, B: int, H: int, N_img: int, N_txt: int, d: int, out, lse, stream=None,
              check: bool = True) -> int:
    """C ABI jattn_fwd.  Tensors: q/k/v/out [B,H,N,d] bf16, gq/gk [d] fp32, lse [B,H,N] fp32."""
    import torch

    lib = load_library()
    N = N_img + N_txt
    e, r = B * H * N * d, B * H * N
    bf, f32 = torch.bfloat16, torch.float32
    rc = lib.jattn_fwd(_ptr(q, "q", bf, e), _ptr(k, "k", bf, e), _ptr(v, "v", bf, e), _ptr(gq, "gq", f32, d),
                       _ptr(gk, "gk", f32, d), B, H, N_img, N_txt, d, _ptr(out, "out", bf, e),
                       _ptr(lse, "lse", f32, r), _stream(stream))
    if check and rc != 0:
        raise JattnError(rc, "jattn_fwd")
    return rc


def jattn_fwd_noalloc(q, k, v, gq, gk, B: int, H: int, N_img: int, N_txt: int, d: int, out, lse, stream=None,
                      check: bool = True) -> int:
    """C ABI jattn_fwd_noalloc: jattn_fwd with its scratch in a fixed device array (no allocation)."""
    import torch

    lib = load_library()
    N = N_img + N_txt
    e, r = B * H * N * d, B * H * N
    bf, f32 = torch.bfloat16, torch.float32
    rc = lib.jattn_fwd_noalloc(_ptr(q, "q", bf, e), _ptr(k, "k", bf, e), _ptr(v, "v", bf, e),
                               _ptr(gq, "gq", f32, d), _ptr(gk, "gk", f32, d), B, H, N_img, N_txt, d,
                               _ptr(out, "out", bf, e), _ptr(lse, "lse", f32, r), _stream(stream))
    if check and rc != 0:
        raise JattnError(rc, "jattn_fwd_noalloc")
    return rc


def jattn_bwd(q, k, v, gq, gk, out, lse, dout, dq, dk, dv, dgq, dgk, B: int, H: int, N_img: int, N_txt: int,
              d: int, stream=None, check: bool = True) -> int:
    """C ABI jattn_bwd.  Gradients dq/dk/dv [B,H,N,d] bf16 and dgq/dgk [d] fp32 are overwritten."""
    import torch

    lib = load_library()
    N = N_img + N_txt
    e, r = B * H * N * d, B * H * N
    bf, f32 = torch.bfloat16, torch.float32
    rc = lib.jattn_bwd(_ptr(q, "q", bf, e), _ptr(k, "k", bf, e), _ptr(v, "v", bf, e), _ptr(gq, "gq", f32, d),
                       _ptr(gk, "gk", f32, d), _ptr(out, "out", bf, e), _ptr(lse, "lse", f32, r),
                       _ptr(dout, "dout", bf, e), _ptr(dq, "dq", bf, e), _ptr(dk, "dk", bf, e),
                       _ptr(dv, "dv", bf, e), _ptr(dgq, "dgq", f32, d), _ptr(dgk, "dgk", f32, d), B, H, N_img,
                       N_txt, d, _stream(stream))
    if check and rc != 0:
        raise JattnError(rc, "jattn_bwd")
    return rc


def _cu_array(cu_seqlens):
    """Host int array (ctypes) of the sequence offsets, and T and the count."""
    vals = [int(x) for x in cu_seqlens]
    arr = (ctypes.c_int * len(vals))(*vals)
    return arr, vals[-1] if vals else 0, len(vals) - 1


def jattn_fwd_varlen(q, k, v, gq, gk, cu_seqlens, H: int, d: int, out, lse, stream=None,
                     check: bool = True) -> int:
    """C ABI jattn_fwd_varlen.  q/k/v/out [H, T, d] bf16 (sequence s = rows cu[s]..cu[s+1]-1 of every
    head), gq/gk [d] fp32, lse [H, T] fp32; cu_seqlens a host sequence of n + 1 ints."""
    import torch

    lib = load_library()
    arr, T, n = _cu_array(cu_seqlens)
    e, r = H * T * d, H * T
    bf, f32 = torch.bfloat16, torch.float32
    rc = lib.jattn_fwd_varlen(_ptr(q, "q", bf, e), _ptr(k, "k", bf, e), _ptr(v, "v", bf, e),
                              _ptr(gq, "gq", f32, d), _ptr(gk, "gk", f32, d), arr, n, H, d,
                              _ptr(out, "out", bf, e), _ptr(lse, "lse", f32, r), _stream(stream))
    if check and rc != 0:
        raise JattnError(rc, "jattn_fwd_varlen")
    return rc


def jattn_bwd_varlen(q, k, v, gq, gk, out, lse, dout, dq, dk, dv, dgq, dgk, cu_seqlens, H: int, d: int,
                     stream=None, check: bool = True) -> int:
    """C ABI jattn_bwd_varlen (layouts as jattn_fwd_varlen)."""
    import torch

    lib = load_library()
    arr, T, n = _cu_array(cu_seqlens)
    e, r = H * T * d, H * T
    bf, f32 = torch.bfloat16, torch.float32
    rc = lib.jattn_bwd_varlen(_ptr(q, "q", bf, e), _ptr(k, "k", bf, e), _ptr(v, "v", bf, e),
                              _ptr(gq, "gq", f32, d), _ptr(gk, "gk", f32, d), _ptr(out, "out", bf, e),
                              _ptr(lse, "lse", f32, r), _ptr(dout, "dout", bf, e), _ptr(dq, "dq", bf, e),
                              _ptr(dk, "dk", bf, e), _ptr(dv, "dv", bf, e), _ptr(dgq, "dgq", f32, d),
                              _ptr(dgk, "dgk", f32, d), arr, n, H, d, _stream(stream))
    if check and rc != 0:
        raise JattnError(rc, "jattn_bwd_varlen")
    return rc


@functools.lru_cache(maxsize=1024)  # a function of the sizes alone, and a library call of 0.8 us
def jattn_saved_bytes(B: int, H: int, N_img: int, N_txt: int, d: int) -> int:
    """C ABI jattn_saved_bytes: size of the activation buffer of jattn_fwd_train / jattn_bwd_train."""
    return int(load_library().jattn_saved_bytes(B, H, N_img, N_txt, d))


def jattn_saved_bytes_varlen(cu_seqlens, H: int, d: int) -> int:
    """C ABI jattn_saved_bytes_varlen."""
    arr, _, n = _cu_array(cu_seqlens)
    return int(load_library().jattn_saved_bytes_varlen(arr, n, H, d))


def _saved_ptr(saved, nbytes: int):
    import torch

    if isinstance(saved, int) or saved is None:
        return saved
    if not isinstance(saved, torch.Tensor) or not saved.is_cuda or not saved.is_contiguous():
        raise ValueError("saved: expected a contiguous CUDA tensor")
    if saved.numel() * saved.element_size() < nbytes:
        raise ValueError(f"saved: needs {nbytes} bytes, got {saved.numel() * saved.element_size()}")
    return saved.data_ptr()


def jattn_fwd_train(q, k, v, gq, gk, B: int, H: int, N_img: int, N_txt: int, d: int, out, lse, saved,
                    stream=None, check: bool = True) -> int:
    """C ABI jattn_fwd_train: jattn_fwd that also fills `saved` (jattn_saved_bytes bytes) for jattn_bwd_train."""
    import torch

    lib = load_library()
    N = N_img + N_txt
    e, r = B * H * N * d, B * H * N
    bf, f32 = torch.bfloat16, torch.float32
    nb = jattn_saved_bytes(B, H, N_img, N_txt, d)
    rc = lib.jattn_fwd_train(_ptr(q, "q", bf, e), _ptr(k, "k", bf, e), _ptr(v, "v", bf, e),
                             _ptr(gq, "gq", f32, d), _ptr(gk, "gk", f32, d), B, H, N_img, N_txt, d,
                             _ptr(out, "out", bf, e), _ptr(lse, "lse", f32, r), _saved_ptr(saved, nb),
                             _stream(stream))
    if check and rc != 0:
        raise JattnError(rc, "jattn_fwd_train")
    return rc


def jattn_bwd_train(q, k, v, gq, gk, out, lse, dout, saved, dq, dk, dv, dgq, dgk, B: int, H: int, N_img: int,
                    N_txt: int, d: int, stream=None, check: bool = True) -> int:
    """C ABI jattn_bwd_train: jattn_bwd reading q_hat, k_hat and 1/rms from the forward's `saved`."""
    import torch

    lib = load_library()
    N = N_img + N_txt
    e, r = B * H * N * d, B * H * N
    bf, f32 = torch.bfloat16, torch.float32
    nb = jattn_saved_bytes(B, H, N_img, N_txt, d)
    rc = lib.jattn_bwd_train(_ptr(q, "q", bf, e), _ptr(k, "k", bf, e), _ptr(v, "v", bf, e),
                             _ptr(gq, "gq", f32, d), _ptr(gk, "gk", f32, d), _ptr(out, "out", bf, e),
                             _ptr(lse, "lse", f32, r), _ptr(dout, "dout", bf, e), _saved_ptr(saved, nb),
                             _ptr(dq, "dq", bf, e), _ptr(dk, "dk", bf, e), _ptr(dv, "dv", bf, e),
                             _ptr(dgq, "dgq", f32, d), _ptr(dgk, "dgk", f32, d), B, H, N_img, N_txt, d,
                             _stream(stream))
    if check and rc != 0:
        raise JattnError(rc, "jattn_bwd_train")
    return rc


def jattn_fwd_train_varlen(q, k, v, gq, gk, cu_seqlens, H: int, d: int, out, lse, saved, stream=None,
                           check: bool = True) -> int:
    """C ABI jattn_fwd_train_varlen (layouts as jattn_fwd_varlen)."""
    import torch

    lib = load_library()
    arr, T, n = _cu_array(cu_seqlens)
    e, r = H * T * d, H * T
    bf, f32 = torch.bfloat16, torch.float32
    nb = jattn_saved_bytes_varlen(cu_seqlens, H, d)
    rc = lib.jattn_fwd_train_varlen(_ptr(q, "q", bf, e), _ptr(k, "k", bf, e), _ptr(v, "v", bf, e),
                                    _ptr(gq, "gq", f32, d), _ptr(gk, "gk", f32, d), arr, n, H, d,
                                    _ptr(out, "out", bf, e), _ptr(lse, "lse", f32, r), _saved_ptr(saved, nb),
                                    _stream(stream))
    if check and rc != 0:
        raise JattnError(rc, "jattn_fwd_train_varlen")
    return rc


def jattn_bwd_train_varlen(q, k, v, gq, gk, out, lse, dout, saved, dq, dk, dv, dgq, dgk, cu_seqlens, H: int,
                           d: int, stream=None, check: bool = True) -> int:
    """C ABI jattn_bwd_train_varlen (layouts as jattn_fwd_varlen)."""
    import torch

    lib = load_library()
    arr, T, n = _cu_array(cu_seqlens)
    e, r = H * T * d, H * T
    bf, f32 = torch.bfloat16, torch.float32
    nb = jattn_saved_bytes_varlen(cu_seqlens, H, d)
    rc = lib.jattn_bwd_train_varlen(_ptr(q, "q", bf, e), _ptr(k, "k", bf, e), _ptr(v, "v", bf, e),
                                    _ptr(gq, "gq", f32, d), _ptr(gk, "gk", f32, d), _ptr(out, "out", bf, e),
                                    _ptr(lse, "lse", f32, r), _ptr(dout, "dout", bf, e), _saved_ptr(saved, nb),
                                    _ptr(dq, "dq", bf, e), _ptr(dk, "dk", bf, e), _ptr(dv, "dv", bf, e),
                                    _ptr(dgq, "dgq", f32, d), _ptr(dgk, "dgk", f32, d), arr, n, H, d,
                                    _stream(stream))
    if check and rc != 0:
        raise JattnError(rc, "jattn_bwd_train_varlen")
    return rc


def jattn_qkv_norm(x_img, w_img, b_img, x_txt, w_txt, b_txt, gq, gk, B: int, H: int, N_img: int, N_txt: int,
                   d: int, C: int, q, k, v, saved, stream=None, check: bool = True) -> int:
    """C ABI jattn_qkv_norm.  x_img [B, N_img, C] / x_txt [B, N_txt, C] bf16 tokens, w_* [3 H d, C] bf16,
    b_* [3 H d] fp32 or None, gq/gk [d] fp32; writes q/k/v [B, H, N, d] bf16 and `saved`."""
    import torch

    lib = load_library()
    N = N_img + N_txt
    e = B * H * N * d
    bf, f32 = torch.bfloat16, torch.float32
    yc = 3 * H * d
    nb = jattn_saved_bytes(B, H, N_img, N_txt, d)
    rc = lib.jattn_qkv_norm(_ptr(x_img, "x_img", bf, B * N_img * C if N_img else None),
                            _ptr(w_img, "w_img", bf, yc * C if N_img else None), _ptr(b_img, "b_img", f32, yc),
                            _ptr(x_txt, "x_txt", bf, B * N_txt * C if N_txt else None),
                            _ptr(w_txt, "w_txt", bf, yc * C if N_txt else None), _ptr(b_txt, "b_txt", f32, yc),
                            _ptr(gq, "gq", f32, d), _ptr(gk, "gk", f32, d), B, H, N_img, N_txt, d, C,
                            _ptr(q, "q", bf, e), _ptr(k, "k", bf, e), _ptr(v, "v", bf, e), _saved_ptr(saved, nb),
                            _stream(stream))
    if check and rc != 0:
        raise JattnError(rc, "jattn_qkv_norm")
    return rc


def jattn_fwd_saved(v, B: int, H: int, N_img: int, N_txt: int, d: int, out, lse, saved, stream=None,
                    check: bool = True) -> int:
    """C ABI jattn_fwd_saved: the attention forward from the q_hat / k_hat already in `saved`."""
    import torch

    lib = load_library()
    N = N_img + N_txt
    e, r = B * H * N * d, B * H * N
    bf, f32 = torch.bfloat16, torch.float32
    nb = jattn_saved_bytes(B, H, N_img, N_txt, d)
    rc = lib.jattn_fwd_saved(_ptr(v, "v", bf, e), B, H, N_img, N_txt, d, _ptr(out, "out", bf, e),
                             _ptr(lse, "lse", f32, r), _saved_ptr(saved, nb), _stream(stream))
    if check and rc != 0:
        raise JattnError(rc, "jattn_fwd_saved")
    return rc


def _size(n: int) -> int:
    """n for a C int: 0, which the library refuses, where ctypes would keep the low 32 bits."""
    return n if -(1 << 31) <= n < 1 << 31 else 0


def jattn_add_norm(x, res, g, T: int, C: int, eps: float, h, y, r, stream=None, check: bool = True) -> int:
    """C ABI jattn_add_norm.  x / res / h / y [T, C] bf16 (res and h both or neither; h may be res),
    g [C] fp32, r [T] fp32 or None."""
    import torch

    bf, f32, e = torch.bfloat16, torch.float32, T * C
    rc = load_library().jattn_add_norm(_ptr(x, "x", bf, e), _ptr(res, "res", bf, e), _ptr(g, "g", f32, C), _size(T),
                                       _size(C), eps, _ptr(h, "h", bf, e), _ptr(y, "y", bf, e), _ptr(r, "r", f32, T),
                                       _stream(stream))
    if check and rc != 0:
        raise JattnError(rc, "jattn_add_norm")
    return rc


def jattn_add_norm_fp8(x, res, g, T: int, C: int, eps: float, h, y8, s, r, stream=None, check: bool = True) -> int:
    """C ABI jattn_add_norm_fp8: jattn_add_norm with y8 [T, C] float8_e4m3fn and the rows' scales s [T] fp32."""
    import torch

    bf, f32, e = torch.bfloat16, torch.float32, T * C
    rc = load_library().jattn_add_norm_fp8(_ptr(x, "x", bf, e), _ptr(res, "res", bf, e), _ptr(g, "g", f32, C),
                                           _size(T), _size(C), eps, _ptr(h, "h", bf, e),
                                           _ptr(y8, "y8", torch.float8_e4m3fn, e), _ptr(s, "s", f32, T),
                                           _ptr(r, "r", f32, T), _stream(stream))
    if check and rc != 0:
        raise JattnError(rc, "jattn_add_norm_fp8")
    return rc


def jattn_quant_rows(x, T: int, C: int, x8, s, stream=None, check: bool = True) -> int:
    """C ABI jattn_quant_rows.  x [T, C] bf16 to x8 [T, C] float8_e4m3fn and s [T] fp32."""
    import torch

    e = T * C
    rc = load_library().jattn_quant_rows(_ptr(x, "x", torch.bfloat16, e), _size(T), _size(C),
                                         _ptr(x8, "x8", torch.float8_e4m3fn, e), _ptr(s, "s", torch.float32, T),
                                         _stream(stream))
    if check and rc != 0:
        raise JattnError(rc, "jattn_quant_rows")
    return rc


@functools.lru_cache(maxsize=1024)  # a function of the sizes alone, and a library call of 0.8 us
def jattn_add_norm_bwd_bytes(T: int, C: int) -> int:
    """C ABI jattn_add_norm_bwd_bytes: size of the work buffer of jattn_add_norm_bwd (0: it rejects the sizes)."""
    return int(load_library().jattn_add_norm_bwd_bytes(_size(T), _size(C)))


def _work_ptr(work, bytes_of, *sizes):
    """Raw pointer of a work buffer of at least bytes_of(*sizes) bytes (any dtype)."""
    if work is None or isinstance(work, int):
        return work
    import torch

    nbytes = bytes_of(*sizes)
    if not isinstance(work, torch.Tensor) or not work.is_cuda or not work.is_contiguous():
        raise ValueError("work: expected a contiguous CUDA tensor")
    if work.numel() * work.element_size() < nbytes:
        raise ValueError(f"work: needs {nbytes} bytes, got {work.numel() * work.element_size()}")
    return work.data_ptr()


def jattn_add_norm_bwd(dy, dh, h, r, g, T: int, C: int, dx, dg, work, stream=None, check: bool = True) -> int:
    """C ABI jattn_add_norm_bwd.  dy / dh (or None) / h / dx [T, C] bf16 (dx may be dh), r [T] fp32,
    g / dg [C] fp32, work jattn_add_norm_bwd_bytes(T, C) bytes."""
    import torch

    bf, f32, e = torch.bfloat16, torch.float32, T * C
    lib = load_library()
    rc = lib.jattn_add_norm_bwd(_ptr(dy, "dy", bf, e), _ptr(dh, "dh", bf, e), _ptr(h, "h", bf, e),
                                _ptr(r, "r", f32, T), _ptr(g, "g", f32, C), _size(T), _size(C), _ptr(dx, "dx", bf, e),
                                _ptr(dg, "dg", f32, C), _work_ptr(work, jattn_add_norm_bwd_bytes, T, C),
                                _stream(stream))
    if check and rc != 0:
        raise JattnError(rc, "jattn_add_norm_bwd")
    return rc


def _saved(saved, *sizes):
    """Raw pointer of a training pair's buffer for a [B, H, N, d] shape."""
    return saved if saved is None or isinstance(saved, int) else _saved_ptr(saved, jattn_saved_bytes(*sizes))


def jattn_qkv_norm_fp8(x_img, sx_img, w_img, sw_img, b_img, x_txt, sx_txt, w_txt, sw_txt, b_txt, gq, gk, B: int,
                       H: int, N_img: int, N_txt: int, d: int, C: int, q, k, v, saved, stream=None,
                       check: bool = True) -> int:
    """C ABI jattn_qkv_norm_fp8: jattn_qkv_norm with tokens and weights in float8_e4m3fn and the fp32 scales
    of their rows, sx_* [B, N_*] and sw_* [3 H d]."""
    import torch

    e = B * H * (N_img + N_txt) * d
    bf, f32, f8 = torch.bfloat16, torch.float32, torch.float8_e4m3fn
    yc = 3 * H * d
    rc = load_library().jattn_qkv_norm_fp8(
        _ptr(x_img, "x_img", f8, B * N_img * C), _ptr(sx_img, "sx_img", f32, B * N_img),
        _ptr(w_img, "w_img", f8, yc * C if N_img else None), _ptr(sw_img, "sw_img", f32, yc if N_img else None),
        _ptr(b_img, "b_img", f32, yc), _ptr(x_txt, "x_txt", f8, B * N_txt * C),
        _ptr(sx_txt, "sx_txt", f32, B * N_txt), _ptr(w_txt, "w_txt", f8, yc * C if N_txt else None),
        _ptr(sw_txt, "sw_txt", f32, yc if N_txt else None), _ptr(b_txt, "b_txt", f32, yc), _ptr(gq, "gq", f32, d),
        _ptr(gk, "gk", f32, d), B, H, N_img, N_txt, d, C, _ptr(q, "q", bf, e), _ptr(k, "k", bf, e),
        _ptr(v, "v", bf, e), _saved(saved, B, H, N_img, N_txt, d), _stream(stream))
    if check and rc != 0:
        raise JattnError(rc, "jattn_qkv_norm_fp8")
    return rc


@functools.lru_cache(maxsize=1024)
def jattn_qkv_norm_lora_bytes(B: int, H: int, N_img: int, N_txt: int, d: int, rank: int) -> int:
    """C ABI jattn_qkv_norm_lora_bytes: size of the work buffer of jattn_qkv_norm_lora (0: it rejects the sizes)."""
    return int(load_library().jattn_qkv_norm_lora_bytes(B, H, N_img, N_txt, d, rank))


def jattn_qkv_norm_lora(x_img, w_img, b_img, x_txt, w_txt, b_txt, gq, gk, down_img, up_img, down_txt, up_txt, scale,
                        index, n_adapters: int, rank: int, B: int, H: int, N_img: int, N_txt: int, d: int, C: int,
                        q, k, v, saved, work, stream=None, check: bool = True) -> int:
    """C ABI jattn_qkv_norm_lora: jattn_qkv_norm with the batch items' adapters.  down_* [n, 3 rank, C] and up_*
    [n, 3 H d, rank] bf16 (None: none in that stream), scale [n] fp32, index [B] int32 (outside 0 .. n - 1:
    no adapter), work jattn_qkv_norm_lora_bytes(...) bytes."""
    import torch

    e = B * H * (N_img + N_txt) * d
    bf, f32 = torch.bfloat16, torch.float32
    yc = 3 * H * d
    rc = load_library().jattn_qkv_norm_lora(
        _ptr(x_img, "x_img", bf, B * N_img * C), _ptr(w_img, "w_img", bf, yc * C if N_img else None),
        _ptr(b_img, "b_img", f32, yc), _ptr(x_txt, "x_txt", bf, B * N_txt * C),
        _ptr(w_txt, "w_txt", bf, yc * C if N_txt else None), _ptr(b_txt, "b_txt", f32, yc), _ptr(gq, "gq", f32, d),
        _ptr(gk, "gk", f32, d), _ptr(down_img, "down_img", bf, n_adapters * 3 * rank * C),
        _ptr(up_img, "up_img", bf, n_adapters * yc * rank), _ptr(down_txt, "down_txt", bf, n_adapters * 3 * rank * C),
        _ptr(up_txt, "up_txt", bf, n_adapters * yc * rank), _ptr(scale, "scale", f32, n_adapters),
        _ptr(index, "index", torch.int32, B), n_adapters, rank, B, H, N_img, N_txt, d, C, _ptr(q, "q", bf, e),
        _ptr(k, "k", bf, e), _ptr(v, "v", bf, e), _saved(saved, B, H, N_img, N_txt, d),
        _work_ptr(work, jattn_qkv_norm_lora_bytes, B, H, N_img, N_txt, d, rank), _stream(stream))
    if check and rc != 0:
        raise JattnError(rc, "jattn_qkv_norm_lora")
    return rc


def jattn_last_device_error(stream=None) -> int:
    return load_library().jattn_last_device_error(_stream(stream))


def jattn_selftest_wait_timeout(stream=None) -> int:
    """Runs the bounded-wait self-test kernel; the next jattn_last_device_error reports the timeout."""
    rc = load_library().jattn_selftest_wait_timeout(_stream(stream))
    if rc != 0:
        raise JattnError(rc, "jattn_selftest_wait_timeout")
    return rc


def jattn_set_sm_limit(max_sms: int) -> int:
    """C ABI jattn_set_sm_limit: cap the persistent kernels' CTAs (0 = every SM)."""
    rc = load_library().jattn_set_sm_limit(int(max_sms))
    if rc != 0:
        raise JattnError(rc, "jattn_set_sm_limit")
    return rc


def jattn_set_deterministic(on: bool) -> int:
    """C ABI jattn_set_deterministic: bitwise-reproducible backward (fixed dQ accumulation order) or not."""
    rc = load_library().jattn_set_deterministic(1 if on else 0)
    if rc != 0:
        raise JattnError(rc, "jattn_set_deterministic")
    return rc


def jattn_status_string(status: int) -> str:
    return load_library().jattn_status_string(int(status)).decode()


def jattn_last_error_message() -> str:
    return load_library().jattn_last_error_message().decode()


def jattn_version() -> int:
    return load_library().jattn_version()
