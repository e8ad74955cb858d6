"""ctypes binding of libfa.so (argument marshalling only).

Every function here passes raw device pointers, sizes and the current CUDA
stream to the C ABI declared in include/fa.h; all the arithmetic runs in the
library's CUDA kernels.  There is no fallback: if libfa.so is missing or
cannot be loaded, or a call returns an error code, a ``FaError`` is raised.

Tensors are torch tensors used as device buffers: q, k, v, o, dout, dq, dk,
dv are contiguous bf16 (B, H, N, d) on a CUDA device, lse is contiguous fp32
(B, H, N).
"""
from __future__ import annotations

import ctypes
import functools
import math
import os
import struct
import threading

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
# FA_CHECKED=1 selects the bounds-checked build (python -m
# io_aware_exact_02_gb300.build --checked), whose kernels range-check every
# tile, mask and row index they compute.
CHECKED = os.environ.get("FA_CHECKED") == "1"
LIB_PATH = os.path.join(_HERE, "libfa_checked.so" if CHECKED else "libfa.so")

FA_OK = 0
FA_ERR_ARG = -1
FA_ERR_UNSUPPORTED_D = -2
FA_ERR_ALIGN = -3
FA_ERR_WORKSPACE = -4
FA_ERR_DEVICE = -5
FA_ERR_LAUNCH = -6
FA_ERR_TIMEOUT = -7
FA_ERR_BOUNDS = -8
FA_ERR_PAGE = -9

# Size of the static scratch array fa_bwd_noalloc uses (FA_NOALLOC_SCRATCH_BYTES).
FA_NOALLOC_SCRATCH_BYTES = 32 << 20

# Every symbol include/fa.h declares, with (restype, argtypes).
_vp, _i, _f, _sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_size_t
_ll = ctypes.c_longlong
_ip = ctypes.POINTER(ctypes.c_int)
SIGNATURES = {
    "fa_fwd": (_i, [_vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _f, _vp]),
    "fa_fwd_gqa": (_i, [_vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _i, _i, _f, _i, _vp, _sz,
                        _vp]),
    "fa_fwd_gqa_workspace_size": (_sz, [_i, _i, _i, _i, _i, _i, _i]),
    "fa_fwd_gqa_splits": (_i, [_i, _i, _i, _i, _i, _i, _i, _i]),
    "fa_bwd_workspace_size": (_sz, [_i, _i, _i, _i]),
    "fa_bwd": (_i, [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _f,
                    _vp, _sz, _vp]),
    "fa_bwd_phases": (_i, [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _f,
                           _vp, _sz, _vp, _i]),
    "fa_bwd_noalloc": (_i, [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _f,
                            _vp]),
    "fa_fwd_blocksparse": (_i, [_vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _f, _vp, _vp]),
    "fa_bwd_blocksparse": (_i, [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i,
                                _f, _vp, _vp, _sz, _vp]),
    "fa_fwd_fp8_workspace_size": (_sz, [_i, _i, _i, _i]),
    "fa_fp8_workspace_offsets": (_i, [_i, _i, _i, _i, ctypes.POINTER(ctypes.c_size_t)]),
    "fa_fp8_quantize": (_i, [_vp, _vp, _vp, _i, _i, _i, _i, _i, _vp, _sz, _vp]),
    "fa_fwd_fp8_quantized": (_i, [_vp, _vp, _i, _i, _i, _i, _i, _f, _i, _vp, _sz, _vp]),
    "fa_fwd_fp8": (_i, [_vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _f, _i, _vp, _sz, _vp]),
    "fa_kv_append": (_i, [_vp] * 10 + [_i] * 5 + [_ll] * 4 + [_i] * 6 + [_vp]),
    "fa_fwd_paged_workspace_size": (_sz, [_i] * 7),
    "fa_fwd_paged": (_i, [_vp] * 8 + [_i] * 5 + [_ll] + [_i] * 5 + [_f, _vp, _sz, _vp]),
    "fa_fwd_paged_prefix": (_i, [_vp] * 9 + [_i] * 6 + [_ll] + [_i] * 5 + [_f, _vp, _sz, _vp]),
    "fa_kv_append_words": (_i, [ctypes.c_char_p, _i]),
    "fa_fwd_paged_words": (_i, [ctypes.c_char_p, _i]),
    "fa_device_status": (_i, [_vp, _ip]),
    "fa_selftest_timeout": (_i, [_i, _vp]),
    "fa_checks_enabled": (_i, []),
    "fa_selftest_bounds": (_i, [_vp]),
    "fa_status_string": (ctypes.c_char_p, [_i]),
    "fa_fwd_schedule": (_i, [_i, _i, _i, _i, _i, _ip, _ip, _ip, _ip, _i]),
    "fa_snake_assign": (_i, [_i, _i, _ip]),
    "fa_version": (_i, []),
}


class FaError(RuntimeError):
    def __init__(self, fn: str, code: int, msg: str):
        super().__init__("%s failed: %s (%d)" % (fn, msg, code))
        self.code = code


_lock = threading.Lock()
_lib = None


def load(path: str | None = None):
    """Load libfa.so (once) and declare its signatures.  Raises if missing."""
    global _lib
    if _lib is not None and path is None:
        return _lib
    with _lock:
        if _lib is not None and path is None:
            return _lib
        p = path or LIB_PATH
        if not os.path.exists(p):
            raise FaError("load", FA_ERR_DEVICE,
                          "%s is missing; build it with python -m io_aware_exact_02_gb300.build" % p)
        lib = ctypes.CDLL(p)
        for name, (res, args) in SIGNATURES.items():
            fn = getattr(lib, name)
            fn.restype = res
            fn.argtypes = args
        if path is None:
            _lib = lib
        return lib


def status_string(code: int) -> str:
    return load().fa_status_string(int(code)).decode()


def _check(fn: str, code: int):
    if code != FA_OK:
        raise FaError(fn, code, status_string(code))


def _stream_of(t: torch.Tensor):
    return ctypes.c_void_p(torch.cuda.current_stream(t.device).cuda_stream)


def _check_qkv(name, t, shape, dtype=torch.bfloat16):
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError("%s must be a CUDA tensor" % name)
    if t.dtype != dtype:
        raise ValueError("%s must be %s" % (name, dtype))
    if tuple(t.shape) != tuple(shape):
        raise ValueError("%s has shape %s, expected %s" % (name, tuple(t.shape), tuple(shape)))
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)


def _on_device(ref, **tensors):
    """Check that every given tensor is on ``ref``'s device and return a
    context manager that makes that device current for the call: the library
    looks up its per-device state (status word, SM count, tensor maps) on the
    current device, and tensor maps built there must address that device's
    memory."""
    for name, t in tensors.items():
        if t is not None and t.device != ref.device:
            raise ValueError("%s is on %s, expected %s (one call's tensors must share a device)"
                             % (name, t.device, ref.device))
    return torch.cuda.device(ref.device)


def default_scale(d: int) -> float:
    return 1.0 / math.sqrt(d)


def fwd(q, k, v, causal: bool = False, scale: float | None = None, out=None, lse=None):
    """O, lse = attention(q, k, v).  Returns (o, lse) (allocated if not given)."""
    B, H, N, d = q.shape
    scale = default_scale(d) if scale is None else float(scale)
    for name, t in (("q", q), ("k", k), ("v", v)):
        _check_qkv(name, t, (B, H, N, d))
    if out is None:
        out = torch.empty_like(q)
    if lse is None:
        lse = torch.empty((B, H, N), dtype=torch.float32, device=q.device)
    _check_qkv("out", out, (B, H, N, d))
    _check_qkv("lse", lse, (B, H, N), torch.float32)
    with _on_device(q, k=k, v=v, out=out, lse=lse):
        rc = load().fa_fwd(q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(),
                           lse.data_ptr(), B, H, N, d, int(bool(causal)), ctypes.c_float(scale),
                           _stream_of(q))
    _check("fa_fwd", rc)
    return out, lse


def fwd_gqa_splits(B, Hq, Hkv, Nq, Nkv, d, causal=False, sm_count=None) -> int:
    """Key splits that fill the device's SMs (fa_fwd_gqa_splits)."""
    if sm_count is None:
        sm_count = torch.cuda.get_device_properties(torch.cuda.current_device()).multi_processor_count
    n = load().fa_fwd_gqa_splits(B, Hq, Hkv, Nq, Nkv, d, int(bool(causal)), int(sm_count))
    if n < 0:
        _check("fa_fwd_gqa_splits", n)
    return n


def fwd_gqa_workspace_size(B, Hq, Hkv, Nq, Nkv, d, num_splits) -> int:
    return int(load().fa_fwd_gqa_workspace_size(B, Hq, Hkv, Nq, Nkv, d, int(num_splits)))


def fwd_gqa(q, k, v, causal: bool = False, scale: float | None = None, num_splits=None,
            out=None, lse=None, workspace=None):
    """General forward: q (B, Hq, Nq, d), k and v (B, Hkv, Nkv, d), Hq a
    multiple of Hkv; causal aligned bottom-right; the keys cut into
    ``num_splits`` ranges (None: fa_fwd_gqa_splits).  Returns (o, lse)."""
    B, Hq, Nq, d = q.shape
    Bk, Hkv, Nkv, dk = k.shape
    scale = default_scale(d) if scale is None else float(scale)
    _check_qkv("q", q, (B, Hq, Nq, d))
    _check_qkv("k", k, (B, Hkv, Nkv, d))
    _check_qkv("v", v, (B, Hkv, Nkv, d))
    if num_splits is None:
        num_splits = fwd_gqa_splits(B, Hq, Hkv, Nq, Nkv, d, causal)
    if out is None:
        out = torch.empty_like(q)
    if lse is None:
        lse = torch.empty((B, Hq, Nq), dtype=torch.float32, device=q.device)
    _check_qkv("out", out, (B, Hq, Nq, d))
    _check_qkv("lse", lse, (B, Hq, Nq), torch.float32)
    need = fwd_gqa_workspace_size(B, Hq, Hkv, Nq, Nkv, d, num_splits)
    if workspace is None and need > 0:
        workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
    ws_ptr = workspace.data_ptr() if workspace is not None else None
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    with _on_device(q, k=k, v=v, out=out, lse=lse, workspace=workspace):
        rc = load().fa_fwd_gqa(q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(),
                               lse.data_ptr(), B, Hq, Hkv, Nq, Nkv, d, int(bool(causal)),
                               ctypes.c_float(scale), int(num_splits), ws_ptr, ws_bytes,
                               _stream_of(q))
    _check("fa_fwd_gqa", rc)
    return out, lse


def bwd_workspace_size(B: int, H: int, N: int, d: int) -> int:
    return int(load().fa_bwd_workspace_size(B, H, N, d))


def bwd(q, k, v, o, dout, lse, causal: bool = False, scale: float | None = None,
        dq=None, dk=None, dv=None, workspace=None, phases: int = 7):
    """dq, dk, dv of L = sum(dout * O).  Returns (dq, dk, dv).

    ``phases`` selects the backward kernels to run (bit 0 prep, bit 1 main,
    bit 2 dQ convert); the default runs all three, as fa_bwd does.
    """
    B, H, N, d = q.shape
    scale = default_scale(d) if scale is None else float(scale)
    for name, t in (("q", q), ("k", k), ("v", v), ("o", o), ("dout", dout)):
        _check_qkv(name, t, (B, H, N, d))
    _check_qkv("lse", lse, (B, H, N), torch.float32)
    dq = torch.empty_like(q) if dq is None else dq
    dk = torch.empty_like(q) if dk is None else dk
    dv = torch.empty_like(q) if dv is None else dv
    for name, t in (("dq", dq), ("dk", dk), ("dv", dv)):
        _check_qkv(name, t, (B, H, N, d))
    need = bwd_workspace_size(B, H, N, d)
    if workspace is None:
        workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
    nbytes = workspace.numel() * workspace.element_size()
    args = (q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), dout.data_ptr(),
            lse.data_ptr(), dq.data_ptr(), dk.data_ptr(), dv.data_ptr(), B, H, N, d,
            int(bool(causal)), ctypes.c_float(scale), workspace.data_ptr(), nbytes, _stream_of(q))
    with _on_device(q, k=k, v=v, o=o, dout=dout, lse=lse, dq=dq, dk=dk, dv=dv,
                    workspace=workspace):
        if phases == 7:
            _check("fa_bwd", load().fa_bwd(*args))
        else:
            _check("fa_bwd_phases", load().fa_bwd_phases(*args, int(phases)))
    return dq, dk, dv


def bwd_noalloc(q, k, v, o, dout, lse, causal: bool = False, scale: float | None = None,
                dq=None, dk=None, dv=None):
    """fa_bwd without a caller workspace: the library's fixed scratch array is
    used instead (for callers that cannot allocate device memory).  Calls
    that overlap on the GPU race on that array.  Returns (dq, dk, dv)."""
    B, H, N, d = q.shape
    scale = default_scale(d) if scale is None else float(scale)
    for name, t in (("q", q), ("k", k), ("v", v), ("o", o), ("dout", dout)):
        _check_qkv(name, t, (B, H, N, d))
    _check_qkv("lse", lse, (B, H, N), torch.float32)
    dq = torch.empty_like(q) if dq is None else dq
    dk = torch.empty_like(q) if dk is None else dk
    dv = torch.empty_like(q) if dv is None else dv
    for name, t in (("dq", dq), ("dk", dk), ("dv", dv)):
        _check_qkv(name, t, (B, H, N, d))
    with _on_device(q, k=k, v=v, o=o, dout=dout, lse=lse, dq=dq, dk=dk, dv=dv):
        rc = load().fa_bwd_noalloc(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(),
                                   dout.data_ptr(), lse.data_ptr(), dq.data_ptr(), dk.data_ptr(),
                                   dv.data_ptr(), B, H, N, d, int(bool(causal)),
                                   ctypes.c_float(scale), _stream_of(q))
    _check("fa_bwd_noalloc", rc)
    return dq, dk, dv


def _check_block_mask(block_mask, N, device):
    nt = (N + 127) // 128
    if not isinstance(block_mask, torch.Tensor) or block_mask.device != device:
        raise ValueError("block_mask must be a tensor on %s" % device)
    if block_mask.dtype not in (torch.uint8, torch.bool) or tuple(block_mask.shape) != (nt, nt):
        raise ValueError("block_mask must be uint8 or bool of shape (%d, %d)" % (nt, nt))
    if not block_mask.is_contiguous():
        raise ValueError("block_mask must be contiguous")


def fwd_blocksparse(q, k, v, block_mask, causal: bool = False, scale: float | None = None,
                    out=None, lse=None):
    """Block-sparse forward: key block c is visible to query block r when
    block_mask[r, c] is nonzero; blocks are 128 rows.  Returns (o, lse)."""
    B, H, N, d = q.shape
    scale = default_scale(d) if scale is None else float(scale)
    for name, t in (("q", q), ("k", k), ("v", v)):
        _check_qkv(name, t, (B, H, N, d))
    _check_block_mask(block_mask, N, q.device)
    out = torch.empty_like(q) if out is None else out
    if lse is None:
        lse = torch.empty((B, H, N), dtype=torch.float32, device=q.device)
    _check_qkv("out", out, (B, H, N, d))
    _check_qkv("lse", lse, (B, H, N), torch.float32)
    with _on_device(q, k=k, v=v, out=out, lse=lse):
        rc = load().fa_fwd_blocksparse(q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(),
                                       lse.data_ptr(), B, H, N, d, int(bool(causal)),
                                       ctypes.c_float(scale), block_mask.data_ptr(),
                                       _stream_of(q))
    _check("fa_fwd_blocksparse", rc)
    return out, lse


def bwd_blocksparse(q, k, v, o, dout, lse, block_mask, causal: bool = False,
                    scale: float | None = None, dq=None, dk=None, dv=None, workspace=None):
    """dq, dk, dv of the block-sparse forward.  Returns (dq, dk, dv)."""
    B, H, N, d = q.shape
    scale = default_scale(d) if scale is None else float(scale)
    for name, t in (("q", q), ("k", k), ("v", v), ("o", o), ("dout", dout)):
        _check_qkv(name, t, (B, H, N, d))
    _check_qkv("lse", lse, (B, H, N), torch.float32)
    _check_block_mask(block_mask, N, q.device)
    dq = torch.empty_like(q) if dq is None else dq
    dk = torch.empty_like(q) if dk is None else dk
    dv = torch.empty_like(q) if dv is None else dv
    for name, t in (("dq", dq), ("dk", dk), ("dv", dv)):
        _check_qkv(name, t, (B, H, N, d))
    if workspace is None:
        workspace = torch.empty(bwd_workspace_size(B, H, N, d), dtype=torch.uint8,
                                device=q.device)
    nbytes = workspace.numel() * workspace.element_size()
    with _on_device(q, k=k, v=v, o=o, dout=dout, lse=lse, dq=dq, dk=dk, dv=dv,
                    workspace=workspace):
        rc = load().fa_bwd_blocksparse(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(),
                                       dout.data_ptr(), lse.data_ptr(), dq.data_ptr(),
                                       dk.data_ptr(), dv.data_ptr(), B, H, N, d,
                                       int(bool(causal)), ctypes.c_float(scale),
                                       block_mask.data_ptr(), workspace.data_ptr(), nbytes,
                                       _stream_of(q))
    _check("fa_bwd_blocksparse", rc)
    return dq, dk, dv


def fwd_fp8_workspace_size(B: int, H: int, N: int, d: int) -> int:
    return int(load().fa_fwd_fp8_workspace_size(B, H, N, d))


def fp8_workspace_offsets(B: int, H: int, N: int, d: int):
    """Byte offsets of (q8, k8, vt8, amax) in the FP8 workspace."""
    off = (ctypes.c_size_t * 4)()
    _check("fa_fp8_workspace_offsets", load().fa_fp8_workspace_offsets(B, H, N, d, off))
    return tuple(int(x) for x in off)


def _fp8_workspace(workspace, B, H, N, d, device):
    need = fwd_fp8_workspace_size(B, H, N, d)
    if workspace is None:
        workspace = torch.empty(max(need, 1), dtype=torch.uint8, device=device)
    return workspace, workspace.numel() * workspace.element_size()


def fp8_quantize(q, k, v, hadamard: bool = True, workspace=None):
    """Quantise bf16 q, k, v to the FP8 workspace (see fa_fp8_quantize).
    Returns the workspace (uint8 tensor)."""
    B, H, N, d = q.shape
    for name, t in (("q", q), ("k", k), ("v", v)):
        _check_qkv(name, t, (B, H, N, d))
    workspace, nbytes = _fp8_workspace(workspace, B, H, N, d, q.device)
    with _on_device(q, k=k, v=v, workspace=workspace):
        rc = load().fa_fp8_quantize(q.data_ptr(), k.data_ptr(), v.data_ptr(), B, H, N, d,
                                    int(bool(hadamard)), workspace.data_ptr(), nbytes,
                                    _stream_of(q))
    _check("fa_fp8_quantize", rc)
    return workspace


def fwd_fp8_quantized(workspace, B, H, N, d, causal: bool = False, scale: float | None = None,
                      hadamard: bool = True, out=None, lse=None):
    """FP8 attention over a workspace written by fp8_quantize.  Returns (o, lse)."""
    scale = default_scale(d) if scale is None else float(scale)
    dev = workspace.device
    out = torch.empty((B, H, N, d), dtype=torch.bfloat16, device=dev) if out is None else out
    if lse is None:
        lse = torch.empty((B, H, N), dtype=torch.float32, device=dev)
    _check_qkv("out", out, (B, H, N, d))
    _check_qkv("lse", lse, (B, H, N), torch.float32)
    with _on_device(workspace, out=out, lse=lse):
        rc = load().fa_fwd_fp8_quantized(out.data_ptr(), lse.data_ptr(), B, H, N, d,
                                         int(bool(causal)), ctypes.c_float(scale),
                                         int(bool(hadamard)), workspace.data_ptr(),
                                         workspace.numel() * workspace.element_size(),
                                         _stream_of(out))
    _check("fa_fwd_fp8_quantized", rc)
    return out, lse


def fwd_fp8(q, k, v, causal: bool = False, scale: float | None = None, hadamard: bool = True,
            out=None, lse=None, workspace=None):
    """FP8 forward pass (quantise, then attention).  Returns (o, lse)."""
    B, H, N, d = q.shape
    scale = default_scale(d) if scale is None else float(scale)
    for name, t in (("q", q), ("k", k), ("v", v)):
        _check_qkv(name, t, (B, H, N, d))
    out = torch.empty_like(q) if out is None else out
    if lse is None:
        lse = torch.empty((B, H, N), dtype=torch.float32, device=q.device)
    _check_qkv("out", out, (B, H, N, d))
    _check_qkv("lse", lse, (B, H, N), torch.float32)
    workspace, nbytes = _fp8_workspace(workspace, B, H, N, d, q.device)
    with _on_device(q, k=k, v=v, out=out, lse=lse, workspace=workspace):
        rc = load().fa_fwd_fp8(q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(),
                               lse.data_ptr(), B, H, N, d, int(bool(causal)),
                               ctypes.c_float(scale), int(bool(hadamard)), workspace.data_ptr(),
                               nbytes, _stream_of(q))
    _check("fa_fwd_fp8", rc)
    return out, lse


def rope_table(length: int, rope_dim: int, base: float = 10000.0, device="cuda"):
    """The rotation table kv_append reads: (length, rope_dim) fp32, row p the
    cosines then the sines of the angles p * base**(-2i / rope_dim), computed
    in fp64.  Any other table of that layout serves as well."""
    half = rope_dim // 2
    freq = float(base) ** (-torch.arange(half, dtype=torch.float64, device=device) / half)
    angle = torch.arange(length, dtype=torch.float64, device=device)[:, None] * freq
    return torch.cat([angle.cos(), angle.sin()], 1).to(torch.float32)


# The paged-cache calls serve single tokens, where the call itself is what a
# step costs: they look at their tensors once, in one condition, and only a
# call that fails it finds out what is wrong (_refuse_call).
_BF16, _I32, _F32 = torch.bfloat16, torch.int32, torch.float32
# The arguments of fa_kv_append, fa_fwd_paged and fa_fwd_paged_prefix as words.
_APPEND_WORDS = struct.Struct("=10Q5q4q6qQ").pack
_PAGED_WORDS = struct.Struct("=8Q5qq5qdQQQ").pack
_PREFIX_WORDS = struct.Struct("=8QQq5qq5qdQQQ").pack
_current_device = torch.cuda.current_device
_current_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _refuse(name, t, shape, dtype, device):
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError("%s must be a CUDA tensor" % name)
    if t.get_device() != device:
        raise ValueError("%s is on %s, expected cuda:%d (one call's tensors must share a device)"
                         % (name, t.device, device))
    if t.dtype != dtype:
        raise ValueError("%s must be %s" % (name, dtype))
    if tuple(t.shape) != tuple(shape):
        raise ValueError("%s has shape %s, expected %s" % (name, tuple(t.shape), tuple(shape)))
    raise ValueError("%s must be contiguous" % name)


def _check_one(name, t, shape, dtype, device):
    if (not isinstance(t, torch.Tensor) or t.dtype is not dtype or t.get_device() != device
            or t.shape != shape or not t.is_contiguous()):
        _refuse(name, t, shape, dtype, device)


def _check_rows(name, t, T, H, d, device):
    if (not isinstance(t, torch.Tensor) or t.dtype is not _BF16 or t.get_device() != device
            or t.shape != (T, H, d)):
        _refuse(name, t, (T, H, d), _BF16, device)
    _, head, one = t.stride()
    if (one != 1 and d > 1) or (head != d and H > 1):
        raise ValueError("%s must have contiguous heads" % name)


def _refuse_call(name, lead, heads, rows, k_pages, v_pages, page_table, seq_lens, cu_q, others):
    """Raises what is wrong with a call of the paged cache.  lead: its first
    rows; heads: their number, None: the cache's; rows, others: more packed
    rows (name, tensor, heads) and contiguous tensors (name, tensor, shape,
    type)."""
    if not isinstance(lead, torch.Tensor) or not lead.is_cuda or lead.dim() != 3:
        raise ValueError("%s must be a CUDA tensor of shape (T, %s, d)" % (name, heads))
    dev, T = lead.get_device(), lead.shape[0]
    if not isinstance(k_pages, torch.Tensor) or k_pages.dim() != 4:
        raise ValueError("k_pages must have shape (num_pages, Hkv, page_size, d)")
    if not isinstance(page_table, torch.Tensor) or page_table.dim() != 2:
        raise ValueError("page_table must have shape (B, max_pages)")
    shape, (B, width) = k_pages.shape, page_table.shape
    _, Hkv, page_size, d = shape
    for n, t, s, dt in (("k_pages", k_pages, shape, _BF16), ("v_pages", v_pages, shape, _BF16),
                        ("page_table", page_table, (B, width), _I32),
                        ("seq_lens", seq_lens, (B,), _I32), ("cu_q", cu_q, (B + 1,), _I32)):
        _check_one(n, t, s, dt, dev)
    _check_rows(name, lead, T, Hkv if heads == "Hkv" else lead.shape[1], d, dev)
    for n, t, h in rows:
        if t is not None:
            if not isinstance(t, torch.Tensor) or t.dim() != 3:
                raise ValueError("%s must have shape (T, %s, d)" % (n, h or "Hq"))
            _check_rows(n, t, T, t.shape[1] if h is None else h, d, dev)
    for n, t, s, dt in others:
        if t is not None:
            if not isinstance(t, torch.Tensor) or t.dim() != len(s):
                raise ValueError("%s must have shape (%s)" % (n, ", ".join(map(str, s))))
            _check_one(n, t, tuple(t.shape[i] if isinstance(x, str) else x
                                   for i, x in enumerate(s)), dt, dev)
    raise ValueError("arguments of other types, shapes or devices than the call takes")


def kv_append(k, v, k_pages, v_pages, page_table, seq_lens, cu_q, q=None, q_out=None, rope=None,
              interleaved: bool = False):
    """Append packed rows k, v (T, Hkv, d) to the paged cache, rotating keys
    (and q, if given) by the table ``rope`` (see rope_table; None: no
    rotation).  Sequence b's rows are cu_q[b] .. cu_q[b+1]-1 and end at
    position seq_lens[b]-1.  Returns the rotated queries (``q_out``,
    allocated if not given; it may be ``q``), or None without q.  Rows of no
    sequence are left as they are; a ``q_out`` of the call's own is filled with
    zeros first, which for one token costs more than the call."""
    Hq = qs = qos = rope_len = rope_dim = 0
    q_ptr = q_out_ptr = rope_ptr = 0
    try:
        dev, pool, table = k.get_device(), k_pages.shape, page_table.shape
        num_pages, Hkv, page_size, d = pool
        B, width = table
        T = k.shape[0]
        rows = (T, Hkv, d)
        ks, head, one = k.stride()
        vs, vhead, vone = v.stride()
        ok = (dev >= 0 and k.shape == rows and v.shape == rows and v_pages.shape == pool
              and seq_lens.shape == (B,) and cu_q.shape == (B + 1,)
              and k.dtype is _BF16 and v.dtype is _BF16 and k_pages.dtype is _BF16
              and v_pages.dtype is _BF16 and page_table.dtype is _I32 and seq_lens.dtype is _I32
              and cu_q.dtype is _I32
              and v.get_device() == dev and k_pages.get_device() == dev
              and v_pages.get_device() == dev and page_table.get_device() == dev
              and seq_lens.get_device() == dev and cu_q.get_device() == dev
              and one == 1 and vone == 1 and (Hkv == 1 or head == vhead == d)
              and k_pages.is_contiguous() and v_pages.is_contiguous()
              and page_table.is_contiguous() and seq_lens.is_contiguous() and cu_q.is_contiguous())
        if ok and q is not None:
            Hq = q.shape[1]
            if q_out is None:  # rows of no sequence are not written
                q_out = torch.zeros((T, Hq, d), dtype=_BF16, device=q.device)
            rows = (T, Hq, d)
            qs, head, one = q.stride()
            qos, ohead, oone = q_out.stride()
            ok = (q.shape == rows and q_out.shape == rows and q.dtype is _BF16
                  and q_out.dtype is _BF16 and q.get_device() == dev and q_out.get_device() == dev
                  and one == 1 and oone == 1 and (Hq == 1 or head == ohead == d))
            q_ptr, q_out_ptr = q.data_ptr(), q_out.data_ptr()
        if ok and rope is not None:
            rope_len, rope_dim = rope.shape
            ok = rope.dtype is _F32 and rope.get_device() == dev and rope.is_contiguous()
            rope_ptr = rope.data_ptr()
    except (AttributeError, TypeError, ValueError, IndexError):
        ok = False
    if not ok:
        h = k_pages.shape[1] if getattr(k_pages, "ndim", 0) == 4 else "Hkv"
        _refuse_call("k", k, "Hkv", (("v", v, h), ("q", q, None),
                                     ("q_out", q_out, q.shape[1] if getattr(q, "ndim", 0) == 3
                                      else None)),
                     k_pages, v_pages, page_table, seq_lens, cu_q,
                     (("rope", rope, ("length", "rope_dim"), _F32),))
    if q is None and q_out is not None:
        raise ValueError("q_out needs q")
    if T == 1:  # a single row has any stride
        ks = vs = Hkv * d
        qs = qos = Hq * d
    if _current_device() != dev:
        with torch.cuda.device(dev):
            return kv_append(k, v, k_pages, v_pages, page_table, seq_lens, cu_q, q, q_out, rope,
                             interleaved)
    rc = (_lib or load()).fa_kv_append_words(_APPEND_WORDS(
        q_ptr, k.data_ptr(), v.data_ptr(), q_out_ptr, k_pages.data_ptr(), v_pages.data_ptr(),
        page_table.data_ptr(), seq_lens.data_ptr(), cu_q.data_ptr(), rope_ptr, T, B, Hq, Hkv, d,
        qs, ks, vs, qos, num_pages, page_size, width, rope_dim, rope_len,
        1 if interleaved else 0, _current_stream(dev)), 26)
    if rc != FA_OK:
        _check("fa_kv_append", rc)
    return q_out


@functools.lru_cache(maxsize=256)
def fwd_paged_workspace_size(T, B, Hq, Hkv, d, max_q, prefix_len=0) -> int:
    """Bytes of workspace for these sizes (0 where they are invalid)."""
    return int(load().fa_fwd_paged_workspace_size(T, B, Hq, Hkv, d, max_q, prefix_len))


def _fwd_paged(fn, q, k_pages, v_pages, page_table, seq_lens, cu_q, prefix_pages, max_q, causal,
               scale, out, lse, workspace):
    prefix_len, prefix = 0, ()
    try:
        dev, pool, table = q.get_device(), k_pages.shape, page_table.shape
        num_pages, Hkv, page_size, d = pool
        B, width = table
        T, Hq, _ = rows = q.shape
        qs, head, one = q.stride()
        ok = (dev >= 0 and rows[2] == d and v_pages.shape == pool
              and seq_lens.shape == (B,) and cu_q.shape == (B + 1,)
              and q.dtype is _BF16 and k_pages.dtype is _BF16 and v_pages.dtype is _BF16
              and page_table.dtype is _I32 and seq_lens.dtype is _I32 and cu_q.dtype is _I32
              and k_pages.get_device() == dev and v_pages.get_device() == dev
              and page_table.get_device() == dev and seq_lens.get_device() == dev
              and cu_q.get_device() == dev and one == 1 and (Hq == 1 or head == d)
              and k_pages.is_contiguous() and v_pages.is_contiguous()
              and page_table.is_contiguous() and seq_lens.is_contiguous() and cu_q.is_contiguous())
        if ok and out is None:  # rows of no sequence are not written
            out = torch.zeros(rows, dtype=_BF16, device=q.device)
        if ok and lse is None:
            lse = torch.full((T, Hq), -math.inf, dtype=_F32, device=q.device)
        ok = (ok and out.shape == rows and out.dtype is _BF16 and out.get_device() == dev
              and out.is_contiguous() and lse.shape == (T, Hq) and lse.dtype is _F32
              and lse.get_device() == dev and lse.is_contiguous())
        if prefix_pages is not None:
            n, = prefix_pages.shape
            prefix_len = n * page_size
            prefix = prefix_pages.data_ptr(), prefix_len
            ok = (ok and prefix_pages.dtype is _I32 and prefix_pages.get_device() == dev
                  and prefix_pages.is_contiguous())
    except (AttributeError, TypeError, ValueError, IndexError):
        ok = False
    if not ok:
        shape = q.shape if getattr(q, "ndim", 0) == 3 else ("T", "Hq", "d")
        _refuse_call("q", q, "Hq", (), k_pages, v_pages, page_table, seq_lens, cu_q,
                     (("out", out, tuple(shape), _BF16), ("lse", lse, tuple(shape[:2]), _F32),
                      ("prefix_pages", prefix_pages, ("pages",), _I32)))
    if workspace is not None and (not isinstance(workspace, torch.Tensor)
                                  or workspace.get_device() != dev
                                  or not workspace.is_contiguous()):
        _refuse("workspace", workspace, getattr(workspace, "shape", ()),
                getattr(workspace, "dtype", None), dev)
    if T == 1:  # a single row has any stride
        qs = Hq * d
    scale = d ** -0.5 if scale is None else float(scale)
    max_q = T if max_q is None else int(max_q)
    if _current_device() != dev:
        with torch.cuda.device(dev):
            return _fwd_paged(fn, q, k_pages, v_pages, page_table, seq_lens, cu_q, prefix_pages,
                              max_q, causal, scale, out, lse, workspace)
    lib, stream = _lib or load(), _current_stream(dev)
    if workspace is None:
        # From torch's allocator without a tensor around it, which costs more
        # than a single-token call's launch; it is the stream's again as soon
        # as the call is enqueued.
        ws_bytes = fwd_paged_workspace_size(T, B, Hq, Hkv, d, max_q, prefix_len)
        ws = torch._C._cuda_cudaCachingAllocator_raw_alloc(max(ws_bytes, 1), stream)
    else:
        ws, ws_bytes = workspace.data_ptr(), workspace.numel() * workspace.element_size()
    try:
        rc = lib.fa_fwd_paged_words((_PREFIX_WORDS if prefix else _PAGED_WORDS)(
            q.data_ptr(), k_pages.data_ptr(), v_pages.data_ptr(), out.data_ptr(), lse.data_ptr(),
            page_table.data_ptr(), seq_lens.data_ptr(), cu_q.data_ptr(), *prefix, T, B, Hq, Hkv, d,
            qs, num_pages, page_size, width, max_q, 1 if causal else 0, scale, ws, ws_bytes,
            stream), 25 if prefix else 23)
    finally:
        if workspace is None:
            torch._C._cuda_cudaCachingAllocator_raw_delete(ws)
    if rc != FA_OK:
        _check(fn, rc)
    return out, lse


def fwd_paged(q, k_pages, v_pages, page_table, seq_lens, cu_q, max_q=None, causal: bool = True,
              scale: float | None = None, out=None, lse=None, workspace=None):
    """Attention of packed query rows q (T, Hq, d) over the paged cache: the
    rows of sequence b are its last cu_q[b+1] - cu_q[b] positions of
    seq_lens[b].  ``max_q``: the most rows of a sequence (None: T), which
    decides the kernel and never the result.  Returns (o, lse), (T, Hq, d)
    and (T, Hq).  Rows of no sequence are left as they are; outputs that are not
    given are filled with 0 and -inf first, which for one token costs more than
    the call."""
    return _fwd_paged("fa_fwd_paged", q, k_pages, v_pages, page_table, seq_lens, cu_q, None,
                      max_q, causal, scale, out, lse, workspace)


def fwd_paged_prefix(q, k_pages, v_pages, page_table, seq_lens, cu_q, prefix_pages, max_q=None,
                     causal: bool = True, scale: float | None = None, out=None, lse=None,
                     workspace=None):
    """fwd_paged for a batch whose sequences all begin with the keys of
    ``prefix_pages`` (int32, in order), whose attention is computed once for
    all rows.  Lengths and positions count the prefix.  Returns (o, lse)."""
    if prefix_pages is None:  # (fwd_paged is the call without a prefix)
        raise ValueError("prefix_pages must be a CUDA tensor of shape (pages,)")
    return _fwd_paged("fa_fwd_paged_prefix", q, k_pages, v_pages, page_table, seq_lens, cu_q,
                      prefix_pages, max_q, causal, scale, out, lse, workspace)


def device_status(stream=None):
    """Synchronise the stream; return (code, site) and clear the status word."""
    s = ctypes.c_void_p(torch.cuda.current_stream().cuda_stream if stream is None else stream)
    site = ctypes.c_int(0)
    code = load().fa_device_status(s, ctypes.byref(site))
    return int(code), int(site.value)


FA_SITE_SELFTEST = 901


def selftest_timeout(timeout_us: int = 20000):
    """Launch the failure-detection self test on the current stream (see
    fa_selftest_timeout); read the result with device_status()."""
    s = ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)
    _check("fa_selftest_timeout", load().fa_selftest_timeout(int(timeout_us), s))


FA_SITE_SELFTEST_BOUNDS = 902


def checks_enabled() -> bool:
    """True for the bounds-checked build of the library."""
    return bool(load().fa_checks_enabled())


def selftest_bounds():
    """Launch the bounds-check self test on the current stream (see
    fa_selftest_bounds); read the result with device_status()."""
    s = ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)
    _check("fa_selftest_bounds", load().fa_selftest_bounds(s))


def check_device_status(stream=None):
    code, site = device_status(stream)
    if code != FA_OK:
        raise FaError("kernel", code, status_string(code) + " (site %d)" % site)


def fwd_schedule(B: int, H: int, N: int, causal: bool, num_ctas: int = 152):
    """The forward kernel's work list: (bh, pair, cost, cta) per item, in list order
    (cta -1: claimed from the work counter at run time)."""
    lib = load()
    n = lib.fa_fwd_schedule(B, H, N, int(bool(causal)), int(num_ctas), None, None, None, None, 0)
    if n < 0:
        _check("fa_fwd_schedule", n)
    bh = (ctypes.c_int * n)()
    pr = (ctypes.c_int * n)()
    cost = (ctypes.c_int * n)()
    cta = (ctypes.c_int * n)()
    lib.fa_fwd_schedule(B, H, N, int(bool(causal)), int(num_ctas), bh, pr, cost, cta, n)
    return list(zip(bh, pr, cost, cta))


def snake_assign(n: int, workers: int):
    """The kernels' static assignment of n listed items to persistent workers."""
    out = (ctypes.c_int * max(n, 1))()
    _check("fa_snake_assign", load().fa_snake_assign(int(n), int(workers), out))
    return list(out)[:n]
