"""GB300-native Ulysses DiT attention: thin Python binding over the ``libuaa.so`` C ABI.

Every step of the computation runs in the library's sm_103a kernels; this module
only marshals arguments (shapes, dtypes, pointers, the current CUDA stream) and
allocates outputs/workspace with PyTorch.  There is no CPU or eager fallback: if
the library is not built, or the tensors are not on a CUDA device, calls raise.

Names follow the C ABI (``include/uaa.h``): ``attn_fwd``, ``attn_bwd``,
``seq_to_head``, ``head_to_seq``, ``assemble_key_mask``; ``Attention`` is the
``torch.autograd.Function`` pairing them (the LSE output is marked
non-differentiable, as in "[attention] Add Ulysses Anything backward", What does
this PR do), and ``ulysses_attention`` composes the Ulysses exchange around it
for P emulated ranks on one device.
"""
from __future__ import annotations

import array
import ctypes
import math
import os
import struct
import threading

import torch

from .build import DEBUG_LIB_PATH, LIB_PATH

__all__ = [
    "UAAError", "lib", "attn_fwd", "attn_bwd", "attn_bwd_workspace_bytes", "attn_bwd_fused_workspace_bytes", "seq_to_head", "head_to_seq",
    "assemble_key_mask", "check_device_status", "watchdog_selftest", "set_wait_timeout_ms", "debug_drop_load",
    "debug_late_warp", "debug_fail_launch",
    "set_bwd_profile_events", "Attention", "attn_fwd_groups", "attn_bwd_groups",
    "attention", "UlyssesAttention", "ulysses_attention", "STATUS", "debug_build", "debug_exp2_fma2",
    "RotaryPlan", "rotary_fwd", "rotary_bwd", "Rotary", "rotary", "shard_positions", "Act8", "act8_pack", "act8_unpack",
    "attn_bwd_act8",
    "diff_attn_fwd", "diff_attn_bwd", "diff_attn_bwd_workspace_bytes", "DiffAttention", "diff_attention",
    "attn_packed_fwd", "attn_packed_bwd", "attn_packed_bwd_workspace_bytes", "attn_seqs_workspace_bytes",
    "PackedAttention", "packed_attention", "attn_paged_fwd", "cache_write", "PagedCache",
]

STATUS = {0: "UAA_OK", -1: "UAA_ERR_INVALID_ARG", -2: "UAA_ERR_UNSUPPORTED", -3: "UAA_ERR_PER_HEAD_MASK",
          -4: "UAA_ERR_CUDA", -5: "UAA_ERR_TIMEOUT", -6: "UAA_ERR_DEBUG_CHECK", -7: "UAA_ERR_NO_PAGES",
          -8: "UAA_ERR_BAD_PAGE"}


class UAAError(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__(f"{STATUS.get(status, status)}: {message}")
        self.status = status


_lib = None
_lib_lock = threading.Lock()

_P = ctypes.c_void_p
_I = ctypes.c_int
_L = ctypes.c_longlong


class _RotaryPlan(ctypes.Structure):  # uaa_rotary_plan
    _fields_ = [("rot", _I), ("layout", _I), ("axes", _I), ("magnitude", ctypes.c_float),
                ("turns", ctypes.c_uint64 * 128), ("axis", ctypes.c_uint8 * 128)]


# uaa_rotary_tensor, as bytes: x, y, their batch, token and head strides, H
_ROTARY_TENSOR = struct.Struct("@PP6qi0q")

# uaa_seqs, uaa_pools and uaa_cache_rows, as bytes
_SEQS = struct.Struct("@10P8q13if0q")
_POOLS = struct.Struct("@4P2i0q")
_CACHE_ROWS = struct.Struct("@8P10q8i0q")

_SIGS = {
    "uaa_attn_seqs_workspace_bytes": (ctypes.c_size_t, [_I, _I, _I, _I, _I]),
    "uaa_attn_packed_fwd": (_I, [_P, _P, ctypes.c_size_t, _P]),
    "uaa_attn_paged_fwd": (_I, [_P, _P, ctypes.c_size_t, _P]),
    "uaa_attn_packed_bwd_workspace_bytes": (ctypes.c_size_t, [_I, _I, _I, _I, _I]),
    "uaa_attn_packed_bwd": (_I, [_P, _P, _P, _P, _P, _P, ctypes.c_size_t, _P]),
    "uaa_pages_create": (_I, [ctypes.POINTER(_P), _I, _I, _I, _I]),
    "uaa_pages_destroy": (None, [_P]),
    "uaa_pages_append": (_I, [_P, _P, _I, _P, _P, _P, _P, _P]),
    "uaa_pages_fork": (_I, [_P, _P, _I, _P, _P, _P]),
    "uaa_pages_truncate": (_I, [_P, _P, _I, _P, _P, _P]),
    "uaa_pages_compact": (_I, [_P, _P, _P]),
    "uaa_pages_row": (_I, [_P, _I, _P, _I]),
    "uaa_pages_free": (_I, [_P]),
    "uaa_cache_write": (_I, [_P, _P]),
    "uaa_rotary_plan_init": (_I, [ctypes.POINTER(_RotaryPlan), _I, _I, _P, ctypes.c_double, _I, ctypes.c_double,
                                  ctypes.c_double, ctypes.c_double, ctypes.c_double]),
    "uaa_rotary": (_I, [ctypes.POINTER(_RotaryPlan), _P, _P, _P,
                        _I, _L, _L, _L, _I, _I, _I, _I, _I, _P]),
    "uaa_attn_bwd_act8_workspace_bytes": (ctypes.c_size_t, [_I, _I, _I, _I, _I]),
    "uaa_attn_bwd_act8": (_I, [_P, _P, _P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I, ctypes.c_float, _P, ctypes.c_size_t,
                               _P]),
    "uaa_act8_pack": (_I, [_I, _P, _P, _P, _P, _I, _I, _P]),
    "uaa_act8_unpack": (_I, [_I, _P, _P, _P, _P, _I, _I, _P]),
    "uaa_diff_attn_fwd": (_I, [_P, _P, _P, _P, _I, _P, _P, _P, _P, _I, _I, _I, _I, _I, ctypes.c_float, _P]),
    "uaa_diff_attn_bwd_workspace_bytes": (ctypes.c_size_t, [_I, _I, _I, _I, _I]),
    "uaa_diff_attn_bwd": (_I, [_P, _P, _P, _P, _I, _P, _P, _P, _P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I,
                               ctypes.c_float, _P, ctypes.c_size_t, _P]),
    "uaa_attn_fwd": (_I, [_P, _P, _P, _P, _P, _P, _I, _I, _I, _I, ctypes.c_float, _P]),
    "uaa_attn_fwd_cross": (_I, [_P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I, ctypes.c_float, _P]),
    "uaa_attn_bwd_workspace_bytes": (ctypes.c_size_t, [_I, _I, _I, _I]),
    "uaa_attn_bwd": (_I, [_P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _I, _I, _I, _I, ctypes.c_float, _P,
                          ctypes.c_size_t, _P]),
    "uaa_attn_bwd_cross": (_I, [_P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I, ctypes.c_float, _P,
                                ctypes.c_size_t, _P]),
    "uaa_attn_bwd_fused_workspace_bytes": (ctypes.c_size_t, [_I, _I, _I, _I]),
    "uaa_attn_bwd_fused": (_I, [_P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _I, _I, _I, _I, ctypes.c_float, _P,
                                ctypes.c_size_t, _P]),
    "uaa_attn_fwd_groups": (_I, [_P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I, ctypes.c_float, _P]),
    "uaa_attn_bwd_groups": (_I, [_P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I, ctypes.c_float, _P,
                                 ctypes.c_size_t, _P]),
    "uaa_attn_bwd_noalloc": (_I, [_P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _I, _I, _I, _I, ctypes.c_float, _P]),
    "uaa_attn_bwd_noalloc_max_bytes": (ctypes.c_size_t, []),
    "uaa_ulysses_attn_fwd": (_I, [_P, _P, _P, _P, _P, _P, _I, _P, _I, _I, _I, _I, ctypes.c_float, _P]),
    "uaa_ulysses_attn_bwd_workspace_bytes": (ctypes.c_size_t, [_I, _P, _I, _I, _I, _I]),
    "uaa_ulysses_attn_bwd": (_I, [_P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _I, _P, _I, _I, _I, _I, ctypes.c_float,
                                  _P, ctypes.c_size_t, _P]),
    "uaa_seq_to_head": (_I, [_P, _P, _I, _P, _I, _I, _I, _I, _I, _P]),
    "uaa_head_to_seq": (_I, [_P, _P, _I, _P, _I, _I, _I, _I, _I, _P]),
    "uaa_assemble_key_mask": (_I, [_P, _P, _I, _P, _I, _I, _P]),
    "uaa_check_device_status": (_I, [_P]),
    "uaa_watchdog_selftest": (_I, [ctypes.c_uint, _P]),
    "uaa_set_wait_timeout_ms": (None, [ctypes.c_uint]),
    "uaa_debug_drop_load": (None, [_I]),
    "uaa_debug_fail_launch": (None, [_I]),
    "uaa_debug_late_warp": (_I, [_I, ctypes.c_uint]),
    "uaa_set_bwd_profile_events": (None, [_P, _P, _P]),
    "uaa_last_error": (ctypes.c_char_p, []),
    "uaa_version": (ctypes.c_char_p, []),
    "uaa_debug_build": (_I, []),
    "uaa_debug_exp2_fma2": (_I, [_P, _P, ctypes.c_longlong, _P]),
}


def lib():
    """Load ``libuaa.so`` (once; ``libuaa_debug.so``, the build with device range checks,
    when the environment sets ``UAA_DEBUG=1``).  Raises if it has not been built."""
    global _lib
    if _lib is None:
        with _lib_lock:
            if _lib is None:
                debug = os.environ.get("UAA_DEBUG", "") == "1"
                path = DEBUG_LIB_PATH if debug else LIB_PATH
                if not os.path.exists(path):
                    how = "--debug " if debug else ""
                    raise RuntimeError(f"{path} is missing: build it with "
                                       f"`python -m ulysses_dit_attention_gb300.build {how}` (no fallback exists)")
                handle = ctypes.CDLL(path)
                for name, (res, args) in _SIGS.items():
                    fn = getattr(handle, name)
                    fn.restype = res
                    fn.argtypes = args
                _lib = handle
    return _lib


def _check(status: int):
    if status != 0:
        raise UAAError(status, lib().uaa_last_error().decode(errors="replace"))


def _stream(device) -> int:
    index = torch.device(device).index
    return torch._C._cuda_getCurrentRawStream(torch.cuda.current_device() if index is None else index)


def _ptr(t):
    return None if t is None else t.data_ptr()


def _need_cuda(*ts):
    for t in ts:
        if t is not None and not t.is_cuda:
            raise ValueError("uaa kernels run on CUDA tensors only (no CPU fallback)")


def _bshd(name, t, ref=None, same_s=True):
    if t.dim() != 4:
        raise ValueError(f"{name} must be (B, S, H, D), got {tuple(t.shape)}")
    if t.dtype != torch.bfloat16:
        raise TypeError(f"{name} must be bfloat16")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous BSHD")
    if ref is not None:
        a, b = tuple(t.shape), tuple(ref.shape)
        if (a != b) if same_s else (a[0] != b[0] or a[2:] != b[2:]):
            raise ValueError(f"{name} shape {a} does not fit {b}")


def normalize_key_mask(mask, B, S):
    """Key mask -> contiguous uint8 ``(B, S)``.

    Accepts ``(B, S)`` or the head-broadcast ``(B, 1, 1, S)`` form; a per-head
    ``(B, H>1, 1, S)`` mask raises ``ValueError`` before any launch ("[attention]
    Add Ulysses Anything backward", What does this PR do: fail fast on per-head
    masks, which Ulysses cannot shard).  A bool mask is reinterpreted as bytes
    (no copy kernel).
    """
    if mask is None:
        return None
    if mask.dim() == 4:
        if mask.shape[1] != 1 or mask.shape[2] != 1:
            raise ValueError(f"per-head attention masks {tuple(mask.shape)} are not supported: only "
                             "head-broadcast (B, 1, 1, S) key masks can be sharded across heads")
        mask = mask.reshape(mask.shape[0], mask.shape[3])
    if mask.dim() != 2 or tuple(mask.shape) != (B, S):
        raise ValueError(f"key mask must be (B, S) = {(B, S)}, got {tuple(mask.shape)}")
    if mask.dtype == torch.bool:
        mask = mask.view(torch.uint8)
    if mask.dtype != torch.uint8:
        raise TypeError("key mask must be bool or uint8")
    if not mask.is_contiguous():
        raise ValueError("key mask must be contiguous")
    return mask


# --------------------------------------------------------------------------- attention
def attn_fwd(q, k, v, key_mask=None, scale=None, out=None, lse=None):
    """``uaa_attn_fwd`` / ``uaa_attn_fwd_cross``: returns ``(out bf16 (B,Sq,H,D), lse fp32 (B,H,Sq))``.

    ``k`` and ``v`` may have another sequence length ``Sk`` than ``q`` (cross-attention);
    ``key_mask`` is then ``(B, Sk)``.
    """
    _bshd("q", q)
    _bshd("k", k, q, same_s=False)
    _bshd("v", v, k)
    _need_cuda(q, k, v)
    B, Sq, H, D = q.shape
    Sk = k.shape[1]
    mask = normalize_key_mask(key_mask, B, Sk)
    if scale is None:
        scale = 1.0 / math.sqrt(D)
    if out is None:
        out = torch.empty_like(q)
    if lse is None:
        lse = torch.empty((B, H, Sq), dtype=torch.float32, device=q.device)
    if Sq == Sk:
        _check(lib().uaa_attn_fwd(_ptr(q), _ptr(k), _ptr(v), _ptr(mask), _ptr(out), _ptr(lse), B, Sq, H, D,
                                  float(scale), _P(_stream(q.device))))
    else:
        _check(lib().uaa_attn_fwd_cross(_ptr(q), _ptr(k), _ptr(v), _ptr(mask), _ptr(out), _ptr(lse), B, Sq, Sk, H,
                                        D, float(scale), _P(_stream(q.device))))
    return out, lse


def attn_bwd_workspace_bytes(B, S, H, D) -> int:
    return int(lib().uaa_attn_bwd_workspace_bytes(B, S, H, D))


def attn_bwd_fused_workspace_bytes(B, S, H, D) -> int:
    return int(lib().uaa_attn_bwd_fused_workspace_bytes(B, S, H, D))


def attn_bwd(q, k, v, out, dout, lse, key_mask=None, scale=None, dq=None, dk=None, dv=None, workspace=None,
             fused=False):
    """``uaa_attn_bwd`` / ``uaa_attn_bwd_cross``: returns ``(dq, dk, dv)`` in bf16 BSHD.

    ``k``, ``v`` (and ``dk``, ``dv``) may have another sequence length than ``q``.  With
    ``fused=True`` (same sequence lengths only) the one-pass ``uaa_attn_bwd_fused`` runs
    instead: five GEMMs instead of seven, dQ by fp32 reductions, so dQ is not bit-for-bit
    reproducible.
    """
    _bshd("q", q)
    _bshd("k", k, q, same_s=False)
    _bshd("v", v, k)
    _bshd("out", out, q)
    _bshd("dout", dout, q)
    _need_cuda(q, k, v, out, dout, lse)
    B, Sq, H, D = q.shape
    Sk = k.shape[1]
    if lse.dtype != torch.float32 or tuple(lse.shape) != (B, H, Sq) or not lse.is_contiguous():
        raise ValueError("lse must be contiguous fp32 (B, H, Sq)")
    mask = normalize_key_mask(key_mask, B, Sk)
    if scale is None:
        scale = 1.0 / math.sqrt(D)
    dq = torch.empty_like(q) if dq is None else dq
    dk = torch.empty_like(k) if dk is None else dk
    dv = torch.empty_like(k) if dv is None else dv
    if fused and Sq != Sk:
        raise ValueError("the fused backward takes equal query and key lengths")
    nbytes = attn_bwd_fused_workspace_bytes(B, Sq, H, D) if fused else attn_bwd_workspace_bytes(B, Sq, H, D)
    if workspace is None:
        workspace = torch.empty(max(nbytes, 1), dtype=torch.uint8, device=q.device)
    wsb = workspace.numel() * workspace.element_size()
    if fused:
        _check(lib().uaa_attn_bwd_fused(_ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(dout), _ptr(lse), _ptr(mask),
                                        _ptr(dq), _ptr(dk), _ptr(dv), B, Sq, H, D, float(scale), _ptr(workspace), wsb,
                                        _P(_stream(q.device))))
    elif Sq == Sk:
        _check(lib().uaa_attn_bwd(_ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(dout), _ptr(lse), _ptr(mask),
                                  _ptr(dq), _ptr(dk), _ptr(dv), B, Sq, H, D, float(scale), _ptr(workspace), wsb,
                                  _P(_stream(q.device))))
    else:
        _check(lib().uaa_attn_bwd_cross(_ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(dout), _ptr(lse), _ptr(mask),
                                        _ptr(dq), _ptr(dk), _ptr(dv), B, Sq, Sk, H, D, float(scale),
                                        _ptr(workspace), wsb, _P(_stream(q.device))))
    return dq, dk, dv


def _groups(name, t, ref=None):
    if t.dim() != 5:
        raise ValueError(f"{name} must be (G, B, S, H, D), got {tuple(t.shape)}")
    if t.dtype != torch.bfloat16:
        raise TypeError(f"{name} must be bfloat16")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous (G, B, S, H, D)")
    if ref is not None and tuple(t.shape) != tuple(ref.shape):
        raise ValueError(f"{name} shape {tuple(t.shape)} does not fit {tuple(ref.shape)}")


def attn_fwd_groups(q, k, v, key_mask=None, scale=None, out=None, lse=None):
    """``uaa_attn_fwd_groups``: attention of G head groups ``(G, B, S, H, D)`` in one launch.

    The ``(B, S)`` key mask is shared by the G groups.  Returns ``(out, lse)`` with ``lse``
    fp32 ``(G, B, H, S)``.
    """
    _groups("q", q)
    _groups("k", k, q)
    _groups("v", v, q)
    _need_cuda(q, k, v)
    G, B, S, H, D = q.shape
    mask = normalize_key_mask(key_mask, B, S)
    if scale is None:
        scale = 1.0 / math.sqrt(D)
    if out is None:
        out = torch.empty_like(q)
    if lse is None:
        lse = torch.empty((G, B, H, S), dtype=torch.float32, device=q.device)
    _check(lib().uaa_attn_fwd_groups(_ptr(q), _ptr(k), _ptr(v), _ptr(mask), _ptr(out), _ptr(lse), G, B, S, H, D,
                                     float(scale), _P(_stream(q.device))))
    return out, lse


def attn_bwd_groups(q, k, v, out, dout, lse, key_mask=None, scale=None, dq=None, dk=None, dv=None, workspace=None):
    """``uaa_attn_bwd_groups``: the backward of :func:`attn_fwd_groups`; returns ``(dq, dk, dv)``."""
    for n, t in (("k", k), ("v", v), ("out", out), ("dout", dout)):
        _groups(n, t, q)
    _groups("q", q)
    _need_cuda(q, k, v, out, dout, lse)
    G, B, S, H, D = q.shape
    if lse.dtype != torch.float32 or tuple(lse.shape) != (G, B, H, S) or not lse.is_contiguous():
        raise ValueError("lse must be contiguous fp32 (G, B, H, S)")
    mask = normalize_key_mask(key_mask, B, S)
    if scale is None:
        scale = 1.0 / math.sqrt(D)
    dq = torch.empty_like(q) if dq is None else dq
    dk = torch.empty_like(q) if dk is None else dk
    dv = torch.empty_like(q) if dv is None else dv
    nbytes = attn_bwd_workspace_bytes(G * B, S, H, D)
    if workspace is None:
        workspace = torch.empty(max(nbytes, 1), dtype=torch.uint8, device=q.device)
    wsb = workspace.numel() * workspace.element_size()
    _check(lib().uaa_attn_bwd_groups(_ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(dout), _ptr(lse), _ptr(mask),
                                     _ptr(dq), _ptr(dk), _ptr(dv), G, B, S, H, D, float(scale), _ptr(workspace), wsb,
                                     _P(_stream(q.device))))
    return dq, dk, dv


def _check_saved(saved):
    if saved not in (None, "int8"):
        raise ValueError(f"saved must be None or 'int8', got {saved!r}")


def _save(ctx, saved, tensors, *others, key_mask):
    """Keeps ``tensors`` for the backward pass, as they are or (``saved="int8"``) as an 8-bit checkpoint, and the key
    mask among the saved tensors, so that a change to it between the passes raises.  (A mask made in inference mode has
    no versions and cannot be saved: it stays on ``ctx``.)"""
    ctx.packed = None
    if saved == "int8" and any(ctx.needs_input_grad):
        packed = act8_pack(tensors)
        ctx.packed = packed._meta()
        tensors = (packed.data,)
    ctx.held_mask = key_mask if key_mask is not None and key_mask.is_inference() else None
    ctx.save_for_backward(*tensors, *others, None if ctx.held_mask is not None else key_mask)


def _kept(ctx):
    """What :func:`_save` kept: the tensors or their checkpoint's buffer, the others, and the key mask."""
    *kept, key_mask = ctx.saved_tensors
    return kept, key_mask if ctx.held_mask is None else ctx.held_mask


def _saved(ctx, n):
    """The ``n`` tensors that :func:`_save` kept, the others, and the key mask."""
    kept, key_mask = _kept(ctx)
    if ctx.packed is None:
        return kept[:n], kept[n:], key_mask
    return act8_unpack(Act8(kept[0], *ctx.packed)), kept[1:], key_mask


class Attention(torch.autograd.Function):
    """Autograd pairing of ``attn_fwd`` / ``attn_bwd``; ``lse`` is non-differentiable.

    ``saved="int8"`` keeps Q, K, V and O for the backward pass as an 8-bit checkpoint
    (:func:`act8_pack`): half the memory, gradients of the values that the codes stand for."""

    @staticmethod
    def forward(ctx, q, k, v, key_mask=None, scale=None, saved=None):
        _check_saved(saved)
        out, lse = attn_fwd(q, k, v, key_mask, scale)
        _save(ctx, saved, (q, k, v, out), lse, key_mask=key_mask)
        ctx.scale = scale
        ctx.mark_non_differentiable(lse)
        ctx.set_materialize_grads(False)  # no zeros for lse
        return out, lse

    @staticmethod
    def backward(ctx, dout, _dlse):
        if dout is None:
            return None, None, None, None, None, None
        kept, key_mask = _kept(ctx)
        if ctx.packed is not None:
            data, lse = kept
            grads = attn_bwd_act8(Act8(data, *ctx.packed), dout.contiguous(), lse, key_mask, ctx.scale)
        else:
            q, k, v, out, lse = kept
            grads = attn_bwd(q, k, v, out, dout.contiguous(), lse, key_mask, ctx.scale)
        return *grads, None, None, None


def attention(q, k, v, key_mask=None, scale=None, saved=None):
    return Attention.apply(q, k, v, key_mask, scale, saved)


# --------------------------------------------------------------------------- shared checks of the calls below
_DTYPES = {torch.bfloat16: 0, torch.float16: 1, torch.float32: 2}


def _same_device(*ts):
    first = None
    for t in ts:
        if t is None:
            continue
        if first is None:
            first = t.device
            if first.type != "cuda":
                raise ValueError("uaa kernels run on CUDA tensors only (no CPU fallback)")
        elif t.device != first:
            raise ValueError(f"tensors are on {first} and {t.device}: uaa kernels run on CUDA tensors of one device")
    return first


def _call(device, name, *args):
    """Calls the library on the tensors' device, on its current stream."""
    i = device.index
    fn = getattr(_lib or lib(), name)
    if i == torch._C._cuda_getDevice():
        st = fn(*args, torch._C._cuda_getCurrentRawStream(i))
    else:
        with torch.cuda.device(device):
            st = fn(*args, torch._C._cuda_getCurrentRawStream(i))
    if st != 0:
        _check(st)


def _result(name, t, shape, dtype, device):
    """An output of the caller's, checked, or a new one."""
    if t is None:
        return torch.empty(shape, dtype=dtype, device=device)
    if tuple(t.shape) != tuple(shape) or t.dtype != dtype or t.device != device or not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous {dtype} {tuple(shape)} on {device}")
    return t


# --------------------------------------------------------------------------- rotary positions
class RotaryPlan:
    """The frequencies of a rotary position code (``uaa_rotary_plan``), made once and kept by the model.

    ``widths``: rotated columns of a head per position axis -- ``[128]`` for one axis, ``[44, 42, 42]``
    for frame, row and column; the columns behind them are copied.  ``layout``: ``"half"`` pairs column
    ``i`` with ``i + R/2`` (``R = sum(widths)``), ``"interleaved"`` pairs ``2i`` with ``2i + 1``.
    ``scaling`` for contexts longer than the trained one: ``"linear"`` divides every frequency by
    ``factor``; ``"ntk"`` raises the base; ``"parts"`` keeps pairs that turn more than ``beta`` times over
    ``original`` positions, divides those below ``alpha`` by ``factor``, blends between, and multiplies
    the result by ``0.1 ln(factor) + 1``.
    """

    LAYOUTS = {"half": 0, "interleaved": 1}
    SCALINGS = {"none": 0, "linear": 1, "ntk": 2, "parts": 3}

    def __init__(self, widths, layout="half", base=10000.0, scaling="none", factor=1.0, original=8192, alpha=1.0,
                 beta=32.0):
        widths = [int(w) for w in ([widths] if isinstance(widths, int) else widths)]
        if layout not in self.LAYOUTS:
            raise ValueError(f"layout must be one of {sorted(self.LAYOUTS)}, got {layout!r}")
        if scaling not in self.SCALINGS:
            raise ValueError(f"scaling must be one of {sorted(self.SCALINGS)}, got {scaling!r}")
        self._c = _RotaryPlan()
        _check(lib().uaa_rotary_plan_init(ctypes.byref(self._c), self.LAYOUTS[layout], len(widths),
                                          (ctypes.c_int * len(widths))(*widths), float(base), self.SCALINGS[scaling],
                                          float(factor), float(original), float(alpha), float(beta)))
        self._bind()

    def _bind(self):
        self._ref = ctypes.byref(self._c)
        self.axes, self.rot, self.magnitude = self._c.axes, self._c.rot, self._c.magnitude

    def __getstate__(self):  # for copies and pickles
        return bytes(self._c)

    def __setstate__(self, state):
        self._c = _RotaryPlan.from_buffer_copy(state)
        self._bind()

    @property
    def turns(self):
        """Turns per position of each pair, as numbers below 1."""
        return [self._c.turns[i] / 2.0 ** 64 for i in range(self.rot // 2)]


def shard_positions(shard_lens, cap, B, device, dtype=torch.int32):
    """Positions ``(P*B, cap)`` of the rows of ``(P, B, cap, H, D)`` shards seen as ``(P*B, cap, H, D)``: row s of
    shard p stands at ``sum(shard_lens[:p]) + s`` (padding rows run on)."""
    starts = torch.tensor([sum(shard_lens[:p]) for p in range(len(shard_lens))], dtype=dtype)
    at = starts[:, None, None] + torch.arange(cap, dtype=dtype)
    return at.expand(len(shard_lens), B, cap).reshape(len(shard_lens) * B, cap).contiguous().to(device)


def _rotary_operand(name, t, ref, out):
    """Checks an operand and its result; returns the library's view of both, and the result."""
    shape, dtype = t.shape, t.dtype
    if len(shape) != 4:
        raise ValueError(f"{name} must be (B, S, H, D), got {tuple(shape)}")
    if dtype not in _DTYPES or dtype != ref.dtype:
        raise TypeError(f"{name} must be bfloat16, float16 or float32, q and k alike")
    if t is not ref and (shape[:2] != ref.shape[:2] or shape[3] != ref.shape[3]):
        raise ValueError(f"{name} shape {tuple(shape)} does not fit {tuple(ref.shape)}")
    x0, x1, x2, x3 = t.stride()
    if x3 != 1 and shape[3] > 1:
        raise ValueError(f"the columns of {name} must be contiguous")
    if out is None:
        out = torch.empty(shape, dtype=dtype, device=t.device)
    elif out.shape != shape or out.dtype != dtype or out.device != t.device or (shape[3] > 1 and out.stride(3) != 1):
        raise ValueError(f"out_{name} must be {dtype} {tuple(shape)} on {t.device} with contiguous columns")
    y0, y1, y2, _ = out.stride()
    return _ROTARY_TENSOR.pack(t.data_ptr(), out.data_ptr(), x0, x1, x2, y0, y1, y2, shape[2]), out


def _rotate(q, k, plan, positions, start, inverse, out_q, out_k):
    if not isinstance(plan, RotaryPlan):
        raise TypeError("plan must be a RotaryPlan")
    dev = _same_device(q, k, positions)
    tq, out_q = _rotary_operand("q", q, q, out_q)
    tk = None
    if k is not None:
        tk, out_k = _rotary_operand("k", k, q, out_k)
    B, S, _, D = q.shape
    pos, wide, pb, ps = None, 0, 0, 0
    if positions is not None:
        if start:
            raise ValueError("start goes with positions=None")
        axes, at, dtype = plan.axes, positions.stride(), positions.dtype
        tail = () if axes == 1 else (axes,)
        if positions.shape == (B, S) + tail:
            pb, ps = at[0], at[1]
        elif positions.shape == (S,) + tail:
            ps = at[0]
        else:
            raise ValueError(f"positions must be {(S,) + tail} or {(B, S) + tail}, got {tuple(positions.shape)}")
        if dtype == torch.int64:
            wide = 1
        elif dtype != torch.int32:
            raise TypeError("positions must be int32 or int64")
        if axes > 1 and at[-1] != 1:
            raise ValueError("the axes of positions must be contiguous")
        pos = positions.data_ptr()
    _call(dev, "uaa_rotary", plan._ref, tq, tk, pos, wide, pb, ps, start, B, S, D, _DTYPES[q.dtype], inverse)
    return out_q, out_k


def rotary_fwd(q, k, plan, positions=None, start=0, out_q=None, out_k=None):
    """``uaa_rotary``: returns ``(q, k)`` rotated; ``k`` may be None or have another head count.

    ``q``, ``k``: ``(B, S, H, D)`` bf16, fp16 or fp32 with contiguous columns -- slices of a packed
    projection are fine.  ``positions``: int32 or int64 ``(S,)`` or ``(B, S)``, with a last dimension of
    ``plan.axes`` when the plan has several; None stands for ``start, start + 1, ...``.  ``out_q=q`` rotates
    in place; otherwise a result must not overlap an operand or the other result.
    """
    return _rotate(q, k, plan, positions, start, 0, out_q, out_k)


def rotary_bwd(dq, dk, plan, positions=None, start=0, out_q=None, out_k=None):
    """The gradients of :func:`rotary_fwd`'s ``q`` and ``k`` from those of its results (the transposed map)."""
    return _rotate(dq, dk, plan, positions, start, 1, out_q, out_k)


class Rotary(torch.autograd.Function):
    """Autograd pairing of ``rotary_fwd`` / ``rotary_bwd``; keeps nothing but the positions."""

    @staticmethod
    def forward(ctx, q, k, plan, positions=None, start=0):
        ctx.plan, ctx.start = plan, start
        ctx.save_for_backward(positions)
        ctx.set_materialize_grads(False)
        return _rotate(q, k, plan, positions, start, 0, None, None)

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dq, dk):
        (positions,) = ctx.saved_tensors
        dq, dk = (t if t is None or t.stride(-1) == 1 else t.contiguous() for t in (dq, dk))
        if dq is None and dk is None:
            return None, None, None, None, None
        if dq is None:
            dk, dq = _rotate(dk, None, ctx.plan, positions, ctx.start, 1, None, None)
        else:
            dq, dk = _rotate(dq, dk, ctx.plan, positions, ctx.start, 1, None, None)
        return dq, dk, None, None, None


def rotary(q, k, plan, positions=None, start=0):
    """Differentiable :func:`rotary_fwd`."""
    return Rotary.apply(q, k, plan, positions, start)


# --------------------------------------------------------------------------- activation checkpoints in 8 bits
class Act8:
    """Tensors kept in 8 bits: one buffer with the codes of all of them, one behind the other, then their steps."""

    __slots__ = ("data", "shapes", "dtype", "single")

    def __init__(self, data, shapes, dtype, single):
        self.data, self.shapes, self.dtype, self.single = data, shapes, dtype, single

    def _meta(self):
        return self.shapes, self.dtype, self.single

    @property
    def _numel(self):
        return sum(s.numel() for s in self.shapes)

    @property
    def codes(self):
        return self.data[:self._numel].view(torch.int8)

    @property
    def steps(self):
        return self.data[self._numel:].view(torch.float32)

    @property
    def nbytes(self):
        return self.data.numel()


_ACT8_ARRAYS = [(ctypes.c_void_p * n, _L * n) for n in range(9)]


def _act8_layout(data, shapes):
    """Arrays of the tensors' code and step pointers and of their rows; D."""
    ptrs, longs = _ACT8_ARRAYS[len(shapes)]
    D = shapes[0][-1]
    rows = [s.numel() // D for s in shapes]
    c = data.data_ptr()
    s, pc, ps = c + sum(rows) * D, [], []
    for r in rows:
        pc.append(c)
        ps.append(s)
        c += r * D
        s += r * 4
    return ptrs(*pc), ptrs(*ps), longs(*rows), D


def act8_pack(x):
    """``uaa_act8_pack``: puts a tensor, or up to eight of one type and last dimension, away in 8 bits.

    Each row of the last dimension D (a multiple of 16 up to 512) becomes int8 codes and one fp32 step,
    ``max|row| / 127``.  Returns an :class:`Act8` for :func:`act8_unpack`.
    """
    single = isinstance(x, torch.Tensor)
    xs = (x,) if single else tuple(x)
    if not 1 <= len(xs) <= 8:
        raise ValueError(f"one to eight tensors at a time, got {len(xs)}")
    dev = _same_device(*xs)
    dtype, shapes = xs[0].dtype, tuple([t.shape for t in xs])
    if dtype not in _DTYPES:
        raise TypeError("tensors must be bfloat16, float16 or float32, all alike")
    if not shapes[0] or not shapes[0][-1]:
        raise ValueError("the last dimension is empty")
    D, total = shapes[0][-1], 0
    for t, s in zip(xs, shapes):
        if t.dtype != dtype:
            raise TypeError("tensors must be bfloat16, float16 or float32, all alike")
        if not s or s[-1] != D or not t.is_contiguous():
            raise ValueError("tensors must be contiguous, with one last dimension")
        total += s.numel()
    data = torch.empty(total + total // D * 4, dtype=torch.uint8, device=dev)
    pc, ps, rows, D = _act8_layout(data, shapes)
    _call(dev, "uaa_act8_pack", len(xs), _ACT8_ARRAYS[len(xs)][0](*[t.data_ptr() for t in xs]), pc, ps, rows, D,
          _DTYPES[dtype])
    return Act8(data, shapes, dtype, single)


def act8_unpack(packed):
    """``uaa_act8_unpack``: the values that the codes stand for, in the shapes and type of the tensors packed."""
    dev, dtype, shapes = _same_device(packed.data), packed.dtype, packed.shapes
    ys = [torch.empty(s, dtype=dtype, device=dev) for s in shapes]
    pc, ps, rows, D = _act8_layout(packed.data, shapes)
    _call(dev, "uaa_act8_unpack", len(ys), pc, ps, _ACT8_ARRAYS[len(ys)][0](*[t.data_ptr() for t in ys]), rows, D,
          _DTYPES[dtype])
    return ys[0] if packed.single else ys


def attn_bwd_act8(packed, dout, lse, key_mask=None, scale=None, dq=None, dk=None, dv=None, workspace=None):
    """``uaa_attn_bwd_act8``: the gradients of :func:`attn_bwd` from an 8-bit checkpoint of ``[q, k, v, out]``."""
    shapes = packed.shapes
    if len(shapes) != 4 or packed.dtype != torch.bfloat16 or any(len(s) != 4 for s in shapes):
        raise ValueError("packed must hold the bf16 BSHD tensors q, k, v and out")
    qs, ks = shapes[0], shapes[1]
    if shapes[2] != ks or shapes[3] != qs or ks[0] != qs[0] or ks[2:] != qs[2:]:
        raise ValueError(f"the packed shapes do not fit: {[tuple(s) for s in shapes]}")
    _bshd("dout", dout)
    B, Sq, H, D = qs
    Sk = ks[1]
    if dout.shape != qs:
        raise ValueError(f"dout shape {tuple(dout.shape)} does not fit {tuple(qs)}")
    if lse.dtype != torch.float32 or lse.shape != (B, H, Sq) or not lse.is_contiguous():
        raise ValueError("lse must be contiguous fp32 (B, H, Sq)")
    mask = normalize_key_mask(key_mask, B, Sk)
    dev = _same_device(packed.data, dout, lse, mask, workspace)
    dq = _result("dq", dq, qs, torch.bfloat16, dev)
    dk = _result("dk", dk, ks, torch.bfloat16, dev)
    dv = _result("dv", dv, ks, torch.bfloat16, dev)
    if workspace is None:
        nbytes = int(lib().uaa_attn_bwd_act8_workspace_bytes(B, Sq, Sk, H, D))
        workspace = torch.empty(max(nbytes, 1), dtype=torch.uint8, device=dev)
    pc, ps, _, _ = _act8_layout(packed.data, shapes)
    _call(dev, "uaa_attn_bwd_act8", pc, ps, dout.data_ptr(), lse.data_ptr(), _ptr(mask), dq.data_ptr(), dk.data_ptr(),
          dv.data_ptr(), B, Sq, Sk, H, D, float(1.0 / math.sqrt(D) if scale is None else scale), workspace.data_ptr(),
          workspace.numel() * workspace.element_size())
    return dq, dk, dv


# --------------------------------------------------------------------------- differential attention
def _diff_args(q, k, v, lam, key_mask, scale):
    _bshd("q", q)
    _bshd("k", k, q, same_s=False)
    _bshd("v", v, k)
    B, Sq, H, D = q.shape
    Sk = k.shape[1]
    if lam.dtype not in (torch.bfloat16, torch.float32):
        raise TypeError("lam must be bfloat16 or float32")
    if tuple(lam.shape) != (H,) or not lam.is_contiguous():
        raise ValueError(f"lam must be contiguous (H,) = ({H},), got {tuple(lam.shape)}")
    mask = normalize_key_mask(key_mask, B, Sk)
    dev = _same_device(q, k, v, lam, mask)
    return B, Sq, Sk, H, D, mask, float(1.0 / math.sqrt(D / 2) if scale is None else scale), dev


def diff_attn_fwd(q, k, v, lam, key_mask=None, scale=None, need_out2=True, out=None, out2=None, lse=None):
    """``uaa_diff_attn_fwd``: returns ``(out, out2, lse)``.

    ``q`` ``(B, Sq, H, D)``, ``k``, ``v`` ``(B, Sk, H, D)``: bf16 BSHD as for :func:`attn_fwd`; the first D/2 columns
    of ``q`` and ``k`` are the first softmax map's, the others the second's.  ``lam`` ``(H,)``: bf16 or fp32.
    ``out = (A1 - lam A2) v``; ``out2 = A2 v`` (None with ``need_out2=False``, when no gradient is wanted);
    ``lse`` fp32 ``(B, H, 2, Sq)``.  ``scale`` defaults to ``1/sqrt(D/2)``.
    """
    B, Sq, Sk, H, D, mask, scale, dev = _diff_args(q, k, v, lam, key_mask, scale)
    out = _result("out", out, q.shape, q.dtype, dev)
    out2 = _result("out2", out2, q.shape, q.dtype, dev) if need_out2 or out2 is not None else None
    lse = _result("lse", lse, (B, H, 2, Sq), torch.float32, dev)
    _call(dev, "uaa_diff_attn_fwd", _ptr(q), _ptr(k), _ptr(v), _ptr(lam), _DTYPES[lam.dtype], _ptr(mask), _ptr(out),
          _ptr(out2), _ptr(lse), B, Sq, Sk, H, D, scale)
    return out, out2, lse


def diff_attn_bwd_workspace_bytes(B, Sq, Sk, H, D) -> int:
    return int(lib().uaa_diff_attn_bwd_workspace_bytes(B, Sq, Sk, H, D))


def diff_attn_bwd(q, k, v, lam, out, out2, dout, lse, key_mask=None, scale=None, dq=None, dk=None, dv=None, dlam=None,
                  workspace=None):
    """``uaa_diff_attn_bwd``: returns ``(dq, dk, dv, dlam)``, ``dlam`` in ``lam``'s type."""
    B, Sq, Sk, H, D, mask, scale, dev = _diff_args(q, k, v, lam, key_mask, scale)
    for n, t in (("out", out), ("out2", out2), ("dout", dout)):
        _bshd(n, t, q)
    if lse.dtype != torch.float32 or tuple(lse.shape) != (B, H, 2, Sq) or not lse.is_contiguous():
        raise ValueError("lse must be contiguous fp32 (B, H, 2, Sq)")
    _same_device(q, out, out2, dout, lse, workspace)
    dq = _result("dq", dq, q.shape, q.dtype, dev)
    dk = _result("dk", dk, k.shape, q.dtype, dev)
    dv = _result("dv", dv, k.shape, q.dtype, dev)
    dlam = _result("dlam", dlam, lam.shape, lam.dtype, dev)
    if B * Sq == 0:
        if Sk and B:
            raise ValueError("keys without queries (Sq = 0)")
        return dq, dk, dv, dlam.zero_()
    nbytes = diff_attn_bwd_workspace_bytes(B, Sq, Sk, H, D)
    if workspace is None:
        workspace = torch.empty(max(nbytes, 1), dtype=torch.uint8, device=dev)
    _call(dev, "uaa_diff_attn_bwd", _ptr(q), _ptr(k), _ptr(v), _ptr(lam), _DTYPES[lam.dtype], _ptr(out), _ptr(out2),
          _ptr(dout), _ptr(lse), _ptr(mask), _ptr(dq), _ptr(dk), _ptr(dv), _ptr(dlam), B, Sq, Sk, H, D, scale,
          _ptr(workspace), workspace.numel() * workspace.element_size())
    return dq, dk, dv, dlam


class DiffAttention(torch.autograd.Function):
    """Autograd pairing of ``diff_attn_fwd`` / ``diff_attn_bwd``; ``lse`` is non-differentiable.

    ``saved="int8"`` keeps Q, K, V, O and O2 for the backward pass as an 8-bit checkpoint."""

    @staticmethod
    def forward(ctx, q, k, v, lam, key_mask=None, scale=None, saved=None):
        _check_saved(saved)
        grad = any(ctx.needs_input_grad)
        out, out2, lse = diff_attn_fwd(q, k, v, lam, key_mask, scale, need_out2=grad)
        if grad:
            _save(ctx, saved, (q, k, v, out, out2), lam, lse, key_mask=key_mask)
        ctx.scale = scale
        ctx.mark_non_differentiable(lse)
        ctx.set_materialize_grads(False)  # no zeros for lse
        return out, lse

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dout, _dlse):
        if dout is None:
            return None, None, None, None, None, None, None
        (q, k, v, out, out2), (lam, lse), key_mask = _saved(ctx, 5)
        dq, dk, dv, dlam = diff_attn_bwd(q, k, v, lam, out, out2, dout.contiguous(), lse, key_mask, ctx.scale)
        return dq, dk, dv, dlam, None, None, None


def diff_attention(q, k, v, lam, key_mask=None, scale=None, saved=None):
    """Differentiable differential attention: returns ``(out, lse)``.

    To capture a step with its gradients in a CUDA graph, warm up on another stream and let no eager autograd graph
    of the same leaves live: PyTorch ties a leaf's gradients to the stream of the first graph that holds it."""
    return DiffAttention.apply(q, k, v, lam, key_mask, scale, saved)


# --------------------------------------------------------------------------- sequences of their own lengths
def _rows16(name, t, dims, D=None):
    """Checks a 16-bit operand (..., heads, D); returns its strides, those of dimensions of one entry as if contiguous."""
    shape, strides = t.shape, t.stride()
    if len(shape) != dims:
        raise ValueError(f"{name} must have {dims} dimensions, got {tuple(shape)}")
    if D is not None and shape[-1] != D:
        raise ValueError(f"{name} has heads of {shape[-1]} columns, not {D}")
    if 1 in shape or 0 in shape:
        strides, dense = list(strides), 1
        for i in range(dims - 1, -1, -1):
            if shape[i] <= 1:
                strides[i] = dense
            dense *= max(shape[i], 1)
    if strides[-1] != 1:
        raise ValueError(f"the columns of {name} must be contiguous")
    return strides


def _starts(name, t, B=None):
    if t.dim() != 1 or t.dtype != torch.int32 or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous int32 vector, got {t.dtype} {tuple(t.shape)}")
    if t.shape[0] < 1 or (B is not None and t.shape[0] != B + 1):
        raise ValueError(f"{name} must have one entry more than there are sequences, got {t.shape[0]}")


def _seqs_common(q, k, v, starts, scale, out, lse, half=True):
    """What packed and paged attention check alike; returns the type's number, the scale and the results."""
    if q.dtype not in (torch.bfloat16, torch.float16) or (q.dtype != torch.bfloat16 and not half):
        raise TypeError("q must be bfloat16 or float16" if half else "gradients are built for bfloat16")
    if k.dtype != q.dtype or v.dtype != q.dtype:
        raise TypeError("q, k and v must have one type")
    T, Hq, D = q.shape
    if k.shape != v.shape:
        raise ValueError(f"k {tuple(k.shape)} and v {tuple(v.shape)} must have one shape")
    _starts("starts", starts)
    dev = q.device
    return (_DTYPES[q.dtype], float(1.0 / math.sqrt(D) if scale is None else scale),
            _result("out", out, (T, Hq, D), q.dtype, dev), _result("lse", lse, (Hq, T), torch.float32, dev))


def attn_seqs_workspace_bytes(B, T, Hq, Hk, D) -> int:
    return int(lib().uaa_attn_seqs_workspace_bytes(B, T, Hq, Hk, D))


def _seqs_workspace(workspace, B, T, Hq, Hk, D, dev):
    if workspace is None:
        workspace = torch.empty(attn_seqs_workspace_bytes(B, T, Hq, Hk, D), dtype=torch.uint8, device=dev)
    return workspace


def _packed_args(q, k, v, starts, starts_k, causal, scale, out, lse, half=True, rest=0):
    (q0, q1, _), (k0, k1, _), (v0, v1, _) = _rows16("q", q, 3), _rows16("k", k, 3, q.shape[-1]), _rows16("v", v, 3)
    dtype, scale, out, lse = _seqs_common(q, k, v, starts, scale, out, lse, half)
    B = starts.shape[0] - 1
    if starts_k is not None:
        _starts("starts_k", starts_k, B)
    elif k.shape[0] != q.shape[0]:
        raise ValueError(f"{q.shape[0]} query and {k.shape[0]} key tokens: starts_k is needed")
    T, Hq, D = q.shape
    packed = _SEQS.pack(q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(), lse.data_ptr(), starts.data_ptr(),
                        0 if starts_k is None else starts_k.data_ptr(), 0, 0, 0, q0, q1, k0, k1, v0, v1, 0, 0, B, T,
                        k.shape[0], Hq, k.shape[1], D, dtype, 1 if causal else 0, 0, 0, 0, 0, rest, scale)
    return packed, out, lse


def attn_packed_fwd(q, k, v, starts, starts_k=None, causal=True, scale=None, out=None, lse=None, workspace=None):
    """``uaa_attn_packed_fwd``: attention of sequences packed one behind the other; returns ``(out, lse)``.

    ``q`` ``(T, Hq, D)``, ``k``, ``v`` ``(Tk, Hk, D)``: bf16 or fp16 with contiguous columns -- slices of a packed
    projection are fine.  ``Hq`` is a multiple of ``Hk``: query head h reads key head ``h // (Hq // Hk)``.
    ``starts``: int32 ``(B + 1)`` on the device, the first token of each sequence and the end of the last;
    ``starts_k`` the keys' where they are others than the queries'.  With ``causal`` a sequence's last query stands at
    its last key and each reads the keys up to its own place.  Returns ``out`` ``(T, Hq, D)`` and ``lse`` fp32
    ``(Hq, T)``; tokens behind ``starts[-1]`` are left as they were (in new results: undefined).
    """
    return _packed_fwd(q, k, v, starts, starts_k, causal, scale, out, lse, workspace, 0)


def _packed_fwd(q, k, v, starts, starts_k, causal, scale, out, lse, workspace, rest):
    dev = _same_device(q, k, v, starts, starts_k, out, lse, workspace)
    args, out, lse = _packed_args(q, k, v, starts, starts_k, causal, scale, out, lse, rest=rest)
    T, Hq, D = q.shape
    workspace = _seqs_workspace(workspace, starts.shape[0] - 1, T, Hq, k.shape[1], D, dev)  # held until the launch
    _call(dev, "uaa_attn_packed_fwd", args, workspace.data_ptr(), workspace.numel() * workspace.element_size())
    return out, lse


def attn_packed_bwd_workspace_bytes(B, T, Hq, Hk, D) -> int:
    return int(lib().uaa_attn_packed_bwd_workspace_bytes(B, T, Hq, Hk, D))


def attn_packed_bwd(q, k, v, out, dout, lse, starts, starts_k=None, causal=True, scale=None, dq=None, dk=None, dv=None,
                    workspace=None):
    """``uaa_attn_packed_bwd``: the gradients ``(dq, dk, dv)`` of :func:`attn_packed_fwd` (bf16).

    ``k`` and ``v`` may be some of the keys that ``out`` and ``lse`` are of: then ``dq`` is a part, ``dk`` and ``dv`` are those
    keys'.
    An infinity or a NaN of a token may show in the gradients of any token of its own sequence; other sequences' stay
    clean."""
    if out is None or lse is None:
        raise ValueError("out and lse are the forward's results")
    return _packed_bwd(q, k, v, out, dout, lse, starts, starts_k, causal, scale, dq, dk, dv, workspace, 0)


def _packed_bwd(q, k, v, out, dout, lse, starts, starts_k, causal, scale, dq, dk, dv, workspace, rest):
    dev = _same_device(q, k, v, out, dout, lse, starts, starts_k, workspace)
    args, out, lse = _packed_args(q, k, v, starts, starts_k, causal, scale, out, lse, half=False, rest=rest)
    dout = _result("dout", dout, q.shape, q.dtype, dev)
    dq = _result("dq", dq, q.shape, q.dtype, dev)
    dk = _result("dk", dk, k.shape, q.dtype, dev)
    dv = _result("dv", dv, k.shape, q.dtype, dev)
    T, Hq, D = q.shape
    if workspace is None:
        nbytes = attn_packed_bwd_workspace_bytes(starts.shape[0] - 1, T, Hq, k.shape[1], D)
        workspace = torch.empty(max(nbytes, 1), dtype=torch.uint8, device=dev)
    _call(dev, "uaa_attn_packed_bwd", args, dout.data_ptr(), dq.data_ptr(), dk.data_ptr(), dv.data_ptr(),
          workspace.data_ptr(), workspace.numel() * workspace.element_size())
    return dq, dk, dv


class PackedAttention(torch.autograd.Function):
    """Autograd pairing of ``attn_packed_fwd`` / ``attn_packed_bwd``; ``lse`` is non-differentiable.

    ``saved="int8"`` keeps Q, K, V and O for the backward pass as an 8-bit checkpoint.  For tokens of no sequence (before
    ``starts[0]``, behind ``starts[-1]``) ``out`` and the gradients are zero."""

    @staticmethod
    def forward(ctx, q, k, v, starts, starts_k=None, causal=True, scale=None, saved=None):
        _check_saved(saved)
        out, lse = _packed_fwd(q, k, v, starts, starts_k, causal, scale, None, None, None, 1)
        if saved == "int8":  # the checkpoint takes contiguous rows
            q, k, v = q.contiguous(), k.contiguous(), v.contiguous()
        # (made in inference mode they have no versions and cannot be saved: they stay on ctx)
        ctx.starts = [t if t is not None and t.is_inference() else None for t in (starts, starts_k)]
        _save(ctx, saved, (q, k, v, out), lse, *(t if c is None else None for t, c in zip((starts, starts_k), ctx.starts)),
              key_mask=None)
        ctx.causal, ctx.scale = causal, scale
        ctx.mark_non_differentiable(lse)
        ctx.set_materialize_grads(False)  # no zeros for lse
        return out, lse

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dout, _dlse):
        if dout is None:
            return (None,) * 8
        (q, k, v, out), (lse, starts, starts_k), _ = _saved(ctx, 4)
        starts, starts_k = (a if b is None else b for a, b in zip((starts, starts_k), ctx.starts))
        dq, dk, dv = _packed_bwd(q, k, v, out, dout.contiguous(), lse, starts, starts_k, ctx.causal, ctx.scale, None, None,
                                 None, None, 1)
        return dq, dk, dv, None, None, None, None, None


def packed_attention(q, k, v, starts, starts_k=None, causal=True, scale=None, saved=None):
    """Differentiable :func:`attn_packed_fwd`: returns ``(out, lse)``.  ``saved`` and tokens of no sequence:
    :class:`PackedAttention`.

    To capture a step with its gradients in a CUDA graph, warm up on another stream and let no eager autograd graph
    of the same leaves live: PyTorch ties a leaf's gradients to the stream of the first graph that holds it."""
    # (asked here: inside of a Function the grad mode is off, and a leaf says that it needs a gradient under no_grad too)
    if q.dtype != torch.bfloat16 and torch.is_grad_enabled() and any(t.requires_grad for t in (q, k, v)):
        raise TypeError("gradients are built for bfloat16")
    return PackedAttention.apply(q, k, v, starts, starts_k, causal, scale, saved)


def _table(table, lens, seqs, B):
    if table.dim() != 2 or table.dtype != torch.int32 or not table.is_contiguous():
        raise ValueError(f"table must be contiguous int32 (sequences, pages), got {table.dtype} {tuple(table.shape)}")
    if lens.dtype != torch.int32 or lens.shape != table.shape[:1] or not lens.is_contiguous():
        raise ValueError(f"lens must be contiguous int32 ({table.shape[0]},), got {lens.dtype} {tuple(lens.shape)}")
    if seqs is not None and (seqs.dtype != torch.int32 or seqs.shape != (B,) or not seqs.is_contiguous()):
        raise ValueError(f"seqs must be contiguous int32 ({B},), got {seqs.dtype} {tuple(seqs.shape)}")


def attn_paged_fwd(q, k_pages, v_pages, starts, table, lens, seqs=None, causal=True, scale=None, out=None, lse=None,
                   workspace=None):
    """``uaa_attn_paged_fwd``: new tokens attend to the pages of a cache; returns ``(out, lse)``.

    ``q`` ``(T, Hq, D)``: the new tokens of B sequences packed one behind the other (``starts`` int32 ``(B + 1)``), one
    or many of each.  ``k_pages``, ``v_pages`` ``(pages, page, Hk, D)``: a layer's pools, which hold the new tokens'
    keys and values already (:func:`cache_write`).  ``table`` int32 ``(rows, width)`` and ``lens`` int32 ``(rows,)``, the
    new tokens counted, are a :class:`PagedCache`'s; sequence b is row ``seqs[b]`` (None: b).  Everything is read on the
    device when the call runs: it may be captured in a graph and replayed with other lengths and pages.
    """
    dev = _same_device(q, k_pages, v_pages, starts, table, lens, seqs, out, lse, workspace)
    q0, q1, _ = _rows16("q", q, 3)
    (k0, k1, k2, _), (v0, v1, v2, _) = _rows16("k_pages", k_pages, 4, q.shape[-1]), _rows16("v_pages", v_pages, 4)
    dtype, scale, out, lse = _seqs_common(q, k_pages, v_pages, starts, scale, out, lse)
    B = starts.shape[0] - 1
    _table(table, lens, seqs, B)
    (T, Hq, D), (N, page, Hk, _), (rows, width) = q.shape, k_pages.shape, table.shape
    args = _SEQS.pack(q.data_ptr(), k_pages.data_ptr(), v_pages.data_ptr(), out.data_ptr(), lse.data_ptr(),
                      starts.data_ptr(), 0, table.data_ptr(), lens.data_ptr(), 0 if seqs is None else seqs.data_ptr(),
                      q0, q1, k1, k2, v1, v2, k0, v0, B, T, 0, Hq, Hk, D, dtype, 1 if causal else 0, N, page, rows,
                      width, 0, scale)
    workspace = _seqs_workspace(workspace, B, T, Hq, Hk, D, dev)  # held until the launch
    _call(dev, "uaa_attn_paged_fwd", args, workspace.data_ptr(), workspace.numel() * workspace.element_size())
    return out, lse


def cache_write(k, v, k_pages, v_pages, starts, table, lens, seqs=None):
    """``uaa_cache_write``: puts the keys and values ``(T, Hk, D)`` of new tokens into the pages of one layer.

    Token ``starts[b] + i`` goes to row ``lens[r] - n + i`` of sequence ``r = seqs[b]`` (None: b), n being the
    sequence's new tokens, which ``lens`` counts.  Any 2-byte type.
    """
    dev = _same_device(k, v, k_pages, v_pages, starts, table, lens, seqs)
    if k.element_size() != 2 or any(t.dtype != k.dtype for t in (v, k_pages, v_pages)):
        raise TypeError("k, v and the pages must have one 2-byte type")
    if (k.shape != v.shape or k_pages.shape != v_pages.shape or k.dim() != 3 or k_pages.dim() != 4 or
            k.shape[1:] != k_pages.shape[2:]):
        raise ValueError(f"k {tuple(k.shape)}, v {tuple(v.shape)} and pages {tuple(k_pages.shape)}, "
                         f"{tuple(v_pages.shape)} do not fit")
    (k0, k1, _), (v0, v1, _) = _rows16("k", k, 3), _rows16("v", v, 3)
    (a0, a1, a2, _), (b0, b1, b2, _) = _rows16("k_pages", k_pages, 4), _rows16("v_pages", v_pages, 4)
    _starts("starts", starts)
    B = starts.shape[0] - 1
    _table(table, lens, seqs, B)
    (T, Hk, D), (N, page, _, _), (rows, width) = k.shape, k_pages.shape, table.shape
    _call(dev, "uaa_cache_write",
          _CACHE_ROWS.pack(k.data_ptr(), v.data_ptr(), k_pages.data_ptr(), v_pages.data_ptr(), starts.data_ptr(),
                           0 if seqs is None else seqs.data_ptr(), table.data_ptr(), lens.data_ptr(), k0, k1, v0, v1,
                           a0, a1, a2, b0, b1, b2, B, T, Hk, D, N, page, rows, width))


class PagedCache:
    """The keys and values of sequences, of all layers, in pages that sequences may share (``uaa_pages``).

    ``k``, ``v`` ``(layers, pages, page, heads, dim)``; ``table`` int32 ``(seqs, width)`` and ``lens`` int32 ``(seqs,)``
    on the device, for :func:`attn_paged_fwd`.  A sequence is a number below ``seqs`` and has ``width`` pages at most.
    The lowest free pages are taken first.  A call that cannot be done raises before anything changes
    (``UAA_ERR_NO_PAGES`` where pages are short).  The device's side is changed on the current stream, by small
    launches that hold their data; these calls are made outside of graph captures, between replays.  Should such a launch
    fail (``UAA_ERR_CUDA``), the device has not followed the host: the cache refuses further changes and is to be given
    up.  A cache is not copied or pickled.  Calls from several threads lock the host's side; the device's follows the order of
    the streams, so a cache is used on one stream or on streams that wait for one another.

    A step of a model::

        starts, seqs = cache.append(ids, [1] * len(ids))
        for layer in range(layers):
            cache.write(layer, k, v, starts, seqs)
            out, _ = cache.attend(layer, q, starts, seqs)
    """

    def __init__(self, layers, pages, page, heads, dim, seqs, width, dtype=torch.bfloat16, device="cuda"):
        if dtype not in (torch.bfloat16, torch.float16):
            raise TypeError("dtype must be bfloat16 or float16")
        if min(layers, heads) < 1 or dim not in (64, 128):
            raise ValueError(f"layers={layers} and heads={heads} must be positive, dim={dim} 64 or 128")
        self._h = _P()
        _check(lib().uaa_pages_create(ctypes.byref(self._h), pages, page, seqs, width))
        self._k, self._v = (torch.empty((layers, pages, page, heads, dim), dtype=dtype, device=device) for _ in range(2))
        self._table = torch.full((seqs, width), -1, dtype=torch.int32, device=device)
        self._lens = torch.zeros(seqs, dtype=torch.int32, device=device)
        self._at = tuple(t.data_ptr() for t in (self._k, self._v, self._table, self._lens))
        self._pools = _POOLS.pack(*self._at, layers, heads * dim * 2)
        self._strides = (page * heads * dim, heads * dim, dim) * 2
        self._rows = (heads, dim, pages, page, seqs, width)
        self._layer_bytes = pages * page * heads * dim * 2

    # The calls hold the tensors' addresses, so other tensors cannot take their places.
    k = property(lambda self: self._k)
    v = property(lambda self: self._v)
    table = property(lambda self: self._table)
    lens = property(lambda self: self._lens)
    page = property(lambda self: self._rows[3])
    seqs = property(lambda self: self._rows[4])

    def __del__(self):
        if getattr(self, "_h", None) and _lib is not None:
            _lib.uaa_pages_destroy(self._h)
            self._h = None

    def __reduce_ex__(self, protocol):  # a copy would share the handle, which either of the two frees
        raise TypeError("a PagedCache cannot be copied or pickled")

    @property
    def free_pages(self):
        return int(lib().uaa_pages_free(self._h))

    def length(self, seq):
        """Tokens of a sequence, as the host knows them."""
        n = int(lib().uaa_pages_row(self._h, seq, None, 0))
        if n < 0:
            _check(n)
        return n

    def pages_of(self, seq):
        """The pages that a sequence holds, in order."""
        n = -(-self.length(seq) // self.page)
        row = (_I * max(n, 1))()
        lib().uaa_pages_row(self._h, seq, row, n)
        return list(row)[:n]

    def _pair(self, name, a, b):
        a, b = array.array("i", a), array.array("i", b)
        if len(a) != len(b):
            raise ValueError(f"{len(a)} and {len(b)} entries")
        _call(self._k.device, name, self._h, self._pools, len(a), a.buffer_info()[0], b.buffer_info()[0])

    def append(self, seqs, counts):
        """Makes room for ``counts[i]`` more tokens of sequence ``seqs[i]``; a shared, partly filled last page is
        copied first.  Returns ``(starts, seqs)`` on the device, for :meth:`write` and :meth:`attend`."""
        a, b = array.array("i", seqs), array.array("i", counts)
        if len(a) != len(b):
            raise ValueError(f"{len(a)} sequences and {len(b)} counts")
        n, dev = len(a), self._k.device
        both = torch.empty(2 * n + 1, dtype=torch.int32, device=dev)
        starts, ids = both[: n + 1], both[n + 1:]
        at = both.data_ptr()
        _call(dev, "uaa_pages_append", self._h, self._pools, n, a.buffer_info()[0], b.buffer_info()[0], at,
              at + 4 * (n + 1))
        return starts, ids

    def fork(self, parents, children):
        """Makes ``children[i]``, an empty sequence, a copy of ``parents[i]``: it shares the pages, none is copied."""
        self._pair("uaa_pages_fork", parents, children)

    def truncate(self, seqs, lens):
        """Cuts sequence ``seqs[i]`` to its first ``lens[i]`` tokens."""
        self._pair("uaa_pages_truncate", seqs, lens)

    def free(self, seqs):
        """Empties sequences; pages that no other sequence shares are free again."""
        seqs = list(seqs)
        self.truncate(seqs, [0] * len(seqs))

    def compact(self):
        """Moves pages so that those in use are the lowest ones."""
        _call(self._k.device, "uaa_pages_compact", self._h, self._pools)

    def write(self, layer, k, v, starts, seqs=None):
        """:func:`cache_write` into a layer."""
        pools, shape = self._k, k.shape
        if k.dtype != pools.dtype or v.dtype != pools.dtype:
            raise TypeError(f"k and v must be {pools.dtype}")
        if shape != v.shape or len(shape) != 3 or shape[1] != self._rows[0] or shape[2] != self._rows[1]:
            raise ValueError(f"k {tuple(shape)} and v {tuple(v.shape)} must be (tokens, {self._rows[0]}, {self._rows[1]})")
        if not 0 <= layer < pools.shape[0]:
            raise IndexError(f"layer {layer} of {pools.shape[0]}")
        dev = _same_device(pools, k, v, starts, seqs)
        (k0, k1, _), (v0, v1, _) = _rows16("k", k, 3), _rows16("v", v, 3)
        _starts("starts", starts)
        B = starts.shape[0] - 1
        if seqs is not None and (seqs.dtype != torch.int32 or seqs.shape != (B,) or not seqs.is_contiguous()):
            raise ValueError(f"seqs must be contiguous int32 ({B},), got {seqs.dtype} {tuple(seqs.shape)}")
        at = layer * self._layer_bytes
        _call(dev, "uaa_cache_write",
              _CACHE_ROWS.pack(k.data_ptr(), v.data_ptr(), self._at[0] + at, self._at[1] + at, starts.data_ptr(),
                               0 if seqs is None else seqs.data_ptr(), self._at[2], self._at[3], k0, k1, v0, v1,
                               *self._strides, B, shape[0], *self._rows))

    def attend(self, layer, q, starts, seqs=None, causal=True, scale=None):
        """:func:`attn_paged_fwd` over a layer."""
        return attn_paged_fwd(q, self.k[layer], self.v[layer], starts, self.table, self.lens, seqs, causal, scale)


# --------------------------------------------------------------------------- Ulysses re-layout
def _lens_array(shard_lens):
    lens = [int(x) for x in shard_lens]
    return (ctypes.c_int * len(lens))(*lens), lens


def seq_to_head(x, shard_lens, out=None):
    """``uaa_seq_to_head``: ``(P, B, cap, H, D)`` shards -> ``(P, B, N, ceil(H/P), D)`` groups.

    When P does not divide H the groups are padded with zero heads.
    """
    _need_cuda(x)
    if x.dim() != 5 or not x.is_contiguous():
        raise ValueError("x must be contiguous (P, B, cap, H, D)")
    P, B, cap, H, D = x.shape
    arr, lens = _lens_array(shard_lens)
    if len(lens) != P:
        raise ValueError("len(shard_lens) must equal P")
    N = sum(lens)
    if out is None:
        out = torch.empty((P, B, N, -(-H // P), D), dtype=x.dtype, device=x.device)
    _check(lib().uaa_seq_to_head(_ptr(x), _ptr(out), P, arr, cap, B, H, D, x.element_size(), _P(_stream(x.device))))
    return out


def head_to_seq(y, shard_lens, cap, H=None, out=None):
    """``uaa_head_to_seq``: ``(P, B, N, Hg, D)`` groups -> ``(P, B, cap, H, D)`` shards (padding zeroed).

    ``H`` is the true head count (default ``P * Hg``); padding heads of the groups are dropped.
    """
    _need_cuda(y)
    if y.dim() != 5 or not y.is_contiguous():
        raise ValueError("y must be contiguous (P, B, N, Hg, D)")
    P, B, N, Hg, D = y.shape
    H = P * Hg if H is None else int(H)
    if not (Hg - 1) * P < H <= Hg * P:
        raise ValueError(f"H={H} does not have ceil(H/P) = {Hg} heads per group")
    arr, lens = _lens_array(shard_lens)
    if len(lens) != P or sum(lens) != N:
        raise ValueError("shard_lens must have P entries summing to N")
    if out is None:
        out = torch.empty((P, B, cap, H, D), dtype=y.dtype, device=y.device)
    _check(lib().uaa_head_to_seq(_ptr(y), _ptr(out), P, arr, cap, B, H, D, y.element_size(),
                                 _P(_stream(y.device))))
    return out


def assemble_key_mask(gathered, shard_lens, out=None):
    """``uaa_assemble_key_mask``: gathered ``(P, B, cap)`` uint8 -> trimmed ``(B, N)`` uint8."""
    _need_cuda(gathered)
    if gathered.dtype == torch.bool:
        gathered = gathered.view(torch.uint8)
    if gathered.dim() != 3 or gathered.dtype != torch.uint8 or not gathered.is_contiguous():
        raise ValueError("gathered must be contiguous uint8 (P, B, cap)")
    P, B, cap = gathered.shape
    arr, lens = _lens_array(shard_lens)
    if len(lens) != P:
        raise ValueError("len(shard_lens) must equal P")
    if out is None:
        out = torch.empty((B, sum(lens)), dtype=torch.uint8, device=gathered.device)
    _check(lib().uaa_assemble_key_mask(_ptr(gathered), _ptr(out), P, arr, cap, B, _P(_stream(gathered.device))))
    return out


def debug_exp2_fma2(x):
    """``uaa_debug_exp2_fma2``: the forward's FMA-pipe 2^x on a contiguous float32 CUDA tensor
    with an even number of elements (a diagnostic for tests)."""
    _need_cuda(x)
    if x.dtype != torch.float32 or not x.is_contiguous() or x.numel() % 2:
        raise ValueError("x must be a contiguous float32 tensor with an even number of elements")
    y = torch.empty_like(x)
    _check(lib().uaa_debug_exp2_fma2(_ptr(x), _ptr(y), x.numel(), _P(_stream(x.device))))
    return y


def debug_build() -> bool:
    """True when the loaded library is the debug build (device range checks)."""
    return bool(lib().uaa_debug_build())


def check_device_status(device=None):
    dev = torch.device("cuda") if device is None else torch.device(device)
    _check(lib().uaa_check_device_status(_P(_stream(dev))))


def watchdog_selftest(timeout_us=2000, device=None):
    dev = torch.device("cuda") if device is None else torch.device(device)
    return lib().uaa_watchdog_selftest(int(timeout_us), _P(_stream(dev)))


def set_wait_timeout_ms(ms: int):
    lib().uaa_set_wait_timeout_ms(int(ms))



def debug_drop_load(n: int):
    """Diagnostic: the attention kernels' producers skip their n-th ring load (-1: off)."""
    lib().uaa_debug_drop_load(int(n))


def debug_fail_launch(n: int = -1):
    """Diagnostic: the n-th launch of every call that changes a :class:`PagedCache` is not made, and the call fails (-1:
    off)."""
    lib().uaa_debug_fail_launch(int(n))


def debug_late_warp(warp: int = -1, ns: int = 0):
    """Diagnostic of the debug build: that warp of the attention kernels comes late to each of its waits (-1: off)."""
    _check(lib().uaa_debug_late_warp(int(warp), int(ns)))


def set_bwd_profile_events(events=None):
    """Record three ``torch.cuda.Event``s around the backward's dK/dV and dQ kernels (None stops)."""
    if events is None:
        lib().uaa_set_bwd_profile_events(None, None, None)
    else:
        a, b, c = (_P(e.cuda_event) for e in events)
        lib().uaa_set_bwd_profile_events(a, b, c)


# --------------------------------------------------------------------------- Ulysses composition
class UlyssesAttention(torch.autograd.Function):
    """Ulysses attention over P emulated ranks on one device.

    Forward: seq->head exchange of Q, K, V; attention per head group (all groups
    share the assembled key mask); head->seq exchange of O.  Backward: seq->head
    exchange of dO; attention backward per group; head->seq exchange of dQ
    (query partition) and dK, dV (key partition).  "[attention] Add Ulysses
    Anything backward", What does this PR do.
    """

    @staticmethod
    def forward(ctx, q_sh, k_sh, v_sh, shard_lens, key_mask=None, scale=None, saved=None):
        _check_saved(saved)
        cap, H = q_sh.shape[2], q_sh.shape[3]
        yq, yk, yv = (seq_to_head(t, shard_lens) for t in (q_sh, k_sh, v_sh))
        P = yq.shape[0]
        # the P groups form one batch of P*B sequences sharing the B mask rows: one launch for all
        # emulated ranks
        o, lse = attn_fwd_groups(yq, yk, yv, key_mask, scale)
        o_sh = head_to_seq(o, shard_lens, cap, H)
        _save(ctx, saved, (yq, yk, yv, o), lse, key_mask=key_mask)
        ctx.shard_lens, ctx.scale, ctx.cap, ctx.H = tuple(shard_lens), scale, cap, H
        ctx.mark_non_differentiable(lse)
        return o_sh, lse

    @staticmethod
    def backward(ctx, do_sh, _dlse):
        (yq, yk, yv, o), (lse,), key_mask = _saved(ctx, 4)
        ydo = seq_to_head(do_sh.contiguous(), ctx.shard_lens)
        dq, dk, dv = attn_bwd_groups(yq, yk, yv, o, ydo, lse, key_mask, ctx.scale)
        return (head_to_seq(dq, ctx.shard_lens, ctx.cap, ctx.H), head_to_seq(dk, ctx.shard_lens, ctx.cap, ctx.H),
                head_to_seq(dv, ctx.shard_lens, ctx.cap, ctx.H), None, None, None, None)


def ulysses_attention(q_sh, k_sh, v_sh, shard_lens, key_mask=None, scale=None, saved=None):
    """Differentiable Ulysses attention; ``saved="int8"`` keeps the head groups of Q, K, V and O for the
    backward pass as an 8-bit checkpoint."""
    return UlyssesAttention.apply(q_sh, k_sh, v_sh, tuple(shard_lens), key_mask, scale, saved)


# --------------------------------------------------------------------------- Ulysses, exchanges fused
def _shards(name, t, ref=None):
    if t.dim() != 5:
        raise ValueError(f"{name} must be (P, B, cap, H, D), got {tuple(t.shape)}")
    if t.dtype != torch.bfloat16:
        raise TypeError(f"{name} must be bfloat16")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous (P, B, cap, H, D)")
    if ref is not None and tuple(t.shape) != tuple(ref.shape):
        raise ValueError(f"{name} shape {tuple(t.shape)} does not fit {tuple(ref.shape)}")


def ulysses_attn_fwd(q_sh, k_sh, v_sh, shard_lens, key_mask=None, scale=None, out=None, lse=None):
    """``uaa_ulysses_attn_fwd``: Ulysses attention straight on the sequence shards.

    ``q_sh``, ``k_sh``, ``v_sh``: ``(P, B, cap, H, D)`` bf16 shards; returns ``(out_sh, lse)`` with
    ``out_sh`` in the same layout (padding rows zero) and ``lse`` fp32 ``(B, H, N)`` in sequence
    order, N = sum(shard_lens).  ``key_mask`` is ``(B, N)`` in sequence order.
    """
    _shards("q_sh", q_sh)
    _shards("k_sh", k_sh, q_sh)
    _shards("v_sh", v_sh, q_sh)
    _need_cuda(q_sh, k_sh, v_sh)
    P, B, cap, H, D = q_sh.shape
    arr, lens = _lens_array(shard_lens)
    if len(lens) != P:
        raise ValueError("len(shard_lens) must equal P")
    N = sum(lens)
    mask = normalize_key_mask(key_mask, B, N)
    if scale is None:
        scale = 1.0 / math.sqrt(D)
    if out is None:
        out = torch.empty_like(q_sh)
    if lse is None:
        lse = torch.empty((B, H, N), dtype=torch.float32, device=q_sh.device)
    _check(lib().uaa_ulysses_attn_fwd(_ptr(q_sh), _ptr(k_sh), _ptr(v_sh), _ptr(mask), _ptr(out), _ptr(lse), P, arr,
                                      cap, B, H, D, float(scale), _P(_stream(q_sh.device))))
    return out, lse


def ulysses_attn_bwd_workspace_bytes(shard_lens, cap, B, H, D) -> int:
    arr, lens = _lens_array(shard_lens)
    return int(lib().uaa_ulysses_attn_bwd_workspace_bytes(len(lens), arr, cap, B, H, D))


def ulysses_attn_bwd(q_sh, k_sh, v_sh, out_sh, dout_sh, lse, shard_lens, key_mask=None, scale=None, dq=None,
                     dk=None, dv=None, workspace=None):
    """``uaa_ulysses_attn_bwd``: the backward of :func:`ulysses_attn_fwd` on the shards."""
    for n, t in (("k_sh", k_sh), ("v_sh", v_sh), ("out_sh", out_sh), ("dout_sh", dout_sh)):
        _shards(n, t, q_sh)
    _shards("q_sh", q_sh)
    _need_cuda(q_sh, k_sh, v_sh, out_sh, dout_sh, lse)
    P, B, cap, H, D = q_sh.shape
    arr, lens = _lens_array(shard_lens)
    if len(lens) != P:
        raise ValueError("len(shard_lens) must equal P")
    N = sum(lens)
    if lse.dtype != torch.float32 or tuple(lse.shape) != (B, H, N) or not lse.is_contiguous():
        raise ValueError("lse must be contiguous fp32 (B, H, N)")
    mask = normalize_key_mask(key_mask, B, N)
    if scale is None:
        scale = 1.0 / math.sqrt(D)
    dq = torch.empty_like(q_sh) if dq is None else dq
    dk = torch.empty_like(q_sh) if dk is None else dk
    dv = torch.empty_like(q_sh) if dv is None else dv
    nbytes = ulysses_attn_bwd_workspace_bytes(lens, cap, B, H, D)
    if workspace is None:
        workspace = torch.empty(max(nbytes, 1), dtype=torch.uint8, device=q_sh.device)
    wsb = workspace.numel() * workspace.element_size()
    _check(lib().uaa_ulysses_attn_bwd(_ptr(q_sh), _ptr(k_sh), _ptr(v_sh), _ptr(out_sh), _ptr(dout_sh), _ptr(lse),
                                      _ptr(mask), _ptr(dq), _ptr(dk), _ptr(dv), P, arr, cap, B, H, D, float(scale),
                                      _ptr(workspace), wsb, _P(_stream(q_sh.device))))
    return dq, dk, dv


class FusedUlyssesAttention(torch.autograd.Function):
    """Ulysses attention with the exchanges fused into the attention kernels (same result as
    :class:`UlyssesAttention` up to rounding; ``lse`` is ``(B, H, N)``, non-differentiable)."""

    @staticmethod
    def forward(ctx, q_sh, k_sh, v_sh, shard_lens, key_mask=None, scale=None, saved=None):
        _check_saved(saved)
        out, lse = ulysses_attn_fwd(q_sh, k_sh, v_sh, shard_lens, key_mask, scale)
        _save(ctx, saved, (q_sh, k_sh, v_sh, out), lse, key_mask=key_mask)
        ctx.shard_lens, ctx.scale = tuple(shard_lens), scale
        ctx.mark_non_differentiable(lse)
        return out, lse

    @staticmethod
    def backward(ctx, dout, _dlse):
        (q_sh, k_sh, v_sh, out), (lse,), key_mask = _saved(ctx, 4)
        dq, dk, dv = ulysses_attn_bwd(q_sh, k_sh, v_sh, out, dout.contiguous(), lse, ctx.shard_lens, key_mask,
                                      ctx.scale)
        return dq, dk, dv, None, None, None, None


def ulysses_attention_fused(q_sh, k_sh, v_sh, shard_lens, key_mask=None, scale=None, saved=None):
    return FusedUlyssesAttention.apply(q_sh, k_sh, v_sh, tuple(shard_lens), key_mask, scale, saved)
