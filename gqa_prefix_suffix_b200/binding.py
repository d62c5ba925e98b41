"""ctypes binding of the C ABI in include/dm05_suffix_attn.h.

Argument marshalling only: every step of the attention runs in the CUDA
library.  If the library is missing the import of the entry points fails
loudly; there is no other implementation behind these names.
"""
from __future__ import annotations

import contextlib
import ctypes
import os
import threading
from typing import NamedTuple, Optional

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libdm05_suffix_attn.so")

DM05_OK = 0
DM05_ERR_NULL = -1
DM05_ERR_SHAPE = -2
DM05_ERR_UNSUPPORTED = -3
DM05_ERR_ALIGN = -4
DM05_ERR_WORKSPACE = -5
DM05_ERR_CUDA = -6
DM05_EW_VALID_LEN_CLAMPED = 0x1
DM05_EW_WAIT_TIMEOUT = 0x2
DM05_EW_BAD_SPLIT = 0x4

DM05_FLAG_PREFIX_STATIC = 0x1

EXPORTS = ("dm05_suffix_attn", "dm05_suffix_attn_ex", "dm05_suffix_attn_workspace_bytes", "dm05_suffix_attn_reserve",
           "dm05_suffix_attn_plan", "dm05_set_split_override", "dm05_set_row_block_override",
           "dm05_get_error_word",
           "dm05_status_string", "dm05_release", "dm05_suffix_attn_noalloc", "dm05_suffix_attn_host",
           "dm05_suffix_attn_host_copy_bytes", "dm05_selftest_wait_timeout", "dm05_prefix_prefill_attn",
           "dm05_prefix_prefill_reserve", "dm05_prefix_prefill_plan", "dm05_suffix_qkv_prologue",
           "dm05_suffix_attn_steps_create", "dm05_suffix_attn_steps_launch", "dm05_suffix_attn_steps_destroy",
           "dm05_post_attention", "dm05_post_attention_reserve", "dm05_kv8_quantize", "dm05_suffix_attn_kv8",
           "dm05_suffix_attn_kv8_plan", "dm05_prefix_attn_mass", "dm05_prefix_attn_mass_kv8", "dm05_prefix_evict",
           "dm05_prefix_evict_kv8")

_lock = threading.Lock()
_lib = None


class Dm05Step(ctypes.Structure):
    """dm05_step: one call's own tensors (device addresses)."""
    _fields_ = [("q", ctypes.c_void_p), ("k_suffix", ctypes.c_void_p), ("v_suffix", ctypes.c_void_p),
                ("out", ctypes.c_void_p), ("lse", ctypes.c_void_p)]


class Dm05Error(RuntimeError):
    def __init__(self, status: int, what: str = ""):
        self.status = status
        super().__init__(f"{what}: {dm05_status_string(status)} ({status})" if what else
                         f"{dm05_status_string(status)} ({status})")


def lib() -> ctypes.CDLL:
    """The loaded library (raises if it has not been built)."""
    global _lib
    with _lock:
        if _lib is None:
            if not os.path.exists(LIB_PATH):
                raise RuntimeError(f"{LIB_PATH} is missing: build it with "
                                   "`python -m gqa_prefix_suffix_b200.build` (nvcc, sm_100a)")
            L = ctypes.CDLL(LIB_PATH)
            p, i, sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t
            L.dm05_suffix_attn.argtypes = [p] * 9 + [i] * 6 + [p]
            L.dm05_suffix_attn.restype = i
            L.dm05_suffix_attn_ex.argtypes = [p] * 9 + [i] * 6 + [ctypes.c_uint, p]
            L.dm05_suffix_attn_ex.restype = i
            L.dm05_suffix_attn_workspace_bytes.argtypes = [i] * 6
            L.dm05_suffix_attn_workspace_bytes.restype = sz
            L.dm05_suffix_attn_reserve.argtypes = [i] * 6 + [p]
            L.dm05_suffix_attn_reserve.restype = i
            L.dm05_suffix_attn_plan.argtypes = [i] * 6 + [ctypes.POINTER(i)] * 3
            L.dm05_suffix_attn_plan.restype = i
            L.dm05_set_split_override.argtypes = [i]
            L.dm05_set_split_override.restype = i
            L.dm05_set_row_block_override.argtypes = [i]
            L.dm05_set_row_block_override.restype = i
            L.dm05_get_error_word.argtypes = [p, ctypes.POINTER(ctypes.c_uint32)]
            L.dm05_get_error_word.restype = i
            L.dm05_status_string.argtypes = [i]
            L.dm05_status_string.restype = ctypes.c_char_p
            L.dm05_release.argtypes = []
            L.dm05_release.restype = None
            L.dm05_suffix_attn_noalloc.argtypes = [p] * 9 + [i] * 6 + [p]
            L.dm05_suffix_attn_noalloc.restype = i
            L.dm05_suffix_attn_host.argtypes = [p] * 9 + [i] * 6 + [p]
            L.dm05_suffix_attn_host.restype = i
            L.dm05_suffix_attn_host_copy_bytes.argtypes = [p] + [i] * 8 + [ctypes.POINTER(sz)] * 2
            L.dm05_suffix_attn_host_copy_bytes.restype = i
            L.dm05_selftest_wait_timeout.argtypes = [i, p]
            L.dm05_selftest_wait_timeout.restype = i
            L.dm05_prefix_prefill_attn.argtypes = [p] * 6 + [i] * 5 + [p]
            L.dm05_prefix_prefill_attn.restype = i
            L.dm05_prefix_prefill_reserve.argtypes = [i] * 5 + [p]
            L.dm05_prefix_prefill_reserve.restype = i
            L.dm05_prefix_prefill_plan.argtypes = [i] * 5 + [ctypes.POINTER(i)] * 3
            L.dm05_prefix_prefill_plan.restype = i
            L.dm05_suffix_qkv_prologue.argtypes = [p] * 8 + [i] * 6 + [ctypes.c_float] * 2 + [p]
            L.dm05_suffix_qkv_prologue.restype = i
            L.dm05_suffix_attn_steps_create.argtypes = [ctypes.POINTER(Dm05Step), i] + [p] * 4 + [i] * 6 + \
                [ctypes.c_uint, ctypes.POINTER(p)]
            L.dm05_suffix_attn_steps_create.restype = i
            L.dm05_suffix_attn_steps_launch.argtypes = [p, p]
            L.dm05_suffix_attn_steps_launch.restype = i
            L.dm05_suffix_attn_steps_destroy.argtypes = [p]
            L.dm05_suffix_attn_steps_destroy.restype = i
            L.dm05_post_attention.argtypes = [p] * 9 + [i] * 6 + [ctypes.c_float, p]
            L.dm05_post_attention.restype = i
            L.dm05_post_attention_reserve.argtypes = [i] * 6 + [p]
            L.dm05_post_attention_reserve.restype = i
            L.dm05_kv8_quantize.argtypes = [p] * 7 + [i] * 6 + [p]
            L.dm05_kv8_quantize.restype = i
            L.dm05_suffix_attn_kv8.argtypes = [p] * 5 + [i] + [p] * 7 + [sz] + [i] * 6 + [p]
            L.dm05_suffix_attn_kv8.restype = i
            L.dm05_suffix_attn_kv8_plan.argtypes = [i] * 6 + [ctypes.POINTER(i)] * 2 + [ctypes.POINTER(sz)]
            L.dm05_suffix_attn_kv8_plan.restype = i
            L.dm05_prefix_attn_mass.argtypes = [p] * 7 + [i] * 6 + [p]
            L.dm05_prefix_attn_mass.restype = i
            L.dm05_prefix_attn_mass_kv8.argtypes = [p] * 3 + [i] + [p] * 5 + [i] * 6 + [p]
            L.dm05_prefix_attn_mass_kv8.restype = i
            L.dm05_prefix_evict.argtypes = [p] * 10 + [i] * 8 + [p]
            L.dm05_prefix_evict.restype = i
            L.dm05_prefix_evict_kv8.argtypes = [p] * 4 + [i] + [p] * 10 + [i] * 8 + [p]
            L.dm05_prefix_evict_kv8.restype = i
            _lib = L
    return _lib


# ---- the C entry points, same names, integer pointers ------------------------

def dm05_suffix_attn(q, k_prefix, v_prefix, prefix_valid_len, prefix_mask, k_suffix, v_suffix,
                     out, lse, B, Hq, Hkv, P, S, D, stream) -> int:
    return lib().dm05_suffix_attn(q, k_prefix, v_prefix, prefix_valid_len, prefix_mask, k_suffix,
                                  v_suffix, out, lse, B, Hq, Hkv, P, S, D, stream)


def dm05_suffix_attn_ex(q, k_prefix, v_prefix, prefix_valid_len, prefix_mask, k_suffix, v_suffix,
                        out, lse, B, Hq, Hkv, P, S, D, flags, stream) -> int:
    """dm05_suffix_attn with option flags (DM05_FLAG_PREFIX_STATIC)."""
    return lib().dm05_suffix_attn_ex(q, k_prefix, v_prefix, prefix_valid_len, prefix_mask, k_suffix,
                                     v_suffix, out, lse, B, Hq, Hkv, P, S, D, flags, stream)


def dm05_suffix_attn_noalloc(q, k_prefix, v_prefix, prefix_valid_len, prefix_mask, k_suffix, v_suffix,
                             out, lse, B, Hq, Hkv, P, S, D, stream) -> int:
    """The allocation-free entry point (for callers that must not allocate
    device memory); same arguments as dm05_suffix_attn."""
    return lib().dm05_suffix_attn_noalloc(q, k_prefix, v_prefix, prefix_valid_len, prefix_mask, k_suffix,
                                          v_suffix, out, lse, B, Hq, Hkv, P, S, D, stream)


def dm05_suffix_attn_host(q, k_prefix, v_prefix, prefix_valid_len, prefix_mask, k_suffix, v_suffix,
                          out, lse, B, Hq, Hkv, P, S, D, stream) -> int:
    """The host-buffer entry point: every pointer is a host address."""
    return lib().dm05_suffix_attn_host(q, k_prefix, v_prefix, prefix_valid_len, prefix_mask, k_suffix,
                                       v_suffix, out, lse, B, Hq, Hkv, P, S, D, stream)


def dm05_suffix_attn_host_copy_bytes(prefix_valid_len, has_prefix_mask, want_lse, B, Hq, Hkv, P, S, D):
    """Returns (status, host-to-device bytes, device-to-host bytes) of one
    dm05_suffix_attn_host call; prefix_valid_len is a host address or None."""
    h, d = ctypes.c_size_t(0), ctypes.c_size_t(0)
    rc = lib().dm05_suffix_attn_host_copy_bytes(prefix_valid_len, int(bool(has_prefix_mask)), int(bool(want_lse)),
                                                B, Hq, Hkv, P, S, D, ctypes.byref(h), ctypes.byref(d))
    return rc, int(h.value), int(d.value)


def dm05_prefix_prefill_attn(q, k, v, valid_len, out, lse, B, Hq, Hkv, P, D, stream) -> int:
    """The prefix-prefill attention under the prefix-causal mask."""
    return lib().dm05_prefix_prefill_attn(q, k, v, valid_len, out, lse, B, Hq, Hkv, P, D, stream)


def dm05_prefix_prefill_reserve(B, Hq, Hkv, P, D, stream) -> int:
    return lib().dm05_prefix_prefill_reserve(B, Hq, Hkv, P, D, stream)


def dm05_prefix_prefill_plan(B, Hq, Hkv, P, D):
    """Returns (status, splits_per_head, query_block, row_blocks)."""
    sp, qb, rb = ctypes.c_int(0), ctypes.c_int(0), ctypes.c_int(0)
    rc = lib().dm05_prefix_prefill_plan(B, Hq, Hkv, P, D, ctypes.byref(sp), ctypes.byref(qb), ctypes.byref(rb))
    return rc, sp.value, qb.value, rb.value


def dm05_suffix_qkv_prologue(x, w, q_norm_w, k_norm_w, positions, q, k, v, B, S, H, Hq, Hkv, D, eps, theta,
                             stream) -> int:
    """QKV projection + QK-Norm + RoPE of the suffix tokens."""
    return lib().dm05_suffix_qkv_prologue(x, w, q_norm_w, k_norm_w, positions, q, k, v, B, S, H, Hq, Hkv, D,
                                          float(eps), float(theta), stream)


def dm05_suffix_attn_steps_create(steps, k_prefix, v_prefix, prefix_valid_len, prefix_mask, B, Hq, Hkv, P, S, D,
                                  flags=0):
    """steps: a list of (q, k_suffix, v_suffix, out, lse) device addresses.
    Returns (status, handle)."""
    arr = (Dm05Step * len(steps))(*[Dm05Step(*st) for st in steps])
    h = ctypes.c_void_p(0)
    rc = lib().dm05_suffix_attn_steps_create(arr, len(steps), k_prefix, v_prefix, prefix_valid_len, prefix_mask,
                                             B, Hq, Hkv, P, S, D, flags, ctypes.byref(h))
    return rc, h.value


def dm05_suffix_attn_steps_launch(handle, stream) -> int:
    return lib().dm05_suffix_attn_steps_launch(handle, stream)


def dm05_suffix_attn_steps_destroy(handle) -> int:
    return lib().dm05_suffix_attn_steps_destroy(handle)


def dm05_post_attention(attn, h, scale, shift, gate, wo, wgu, wd, out, B, S, Hq, D, Hd, F, eps, stream) -> int:
    """Output projection + residual, Adarms, GEGLU, MLP down + gated residual."""
    return lib().dm05_post_attention(attn, h, scale, shift, gate, wo, wgu, wd, out, B, S, Hq, D, Hd, F,
                                     float(eps), stream)


def dm05_post_attention_reserve(B, S, Hq, D, Hd, F, stream) -> int:
    return lib().dm05_post_attention_reserve(B, S, Hq, D, Hd, F, stream)


def dm05_kv8_quantize(k, v, valid_len, k8, v8, k_scale, v_scale, B, Hkv, P, D, block, first, stream) -> int:
    """The 8-bit form (e4m3 codes, a scale per block of tokens and KV head) of a prefix cache."""
    return lib().dm05_kv8_quantize(k, v, valid_len, k8, v8, k_scale, v_scale, B, Hkv, P, D, block, first, stream)


def dm05_suffix_attn_kv8(q, k8, v8, k_scale, v_scale, block, prefix_valid_len, prefix_mask, k_suffix, v_suffix, out,
                         lse, workspace, workspace_bytes, B, Hq, Hkv, P, S, D, stream) -> int:
    """The suffix attention over an 8-bit prefix cache."""
    return lib().dm05_suffix_attn_kv8(q, k8, v8, k_scale, v_scale, block, prefix_valid_len, prefix_mask, k_suffix,
                                      v_suffix, out, lse, workspace, workspace_bytes, B, Hq, Hkv, P, S, D, stream)


def dm05_suffix_attn_kv8_plan(B, Hq, Hkv, P, S, D):
    """Returns (status, splits_per_head, tile_rows, workspace_bytes)."""
    sp, tr, ws = ctypes.c_int(0), ctypes.c_int(0), ctypes.c_size_t(0)
    rc = lib().dm05_suffix_attn_kv8_plan(B, Hq, Hkv, P, S, D, ctypes.byref(sp), ctypes.byref(tr), ctypes.byref(ws))
    return rc, sp.value, tr.value, ws.value


def dm05_prefix_attn_mass(q, k_prefix, prefix_valid_len, prefix_mask, lse, mass_in, mass, B, Hq, Hkv, P, S, D,
                          stream) -> int:
    """The attention weight each prefix position received, from a bf16 cache."""
    return lib().dm05_prefix_attn_mass(q, k_prefix, prefix_valid_len, prefix_mask, lse, mass_in, mass, B, Hq, Hkv, P,
                                       S, D, stream)


def dm05_prefix_attn_mass_kv8(q, k8, k_scale, block, prefix_valid_len, prefix_mask, lse, mass_in, mass, B, Hq, Hkv,
                              P, S, D, stream) -> int:
    """The same from an 8-bit cache."""
    return lib().dm05_prefix_attn_mass_kv8(q, k8, k_scale, block, prefix_valid_len, prefix_mask, lse, mass_in, mass,
                                           B, Hq, Hkv, P, S, D, stream)


def dm05_prefix_evict(k, v, mass, valid_len, mask, k_out, v_out, mass_out, positions, valid_out, B, Hkv, P, P_out, D,
                      n_keep, n_first, n_last, stream) -> int:
    """Keeps the positions of largest mass in a smaller bf16 cache."""
    return lib().dm05_prefix_evict(k, v, mass, valid_len, mask, k_out, v_out, mass_out, positions, valid_out, B, Hkv,
                                   P, P_out, D, n_keep, n_first, n_last, stream)


def dm05_prefix_evict_kv8(k8, v8, k_scale, v_scale, block, mass, valid_len, mask, k8_out, v8_out, k_scale_out,
                          v_scale_out, mass_out, positions, valid_out, B, Hkv, P, P_out, D, n_keep, n_first, n_last,
                          stream) -> int:
    """The same on an 8-bit cache."""
    return lib().dm05_prefix_evict_kv8(k8, v8, k_scale, v_scale, block, mass, valid_len, mask, k8_out, v8_out,
                                       k_scale_out, v_scale_out, mass_out, positions, valid_out, B, Hkv, P, P_out, D,
                                       n_keep, n_first, n_last, stream)


def post_attention(attn, h, scale, shift, gate, wo, wgu, wd, eps=1e-6, out=None, stream=None):
    """The post-attention block on CUDA torch tensors; returns out [B*S, Hd] bf16."""
    import torch
    B, Hq, S, D = attn.shape
    Hd = h.shape[1]
    F = wgu.shape[0] // 2
    for name, t, shape in (("attn", attn, (B, Hq, S, D)), ("h", h, (B * S, Hd)), ("scale", scale, (B, Hd)),
                           ("shift", shift, (B, Hd)), ("gate", gate, (B, Hd)), ("wo", wo, (Hd, Hq * D)),
                           ("wgu", wgu, (2 * F, Hd)), ("wd", wd, (Hd, F))):
        if (not t.is_cuda or t.dtype != torch.bfloat16 or tuple(t.shape) != shape or not t.is_contiguous()
                or t.device != attn.device):
            raise ValueError(f"{name} must be a contiguous CUDA bfloat16 tensor {list(shape)} on {attn.device}")
    if out is None:
        out = torch.empty((B * S, Hd), dtype=torch.bfloat16, device=attn.device)
    if (not out.is_cuda or out.dtype != torch.bfloat16 or tuple(out.shape) != (B * S, Hd) or not out.is_contiguous()):
        raise ValueError(f"out must be a contiguous CUDA bfloat16 tensor {[B * S, Hd]}")
    rc = dm05_post_attention(attn.data_ptr(), h.data_ptr(), scale.data_ptr(), shift.data_ptr(), gate.data_ptr(),
                             wo.data_ptr(), wgu.data_ptr(), wd.data_ptr(), out.data_ptr(), B, S, Hq, D, Hd, F, eps,
                             _stream_handle(stream))
    if rc != DM05_OK:
        raise Dm05Error(rc, "dm05_post_attention")
    return out


def dm05_suffix_attn_workspace_bytes(B, Hq, Hkv, P, S, D) -> int:
    return int(lib().dm05_suffix_attn_workspace_bytes(B, Hq, Hkv, P, S, D))


def dm05_suffix_attn_reserve(B, Hq, Hkv, P, S, D, stream) -> int:
    return lib().dm05_suffix_attn_reserve(B, Hq, Hkv, P, S, D, stream)


def dm05_suffix_attn_plan(B, Hq, Hkv, P, S, D):
    """Returns (status, splits_per_head, tile_rows, row_blocks)."""
    sp, tr, rb = ctypes.c_int(0), ctypes.c_int(0), ctypes.c_int(0)
    rc = lib().dm05_suffix_attn_plan(B, Hq, Hkv, P, S, D, ctypes.byref(sp), ctypes.byref(tr), ctypes.byref(rb))
    return rc, sp.value, tr.value, rb.value


def dm05_set_split_override(splits_per_head: int) -> int:
    _kv8_workspace_bytes.clear()
    return lib().dm05_set_split_override(splits_per_head)


def dm05_set_row_block_override(row_blocks: int) -> int:
    return lib().dm05_set_row_block_override(row_blocks)


def dm05_selftest_wait_timeout(limit_ms: int, stream) -> int:
    """Launches the bounded-wait self-test (a wait that must run out)."""
    return lib().dm05_selftest_wait_timeout(limit_ms, stream)


def dm05_get_error_word(stream):
    """Returns (status, error bits); synchronises the stream and clears the bits."""
    w = ctypes.c_uint32(0)
    rc = lib().dm05_get_error_word(stream, ctypes.byref(w))
    return rc, int(w.value)


def dm05_status_string(status: int) -> str:
    return lib().dm05_status_string(status).decode()


def dm05_release() -> None:
    lib().dm05_release()


# ---- torch front end (marshalling only) -------------------------------------

def _stream_handle(stream):
    import torch
    if stream is None:
        stream = torch.cuda.current_stream()
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def suffix_attn(q, k_prefix, v_prefix, k_suffix, v_suffix, prefix_valid_len=None, prefix_mask=None,
                out=None, lse=None, want_lse: bool = True, stream=None, prefix_static: bool = False):
    """Suffix attention on CUDA torch tensors; returns (out, lse or None).

    q [B,Hq,S,D] bf16; k_prefix/v_prefix [B,Hkv,P,D] bf16; k_suffix/v_suffix
    [B,Hkv,S,D] bf16; prefix_valid_len int32 [B] or None; prefix_mask uint8
    [B,P] or None.  out (bf16 [B,Hq,S,D]) and lse (fp32 [B,Hq,S]) are
    allocated when not given."""
    import torch
    B, Hq, S, D = q.shape
    Hkv, P = k_prefix.shape[1], k_prefix.shape[2]
    for name, t, dt in (("q", q, torch.bfloat16), ("k_prefix", k_prefix, torch.bfloat16),
                        ("v_prefix", v_prefix, torch.bfloat16), ("k_suffix", k_suffix, torch.bfloat16),
                        ("v_suffix", v_suffix, torch.bfloat16)):
        if not t.is_cuda or t.dtype != dt or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous CUDA {dt} tensor")
    if tuple(k_prefix.shape) != (B, Hkv, P, D) or tuple(v_prefix.shape) != (B, Hkv, P, D):
        raise ValueError("k_prefix/v_prefix must be [B,Hkv,P,D]")
    if tuple(k_suffix.shape) != (B, Hkv, S, D) or tuple(v_suffix.shape) != (B, Hkv, S, D):
        raise ValueError("k_suffix/v_suffix must be [B,Hkv,S,D]")
    if prefix_valid_len is not None:
        if (not prefix_valid_len.is_cuda or prefix_valid_len.dtype != torch.int32 or prefix_valid_len.numel() != B
                or not prefix_valid_len.is_contiguous()):
            raise ValueError("prefix_valid_len must be a contiguous CUDA int32 tensor of B values")
    if prefix_mask is not None:
        if (not prefix_mask.is_cuda or prefix_mask.dtype != torch.uint8 or tuple(prefix_mask.shape) != (B, P)
                or not prefix_mask.is_contiguous()):
            raise ValueError("prefix_mask must be a contiguous CUDA uint8 tensor [B,P]")
    if out is None:
        out = torch.empty((B, Hq, S, D), dtype=torch.bfloat16, device=q.device)
    if lse is None and want_lse:
        lse = torch.empty((B, Hq, S), dtype=torch.float32, device=q.device)
    # the library writes B*Hq*S rows through these pointers: a smaller or
    # strided buffer would be overrun
    for name, t, shape, dt in (("out", out, (B, Hq, S, D), torch.bfloat16), ("lse", lse, (B, Hq, S), torch.float32)):
        if t is not None and (not t.is_cuda or t.dtype != dt or tuple(t.shape) != shape or not t.is_contiguous()):
            raise ValueError(f"{name} must be a contiguous CUDA {dt} tensor {list(shape)}")
    for name, t in (("k_prefix", k_prefix), ("v_prefix", v_prefix), ("k_suffix", k_suffix), ("v_suffix", v_suffix),
                    ("prefix_valid_len", prefix_valid_len), ("prefix_mask", prefix_mask), ("out", out), ("lse", lse)):
        if t is not None and t.device != q.device:
            raise ValueError(f"{name} must be on {q.device} like q")
    ptr = lambda t: None if t is None else t.data_ptr()
    rc = dm05_suffix_attn_ex(ptr(q), ptr(k_prefix), ptr(v_prefix), ptr(prefix_valid_len), ptr(prefix_mask),
                             ptr(k_suffix), ptr(v_suffix), ptr(out), ptr(lse), B, Hq, Hkv, P, S, D,
                             DM05_FLAG_PREFIX_STATIC if prefix_static else 0, _stream_handle(stream))
    if rc != DM05_OK:
        raise Dm05Error(rc, "dm05_suffix_attn")
    return out, lse


def suffix_attn_host(q, k_prefix, v_prefix, k_suffix, v_suffix, prefix_valid_len=None, prefix_mask=None,
                     out=None, lse=None, want_lse: bool = True, stream=None):
    """Suffix attention on CPU torch tensors (page-locked for asynchronous
    copies) through dm05_suffix_attn_host; returns (out, lse or None), host
    tensors that hold the result once `stream` has passed the call.

    Shapes and dtypes are those of suffix_attn; every tensor, out and lse
    included, must be a contiguous CPU tensor."""
    import torch
    B, Hq, S, D = q.shape
    Hkv, P = k_prefix.shape[1], k_prefix.shape[2]
    for name, t, dt in (("q", q, torch.bfloat16), ("k_prefix", k_prefix, torch.bfloat16),
                        ("v_prefix", v_prefix, torch.bfloat16), ("k_suffix", k_suffix, torch.bfloat16),
                        ("v_suffix", v_suffix, torch.bfloat16)):
        if t.is_cuda or t.dtype != dt or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous CPU {dt} tensor")
    if tuple(k_prefix.shape) != (B, Hkv, P, D) or tuple(v_prefix.shape) != (B, Hkv, P, D):
        raise ValueError("k_prefix/v_prefix must be [B,Hkv,P,D]")
    if tuple(k_suffix.shape) != (B, Hkv, S, D) or tuple(v_suffix.shape) != (B, Hkv, S, D):
        raise ValueError("k_suffix/v_suffix must be [B,Hkv,S,D]")
    if prefix_valid_len is not None and (prefix_valid_len.is_cuda or prefix_valid_len.dtype != torch.int32
                                         or prefix_valid_len.numel() != B or not prefix_valid_len.is_contiguous()):
        raise ValueError("prefix_valid_len must be a contiguous CPU int32 tensor of B values")
    if prefix_mask is not None and (prefix_mask.is_cuda or prefix_mask.dtype != torch.uint8
                                    or tuple(prefix_mask.shape) != (B, P) or not prefix_mask.is_contiguous()):
        raise ValueError("prefix_mask must be a contiguous CPU uint8 tensor [B,P]")
    pin = q.is_pinned()
    if out is None:
        out = torch.empty((B, Hq, S, D), dtype=torch.bfloat16, pin_memory=pin)
    if lse is None and want_lse:
        lse = torch.empty((B, Hq, S), dtype=torch.float32, pin_memory=pin)
    for name, t, shape, dt in (("out", out, (B, Hq, S, D), torch.bfloat16), ("lse", lse, (B, Hq, S), torch.float32)):
        if t is not None and (t.is_cuda or t.dtype != dt or tuple(t.shape) != shape or not t.is_contiguous()):
            raise ValueError(f"{name} must be a contiguous CPU {dt} tensor {list(shape)}")
    ptr = lambda t: None if t is None else t.data_ptr()
    rc = dm05_suffix_attn_host(ptr(q), ptr(k_prefix), ptr(v_prefix), ptr(prefix_valid_len), ptr(prefix_mask),
                               ptr(k_suffix), ptr(v_suffix), ptr(out), ptr(lse), B, Hq, Hkv, P, S, D,
                               _stream_handle(stream))
    if rc != DM05_OK:
        raise Dm05Error(rc, "dm05_suffix_attn_host")
    return out, lse


def prefix_prefill_attn(q, k, v, valid_len=None, out=None, lse=None, want_lse: bool = True, stream=None):
    """Prefix-prefill attention on CUDA torch tensors; returns (out, lse or None).

    q [B,Hq,P,D] bf16; k/v [B,Hkv,P,D] bf16; valid_len int32 [B] or None.
    Rows at or past a sample's valid length are not written (a fresh out /
    lse is allocated uninitialised when not given)."""
    import torch
    B, Hq, P, D = q.shape
    Hkv = k.shape[1]
    for name, t in (("q", q), ("k", k), ("v", v)):
        if not t.is_cuda or t.dtype != torch.bfloat16 or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous CUDA bfloat16 tensor")
    if tuple(k.shape) != (B, Hkv, P, D) or tuple(v.shape) != (B, Hkv, P, D):
        raise ValueError("k/v must be [B,Hkv,P,D]")
    if valid_len is not None and (not valid_len.is_cuda or valid_len.dtype != torch.int32 or valid_len.numel() != B
                                  or not valid_len.is_contiguous()):
        raise ValueError("valid_len must be a contiguous CUDA int32 tensor of B values")
    if out is None:
        out = torch.empty((B, Hq, P, D), dtype=torch.bfloat16, device=q.device)
    if lse is None and want_lse:
        lse = torch.empty((B, Hq, P), dtype=torch.float32, device=q.device)
    for name, t, shape, dt in (("out", out, (B, Hq, P, D), torch.bfloat16), ("lse", lse, (B, Hq, P), torch.float32)):
        if t is not None and (not t.is_cuda or t.dtype != dt or tuple(t.shape) != shape or not t.is_contiguous()):
            raise ValueError(f"{name} must be a contiguous CUDA {dt} tensor {list(shape)}")
    for name, t in (("k", k), ("v", v), ("valid_len", valid_len), ("out", out), ("lse", lse)):
        if t is not None and t.device != q.device:
            raise ValueError(f"{name} must be on {q.device} like q")
    ptr = lambda t: None if t is None else t.data_ptr()
    rc = dm05_prefix_prefill_attn(ptr(q), ptr(k), ptr(v), ptr(valid_len), ptr(out), ptr(lse), B, Hq, Hkv, P, D,
                                  _stream_handle(stream))
    if rc != DM05_OK:
        raise Dm05Error(rc, "dm05_prefix_prefill_attn")
    return out, lse


def suffix_qkv_prologue(x, w, q_norm_w, k_norm_w, positions, B, S, Hq=8, Hkv=4, D=256, eps=1e-6, theta=10000.0,
                        q=None, k=None, v=None, stream=None):
    """QKV projection + QK-Norm + RoPE on CUDA torch tensors; returns (q, k, v)
    in the suffix attention's layout.  x [B*S, H] bf16, w [(Hq+2Hkv)*D, H]
    bf16, norm weights [D] bf16, positions int32 [B*S]."""
    import torch
    H = x.shape[1]
    for name, t, shape, dt in (("x", x, (B * S, H), torch.bfloat16), ("w", w, ((Hq + 2 * Hkv) * D, H), torch.bfloat16),
                               ("q_norm_w", q_norm_w, (D,), torch.bfloat16), ("k_norm_w", k_norm_w, (D,), torch.bfloat16),
                               ("positions", positions, (B * S,), torch.int32)):
        if not t.is_cuda or t.dtype != dt or tuple(t.shape) != shape or not t.is_contiguous() or t.device != x.device:
            raise ValueError(f"{name} must be a contiguous CUDA {dt} tensor {list(shape)} on {x.device}")
    if q is None:
        q = torch.empty((B, Hq, S, D), dtype=torch.bfloat16, device=x.device)
    if k is None:
        k = torch.empty((B, Hkv, S, D), dtype=torch.bfloat16, device=x.device)
    if v is None:
        v = torch.empty((B, Hkv, S, D), dtype=torch.bfloat16, device=x.device)
    for name, t, shape in (("q", q, (B, Hq, S, D)), ("k", k, (B, Hkv, S, D)), ("v", v, (B, Hkv, S, D))):
        if not t.is_cuda or t.dtype != torch.bfloat16 or tuple(t.shape) != shape or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous CUDA bfloat16 tensor {list(shape)}")
    rc = dm05_suffix_qkv_prologue(x.data_ptr(), w.data_ptr(), q_norm_w.data_ptr(), k_norm_w.data_ptr(),
                                  positions.data_ptr(), q.data_ptr(), k.data_ptr(), v.data_ptr(), B, S, H, Hq, Hkv, D,
                                  eps, theta, _stream_handle(stream))
    if rc != DM05_OK:
        raise Dm05Error(rc, "dm05_suffix_qkv_prologue")
    return q, k, v


def reserve_for(q, k_prefix, stream=None) -> None:
    """dm05_suffix_attn_reserve for the sizes of these tensors (call before graph capture)."""
    B, Hq, S, D = q.shape
    rc = dm05_suffix_attn_reserve(B, Hq, k_prefix.shape[1], k_prefix.shape[2], S, D, _stream_handle(stream))
    if rc != DM05_OK:
        raise Dm05Error(rc, "dm05_suffix_attn_reserve")


# ---- prefix-cache compression -----------------------------------------------

class Kv8Cache(NamedTuple):
    """A prefix cache held in 8 bits: row j of k stands for
    k_scale[..., j // block] * k[..., j, :], and the same for v.

    k, v: float8_e4m3fn [B, Hkv, P, D]; k_scale, v_scale: fp32
    [B, Hkv, ceil(P / block)]; block: 16, 32, 64 or 128 positions."""
    k: "torch.Tensor"
    v: "torch.Tensor"
    k_scale: "torch.Tensor"
    v_scale: "torch.Tensor"
    block: int


class EvictedPrefix(NamedTuple):
    """What prefix_evict keeps: the smaller cache, the kept positions' mass
    (fp32 [B, Hkv, P_out], 0 behind the kept rows), where each row came from
    (int32 [B, Hkv, P_out], -1 behind them) and its valid lengths (int32 [B])."""
    k: "torch.Tensor"
    v: "torch.Tensor"
    mass: "torch.Tensor"
    positions: "torch.Tensor"
    valid_len: "torch.Tensor"


class EvictedPrefixKv8(NamedTuple):
    """The same for an 8-bit cache."""
    cache: Kv8Cache
    mass: "torch.Tensor"
    positions: "torch.Tensor"
    valid_len: "torch.Tensor"


def _need(name, t, dtype, shape, index):
    """A dense tensor of this type and shape on CUDA device `index`, or ValueError."""
    if t.dtype != dtype or t.shape != shape or t.get_device() != index or index < 0 or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous CUDA {dtype} tensor {list(shape)}"
                         + (f" on cuda:{index}" if index >= 0 else ""))


def _need_prefix(valid_len, mask, B, P, index):
    import torch
    if valid_len is not None:
        _need("prefix_valid_len", valid_len, torch.int32, (B,), index)
    if mask is not None:
        _need("prefix_mask", mask, torch.uint8, (B, P), index)


def _need_cache(name, cache, index):
    """Checks an 8-bit cache; returns its (B, Hkv, P, D)."""
    import torch
    k, v, ks, vs, block = cache
    if k.dim() != 4:
        raise ValueError(f"{name}.k must be [B,Hkv,P,D]")
    shape = k.shape
    B, Hkv, P, D = shape
    if block not in (16, 32, 64, 128):
        raise ValueError(f"{name}.block must be 16, 32, 64 or 128")
    scales = (B, Hkv, -(-P // block))
    _need(f"{name}.k", k, torch.float8_e4m3fn, shape, index)
    _need(f"{name}.v", v, torch.float8_e4m3fn, shape, index)
    _need(f"{name}.k_scale", ks, torch.float32, scales, index)
    _need(f"{name}.v_scale", vs, torch.float32, scales, index)
    return B, Hkv, P, D


def _current_stream_handle(index):
    """Handle of the current stream of CUDA device `index`."""
    import torch
    raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)  # without building a Stream object (3 us)
    return raw(index) if raw is not None else torch.cuda.current_stream(index).cuda_stream


def _on(index, stream, call):
    """call(stream handle) with the tensors' device current and `stream` the
    stream that newly allocated tensors belong to."""
    import torch
    if stream is None and torch.cuda.current_device() == index:
        return call(_current_stream_handle(index))
    with torch.cuda.device(index):
        if stream is None:
            return call(_current_stream_handle(index))
        if not hasattr(stream, "cuda_stream"):
            h = int(stream)
            stream = torch.cuda.ExternalStream(h, device=index) if h else torch.cuda.default_stream(index)
        if stream.device.index != index:
            raise ValueError(f"stream must be on cuda:{index} like the tensors")
        with torch.cuda.stream(stream):
            return call(stream.cuda_stream)


def _ptr(t):
    return None if t is None else t.data_ptr()


def _check(rc, what):
    if rc != DM05_OK:
        raise Dm05Error(rc, what)


def _codes(shape, index):
    import torch
    return torch.zeros(shape, dtype=torch.uint8, device=index).view(torch.float8_e4m3fn)


def _empty_cache(B, Hkv, P, D, block, index):
    """Zero codes and unit scales."""
    import torch
    shape, scales = (B, Hkv, P, D), (B, Hkv, -(-P // block))
    ones = [torch.ones(scales, dtype=torch.float32, device=index) for _ in range(2)]
    return Kv8Cache(_codes(shape, index), _codes(shape, index), ones[0], ones[1], block)


def kv8_quantize(k, v, block: int = 64, valid_len=None, first: int = 0, out: Optional[Kv8Cache] = None, stream=None):
    """The 8-bit form of a bf16 prefix cache [B,Hkv,P,D]; returns the Kv8Cache.

    Rows [first, valid_len) are written (first a multiple of the block, for a
    prefix that is quantised in pieces); a fresh cache has zero codes and unit
    scales elsewhere.  With `out` given, its block is used and everything else
    in it is left as it was."""
    import torch
    if k.dim() != 4:
        raise ValueError("k must be [B,Hkv,P,D]")
    shape = k.shape
    B, Hkv, P, D = shape
    dev = k.get_device()
    _need("k", k, torch.bfloat16, shape, dev)
    _need("v", v, torch.bfloat16, shape, dev)
    if valid_len is not None:
        _need("valid_len", valid_len, torch.int32, (B,), dev)
    if out is None:
        if block not in (16, 32, 64, 128):
            raise ValueError("block must be 16, 32, 64 or 128")
    elif _need_cache("out", out, dev) != (B, Hkv, P, D):
        raise ValueError("out must be a cache of k's sizes")

    def call(s):
        c = _empty_cache(B, Hkv, P, D, block, dev) if out is None else out
        _check(dm05_kv8_quantize(k.data_ptr(), v.data_ptr(), _ptr(valid_len), c.k.data_ptr(), c.v.data_ptr(),
                                 c.k_scale.data_ptr(), c.v_scale.data_ptr(), B, Hkv, P, D, c.block, first, s),
               "dm05_kv8_quantize")
        return c
    return _on(dev, stream, call)


_kv8_workspace_bytes: dict = {}  # sizes and device -> bytes; a split override changes plans and clears it


def _kv8_workspace(key):
    need = _kv8_workspace_bytes.get(key)
    if need is None:
        rc, _, _, need = dm05_suffix_attn_kv8_plan(*key[:6])
        _check(rc, "dm05_suffix_attn_kv8")
        if len(_kv8_workspace_bytes) > 4096:
            _kv8_workspace_bytes.clear()
        _kv8_workspace_bytes[key] = need
    return need


def suffix_attn_kv8(q, cache: Kv8Cache, k_suffix, v_suffix, prefix_valid_len=None, prefix_mask=None, out=None,
                    lse=None, want_lse: bool = True, workspace=None, stream=None):
    """Suffix attention over an 8-bit prefix cache; returns (out, lse or None).

    As suffix_attn, with the prefix in a Kv8Cache.  workspace: a contiguous
    uint8 CUDA tensor of at least dm05_suffix_attn_kv8_plan's bytes that no
    call running at the same time uses; allocated for the call when not given."""
    import torch
    if q.dim() != 4:
        raise ValueError("q must be [B,Hq,S,D]")
    shape = q.shape
    B, Hq, S, D = shape
    dev = q.get_device()
    bf = torch.bfloat16
    _need("q", q, bf, shape, dev)
    Bc, Hkv, P, Dc = _need_cache("cache", cache, dev)
    if Bc != B or Dc != D:
        raise ValueError("cache must have q's batch and head size")
    suffix = (B, Hkv, S, D)
    _need("k_suffix", k_suffix, bf, suffix, dev)
    _need("v_suffix", v_suffix, bf, suffix, dev)
    _need_prefix(prefix_valid_len, prefix_mask, B, P, dev)
    if out is not None:
        _need("out", out, bf, shape, dev)
    if lse is not None:
        _need("lse", lse, torch.float32, (B, Hq, S), dev)
    if workspace is not None:
        _need("workspace", workspace, torch.uint8, (workspace.numel(),), dev)

    def call(s):
        o = torch.empty(shape, dtype=bf, device=dev) if out is None else out
        ls = torch.empty((B, Hq, S), dtype=torch.float32, device=dev) if lse is None and want_lse else lse
        key = (B, Hq, Hkv, P, S, D, dev)
        for attempt in range(2):
            ws = workspace
            if ws is None:
                need = _kv8_workspace(key)
                ws = torch.empty(need, dtype=torch.uint8, device=dev) if need else None
            rc = dm05_suffix_attn_kv8(q.data_ptr(), cache.k.data_ptr(), cache.v.data_ptr(), cache.k_scale.data_ptr(),
                                      cache.v_scale.data_ptr(), cache.block, _ptr(prefix_valid_len), _ptr(prefix_mask),
                                      k_suffix.data_ptr(), v_suffix.data_ptr(), o.data_ptr(), _ptr(ls), _ptr(ws),
                                      0 if ws is None else ws.numel(), B, Hq, Hkv, P, S, D, s)
            if rc != DM05_ERR_WORKSPACE or workspace is not None or _kv8_workspace_bytes.pop(key, None) is None:
                break  # else a plan was forced past this module: ask for its workspace again
        _check(rc, "dm05_suffix_attn_kv8")
        return o, ls
    return _on(dev, stream, call)


def _mass(q, k, k_scale, block, lse, valid_len, mask, mass_in, mass, stream):
    import torch
    if q.dim() != 4 or k.dim() != 4:
        raise ValueError("q must be [B,Hq,S,D] and the keys [B,Hkv,P,D]")
    B, Hq, S, D = q.shape
    Hkv, P = k.shape[1], k.shape[2]
    dev = q.get_device()
    _need("q", q, torch.bfloat16, (B, Hq, S, D), dev)
    if k_scale is None:
        _need("k_prefix", k, torch.bfloat16, (B, Hkv, P, D), dev)
    else:
        if block not in (16, 32, 64, 128):
            raise ValueError("block must be 16, 32, 64 or 128")
        _need("k8", k, torch.float8_e4m3fn, (B, Hkv, P, D), dev)
        _need("k_scale", k_scale, torch.float32, (B, Hkv, -(-P // block)), dev)
    _need("lse", lse, torch.float32, (B, Hq, S), dev)
    _need_prefix(valid_len, mask, B, P, dev)
    if mass_in is not None:
        _need("mass_in", mass_in, torch.float32, (B, Hkv, P), dev)
    if mass is not None:
        _need("mass", mass, torch.float32, (B, Hkv, P), dev)

    def call(s):
        m = torch.empty((B, Hkv, P), dtype=torch.float32, device=dev) if mass is None else mass
        if k_scale is None:
            rc = dm05_prefix_attn_mass(q.data_ptr(), k.data_ptr(), _ptr(valid_len), _ptr(mask), lse.data_ptr(),
                                       _ptr(mass_in), m.data_ptr(), B, Hq, Hkv, P, S, D, s)
        else:
            rc = dm05_prefix_attn_mass_kv8(q.data_ptr(), k.data_ptr(), k_scale.data_ptr(), block, _ptr(valid_len),
                                           _ptr(mask), lse.data_ptr(), _ptr(mass_in), m.data_ptr(), B, Hq, Hkv, P, S,
                                           D, s)
        _check(rc, "dm05_prefix_attn_mass")
        return m
    return _on(dev, stream, call)


def prefix_attn_mass(q, k_prefix, lse, prefix_valid_len=None, prefix_mask=None, mass_in=None, mass=None, stream=None):
    """The attention weight that each prefix position received in a
    suffix_attn call with this q, lse and masks, summed over the queries of
    each KV head and added to mass_in; returns fp32 [B,Hkv,P] (`mass`, which
    may be mass_in itself, when given)."""
    return _mass(q, k_prefix, None, 0, lse, prefix_valid_len, prefix_mask, mass_in, mass, stream)


def prefix_attn_mass_kv8(q, k8, k_scale, block, lse, prefix_valid_len=None, prefix_mask=None, mass_in=None, mass=None,
                         stream=None):
    """prefix_attn_mass over the keys of an 8-bit cache (its k, k_scale and block)."""
    if k_scale is None:
        raise ValueError("k_scale must be given")
    return _mass(q, k8, k_scale, block, lse, prefix_valid_len, prefix_mask, mass_in, mass, stream)


def _need_evicted(mass, B, Hkv, P, P_out, valid_len_in, mask, mass_out, positions, valid_len, index):
    import torch
    _need("mass", mass, torch.float32, (B, Hkv, P), index)
    _need_prefix(valid_len_in, mask, B, P, index)
    if mass_out is not None:
        _need("mass_out", mass_out, torch.float32, (B, Hkv, P_out), index)
    if positions is not None:
        _need("positions", positions, torch.int32, (B, Hkv, P_out), index)
    if valid_len is not None:
        _need("valid_len", valid_len, torch.int32, (B,), index)


def _evict_outputs(B, Hkv, P_out, mass_out, positions, valid_len, index):
    import torch
    if mass_out is None:
        mass_out = torch.empty((B, Hkv, P_out), dtype=torch.float32, device=index)
    if positions is None:
        positions = torch.empty((B, Hkv, P_out), dtype=torch.int32, device=index)
    if valid_len is None:
        valid_len = torch.empty((B,), dtype=torch.int32, device=index)
    return mass_out, positions, valid_len


def prefix_evict(k, v, mass, n_keep: int, n_first: int = 0, n_last: int = 0, prefix_valid_len=None, prefix_mask=None,
                 bucket: Optional[int] = None, k_out=None, v_out=None, mass_out=None, positions=None, valid_len=None,
                 stream=None) -> EvictedPrefix:
    """Keeps the n_keep visible positions of largest mass per (sample, KV
    head), the first n_first and the last n_last in range before all others,
    in a cache of `bucket` rows (n_keep, or k_out's, when not given).  Fresh
    outputs hold zeros behind the kept rows; given ones keep what they held
    there."""
    import torch
    if k.dim() != 4:
        raise ValueError("k must be [B,Hkv,P,D]")
    B, Hkv, P, D = k.shape
    dev = k.get_device()
    bf = torch.bfloat16
    if (k_out is None) != (v_out is None):
        raise ValueError("k_out and v_out must be given together")
    if k_out is not None and k_out.dim() == 4 and bucket is None:
        bucket = k_out.shape[2]
    bucket = n_keep if bucket is None else bucket
    _need("k", k, bf, (B, Hkv, P, D), dev)
    _need("v", v, bf, (B, Hkv, P, D), dev)
    if k_out is not None:
        _need("k_out", k_out, bf, (B, Hkv, bucket, D), dev)
        _need("v_out", v_out, bf, (B, Hkv, bucket, D), dev)
    _need_evicted(mass, B, Hkv, P, bucket, prefix_valid_len, prefix_mask, mass_out, positions, valid_len, dev)

    def call(s):
        ko, vo = k_out, v_out
        if ko is None:
            ko, vo = [torch.zeros((B, Hkv, max(bucket, 0), D), dtype=bf, device=dev) for _ in range(2)]
        mo, po, vl = _evict_outputs(B, Hkv, max(bucket, 0), mass_out, positions, valid_len, dev)
        _check(dm05_prefix_evict(k.data_ptr(), v.data_ptr(), mass.data_ptr(), _ptr(prefix_valid_len),
                                 _ptr(prefix_mask), ko.data_ptr(), vo.data_ptr(), mo.data_ptr(), po.data_ptr(),
                                 vl.data_ptr(), B, Hkv, P, bucket, D, n_keep, n_first, n_last, s), "dm05_prefix_evict")
        return EvictedPrefix(ko, vo, mo, po, vl)
    return _on(dev, stream, call)


def prefix_evict_kv8(cache: Kv8Cache, mass, n_keep: int, n_first: int = 0, n_last: int = 0, prefix_valid_len=None,
                     prefix_mask=None, bucket: Optional[int] = None, out: Optional[Kv8Cache] = None, mass_out=None,
                     positions=None, valid_len=None, stream=None) -> EvictedPrefixKv8:
    """prefix_evict on an 8-bit cache: the kept rows form blocks of the same
    size with scales of their own (a fresh `out` has zero codes and unit
    scales behind them)."""
    dev = cache.k.get_device()
    B, Hkv, P, D = _need_cache("cache", cache, dev)
    if out is not None and bucket is None and out.k.dim() == 4:
        bucket = out.k.shape[2]
    bucket = n_keep if bucket is None else bucket
    if out is not None and (_need_cache("out", out, dev) != (B, Hkv, bucket, D) or out.block != cache.block):
        raise ValueError(f"out must be a cache of {bucket} rows with cache's other sizes and block")
    _need_evicted(mass, B, Hkv, P, bucket, prefix_valid_len, prefix_mask, mass_out, positions, valid_len, dev)

    def call(s):
        c = _empty_cache(B, Hkv, max(bucket, 0), D, cache.block, dev) if out is None else out
        mo, po, vl = _evict_outputs(B, Hkv, max(bucket, 0), mass_out, positions, valid_len, dev)
        _check(dm05_prefix_evict_kv8(cache.k.data_ptr(), cache.v.data_ptr(), cache.k_scale.data_ptr(),
                                     cache.v_scale.data_ptr(), cache.block, mass.data_ptr(), _ptr(prefix_valid_len),
                                     _ptr(prefix_mask), c.k.data_ptr(), c.v.data_ptr(), c.k_scale.data_ptr(),
                                     c.v_scale.data_ptr(), mo.data_ptr(), po.data_ptr(), vl.data_ptr(), B, Hkv, P,
                                     bucket, D, n_keep, n_first, n_last, s), "dm05_prefix_evict_kv8")
        return EvictedPrefixKv8(c, mo, po, vl)
    return _on(dev, stream, call)
