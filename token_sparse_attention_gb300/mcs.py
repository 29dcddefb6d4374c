"""Thin Python binding of libmcs.so (the C ABI declared in include/mcs.h).

Argument marshalling only: every function takes torch tensors that already
live on a CUDA device, checks dtype/shape/contiguity, and passes raw device
pointers and the current CUDA stream to the C entry point of the same name.
Every step of the computation runs in the library's kernels; there is no
fallback of any kind.  If libmcs.so is missing or fails to load, the first
call raises.
"""

from __future__ import annotations

import ctypes
import math
import os

import torch

__all__ = [
    "McsError", "Params", "params", "lib", "library_path", "EXPORTED",
    "mcs_status_string", "mcs_last_cuda_error", "mcs_device_status",
    "mcs_group_workspace", "mcs_anchor_workspace", "mcs_group", "mcs_dense_attn",
    "mcs_group_mass", "mcs_topk", "mcs_select", "mcs_sparse_attn", "mcs_sparse_attn_record",
    "mcs_anchor_select", "mcs_group_noalloc", "mcs_meta_bytes", "mcs_meta_offsets",
    "meta_views", "mcs_meta_pack", "mcs_meta_unpack", "Stager", "mcs_block_workspace", "mcs_block_topk", "mcs_pooled_block_select",
    "mcs_gather_mass", "mcs_rel_l1", "mcs_pair_bytes", "empty_pairs", "mcs_pair_lists",
    "mcs_sparse_attn_pairs", "mcs_sparse_attn_pairs_record", "mcs_quantize_e4m3",
    "mcs_sparse_attn_e4m3", "Paged", "paged", "KV_BF16", "KV_E4M3", "mcs_paged_plan",
    "mcs_paged_write", "mcs_paged_decode_workspace", "mcs_paged_decode",
    "mcs_paged_select_workspace", "mcs_paged_select", "mcs_paged_decode_sparse",
    "mcs_paged_attn_workspace", "mcs_paged_attn", "mcs_paged_decode_shared_workspace",
    "mcs_paged_decode_shared", "mcs_paged_fork_workspace", "mcs_paged_fork",
    "mcs_paged_compact_workspace", "mcs_paged_compact", "mcs_paged_copy", "Rope",
    "rope_params", "mcs_qk_norm_rope", "mcs_qk_norm_rope_backward_workspace",
    "mcs_qk_norm_rope_backward",
]

# Every symbol include/mcs.h declares.
EXPORTED = (
    "mcs_status_string", "mcs_last_cuda_error", "mcs_device_status", "mcs_group_workspace",
    "mcs_anchor_workspace", "mcs_group", "mcs_dense_attn", "mcs_group_mass", "mcs_topk",
    "mcs_select", "mcs_sparse_attn", "mcs_sparse_attn_record", "mcs_anchor_select", "mcs_group_noalloc",
    "mcs_pair_bytes", "mcs_pair_lists", "mcs_sparse_attn_pairs", "mcs_sparse_attn_pairs_record",
    "mcs_meta_bytes", "mcs_meta_offsets", "mcs_meta_pack", "mcs_meta_unpack",
    "mcs_stager_create", "mcs_stager_destroy",
    "mcs_stager_prefetch", "mcs_stager_offload", "mcs_stager_wait", "mcs_block_workspace",
    "mcs_block_topk", "mcs_pooled_block_select", "mcs_gather_mass", "mcs_rel_l1",
    "mcs_quantize_e4m3", "mcs_sparse_attn_e4m3",
    "mcs_paged_plan", "mcs_paged_write", "mcs_paged_decode_workspace", "mcs_paged_decode",
    "mcs_paged_select_workspace", "mcs_paged_select", "mcs_paged_decode_sparse",
    "mcs_paged_attn_workspace", "mcs_paged_attn", "mcs_paged_decode_shared_workspace",
    "mcs_paged_decode_shared", "mcs_paged_fork_workspace", "mcs_paged_fork",
    "mcs_paged_compact_workspace", "mcs_paged_compact", "mcs_paged_copy",
    "mcs_qk_norm_rope", "mcs_qk_norm_rope_backward_workspace", "mcs_qk_norm_rope_backward",
)

STATUS_NAMES = {0: "MCS_OK", 1: "MCS_ERR_INVALID_ARG", 2: "MCS_ERR_UNSUPPORTED",
                3: "MCS_ERR_WORKSPACE", 4: "MCS_ERR_CUDA", 5: "MCS_ERR_TIMEOUT",
                6: "MCS_ERR_BOUNDS"}


class McsError(RuntimeError):
    def __init__(self, status: int, where: str, detail: str = ""):
        self.status = status
        name = STATUS_NAMES.get(status, str(status))
        super().__init__(f"{where}: {name}" + (f" ({detail})" if detail else ""))


class Params(ctypes.Structure):
    """mcs_params: B, H, N, D, C, K, scale (0 -> 1/sqrt(D)), pddp_iters (0 -> 32),
    layout (0: activations [B, H, N, D]; 1: [B, N, H, D])."""

    _fields_ = [("B", ctypes.c_int), ("H", ctypes.c_int), ("N", ctypes.c_int),
                ("D", ctypes.c_int), ("C", ctypes.c_int), ("K", ctypes.c_int),
                ("scale", ctypes.c_float), ("pddp_iters", ctypes.c_int), ("layout", ctypes.c_int)]

    @property
    def G(self) -> int:
        return -(-self.N // self.C)


LAYOUT_BHND, LAYOUT_BNHD = 0, 1


def params(B, H, N, D, C=128, K=None, scale=0.0, pddp_iters=0, layout=LAYOUT_BHND) -> Params:
    return Params(B, H, N, D, C, N if K is None else K, scale, pddp_iters, layout)


class Paged(ctypes.Structure):
    """mcs_paged: B, Hq, Hkv, D, page, num_pages, max_pages, kv (KV_BF16 or KV_E4M3),
    scale (0 -> 1/sqrt(D)), k_scale, v_scale, q_stride, kv_stride (elements between
    consecutive tokens' rows; 0: contiguous)."""

    _fields_ = [("B", ctypes.c_int), ("Hq", ctypes.c_int), ("Hkv", ctypes.c_int),
                ("D", ctypes.c_int), ("page", ctypes.c_int), ("num_pages", ctypes.c_int),
                ("max_pages", ctypes.c_int), ("kv", ctypes.c_int), ("scale", ctypes.c_float),
                ("k_scale", ctypes.c_float), ("v_scale", ctypes.c_float),
                ("q_stride", ctypes.c_int), ("kv_stride", ctypes.c_int)]


KV_BF16, KV_E4M3 = 0, 1


def paged(B, Hq, Hkv, D, page, num_pages, max_pages, kv=KV_BF16, scale=0.0, k_scale=1.0,
          v_scale=1.0, q_stride=0, kv_stride=0) -> Paged:
    return Paged(B, Hq, Hkv, D, page, num_pages, max_pages, kv, scale, k_scale, v_scale,
                 q_stride, kv_stride)


class Rope(ctypes.Structure):
    """mcs_rope: B, N, Hq, Hkv, D, rot, interleaved, table_rows, layout, eps, q_stride,
    k_stride (elements between consecutive tokens' rows; 0: contiguous)."""

    _fields_ = [("B", ctypes.c_int), ("N", ctypes.c_int), ("Hq", ctypes.c_int),
                ("Hkv", ctypes.c_int), ("D", ctypes.c_int), ("rot", ctypes.c_int),
                ("interleaved", ctypes.c_int), ("table_rows", ctypes.c_int),
                ("layout", ctypes.c_int), ("eps", ctypes.c_float), ("q_stride", ctypes.c_int),
                ("k_stride", ctypes.c_int)]


def rope_params(B, N, Hq, Hkv, D, rot, table_rows, interleaved=False, layout=LAYOUT_BHND,
                eps=1e-6, q_stride=0, k_stride=0) -> Rope:
    return Rope(B, N, Hq, Hkv, D, rot, int(interleaved), table_rows, layout, eps, q_stride,
                k_stride)


def library_path() -> str:
    return os.path.join(os.path.dirname(os.path.abspath(__file__)), "libmcs.so")


_LIB = None
_vp, _sz, _i, _st = ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int, ctypes.c_int
_pp = ctypes.POINTER(Params)
_gp, _rp = ctypes.POINTER(Paged), ctypes.POINTER(Rope)

_SIGS = {
    "mcs_status_string": ([_st], ctypes.c_char_p),
    "mcs_last_cuda_error": ([], ctypes.c_char_p),
    "mcs_device_status": ([_vp], _st),
    "mcs_group_workspace": ([_pp], _sz),
    "mcs_anchor_workspace": ([_pp], _sz),
    "mcs_group": ([_pp, _vp, _vp, _vp, _sz, _vp], _st),
    "mcs_dense_attn": ([_pp, _vp, _vp, _vp, _vp, _vp, _vp], _st),
    "mcs_group_mass": ([_pp, _vp, _vp, _vp, _vp, _i, _i, _vp, _vp], _st),
    "mcs_topk": ([_pp, _vp, _i, _vp, _vp, _vp], _st),
    "mcs_select": ([_pp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _sz, _vp], _st),
    "mcs_sparse_attn": ([_pp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp], _st),
    "mcs_sparse_attn_record": ([_pp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp], _st),
    "mcs_pair_bytes": ([_pp], _sz),
    "mcs_pair_lists": ([_pp, _vp, _vp, _sz, _vp], _st),
    "mcs_sparse_attn_pairs": ([_pp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp], _st),
    "mcs_sparse_attn_pairs_record": ([_pp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp], _st),
    "mcs_anchor_select": ([_pp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _sz, _vp], _st),
    "mcs_group_noalloc": ([_pp, _vp, _vp, _vp], _st),
    "mcs_meta_bytes": ([_pp], _sz),
    "mcs_meta_offsets": ([_pp, ctypes.POINTER(_sz), ctypes.POINTER(_sz), ctypes.POINTER(_sz)], _st),
    "mcs_meta_pack": ([_pp, _vp, _vp, _vp], _st),
    "mcs_meta_unpack": ([_pp, _vp, _vp, _vp], _st),
    "mcs_stager_create": ([_pp, _i, ctypes.POINTER(_vp), _vp, ctypes.POINTER(_vp)], _st),
    "mcs_stager_destroy": ([_vp], None),
    "mcs_stager_prefetch": ([_vp, _i, _vp, _vp], _st),
    "mcs_stager_offload": ([_vp, _i, _vp, _vp], _st),
    "mcs_stager_wait": ([_vp, _i, _vp], _st),
    "mcs_block_workspace": ([_pp, _i], _sz),
    "mcs_block_topk": ([_pp, _vp, _i, _i, _vp, _vp, _vp, _sz, _vp], _st),
    "mcs_pooled_block_select": ([_pp, _vp, _vp, _vp, _i, _vp, _vp, _sz, _vp], _st),
    "mcs_gather_mass": ([_pp, _vp, _i, _vp, _vp, _vp], _st),
    "mcs_rel_l1": ([_pp, _vp, _vp, _vp, _i, _vp, _vp], _st),
    "mcs_quantize_e4m3": ([_vp, _sz, ctypes.c_float, _vp, _vp], _st),
    "mcs_sparse_attn_e4m3": ([_pp, _vp, _vp, _vp, ctypes.c_float, ctypes.c_float, _vp, _vp,
                              _vp, _vp, _vp], _st),
    "mcs_paged_plan": ([_gp, _vp, _vp, _vp, _i, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _i, _vp], _st),
    "mcs_paged_write": ([_gp, _i, _vp, _vp, _vp, _vp, _vp, _vp, _vp], _st),
    "mcs_paged_decode_workspace": ([_gp], _sz),
    "mcs_paged_decode": ([_gp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _sz, _vp], _st),
    "mcs_paged_select_workspace": ([_gp], _sz),
    "mcs_paged_select": ([_gp, _vp, _vp, _vp, _vp, _i, _i, _i, _vp, _vp, _sz, _vp], _st),
    "mcs_paged_decode_sparse": ([_gp, _vp, _vp, _vp, _vp, _vp, _vp, _i, _vp, _vp, _vp, _sz, _vp],
                                _st),
    "mcs_paged_attn_workspace": ([_gp], _sz),
    "mcs_paged_attn": ([_gp, _i] + [_vp] * 9 + [_sz, _vp], _st),
    "mcs_paged_decode_shared_workspace": ([_gp], _sz),
    "mcs_paged_decode_shared": ([_gp, _i] + [_vp] * 10 + [_sz, _vp], _st),
    "mcs_paged_fork_workspace": ([_gp], _sz),
    "mcs_paged_fork": ([_gp, _i] + [_vp] * 5 + [_i] + [_vp] * 8 + [_sz, _vp], _st),
    "mcs_paged_compact_workspace": ([_gp], _sz),
    "mcs_paged_compact": ([_gp] + [_vp] * 6 + [_i, _vp, _vp, _i, _vp, _sz, _vp], _st),
    "mcs_paged_copy": ([_gp, _i] + [_vp] * 5, _st),
    "mcs_qk_norm_rope": ([_rp] + [_vp] * 10, _st),
    "mcs_qk_norm_rope_backward_workspace": ([_rp], _sz),
    "mcs_qk_norm_rope_backward": ([_rp] + [_vp] * 14 + [_sz, _vp], _st),
}


def lib() -> ctypes.CDLL:
    """Load libmcs.so (built in-tree by build.py).  Raises if absent."""
    global _LIB
    if _LIB is None:
        path = library_path()
        if not os.path.exists(path):
            raise RuntimeError(f"{path} is not built; run __graft_entry__.build() first")
        L = ctypes.CDLL(path)
        for name, (args, res) in _SIGS.items():
            f = getattr(L, name)
            f.argtypes = args
            f.restype = res
        _LIB = L
    return _LIB


# ---------------------------------------------------------------- helpers

def _stream(stream) -> int:
    if stream is None:
        return torch.cuda.current_stream().cuda_stream
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _ptr(t, dtype, shape=None, name="tensor", optional=False):
    if t is None:
        if optional:
            return None
        raise ValueError(f"{name} is required")
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor (the library has no CPU path)")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    return t.data_ptr()


def _check(status: int, where: str):
    if status != 0:
        detail = lib().mcs_last_cuda_error().decode() if status == 4 else ""
        raise McsError(status, where, detail)


def _qkv_shape(p: Params):
    return (p.B, p.N, p.H, p.D) if p.layout == LAYOUT_BNHD else (p.B, p.H, p.N, p.D)


# ---------------------------------------------------------------- entry points

def mcs_status_string(status: int) -> str:
    return lib().mcs_status_string(status).decode()


def mcs_last_cuda_error() -> str:
    return lib().mcs_last_cuda_error().decode()


def mcs_device_status(stream=None) -> int:
    """Synchronise the stream and return (and clear) the device status code."""
    return lib().mcs_device_status(_stream(stream))


def mcs_group_workspace(p: Params) -> int:
    return lib().mcs_group_workspace(ctypes.byref(p))


def mcs_anchor_workspace(p: Params) -> int:
    return lib().mcs_anchor_workspace(ctypes.byref(p))


def mcs_group(p: Params, q, perm, ws, stream=None):
    bf = torch.bfloat16
    _check(lib().mcs_group(ctypes.byref(p), _ptr(q, bf, _qkv_shape(p), "q"),
                           _ptr(perm, torch.int32, (p.B, p.H, p.G * p.C), "perm"),
                           _ptr(ws, torch.uint8, None, "ws"), ws.numel(), _stream(stream)),
           "mcs_group")


def mcs_group_noalloc(p: Params, q, perm, stream=None):
    """mcs_group for callers that cannot allocate: uses the library's built-in
    64 MiB scratch instead of a workspace (see include/mcs.h)."""
    bf = torch.bfloat16
    _check(lib().mcs_group_noalloc(ctypes.byref(p), _ptr(q, bf, _qkv_shape(p), "q"),
                                   _ptr(perm, torch.int32, (p.B, p.H, p.G * p.C), "perm"),
                                   _stream(stream)), "mcs_group_noalloc")


def mcs_dense_attn(p: Params, q, k, v, out, lse=None, stream=None):
    bf, s = torch.bfloat16, _qkv_shape(p)
    _check(lib().mcs_dense_attn(ctypes.byref(p), _ptr(q, bf, s, "q"), _ptr(k, bf, s, "k"),
                                _ptr(v, bf, s, "v"), _ptr(out, bf, s, "out"),
                                _ptr(lse, torch.float32, (p.B, p.H, p.N), "lse", optional=True),
                                _stream(stream)), "mcs_dense_attn")


def mcs_group_mass(p: Params, q, k, lse, perm, head_begin, head_count, mass, stream=None):
    bf, s = torch.bfloat16, _qkv_shape(p)
    _check(lib().mcs_group_mass(ctypes.byref(p), _ptr(q, bf, s, "q"), _ptr(k, bf, s, "k"),
                                _ptr(lse, torch.float32, (p.B, p.H, p.N), "lse"),
                                _ptr(perm, torch.int32, (p.B, p.H, p.G * p.C), "perm"),
                                int(head_begin), int(head_count),
                                _ptr(mass, torch.float32, (head_count, p.G, p.N), "mass"),
                                _stream(stream)), "mcs_group_mass")


def mcs_topk(p: Params, mass, idx, retained=None, stream=None):
    rows = mass.numel() // p.N
    _check(lib().mcs_topk(ctypes.byref(p), _ptr(mass, torch.float32, None, "mass"), rows,
                          _ptr(idx, torch.int32, None, "idx"),
                          _ptr(retained, torch.float32, None, "retained", optional=True),
                          _stream(stream)), "mcs_topk")
    if idx.numel() != rows * p.K:
        raise ValueError("idx must hold rows * K entries")


def mcs_sparse_attn(p: Params, q, k, v, perm, idx, residual, out, stream=None):
    bf, s = torch.bfloat16, _qkv_shape(p)
    _check(lib().mcs_sparse_attn(ctypes.byref(p), _ptr(q, bf, s, "q"), _ptr(k, bf, s, "k"),
                                 _ptr(v, bf, s, "v"),
                                 _ptr(perm, torch.int32, (p.B, p.H, p.G * p.C), "perm"),
                                 _ptr(idx, torch.int32, (p.B, p.H, p.G, p.K), "idx"),
                                 _ptr(residual, bf, s, "residual", optional=True),
                                 _ptr(out, bf, s, "out"), _stream(stream)), "mcs_sparse_attn")


def mcs_sparse_attn_record(p: Params, q, k, v, perm, idx, dense_out, residual, stream=None):
    bf, s = torch.bfloat16, _qkv_shape(p)
    _check(lib().mcs_sparse_attn_record(
        ctypes.byref(p), _ptr(q, bf, s, "q"), _ptr(k, bf, s, "k"), _ptr(v, bf, s, "v"),
        _ptr(perm, torch.int32, (p.B, p.H, p.G * p.C), "perm"),
        _ptr(idx, torch.int32, (p.B, p.H, p.G, p.K), "idx"),
        _ptr(dense_out, bf, s, "dense_out"), _ptr(residual, bf, s, "residual"),
        _stream(stream)), "mcs_sparse_attn_record")


def _bytes8(t, name, numel):
    """E4M3 tensors: torch.float8_e4m3fn or their uint8 view."""
    if isinstance(t, torch.Tensor) and t.dtype == torch.float8_e4m3fn:
        t = t.view(torch.uint8)
    ptr = _ptr(t, torch.uint8, None, name)
    if t.numel() != numel:
        raise ValueError(f"{name} must hold {numel} bytes, got {t.numel()}")
    return ptr


def mcs_quantize_e4m3(x, scale: float, x8, stream=None):
    """x8 = E4M3(x / scale), elementwise (x bf16; x8 uint8 or float8_e4m3fn)."""
    n = x.numel()
    _check(lib().mcs_quantize_e4m3(_ptr(x, torch.bfloat16, None, "x"), n, float(scale),
                                   _bytes8(x8, "x8", n), _stream(stream)), "mcs_quantize_e4m3")


def mcs_sparse_attn_e4m3(p: Params, q, k8, v8, k_scale: float, v_scale: float, perm, idx,
                         residual, out, stream=None):
    bf, s = torch.bfloat16, _qkv_shape(p)
    n = math.prod(s)
    _check(lib().mcs_sparse_attn_e4m3(
        ctypes.byref(p), _ptr(q, bf, s, "q"), _bytes8(k8, "k8", n), _bytes8(v8, "v8", n),
        float(k_scale), float(v_scale),
        _ptr(perm, torch.int32, (p.B, p.H, p.G * p.C), "perm"),
        _ptr(idx, torch.int32, (p.B, p.H, p.G, p.K), "idx"),
        _ptr(residual, bf, s, "residual", optional=True), _ptr(out, bf, s, "out"),
        _stream(stream)), "mcs_sparse_attn_e4m3")


def mcs_pair_bytes(p: Params) -> int:
    """Bytes of the sibling-pair key-list buffer (0: unsupported for p)."""
    return lib().mcs_pair_bytes(ctypes.byref(p))


def empty_pairs(p: Params, device="cuda"):
    """A device buffer for mcs_pair_lists (uint8, 256-byte aligned)."""
    n = mcs_pair_bytes(p)
    if n == 0:
        raise ValueError("pair lists need C = 64, K <= 16384 and N < 2^28")
    return empty_workspace(n, device)


def mcs_pair_lists(p: Params, idx, pairs, stream=None):
    _check(lib().mcs_pair_lists(
        ctypes.byref(p), _ptr(idx, torch.int32, (p.B, p.H, p.G, p.K), "idx"),
        _ptr(pairs, torch.uint8, None, "pairs"), pairs.numel(), _stream(stream)),
        "mcs_pair_lists")


def mcs_sparse_attn_pairs(p: Params, q, k, v, perm, pairs, residual, out, stream=None):
    bf, s = torch.bfloat16, _qkv_shape(p)
    _check(lib().mcs_sparse_attn_pairs(
        ctypes.byref(p), _ptr(q, bf, s, "q"), _ptr(k, bf, s, "k"), _ptr(v, bf, s, "v"),
        _ptr(perm, torch.int32, (p.B, p.H, p.G * p.C), "perm"),
        _ptr(pairs, torch.uint8, None, "pairs"),
        _ptr(residual, bf, s, "residual", optional=True), _ptr(out, bf, s, "out"),
        _stream(stream)), "mcs_sparse_attn_pairs")


def mcs_sparse_attn_pairs_record(p: Params, q, k, v, perm, pairs, dense_out, residual,
                                 stream=None):
    bf, s = torch.bfloat16, _qkv_shape(p)
    _check(lib().mcs_sparse_attn_pairs_record(
        ctypes.byref(p), _ptr(q, bf, s, "q"), _ptr(k, bf, s, "k"), _ptr(v, bf, s, "v"),
        _ptr(perm, torch.int32, (p.B, p.H, p.G * p.C), "perm"),
        _ptr(pairs, torch.uint8, None, "pairs"),
        _ptr(dense_out, bf, s, "dense_out"), _ptr(residual, bf, s, "residual"),
        _stream(stream)), "mcs_sparse_attn_pairs_record")


def mcs_select(p: Params, q, k, lse, perm, idx, ws, retained=None, stream=None):
    bf, s = torch.bfloat16, _qkv_shape(p)
    _check(lib().mcs_select(
        ctypes.byref(p), _ptr(q, bf, s, "q"), _ptr(k, bf, s, "k"),
        _ptr(lse, torch.float32, (p.B, p.H, p.N), "lse"),
        _ptr(perm, torch.int32, (p.B, p.H, p.G * p.C), "perm"),
        _ptr(idx, torch.int32, (p.B, p.H, p.G, p.K), "idx"),
        _ptr(retained, torch.float32, (p.B, p.H, p.G), "retained", optional=True),
        _ptr(ws, torch.uint8, None, "ws"), ws.numel(), _stream(stream)), "mcs_select")


def mcs_anchor_select(p: Params, q, k, v, perm, idx, dense_out, lse, residual, ws,
                      retained=None, stream=None):
    bf, s = torch.bfloat16, _qkv_shape(p)
    _check(lib().mcs_anchor_select(
        ctypes.byref(p), _ptr(q, bf, s, "q"), _ptr(k, bf, s, "k"), _ptr(v, bf, s, "v"),
        _ptr(perm, torch.int32, (p.B, p.H, p.G * p.C), "perm"),
        _ptr(idx, torch.int32, (p.B, p.H, p.G, p.K), "idx"),
        _ptr(dense_out, bf, s, "dense_out"), _ptr(lse, torch.float32, (p.B, p.H, p.N), "lse"),
        _ptr(residual, bf, s, "residual"),
        _ptr(retained, torch.float32, (p.B, p.H, p.G), "retained", optional=True),
        _ptr(ws, torch.uint8, None, "ws"), ws.numel(), _stream(stream)), "mcs_anchor_select")


def mcs_meta_bytes(p: Params) -> int:
    return lib().mcs_meta_bytes(ctypes.byref(p))


def mcs_meta_offsets(p: Params) -> tuple[int, int, int]:
    o = [_sz(0), _sz(0), _sz(0)]
    _check(lib().mcs_meta_offsets(ctypes.byref(p), *[ctypes.byref(x) for x in o]),
           "mcs_meta_offsets")
    return tuple(x.value for x in o)


def meta_views(p: Params, entry: torch.Tensor):
    """(perm, bits, residual) views into a metadata entry (uint8, host or
    device); bits [B, H, G, ceil(N/32)] holds the index bitmaps (as int32)."""
    if entry.dtype != torch.uint8 or not entry.is_contiguous() or entry.dim() != 1:
        raise ValueError("entry must be a contiguous 1-D uint8 tensor")
    if entry.numel() < mcs_meta_bytes(p):
        raise ValueError("entry is smaller than mcs_meta_bytes(p)")
    po, io, ro = mcs_meta_offsets(p)
    n_perm = p.B * p.H * p.G * p.C * 4
    W = -(-p.N // 32)
    n_idx = p.B * p.H * p.G * W * 4
    n_res = p.B * p.H * p.N * p.D * 2
    perm = entry[po:po + n_perm].view(torch.int32).view(p.B, p.H, p.G * p.C)
    idx = entry[io:io + n_idx].view(torch.int32).view(p.B, p.H, p.G, W)
    res = entry[ro:ro + n_res].view(torch.bfloat16).view(*_qkv_shape(p))
    return perm, idx, res


def mcs_meta_pack(p: Params, idx, entry, stream=None):
    _check(lib().mcs_meta_pack(ctypes.byref(p),
                               _ptr(idx, torch.int32, (p.B, p.H, p.G, p.K), "idx"),
                               _ptr(entry, torch.uint8, None, "entry"), _stream(stream)),
           "mcs_meta_pack")


def mcs_meta_unpack(p: Params, entry, idx, stream=None):
    _check(lib().mcs_meta_unpack(ctypes.byref(p), _ptr(entry, torch.uint8, None, "entry"),
                                 _ptr(idx, torch.int32, (p.B, p.H, p.G, p.K), "idx"),
                                 _stream(stream)), "mcs_meta_unpack")


class Stager:
    """Moves metadata entries between host memory and device slots (mcs_stager_*)."""

    def __init__(self, p: Params, slots, copy_stream):
        for t in slots:
            _ptr(t, torch.uint8, None, "slot")
            if t.numel() < mcs_meta_bytes(p):
                raise ValueError("slot is smaller than mcs_meta_bytes(p)")
        self.slots = list(slots)
        self._h = _vp()
        arr = (_vp * len(slots))(*[t.data_ptr() for t in slots])
        _check(lib().mcs_stager_create(ctypes.byref(p), len(slots), arr, _stream(copy_stream),
                                       ctypes.byref(self._h)), "mcs_stager_create")

    @staticmethod
    def _host(t):
        if not isinstance(t, torch.Tensor) or t.is_cuda or t.dtype != torch.uint8 or \
                not t.is_contiguous():
            raise ValueError("host entry must be a contiguous uint8 CPU tensor (pinned)")
        return t.data_ptr()

    def prefetch(self, slot: int, host_entry, after=None):
        _check(lib().mcs_stager_prefetch(self._h, slot, self._host(host_entry), _stream(after)),
               "mcs_stager_prefetch")

    def offload(self, slot: int, host_entry, after=None):
        _check(lib().mcs_stager_offload(self._h, slot, self._host(host_entry), _stream(after)),
               "mcs_stager_offload")

    def wait(self, slot: int, stream=None):
        _check(lib().mcs_stager_wait(self._h, slot, _stream(stream)), "mcs_stager_wait")

    def close(self):
        if self._h:
            lib().mcs_stager_destroy(self._h)
            self._h = _vp()

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def mcs_block_workspace(p: Params, block: int) -> int:
    return lib().mcs_block_workspace(ctypes.byref(p), block)


def mcs_block_topk(p: Params, mass, block: int, idx, ws, retained=None, stream=None):
    rows = mass.numel() // p.N
    _ptr(idx, torch.int32, None, "idx")
    if idx.numel() != rows * p.K:
        raise ValueError("idx must hold rows * K entries")
    _check(lib().mcs_block_topk(ctypes.byref(p), _ptr(mass, torch.float32, None, "mass"), rows,
                                block, idx.data_ptr(),
                                _ptr(retained, torch.float32, (rows,), "retained", optional=True),
                                _ptr(ws, torch.uint8, None, "ws"), ws.numel(), _stream(stream)),
           "mcs_block_topk")


def mcs_pooled_block_select(p: Params, q, k, perm, block: int, idx, ws, stream=None):
    bf, s = torch.bfloat16, _qkv_shape(p)
    _check(lib().mcs_pooled_block_select(
        ctypes.byref(p), _ptr(q, bf, s, "q"), _ptr(k, bf, s, "k"),
        _ptr(perm, torch.int32, (p.B, p.H, p.G * p.C), "perm"), block,
        _ptr(idx, torch.int32, (p.B, p.H, p.G, p.K), "idx"),
        _ptr(ws, torch.uint8, None, "ws"), ws.numel(), _stream(stream)), "mcs_pooled_block_select")


def mcs_gather_mass(p: Params, mass, idx, retained, stream=None):
    rows = mass.numel() // p.N
    _ptr(idx, torch.int32, None, "idx")
    if idx.numel() != rows * p.K:
        raise ValueError("idx must hold rows * K entries")
    _check(lib().mcs_gather_mass(ctypes.byref(p), _ptr(mass, torch.float32, None, "mass"), rows,
                                 idx.data_ptr(), _ptr(retained, torch.float32, (rows,), "retained"),
                                 _stream(stream)), "mcs_gather_mass")


def mcs_rel_l1(p: Params, got, want, rows=None, stream=None) -> tuple:
    """(sum |got - want|, sum |want|) over the listed rows (all when None);
    synchronises the stream to read the two sums."""
    bf, s = torch.bfloat16, _qkv_shape(p)
    sums = torch.empty(2, dtype=torch.float64, device=got.device)
    nrows = 0 if rows is None else rows.numel()
    _check(lib().mcs_rel_l1(ctypes.byref(p), _ptr(got, bf, s, "got"), _ptr(want, bf, s, "want"),
                            _ptr(rows, torch.int32, None, "rows", optional=True), nrows,
                            sums.data_ptr(), _stream(stream)), "mcs_rel_l1")
    v = sums.cpu()
    return float(v[0]), float(v[1])


# ---------------------------------------------------------------- paged cache

# A decoding step makes these calls for every layer, and their checks stand
# beside kernels of a few microseconds: each tensor is looked at once, by the
# cheapest expression that says whether it fits, and only one that does not is
# taken apart for the message.

def _device(stream) -> int:
    """The device a call runs on: the current one, which the stream must belong to."""
    current = torch.cuda.current_device()
    if stream is not None and getattr(stream, "device_index", current) != current:
        raise ValueError("stream belongs to another device than the current one")
    return current


def _queue(stream, dev) -> int:
    return torch._C._cuda_getCurrentRawStream(dev) if stream is None else _stream(stream)


def _refuse(dev, t, dtype, shape, name):
    _ptr(t, dtype, shape, name)
    raise ValueError(f"{name} is on {t.device}, the call runs on cuda:{dev}")


def _at(dev, t, dtype, shape, name):
    """As _ptr, and on device `dev`."""
    try:
        if t.dtype is dtype and t.get_device() == dev and t.shape == shape and t.is_contiguous():
            return t.data_ptr()
    except AttributeError:
        pass
    return _refuse(dev, t, dtype, shape, name)


def _bytes_at(dev, t, name):
    """(pointer, size) of a workspace."""
    try:
        if t.dtype is _U8 and t.get_device() == dev and t.is_contiguous():
            return t.data_ptr(), t.numel()
    except AttributeError:
        pass
    return _refuse(dev, t, _U8, None, name)


def _rows_at(dev, t, dtype, shape, stride, name):
    """Rows [..., H, D] whose consecutive tokens stand `stride` elements apart (0: H * D)."""
    D = shape[-1]
    try:
        if t.dtype is dtype and t.get_device() == dev and t.shape == shape:
            if stride == 0:
                if t.is_contiguous():
                    return t.data_ptr()
            elif t.stride() == ((stride, D, 1) if len(shape) == 3 else
                                (shape[1] * stride, stride, D, 1)):
                return t.data_ptr()
    except AttributeError:
        pass
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor (the library has no CPU path)")
    if t.dtype is not dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if t.get_device() != dev:
        raise ValueError(f"{name} is on {t.device}, the call runs on cuda:{dev}")
    want, n = (D, 1), stride or D * shape[-2]
    for size in shape[-3::-1]:
        want = (n,) + want
        n *= size
    # (a dimension of one element may have any stride)
    if any(x > 1 and h != w for x, h, w in zip(shape, t.stride(), want)):
        raise ValueError(f"{name} must have strides {want}, got {t.stride()}")
    return t.data_ptr()


def _count(n, name):
    """A size the library takes as an int (ctypes would cut it to 32 bits without a word)."""
    if n > 0x7FFFFFFF:
        raise ValueError(f"{name}: {n} elements are more than a call takes")
    return n


def _cache_at(dev, t, kv, shape, name):
    dtype = _BF
    if kv == KV_E4M3:  # codes as bytes or as what they stand for
        dtype = _F8 if getattr(t, "dtype", None) is _F8 else _U8
    return _at(dev, t, dtype, shape, name)


_BF, _I32, _F32 = torch.bfloat16, torch.int32, torch.float32
_U8, _F8 = torch.uint8, torch.float8_e4m3fn


def mcs_paged_plan(p: Paged, new_lens, lens, free_pages, free_head, block_table, lens_out,
                   head_out, cu_new, slots, positions=None, stream=None):
    T, n_free = _count(slots.numel(), "slots"), _count(free_pages.numel(), "free_pages")
    dev, B, one = _device(stream), (p.B,), (1,)
    _check(lib().mcs_paged_plan(
        ctypes.byref(p), _at(dev, new_lens, _I32, B, "new_lens"), _at(dev, lens, _I32, B, "lens"),
        _at(dev, free_pages, _I32, (n_free,), "free_pages"), n_free,
        _at(dev, free_head, _I32, one, "free_head"),
        _at(dev, block_table, _I32, (p.B, p.max_pages), "block_table"),
        _at(dev, lens_out, _I32, B, "lens_out"), _at(dev, head_out, _I32, one, "head_out"),
        _at(dev, cu_new, _I32, (p.B + 1,), "cu_new"), _at(dev, slots, _I32, (T,), "slots"),
        None if positions is None else _at(dev, positions, _I32, (T,), "positions"), T, _queue(stream, dev)),
        "mcs_paged_plan")


def mcs_paged_write(p: Paged, k, v, slots, k_cache, v_cache, k_mean=None, stream=None):
    T = _count(slots.numel(), "slots")
    dev, Hkv, D, pages, kv = _device(stream), p.Hkv, p.D, p.num_pages, p.kv
    rows, cache, stride = (T, Hkv, D), (pages, Hkv, p.page, D), p.kv_stride
    _check(lib().mcs_paged_write(
        ctypes.byref(p), T, _rows_at(dev, k, _BF, rows, stride, "k"),
        _rows_at(dev, v, _BF, rows, stride, "v"), _at(dev, slots, _I32, (T,), "slots"),
        _cache_at(dev, k_cache, kv, cache, "k_cache"),
        _cache_at(dev, v_cache, kv, cache, "v_cache"),
        None if k_mean is None else _at(dev, k_mean, _BF, (pages, Hkv, D), "k_mean"), _queue(stream, dev)),
        "mcs_paged_write")


def mcs_paged_decode_workspace(p: Paged) -> int:
    return lib().mcs_paged_decode_workspace(ctypes.byref(p))


def mcs_paged_decode(p: Paged, q, k_cache, v_cache, block_table, lens, out, ws, lse=None,
                     stream=None):
    dev, B, Hq, D, kv = _device(stream), p.B, p.Hq, p.D, p.kv
    cache, rows = (p.num_pages, p.Hkv, p.page, D), (B, Hq, D)
    _check(lib().mcs_paged_decode(
        ctypes.byref(p), _rows_at(dev, q, _BF, rows, p.q_stride, "q"),
        _cache_at(dev, k_cache, kv, cache, "k_cache"),
        _cache_at(dev, v_cache, kv, cache, "v_cache"),
        _at(dev, block_table, _I32, (B, p.max_pages), "block_table"),
        _at(dev, lens, _I32, (B,), "lens"), _at(dev, out, _BF, rows, "out"),
        None if lse is None else _at(dev, lse, _F32, (B, Hq), "lse"), *_bytes_at(dev, ws, "ws"),
        _queue(stream, dev)), "mcs_paged_decode")


def mcs_paged_select_workspace(p: Paged) -> int:
    return lib().mcs_paged_select_workspace(ctypes.byref(p))


def _select_of(sel) -> int:
    if not isinstance(sel, torch.Tensor) or sel.dim() != 3:
        raise ValueError("sel must be a [B, Hkv, select] tensor")
    return _count(sel.shape[2], "sel")


def mcs_paged_select(p: Paged, q, k_mean, block_table, lens, sel, ws, sink=1, recent=1,
                     stream=None):
    """sel [B, Hkv, select]: the last dimension says how many pages are kept."""
    keep, sink, recent = _select_of(sel), _count(sink, "sink"), _count(recent, "recent")
    dev, B, Hkv, D = _device(stream), p.B, p.Hkv, p.D
    _check(lib().mcs_paged_select(
        ctypes.byref(p), _rows_at(dev, q, _BF, (B, p.Hq, D), p.q_stride, "q"),
        _at(dev, k_mean, _BF, (p.num_pages, Hkv, D), "k_mean"),
        _at(dev, block_table, _I32, (B, p.max_pages), "block_table"),
        _at(dev, lens, _I32, (B,), "lens"), keep, sink, recent,
        _at(dev, sel, _I32, (B, Hkv, keep), "sel"), *_bytes_at(dev, ws, "ws"),
        _queue(stream, dev)), "mcs_paged_select")


def mcs_paged_decode_sparse(p: Paged, q, k_cache, v_cache, block_table, lens, sel, out, ws,
                            lse=None, stream=None):
    keep = _select_of(sel)
    dev, B, Hq, Hkv, D, kv = _device(stream), p.B, p.Hq, p.Hkv, p.D, p.kv
    cache, rows = (p.num_pages, Hkv, p.page, D), (B, Hq, D)
    _check(lib().mcs_paged_decode_sparse(
        ctypes.byref(p), _rows_at(dev, q, _BF, rows, p.q_stride, "q"),
        _cache_at(dev, k_cache, kv, cache, "k_cache"),
        _cache_at(dev, v_cache, kv, cache, "v_cache"),
        _at(dev, block_table, _I32, (B, p.max_pages), "block_table"),
        _at(dev, lens, _I32, (B,), "lens"), _at(dev, sel, _I32, (B, Hkv, keep), "sel"), keep,
        _at(dev, out, _BF, rows, "out"), None if lse is None else _at(dev, lse, _F32, (B, Hq), "lse"),
        *_bytes_at(dev, ws, "ws"), _queue(stream, dev)), "mcs_paged_decode_sparse")


def mcs_paged_attn_workspace(p: Paged) -> int:
    return lib().mcs_paged_attn_workspace(ctypes.byref(p))


def mcs_paged_attn(p: Paged, q, k_cache, v_cache, block_table, lens, cu_new, out, ws, lse=None,
                   stream=None):
    """q, out [T, Hq, D]: the new tokens of all sequences, one behind another."""
    if not isinstance(q, torch.Tensor) or q.dim() != 3:
        raise ValueError("q must be a [T, Hq, D] tensor")
    T = _count(q.shape[0], "q")
    dev, B, Hq, D, kv = _device(stream), p.B, p.Hq, p.D, p.kv
    cache, rows = (p.num_pages, p.Hkv, p.page, D), (T, Hq, D)
    _check(lib().mcs_paged_attn(
        ctypes.byref(p), T, _rows_at(dev, q, _BF, rows, p.q_stride, "q"),
        _cache_at(dev, k_cache, kv, cache, "k_cache"),
        _cache_at(dev, v_cache, kv, cache, "v_cache"),
        _at(dev, block_table, _I32, (B, p.max_pages), "block_table"),
        _at(dev, lens, _I32, (B,), "lens"), _at(dev, cu_new, _I32, (B + 1,), "cu_new"),
        _at(dev, out, _BF, rows, "out"),
        None if lse is None else _at(dev, lse, _F32, (T, Hq), "lse"), *_bytes_at(dev, ws, "ws"),
        _queue(stream, dev)), "mcs_paged_attn")


def mcs_paged_decode_shared_workspace(p: Paged) -> int:
    return lib().mcs_paged_decode_shared_workspace(ctypes.byref(p))


def mcs_paged_decode_shared(p: Paged, q, k_cache, v_cache, block_table, lens, group_start,
                            shared_pages, out, ws, lse=None, stream=None):
    """Sequences group_start[g] .. group_start[g + 1] - 1 have their first shared_pages[g] pages in
    common."""
    if not isinstance(shared_pages, torch.Tensor) or shared_pages.dim() != 1:
        raise ValueError("shared_pages must be a [groups] tensor")
    G = _count(shared_pages.shape[0], "shared_pages")
    dev, B, Hq, D, kv = _device(stream), p.B, p.Hq, p.D, p.kv
    cache, rows = (p.num_pages, p.Hkv, p.page, D), (B, Hq, D)
    _check(lib().mcs_paged_decode_shared(
        ctypes.byref(p), G, _rows_at(dev, q, _BF, rows, p.q_stride, "q"),
        _cache_at(dev, k_cache, kv, cache, "k_cache"),
        _cache_at(dev, v_cache, kv, cache, "v_cache"),
        _at(dev, block_table, _I32, (B, p.max_pages), "block_table"),
        _at(dev, lens, _I32, (B,), "lens"), _at(dev, group_start, _I32, (G + 1,), "group_start"),
        _at(dev, shared_pages, _I32, (G,), "shared_pages"), _at(dev, out, _BF, rows, "out"),
        None if lse is None else _at(dev, lse, _F32, (B, Hq), "lse"), *_bytes_at(dev, ws, "ws"),
        _queue(stream, dev)), "mcs_paged_decode_shared")


def mcs_paged_fork_workspace(p: Paged) -> int:
    return lib().mcs_paged_fork_workspace(ctypes.byref(p))


def mcs_paged_fork(p: Paged, parents, lens, block_table, extra, free_pages, free_head, lens_out,
                   table_out, extra_out, free_out, head_out, moves, ws, stream=None):
    """parents [n]: which of the B sequences each new one continues (-1: an empty one); moves
    [n, 3] says what mcs_paged_copy has to copy."""
    n, n_free = _count(parents.numel(), "parents"), _count(free_pages.numel(), "free_pages")
    dev, B, P, one, pages = _device(stream), p.B, p.max_pages, (1,), (p.num_pages,)
    _check(lib().mcs_paged_fork(
        ctypes.byref(p), n, _at(dev, parents, _I32, (n,), "parents"),
        _at(dev, lens, _I32, (B,), "lens"), _at(dev, block_table, _I32, (B, P), "block_table"),
        _at(dev, extra, _I32, pages, "extra"), _at(dev, free_pages, _I32, (n_free,), "free_pages"),
        n_free, _at(dev, free_head, _I32, one, "free_head"),
        _at(dev, lens_out, _I32, (n,), "lens_out"),
        _at(dev, table_out, _I32, (n, P), "table_out"),
        _at(dev, extra_out, _I32, pages, "extra_out"),
        _at(dev, free_out, _I32, (n_free,), "free_out"),
        _at(dev, head_out, _I32, one, "head_out"), _at(dev, moves, _I32, (n, 3), "moves"),
        *_bytes_at(dev, ws, "ws"), _queue(stream, dev)), "mcs_paged_fork")


def mcs_paged_compact_workspace(p: Paged) -> int:
    return lib().mcs_paged_compact_workspace(ctypes.byref(p))


def _moves_of(moves) -> int:
    if not isinstance(moves, torch.Tensor) or moves.dim() != 2:
        raise ValueError("moves must be a [n, 3] tensor")
    return _count(moves.shape[0], "moves")


def mcs_paged_compact(p: Paged, lens, block_table, extra, table_out, extra_out, free_out, head_out,
                      moves, ws, stream=None):
    """moves [most, 3]: the first dimension says how many pages are moved at most; none: the free list is
    made anew, as after tokens that were taken back by lowering lens."""
    most, n_free = _moves_of(moves), _count(free_out.numel(), "free_out")
    dev, B, pages = _device(stream), p.B, (p.num_pages,)
    table = (B, p.max_pages)
    _check(lib().mcs_paged_compact(
        ctypes.byref(p), _at(dev, lens, _I32, (B,), "lens"),
        _at(dev, block_table, _I32, table, "block_table"), _at(dev, extra, _I32, pages, "extra"),
        _at(dev, table_out, _I32, table, "table_out"),
        _at(dev, extra_out, _I32, pages, "extra_out"),
        _at(dev, free_out, _I32, (n_free,), "free_out"), n_free,
        _at(dev, head_out, _I32, (1,), "head_out"), _at(dev, moves, _I32, (most, 3), "moves"), most,
        *_bytes_at(dev, ws, "ws"), _queue(stream, dev)), "mcs_paged_compact")


def mcs_paged_copy(p: Paged, moves, k_cache, v_cache, k_mean=None, stream=None):
    """The first rows of pages to other pages, in both caches: moves [n, 3] (from, to, rows)."""
    n = _moves_of(moves)
    dev, Hkv, pages, kv = _device(stream), p.Hkv, p.num_pages, p.kv
    cache = (pages, Hkv, p.page, p.D)
    _check(lib().mcs_paged_copy(
        ctypes.byref(p), n, _at(dev, moves, _I32, (n, 3), "moves"),
        _cache_at(dev, k_cache, kv, cache, "k_cache"),
        _cache_at(dev, v_cache, kv, cache, "v_cache"),
        None if k_mean is None else _at(dev, k_mean, _BF, (pages, Hkv, p.D), "k_mean"),
        _queue(stream, dev)), "mcs_paged_copy")


# ---------------------------------------------------------------- norm and rotation

def _rope_args(dev, p: Rope, q, k, wq, wk, cos, sin, positions, q_out, k_out, names):
    """(pointers of q, k, wq, wk, cos, sin, positions, pointers of the two tensors in the layout of
    q_out and k_out); k's are null when Hkv = 0."""
    B, N, Hq, Hkv, D, rot = p.B, p.N, p.Hq, p.Hkv, p.D, p.rot
    by_token, vector = p.layout == LAYOUT_BNHD, (D,)
    pk = pwk = pko = pc = ps = None
    pq = _rows_at(dev, q, _BF, (B, N, Hq, D), p.q_stride, "q")
    pwq = None if wq is None else _at(dev, wq, _F32, vector, "wq")
    pqo = _at(dev, q_out, _BF, (B, N, Hq, D) if by_token else (B, Hq, N, D), names[0])
    if Hkv:
        pk = _rows_at(dev, k, _BF, (B, N, Hkv, D), p.k_stride, "k")
        pwk = None if wk is None else _at(dev, wk, _F32, vector, "wk")
        pko = _at(dev, k_out, _BF, (B, N, Hkv, D) if by_token else (B, Hkv, N, D), names[1])
    if rot:
        table = (p.table_rows, rot // 2)
        pc, ps = _at(dev, cos, _F32, table, "cos"), _at(dev, sin, _F32, table, "sin")
    pp = None if positions is None else _at(dev, positions, _I32, (B, N), "positions")
    return (pq, pk, pwq, pwk, pc, ps, pp), (pqo, pko)


def mcs_qk_norm_rope(p: Rope, q, k, wq, wk, cos, sin, positions, q_out, k_out, stream=None):
    dev = _device(stream)
    ins, outs = _rope_args(dev, p, q, k, wq, wk, cos, sin, positions, q_out, k_out,
                           ("q_out", "k_out"))
    _check(lib().mcs_qk_norm_rope(ctypes.byref(p), *ins, *outs, _queue(stream, dev)),
           "mcs_qk_norm_rope")


def mcs_qk_norm_rope_backward_workspace(p: Rope) -> int:
    return lib().mcs_qk_norm_rope_backward_workspace(ctypes.byref(p))


def mcs_qk_norm_rope_backward(p: Rope, dq_out, dk_out, q, k, wq, wk, cos, sin, positions, dq, dk,
                              dwq, dwk, ws, stream=None):
    dev, Hkv = _device(stream), p.Hkv
    ins, grads = _rope_args(dev, p, q, k, wq, wk, cos, sin, positions, dq_out, dk_out,
                            ("dq_out", "dk_out"))
    _check(lib().mcs_qk_norm_rope_backward(
        ctypes.byref(p), *grads, *ins,
        _rows_at(dev, dq, _BF, (p.B, p.N, p.Hq, p.D), p.q_stride, "dq"),
        _rows_at(dev, dk, _BF, (p.B, p.N, Hkv, p.D), p.k_stride, "dk") if Hkv else None,
        None if dwq is None else _at(dev, dwq, _F32, (p.D,), "dwq"),
        None if dwk is None or not Hkv else _at(dev, dwk, _F32, (p.D,), "dwk"),
        *_bytes_at(dev, ws, "ws"), _queue(stream, dev)), "mcs_qk_norm_rope_backward")


def empty_workspace(nbytes: int, device="cuda") -> torch.Tensor:
    """A device byte buffer of at least nbytes (256-byte aligned by torch)."""
    return torch.empty(max(int(nbytes), 256), dtype=torch.uint8, device=device)


def default_scale(D: int) -> float:
    return 1.0 / math.sqrt(D)
