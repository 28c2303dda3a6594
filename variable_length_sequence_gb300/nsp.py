"""Thin Python binding of ``libnsp.so`` (C ABI declared in ``include/nsp.h``).

Argument marshalling only: every function named like the C entry point takes
torch tensors (or raw integers) and passes their data pointers, sizes and the
current CUDA stream to the library.  All computation happens in the
library's kernels; there is no Python or CPU fallback, and loading fails
loudly when the library has not been built.
"""
from __future__ import annotations

import array
import ctypes as C
import operator
import os
import re
from typing import Optional, Sequence

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libnsp.so")
HEADER = os.path.join(os.path.dirname(_PKG), "include", "nsp.h")

NSP_OK, NSP_ERR_INVALID, NSP_ERR_UNSUPPORTED, NSP_ERR_WORKSPACE = 0, 1, 2, 3
NSP_ERR_CUDA, NSP_ERR_TIMEOUT, NSP_ERR_ALIGN = 4, 5, 6
NSP_F32, NSP_BF16 = 0, 1

_lib: Optional[C.CDLL] = None

_vp, _i32, _i64, _f32, _sz = C.c_void_p, C.c_int32, C.c_int64, C.c_float, C.c_size_t
_f64 = C.c_double

_SIGNATURES = {
    "nsp_status_str": (C.c_char_p, [_i32]),
    "nsp_version": (C.c_char_p, []),
    "nsp_kernel_launches": (_i64, []),
    "nsp_set_wait_timeout_cycles": (_i64, [_i64]),
    "nsp_path_launches": (_i64, [_i32]),
    "nsp_attn_fwd_workspace_size": (_sz, [_i64, _i64, _i32, _i32, _i32]),
    "nsp_attn_fwd": (_i32, [_vp, _vp, _vp, _vp, _i32, _i64, _i64, _i64, _i64, _i32, _i32, _i32,
                            _f32, _i32, _i32, _vp, _i32, _vp, _vp, _sz, _vp]),
    "nsp_attn_fwd_accumulate": (_i32, [_vp, _vp, _vp, _vp, _i32, _i64, _i64, _i64, _i64, _i32,
                                       _i32, _i32, _f32, _i32, _i32, _vp, _vp, _vp, _sz, _vp]),
    "nsp_attn_fwd_headgroups": (_i32, [_vp, _vp, _vp, _vp, _i32, _i64, _i32, _i32, _i32, _i32,
                                       _f32, _i32, _i32, _vp, _i32, _vp, _vp, _sz, _vp]),
    "nsp_attn_fwd_blocks_workspace_size": (_sz, [_i32, _vp, _i32, _i32, _i32]),
    "nsp_attn_fwd_blocks": (_i32, [_vp, _vp, _vp, _vp, _i32, _i64, _i32, _vp, _i32, _i32, _i32, _f32,
                                   _i32, _i32, _i32, _vp, _sz, _vp]),
    "nsp_attn_bwd_blocks_workspace_size": (_sz, [_i64, _i32, _vp, _i32, _i32, _i32]),
    "nsp_attn_bwd_blocks": (_i32, [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _i32, _i64, _i32, _vp, _i32,
                                   _i32, _i32, _f32, _i32, _i32, _vp, _vp, _vp, _vp, _sz, _vp]),
    "nsp_attn_fwd_validate": (_i32, [_vp, _vp, _vp, _vp, _i32, _i64, _i64, _i64, _i64, _i32,
                                     _i32, _i32, _i32, _i32, _vp, _i32, _vp, _sz]),
    "nsp_attn_fwd_noalloc": (_i32, [_vp, _vp, _vp, _vp, _i32, _i64, _i64, _i64, _i64, _i32,
                                    _i32, _i32, _f32, _i32, _i32, _vp, _i32, _vp, _vp, _vp]),
    "nsp_attn_bwd_workspace_size": (_sz, [_i64, _i32, _i32, _i32, _i32]),
    "nsp_attn_bwd": (_i32, [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _i32, _i64, _i32, _i32, _i32,
                            _f32, _i32, _i32, _vp, _vp, _vp, _vp, _sz, _vp]),
    "nsp_attn_bwd_validate": (_i32, [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _i32, _i64, _i32, _i32,
                                     _i32, _i32, _i32, _vp, _vp, _vp, _vp, _sz]),
    "nsp_attn_bwd_headgroups": (_i32, [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _i32, _i64, _i32, _i32,
                                       _i32, _i32, _f32, _i32, _i32, _vp, _vp, _vp, _vp, _sz,
                                       _vp]),
    "nsp_attn_bwd_accumulate_workspace_size": (_sz, [_i64, _i64, _i32, _i32, _i32, _i32]),
    "nsp_attn_bwd_accumulate": (_i32, [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _i32, _i64, _i64, _i64,
                                       _i64, _i32, _i32, _i32, _f32, _i32, _i32, _vp, _vp, _vp,
                                       _vp, _sz, _vp]),
    "nsp_lse_merge": (_i32, [_vp, _vp, _i32, _i64, _i32, _i32, _vp, _i32, _vp, _vp]),
    "nsp_lse_merge_batch": (_i32, [_i32, _vp, _vp, _vp, _i64, _i32, _i32, _vp, _i32, _vp, _vp]),
    "nsp_lse_merge_validate": (_i32, [_vp, _vp, _i32, _i64, _i32, _i32, _vp, _i32, _vp]),
    "nsp_seq2head_permute": (_i32, [_vp, _vp, _i64, _i32, _i32, _i32, _i32, _i32, _vp]),
    "nsp_seq2head_permute_validate": (_i32, [_vp, _vp, _i64, _i32, _i32, _i32, _i32]),
    "nsp_seq2head_permute_groups": (_i32, [_vp, _vp, _i32, _i64, _i32, _i32, _i32, _i32, _i32,
                                           _vp]),
    "nsp_rope": (_i32, [_vp, _i32, _vp, _i32, _vp, _i64, _i64, _i32, _i32, _vp, _i32, _f32, _i32,
                        _i32, _vp]),
    "nsp_rope_freqs": (_i32, [_i32, _f64, _i32, _f64, _f64, _f64, _f64, _vp]),
    "nsp_diff_lambda_fwd": (_i32, [_vp, _vp, _vp, _vp, _i32, _i32, _i32, _f32, _i32, _vp, _vp]),
    "nsp_diff_lambda_bwd": (_i32, [_vp, _vp, _vp, _vp, _vp, _i32, _i32, _i32, _i32, _vp, _vp, _vp,
                                   _vp, _vp]),
    "nsp_diff_attn_fwd_workspace_size": (_sz, [_i64]),
    "nsp_diff_attn_fwd": (_i32, [_vp, _vp, _vp, _vp, _i64, _vp, _i32, _i64, _i32, _i32, _i32, _f32,
                                 _i32, _i32, _vp, _vp, _vp, _vp, _sz, _vp]),
    "nsp_diff_attn_bwd_workspace_size": (_sz, [_i64, _i32, _i32, _i32, _i32]),
    "nsp_diff_attn_bwd": (_i32, [_vp, _vp, _vp, _vp, _i64, _vp, _vp, _vp, _vp, _vp, _i32, _i64, _i32,
                                 _i32, _i32, _f32, _i32, _i32, _vp, _vp, _vp, _vp, _vp, _sz, _vp]),
    "nsp_head_norm_fwd": (_i32, [_vp, _i64, _vp, _vp, _i64, _i32, _i32, _f32, _f32, _i32, _vp,
                                 _vp]),
    "nsp_head_norm_bwd_workspace_size": (_sz, [_i64, _i32, _i32]),
    "nsp_head_norm_bwd": (_i32, [_vp, _i64, _vp, _vp, _vp, _i64, _i32, _i32, _f32, _f32, _i32, _vp,
                                 _vp, _vp, _vp, _sz, _vp]),
    "nsp_qk_norm_rope_fwd": (_i32, [_vp, _i32, _vp, _i32, _vp, _i64, _i64, _i32, _i32, _vp, _i32,
                                    _f32, _f32, _i32, _vp]),
    "nsp_qk_norm_rope_bwd_workspace_size": (_sz, [_vp, _i32, _i64, _i32]),
    "nsp_qk_norm_rope_bwd": (_i32, [_vp, _i32, _vp, _i32, _vp, _i64, _i64, _i32, _i32, _vp, _i32,
                                    _f32, _f32, _i32, _vp, _sz, _vp]),
    "nsp_token_logp_workspace_size": (_sz, [_i64]),
    "nsp_token_logp_fwd": (_i32, [_vp, _i64, _vp, _i64, _i32, _f64, _i32, _vp, _vp, _vp, _sz, _vp]),
    "nsp_token_logp_bwd": (_i32, [_vp, _i64, _vp, _vp, _vp, _i64, _i32, _f64, _i32, _vp, _i64, _vp]),
    "nsp_policy_loss_workspace_size": (_sz, [_i64, _i32, _i32]),
    "nsp_policy_loss": (_i32, [_vp, _vp, _vp, _i32, _i64, _vp, _vp, _vp, _vp, _sz, _vp]),
    "nsp_policy_loss_logits": (_i32, [_vp, _i64, _vp, _vp, _i32, _i64, _i32, _f64, _i32, _vp, _vp, _vp,
                                      _vp, _i64, _vp, _sz, _vp]),
    "nsp_preference_loss_workspace_size": (_sz, [_i32]),
    "nsp_preference_loss": (_i32, [_vp, _vp, _vp, _vp, _i32, _i64, _i32, _f32, _f32, _f32, _i32, _vp,
                                   _vp, _vp, _vp, _sz, _vp]),
    "nsp_grad_norm_workspace_size": (_sz, [_vp, _i32]),
    "nsp_grad_norm": (_i32, [_vp, _vp, _vp, _i32, _i32, _f32, _vp, _vp, _sz, _vp]),
    "nsp_grad_clip": (_i32, [_vp, _vp, _vp, _vp, _vp, _i32, _i32, _f32, _f32, _f32, _vp, _vp, _sz, _vp]),
    "nsp_status_query": (_i32, [_vp, _vp]),
    "nsp_attn_bwd_ds_cache_size": (_sz, [_vp, _i32, _i32, _i32]),
    "nsp_attn_bwd_blocks_ds_cache_size": (_sz, [_vp, _i32, _i32, _vp, _i32, _i32]),
    "nsp_bwd_ds_cache_used": (_i32, [_vp, C.POINTER(C.c_int32), _vp]),
    "nsp_attn_pairs": (_i32, [_vp, _i32, _i32, C.POINTER(C.c_double)]),
    "nsp_attn_cost": (_i32, [_vp, _i32, _i64, _i64, _i64, _i64, _i32, _i32, _i32, _i32, _i32,
                             _vp]),
}


class Block(C.Structure):
    """nsp_block_t: one (query range, key range) block of a batched forward."""
    _fields_ = [("q_start", C.c_int64), ("q_len", C.c_int64), ("kv_start", C.c_int64),
                ("kv_len", C.c_int64), ("out", C.c_void_p), ("lse", C.c_void_p)]


class Range(C.Structure):
    """nsp_range_t: one (query range, key range) block of a batched backward."""
    _fields_ = [("q_start", C.c_int64), ("q_len", C.c_int64), ("kv_start", C.c_int64),
                ("kv_len", C.c_int64)]


class RopeTensor(C.Structure):
    """nsp_rope_tensor_t: one tensor of a rotation."""
    _fields_ = [("in_", C.c_void_p), ("out", C.c_void_p), ("in_stride", C.c_int64),
                ("out_stride", C.c_int64), ("heads", C.c_int32), ("groups", C.c_int32)]


class QkTensor(C.Structure):
    """nsp_qk_tensor_t: one tensor of a head norm with rotation."""
    _fields_ = [("x", C.c_void_p), ("weight", C.c_void_p), ("y", C.c_void_p), ("dy", C.c_void_p),
                ("dx", C.c_void_p), ("dweight", C.c_void_p), ("x_stride", C.c_int64),
                ("y_stride", C.c_int64), ("dx_stride", C.c_int64), ("heads", C.c_int32),
                ("groups", C.c_int32)]


class Policy(C.Structure):
    """nsp_policy_t: what a clipped policy loss goes by."""
    _fields_ = [("old_logp", C.c_void_p), ("ref_logp", C.c_void_p), ("advantages", C.c_void_p),
                ("per_token", C.c_int32), ("mean", C.c_int32), ("clip_low", C.c_float),
                ("clip_high", C.c_float), ("kl_coef", C.c_float), ("total", C.c_float)]


class AttnCost(C.Structure):
    """nsp_attn_cost_t."""
    _fields_ = [(n, C.c_double) for n in ("pairs", "fwd_flop", "bwd_flop", "tiles",
                                           "fwd_bytes", "bwd_bytes")]


class NspError(RuntimeError):
    def __init__(self, fn: str, status: int):
        self.status = status
        super().__init__(f"{fn} failed: {status_str(status)} ({status})")


def header_functions() -> list:
    """Names of the functions declared in include/nsp.h."""
    with open(HEADER) as f:
        src = f.read()
    src = re.sub(r"/\*.*?\*/", "", src, flags=re.S)
    return sorted(set(re.findall(r"\b(nsp_[a-z0-9_]+)\s*\(", src)))


def load(path: str = LIB_PATH) -> C.CDLL:
    """Load libnsp.so (raises if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise RuntimeError(f"{path} is missing: build the CUDA library first "
                           "(python -c 'import __graft_entry__ as g; g.build()')")
    lib = C.CDLL(path)
    for name, (res, args) in _SIGNATURES.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    _lib = lib
    return lib


def status_str(status: int) -> str:
    return load().nsp_status_str(int(status)).decode()


def _ptr(t: Optional[torch.Tensor]) -> Optional[int]:
    if t is None:
        return None
    if not t.is_contiguous():
        raise ValueError("libnsp takes contiguous tensors only")
    return t.data_ptr() or None


def _stream(stream) -> int:
    if stream is None:
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, torch.cuda.Stream):
        return stream.cuda_stream
    return int(stream)


def _dtype(t: torch.Tensor) -> int:
    if t.dtype == torch.bfloat16:
        return NSP_BF16
    if t.dtype == torch.float32:
        return NSP_F32
    raise TypeError(f"unsupported dtype {t.dtype}")


def _check(fn: str, st: int) -> int:
    if st != NSP_OK:
        raise NspError(fn, st)
    return st


# ----------------------------------------------------------------------------- raw entry points

def nsp_attn_fwd_workspace_size(q_len: int, kv_len: int, Hq: int, Hkv: int, d: int) -> int:
    return int(load().nsp_attn_fwd_workspace_size(q_len, kv_len, Hq, Hkv, d))


def _block_array(blocks):
    """blocks: sequence of (q_start, q_len, kv_start, kv_len, out, lse)."""
    arr = (Block * len(blocks))()
    for i, (qs, ql, ks, kl, out, lse) in enumerate(blocks):
        arr[i] = Block(int(qs), int(ql), int(ks), int(kl), _ptr(out), _ptr(lse))
    return arr


def nsp_attn_fwd_blocks_workspace_size(blocks, Hq: int, Hkv: int, d: int) -> int:
    arr = _block_array(blocks)
    return int(load().nsp_attn_fwd_blocks_workspace_size(len(blocks), C.cast(arr, C.c_void_p),
                                                         int(Hq), int(Hkv), int(d)))


def nsp_attn_fwd_blocks(q, k, v, cu_seqlens, ndoc, T, blocks, Hq, Hkv, d, scale, causal,
                        accumulate, workspace, stream=None) -> int:
    arr = _block_array(blocks)
    st = load().nsp_attn_fwd_blocks(_ptr(q), _ptr(k), _ptr(v), _ptr(cu_seqlens), int(ndoc),
                                    int(T), len(blocks), C.cast(arr, C.c_void_p), int(Hq),
                                    int(Hkv), int(d), float(scale), int(bool(causal)), _dtype(q),
                                    int(bool(accumulate)), _ptr(workspace),
                                    workspace.numel() * workspace.element_size(), _stream(stream))
    return _check("nsp_attn_fwd_blocks", st)


def _range_array(ranges):
    arr = (Range * len(ranges))()
    for i, (qs, ql, ks, kl) in enumerate(ranges):
        arr[i] = Range(int(qs), int(ql), int(ks), int(kl))
    return arr


def nsp_attn_bwd_blocks_workspace_size(T: int, ranges, Hq: int, Hkv: int, d: int) -> int:
    arr = _range_array(ranges)
    return int(load().nsp_attn_bwd_blocks_workspace_size(int(T), len(ranges),
                                                         C.cast(arr, C.c_void_p), int(Hq),
                                                         int(Hkv), int(d)))


def nsp_attn_bwd_blocks(q, k, v, out, dout, lse, cu_seqlens, ndoc, T, ranges, Hq, Hkv, d, scale,
                        causal, dq_acc, dk_acc, dv_acc, workspace, stream=None) -> int:
    arr = _range_array(ranges)
    st = load().nsp_attn_bwd_blocks(_ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(dout), _ptr(lse),
                                    _ptr(cu_seqlens), int(ndoc), int(T), len(ranges),
                                    C.cast(arr, C.c_void_p), int(Hq), int(Hkv), int(d),
                                    float(scale), int(bool(causal)), _dtype(q), _ptr(dq_acc),
                                    _ptr(dk_acc), _ptr(dv_acc), _ptr(workspace),
                                    workspace.numel() * workspace.element_size(), _stream(stream))
    return _check("nsp_attn_bwd_blocks", st)


def nsp_attn_bwd_workspace_size(T: int, Hq: int, Hkv: int, d: int, io_dtype: int = NSP_BF16) -> int:
    return int(load().nsp_attn_bwd_workspace_size(T, Hq, Hkv, d, int(io_dtype)))


def nsp_attn_fwd(q, k, v, cu_seqlens, ndoc, q_start, q_len, kv_start, kv_len, Hq, Hkv, d,
                 scale, causal, out, lse, workspace, stream=None) -> int:
    st = load().nsp_attn_fwd(_ptr(q), _ptr(k), _ptr(v), _ptr(cu_seqlens), int(ndoc),
                             int(q_start), int(q_len), int(kv_start), int(kv_len), int(Hq),
                             int(Hkv), int(d), float(scale), int(bool(causal)), _dtype(q),
                             _ptr(out), _dtype(out), _ptr(lse), _ptr(workspace),
                             workspace.numel() * workspace.element_size(), _stream(stream))
    return _check("nsp_attn_fwd", st)


def nsp_attn_fwd_accumulate(q, k, v, cu_seqlens, ndoc, q_start, q_len, kv_start, kv_len, Hq,
                            Hkv, d, scale, causal, acc, lse_acc, workspace, stream=None) -> int:
    st = load().nsp_attn_fwd_accumulate(_ptr(q), _ptr(k), _ptr(v), _ptr(cu_seqlens), int(ndoc),
                                        int(q_start), int(q_len), int(kv_start), int(kv_len),
                                        int(Hq), int(Hkv), int(d), float(scale),
                                        int(bool(causal)), _dtype(q), _ptr(acc), _ptr(lse_acc),
                                        _ptr(workspace),
                                        workspace.numel() * workspace.element_size(),
                                        _stream(stream))
    return _check("nsp_attn_fwd_accumulate", st)


def nsp_attn_fwd_headgroups(q, k, v, cu_seqlens, ndoc, T, Hq, Hkv, d, P, scale, causal, out, lse,
                            workspace, stream=None) -> int:
    st = load().nsp_attn_fwd_headgroups(_ptr(q), _ptr(k), _ptr(v), _ptr(cu_seqlens), int(ndoc),
                                        int(T), int(Hq), int(Hkv), int(d), int(P), float(scale),
                                        int(bool(causal)), _dtype(q), _ptr(out), _dtype(out),
                                        _ptr(lse), _ptr(workspace),
                                        workspace.numel() * workspace.element_size(),
                                        _stream(stream))
    return _check("nsp_attn_fwd_headgroups", st)


def nsp_attn_fwd_noalloc(q, k, v, cu_seqlens, ndoc, q_start, q_len, kv_start, kv_len, Hq, Hkv,
                         d, scale, causal, out, lse, device_status=None, stream=None) -> int:
    """nsp_attn_fwd for callers that cannot allocate: no workspace argument
    (the library's static device scratch is used; see include/nsp.h)."""
    st = load().nsp_attn_fwd_noalloc(_ptr(q), _ptr(k), _ptr(v), _ptr(cu_seqlens), int(ndoc),
                                     int(q_start), int(q_len), int(kv_start), int(kv_len),
                                     int(Hq), int(Hkv), int(d), float(scale), int(bool(causal)),
                                     _dtype(q), _ptr(out), _dtype(out), _ptr(lse),
                                     _ptr(device_status), _stream(stream))
    return _check("nsp_attn_fwd_noalloc", st)


def nsp_attn_bwd(q, k, v, out, dout, lse, cu_seqlens, ndoc, T, Hq, Hkv, d, scale, causal,
                 dq, dk, dv, workspace, stream=None) -> int:
    st = load().nsp_attn_bwd(_ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(dout), _ptr(lse),
                             _ptr(cu_seqlens), int(ndoc), int(T), int(Hq), int(Hkv), int(d),
                             float(scale), int(bool(causal)), _dtype(q), _ptr(dq), _ptr(dk),
                             _ptr(dv), _ptr(workspace),
                             workspace.numel() * workspace.element_size(), _stream(stream))
    return _check("nsp_attn_bwd", st)


def nsp_attn_bwd_headgroups(q, k, v, out, dout, lse, cu_seqlens, ndoc, T, Hq, Hkv, d, P, scale,
                            causal, dq, dk, dv, workspace, stream=None) -> int:
    st = load().nsp_attn_bwd_headgroups(_ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(dout),
                                        _ptr(lse), _ptr(cu_seqlens), int(ndoc), int(T), int(Hq),
                                        int(Hkv), int(d), int(P), float(scale),
                                        int(bool(causal)), _dtype(q), _ptr(dq), _ptr(dk),
                                        _ptr(dv), _ptr(workspace),
                                        workspace.numel() * workspace.element_size(),
                                        _stream(stream))
    return _check("nsp_attn_bwd_headgroups", st)


def nsp_attn_bwd_accumulate_workspace_size(q_len: int, kv_len: int, Hq: int, Hkv: int, d: int,
                                           io_dtype: int = NSP_BF16) -> int:
    return int(load().nsp_attn_bwd_accumulate_workspace_size(q_len, kv_len, Hq, Hkv, d,
                                                             int(io_dtype)))


def nsp_attn_bwd_accumulate(q, k, v, out, dout, lse, cu_seqlens, ndoc, q_start, q_len, kv_start,
                            kv_len, Hq, Hkv, d, scale, causal, dq_acc, dk_acc, dv_acc, workspace,
                            stream=None) -> int:
    st = load().nsp_attn_bwd_accumulate(
        _ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(dout), _ptr(lse), _ptr(cu_seqlens),
        int(ndoc), int(q_start), int(q_len), int(kv_start), int(kv_len), int(Hq), int(Hkv),
        int(d), float(scale), int(bool(causal)), _dtype(q), _ptr(dq_acc), _ptr(dk_acc),
        _ptr(dv_acc), _ptr(workspace), workspace.numel() * workspace.element_size(),
        _stream(stream))
    return _check("nsp_attn_bwd_accumulate", st)


def nsp_lse_merge(outs: Sequence[torch.Tensor], lses: Sequence[torch.Tensor], out, lse,
                  stream=None) -> int:
    n = len(outs)
    T, H, d = outs[0].shape
    po = (C.c_void_p * n)(*[_ptr(o) for o in outs])
    pl = (C.c_void_p * n)(*[_ptr(l) for l in lses])
    st = load().nsp_lse_merge(C.cast(po, C.c_void_p), C.cast(pl, C.c_void_p), n, T, H, d,
                              _ptr(out), _dtype(out), _ptr(lse), _stream(stream))
    return _check("nsp_lse_merge", st)


def nsp_lse_merge_batch(segments, outs_merged, lses_merged=None, stream=None) -> int:
    """segments: list of (outs, lses) partial lists; outs_merged / lses_merged:
    one tensor per segment (lses_merged entries may be None)."""
    nseg = len(segments)
    if len({o.dtype for o in outs_merged}) != 1:
        raise ValueError("nsp_lse_merge_batch: every merged output must have the same dtype")
    counts = (C.c_int32 * nseg)(*[len(o) for o, _ in segments])
    po = [_ptr(o) for os_, _ in segments for o in os_]
    pl = [_ptr(l) for _, ls in segments for l in ls]
    T, H, d = segments[0][0][0].shape
    a_o = (C.c_void_p * len(po))(*po)
    a_l = (C.c_void_p * len(pl))(*pl)
    a_d = (C.c_void_p * nseg)(*[_ptr(o) for o in outs_merged])
    a_dl = None
    if lses_merged is not None:
        a_dl = C.cast((C.c_void_p * nseg)(*[_ptr(l) if l is not None else None
                                             for l in lses_merged]), C.c_void_p)
    st = load().nsp_lse_merge_batch(nseg, C.cast(counts, C.c_void_p), C.cast(a_o, C.c_void_p),
                                    C.cast(a_l, C.c_void_p), T, H, d, C.cast(a_d, C.c_void_p),
                                    _dtype(outs_merged[0]), a_dl, _stream(stream))
    return _check("nsp_lse_merge_batch", st)


def nsp_seq2head_permute(inp, out, T, H, d, P, inverse=False, stream=None) -> int:
    st = load().nsp_seq2head_permute(_ptr(inp), _ptr(out), int(T), int(H), int(d), int(P),
                                     inp.element_size(), int(bool(inverse)), _stream(stream))
    return _check("nsp_seq2head_permute", st)


def nsp_seq2head_permute_groups(inp, out, B, L, H, d, K, inverse=False, stream=None) -> int:
    st = load().nsp_seq2head_permute_groups(_ptr(inp), _ptr(out), int(B), int(L), int(H), int(d),
                                            int(K), inp.element_size(), int(bool(inverse)),
                                            _stream(stream))
    return _check("nsp_seq2head_permute_groups", st)


def nsp_kernel_launches() -> int:
    return int(load().nsp_kernel_launches())


def nsp_path_launches(tensor_core: bool) -> int:
    """Attention kernels launched so far on the tensor-core (True) or the
    CUDA-core (False) path."""
    return int(load().nsp_path_launches(int(bool(tensor_core))))


def nsp_set_wait_timeout_cycles(cycles: int) -> int:
    """Bound of the kernels' device waits in GPU cycles (< 0: the default);
    returns the previous bound."""
    return int(load().nsp_set_wait_timeout_cycles(int(cycles)))


def nsp_status_query(workspace, stream=None) -> int:
    return int(load().nsp_status_query(_ptr(workspace), _stream(stream)))


def nsp_attn_bwd_ds_cache_size(cu_seqlens_host, Hq, causal=True) -> int:
    import numpy as np
    cu = np.ascontiguousarray(np.asarray(cu_seqlens_host, dtype=np.int32))
    return int(load().nsp_attn_bwd_ds_cache_size(cu.ctypes.data, len(cu) - 1, int(Hq),
                                                 int(bool(causal))))


def nsp_attn_bwd_blocks_ds_cache_size(cu_seqlens_host, ranges, Hq, causal=True) -> int:
    import numpy as np
    cu = np.ascontiguousarray(np.asarray(cu_seqlens_host, dtype=np.int32))
    arr = _range_array(ranges)
    return int(load().nsp_attn_bwd_blocks_ds_cache_size(cu.ctypes.data, len(cu) - 1, len(ranges),
                                                        C.cast(arr, C.c_void_p), int(Hq),
                                                        int(bool(causal))))


def nsp_bwd_ds_cache_used(workspace, stream=None) -> bool:
    used = C.c_int32(0)
    _check("nsp_bwd_ds_cache_used",
           load().nsp_bwd_ds_cache_used(_ptr(workspace), C.byref(used), _stream(stream)))
    return bool(used.value)


def bwd_workspace(T, Hq, Hkv, d, device, io_dtype=NSP_BF16, ds_cache_bytes=0):
    """A backward workspace; ds_cache_bytes > 0 appends a dS cache of that
    size (nsp_attn_bwd_ds_cache_size gives the size that holds every tile)."""
    base = nsp_attn_bwd_workspace_size(T, Hq, Hkv, d, io_dtype)
    if ds_cache_bytes > 0:
        base = (base + 1023) // 1024 * 1024 + int(ds_cache_bytes)
    return torch.empty(base, dtype=torch.uint8, device=device)


def nsp_attn_pairs(cu_seqlens_host, causal=True) -> float:
    import numpy as np
    cu = np.ascontiguousarray(np.asarray(cu_seqlens_host, dtype=np.int32))
    out = C.c_double(0.0)
    st = load().nsp_attn_pairs(cu.ctypes.data, len(cu) - 1, int(bool(causal)), C.byref(out))
    _check("nsp_attn_pairs", st)
    return out.value


def nsp_attn_cost(cu_seqlens_host, Hq, Hkv, d, causal=True, io_dtype=NSP_BF16, q_start=0,
                  q_len=None, kv_start=0, kv_len=None) -> dict:
    """Cost of one attention call (whole stream by default) as a dict."""
    import numpy as np
    cu = np.ascontiguousarray(np.asarray(cu_seqlens_host, dtype=np.int32))
    T = int(cu[-1])
    q_len = T - q_start if q_len is None else q_len
    kv_len = T - kv_start if kv_len is None else kv_len
    c = AttnCost()
    st = load().nsp_attn_cost(cu.ctypes.data, len(cu) - 1, int(q_start), int(q_len),
                              int(kv_start), int(kv_len), int(Hq), int(Hkv), int(d),
                              int(bool(causal)), int(io_dtype), C.cast(C.pointer(c), C.c_void_p))
    _check("nsp_attn_cost", st)
    return {n: getattr(c, n) for n, _ in AttnCost._fields_}


# ----------------------------------------------------------------------------- conveniences

def attn_fwd(q, k, v, cu_seqlens, scale=None, causal=True, out_dtype=None, q_start=0,
             kv_start=0, workspace=None, stream=None):
    """Allocate out/lse/workspace with torch and call nsp_attn_fwd.

    q [q_len, Hq, d], k/v [kv_len, Hkv, d] on the GPU, cu_seqlens int32 on the GPU.
    """
    q_len, Hq, d = q.shape
    kv_len, Hkv, _ = k.shape
    scale = d ** -0.5 if scale is None else scale
    out = torch.empty((q_len, Hq, d), dtype=out_dtype or q.dtype, device=q.device)
    lse = torch.empty((Hq, q_len), dtype=torch.float32, device=q.device)
    if workspace is None:
        workspace = torch.empty(nsp_attn_fwd_workspace_size(q_len, kv_len, Hq, Hkv, d),
                                dtype=torch.uint8, device=q.device)
    nsp_attn_fwd(q, k, v, cu_seqlens, cu_seqlens.numel() - 1, q_start, q_len, kv_start, kv_len,
                 Hq, Hkv, d, scale, causal, out, lse, workspace, stream)
    return out, lse


def attn_fwd_headgroups(qg, k, v, cu_seqlens, scale=None, causal=True, out_dtype=None,
                        workspace=None, stream=None):
    """Forward on q in the head-group-major layout qg [P, T, Hq/P, d]; returns
    out in the same layout and lse [Hq, T]."""
    P, T, hpg, d = qg.shape
    Hq, Hkv = P * hpg, k.shape[1]
    scale = d ** -0.5 if scale is None else scale
    out = torch.empty(qg.shape, dtype=out_dtype or qg.dtype, device=qg.device)
    lse = torch.empty((Hq, T), dtype=torch.float32, device=qg.device)
    if workspace is None:
        workspace = torch.empty(nsp_attn_fwd_workspace_size(T, T, Hq, Hkv, d), dtype=torch.uint8,
                                device=qg.device)
    nsp_attn_fwd_headgroups(qg, k, v, cu_seqlens, cu_seqlens.numel() - 1, T, Hq, Hkv, d, P, scale,
                            causal, out, lse, workspace, stream)
    return out, lse


def attn_bwd_headgroups(qg, k, v, outg, doutg, lse, cu_seqlens, scale=None, causal=True,
                        workspace=None, stream=None):
    """Backward with q, out, dout (and the returned dq) in [P, T, Hq/P, d]."""
    P, T, hpg, d = qg.shape
    Hq, Hkv = P * hpg, k.shape[1]
    scale = d ** -0.5 if scale is None else scale
    dq, dk, dv = torch.empty_like(qg), torch.empty_like(k), torch.empty_like(v)
    if workspace is None:
        workspace = torch.empty(nsp_attn_bwd_workspace_size(T, Hq, Hkv, d, _dtype(qg)),
                                dtype=torch.uint8, device=qg.device)
    nsp_attn_bwd_headgroups(qg, k, v, outg, doutg, lse, cu_seqlens, cu_seqlens.numel() - 1, T,
                            Hq, Hkv, d, P, scale, causal, dq, dk, dv, workspace, stream)
    return dq, dk, dv


def ring_accumulate_init(q_len, Hq, d, device):
    """A fresh ring accumulator: acc = 0 [q_len, Hq, d] float32, lse_acc = -inf [Hq, q_len]."""
    acc = torch.zeros((q_len, Hq, d), dtype=torch.float32, device=device)
    lse = torch.full((Hq, q_len), float("-inf"), dtype=torch.float32, device=device)
    return acc, lse


def attn_fwd_accumulate(q, k, v, cu_seqlens, acc, lse_acc, scale=None, causal=True, q_start=0,
                        kv_start=0, workspace=None, stream=None):
    """Merge the block (q rows from q_start) x (keys from kv_start) into acc/lse_acc in place."""
    q_len, Hq, d = q.shape
    kv_len, Hkv, _ = k.shape
    scale = d ** -0.5 if scale is None else scale
    if workspace is None:
        workspace = torch.empty(nsp_attn_fwd_workspace_size(q_len, kv_len, Hq, Hkv, d),
                                dtype=torch.uint8, device=q.device)
    nsp_attn_fwd_accumulate(q, k, v, cu_seqlens, cu_seqlens.numel() - 1, q_start, q_len,
                            kv_start, kv_len, Hq, Hkv, d, scale, causal, acc, lse_acc,
                            workspace, stream)
    return acc, lse_acc


def attn_fwd_blocks(q, k, v, cu_seqlens, blocks, scale=None, causal=True, accumulate=False,
                    workspace=None, stream=None):
    """Batched blocks of the whole stream q [T, Hq, d], k/v [T, Hkv, d]:
    blocks = [(q_start, q_len, kv_start, kv_len, out, lse), ...] with float32
    out [q_len, Hq, d] and lse [Hq, q_len] written (accumulate=False) or
    merged into (accumulate=True)."""
    T, Hq, d = q.shape
    Hkv = k.shape[1]
    scale = d ** -0.5 if scale is None else scale
    if workspace is None:
        workspace = torch.empty(nsp_attn_fwd_blocks_workspace_size(blocks, Hq, Hkv, d),
                                dtype=torch.uint8, device=q.device)
    nsp_attn_fwd_blocks(q, k, v, cu_seqlens, cu_seqlens.numel() - 1, T, blocks, Hq, Hkv, d, scale,
                        causal, accumulate, workspace, stream)


def attn_bwd_blocks(q, k, v, out, dout, lse, cu_seqlens, ranges, dq_acc, dk_acc, dv_acc,
                    scale=None, causal=True, workspace=None, stream=None, ds_cache_bytes=0):
    """Add the backward contributions of blocks [(q_start, q_len, kv_start,
    kv_len), ...] of the whole stream into float32 dq_acc [T, Hq, d] and
    dk_acc / dv_acc [T, Hkv, d] (lse [Hq, T], the rows' final lse).  A new
    workspace gets ds_cache_bytes of dS cache appended."""
    T, Hq, d = q.shape
    Hkv = k.shape[1]
    scale = d ** -0.5 if scale is None else scale
    if workspace is None:
        n = nsp_attn_bwd_blocks_workspace_size(T, ranges, Hq, Hkv, d)
        if ds_cache_bytes > 0:
            n = (n + 1023) // 1024 * 1024 + int(ds_cache_bytes)
        workspace = torch.empty(n, dtype=torch.uint8, device=q.device)
    nsp_attn_bwd_blocks(q, k, v, out, dout, lse, cu_seqlens, cu_seqlens.numel() - 1, T, ranges,
                        Hq, Hkv, d, scale, causal, dq_acc, dk_acc, dv_acc, workspace, stream)


def attn_bwd(q, k, v, out, dout, lse, cu_seqlens, scale=None, causal=True, workspace=None,
             stream=None):
    T, Hq, d = q.shape
    Hkv = k.shape[1]
    scale = d ** -0.5 if scale is None else scale
    dq, dk, dv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
    if workspace is None:
        workspace = torch.empty(nsp_attn_bwd_workspace_size(T, Hq, Hkv, d, _dtype(q)),
                                dtype=torch.uint8, device=q.device)
    nsp_attn_bwd(q, k, v, out, dout, lse, cu_seqlens, cu_seqlens.numel() - 1, T, Hq, Hkv, d,
                 scale, causal, dq, dk, dv, workspace, stream)
    return dq, dk, dv


def attn_bwd_accumulate(q, k, v, out, dout, lse, cu_seqlens, dq_acc, dk_acc, dv_acc, scale=None,
                        causal=True, q_start=0, kv_start=0, workspace=None, stream=None):
    """Add the block (q rows from q_start) x (keys from kv_start) into the
    float32 gradient accumulators in place."""
    q_len, Hq, d = q.shape
    kv_len, Hkv, _ = k.shape
    scale = d ** -0.5 if scale is None else scale
    if workspace is None:
        workspace = torch.empty(nsp_attn_bwd_accumulate_workspace_size(q_len, kv_len, Hq, Hkv, d,
                                                                       _dtype(q)),
                                dtype=torch.uint8, device=q.device)
    nsp_attn_bwd_accumulate(q, k, v, out, dout, lse, cu_seqlens, cu_seqlens.numel() - 1, q_start,
                            q_len, kv_start, kv_len, Hq, Hkv, d, scale, causal, dq_acc, dk_acc,
                            dv_acc, workspace, stream)
    return dq_acc, dk_acc, dv_acc


def lse_merge(outs, lses, out_dtype=torch.float32, stream=None):
    T, H, d = outs[0].shape
    out = torch.empty((T, H, d), dtype=out_dtype, device=outs[0].device)
    lse = torch.empty((H, T), dtype=torch.float32, device=outs[0].device)
    nsp_lse_merge(outs, lses, out, lse, stream)
    return out, lse


def seq2head(x, P, stream=None):
    T, H, d = x.shape
    out = torch.empty((P, T, H // P, d), dtype=x.dtype, device=x.device)
    nsp_seq2head_permute(x, out, T, H, d, P, False, stream)
    return out


def seq2head_groups(x, B, K, stream=None):
    """[B L, H, d] -> [B, K, L, H / K, d]: the receive side of B independent
    K-way (batch-aware subgroup) all-to-alls."""
    BL, H, d = x.shape
    L = BL // B
    out = torch.empty((B, K, L, H // K, d), dtype=x.dtype, device=x.device)
    nsp_seq2head_permute_groups(x, out, B, L, H, d, K, False, stream)
    return out


def head2seq_groups(y, stream=None):
    B, K, L, h, d = y.shape
    out = torch.empty((B * L, K * h, d), dtype=y.dtype, device=y.device)
    nsp_seq2head_permute_groups(y, out, B, L, K * h, d, K, True, stream)
    return out


def head2seq(y, stream=None):
    P, T, h, d = y.shape
    out = torch.empty((T, P * h, d), dtype=y.dtype, device=y.device)
    nsp_seq2head_permute(y, out, T, P * h, d, P, True, stream)
    return out


# ----------------------------------------------------------------------------- differential attention layer
#
# These calls are short enough on the GPU for the host's share to matter, so
# each tensor is looked at once and the common case takes no detours.

ROPE_SCALINGS = {None: 0, "linear": 1, "base": 2, "parts": 3}
_DTYPES = {torch.bfloat16: NSP_BF16, torch.float32: NSP_F32}
_Rope1, _Rope2 = RopeTensor * 1, RopeTensor * 2


def _io(fn: str, dtype) -> int:
    io = _DTYPES.get(dtype)
    if io is None:
        raise TypeError(f"{fn}: unsupported dtype {dtype}")
    return io


_current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device


def _on_device(fn: str, dtype, **tensors) -> int:
    """Every given tensor is of `dtype` and on the current CUDA device (the
    library takes bare pointers).  Returns that device's index."""
    dev = -2
    for name, t in tensors.items():
        if t is None:
            continue
        at = t.get_device()
        if at != dev:
            if at < 0:
                raise ValueError(f"{fn}: {name} is not on a CUDA device")
            dev = _current_device()
            if at != dev:
                raise ValueError(f"{fn}: {name} is on device {at}, the current one is {dev}")
        if t.dtype is not dtype:
            raise TypeError(f"{fn}: {name} is {t.dtype}, expected {dtype}")
    return dev


def _shape(fn: str, name: str, t, shape) -> None:
    if t is not None and t.shape != shape:
        raise ValueError(f"{fn}: {name} has shape {tuple(t.shape)}, expected {tuple(shape)}")


_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream_of(stream, dev: int) -> int:
    """The address of `stream`, or of the current stream of device `dev`."""
    if stream is None and _raw_stream is not None:
        return _raw_stream(dev)
    return _stream(stream)


def _owner(stream):
    """A context whose new tensors belong to `stream` (not None)."""
    if not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(int(stream))
    return torch.cuda.stream(stream)


def _new(stream, like, shape, dtype=None):
    """A new tensor beside `like` that belongs to `stream` (None: the current one)."""
    if stream is not None:
        with _owner(stream):
            return torch.empty(shape, dtype=dtype or like.dtype, device=like.device)
    return torch.empty(shape, dtype=dtype or like.dtype, device=like.device)


def _new_like(stream, like):
    """A new packed tensor of `like`'s shape and type that belongs to `stream`."""
    if stream is not None:
        return _new(stream, like, like.shape)
    return torch.empty_like(like, memory_format=torch.contiguous_format)


def _token_stride(fn: str, name: str, t) -> int:
    """Elements between tokens of [tokens, heads, d] whose heads are packed."""
    T, H, d = t.shape
    if t.is_contiguous():
        return H * d
    if (d > 1 and t.stride(2) != 1) or (H > 1 and t.stride(1) != d):
        raise ValueError(f"{fn}: the heads of {name} are not packed")
    if T <= 1:
        return H * d
    if t.stride(0) < H * d:
        raise ValueError(f"{fn}: the tokens of {name} overlap")
    return t.stride(0)


def rope_freqs(rot, base=10000.0, scaling=None, factor=1.0, low=1.0, high=32.0, orig_len=0,
               device=None):
    """Rotary frequencies [rot / 2], float64 (radians per position), on
    `device`: base^(-2 i / rot), scaled for long contexts by `scaling` (None,
    "linear", "base" or "parts", see nsp_rope_freqs)."""
    if scaling not in ROPE_SCALINGS:
        raise ValueError(f"rope_freqs: unknown scaling {scaling!r}")
    out = torch.empty(max(int(rot) // 2, 0), dtype=torch.float64)
    st = load().nsp_rope_freqs(int(rot), float(base), ROPE_SCALINGS[scaling], float(factor),
                               float(low), float(high), float(orig_len), out.data_ptr() or None)
    _check("nsp_rope_freqs", st)
    return out if device is None else out.to(device)


def rope(q, k, cu_seqlens, freqs, layout="half", mscale=1.0, inverse=False, start=0,
         positions=None, q_groups=1, out=None, stream=None):
    """Rotate q [T, Hq, d] and k [T, Hkv, d] (k may be None) by their tokens'
    positions: those of row start + t in its document of cu_seqlens, or
    `positions` (int32 [T]; cu_seqlens may then be None).

    freqs: rope_freqs(rot): the first rot = 2 len(freqs) columns of a head are
    rotated, as halves or as interleaved pairs (layout "half", "interleaved").
    q and k may have tokens any stride apart (columns of a fused projection).
    q_groups = P > 1: the rotated q is returned as [P, T, Hq / P, d], the
    layout attn_fwd_headgroups takes; with inverse=True q is given in it.
    inverse=True is the backward: it takes gradients of the rotated q and k to
    gradients of q and k.  out: (q_out, k_out) to write (q and k themselves to
    rotate in place), default new tensors.  Rows at or past cu_seqlens[-1] are
    not written."""
    fn, dt = "rope", q.dtype
    io = _io(fn, dt)
    qo, ko = out if out is not None else (None, None)
    dev = _on_device(fn, dt, q=q, k=k, q_out=qo, k_out=ko)
    _on_device(fn, torch.int32, cu_seqlens=cu_seqlens, positions=positions)
    _on_device(fn, torch.float64, freqs=freqs)
    if layout not in ("half", "interleaved"):
        raise ValueError(f"rope: unknown layout {layout!r}")
    P = int(q_groups)
    grouped_in, grouped_out = inverse and P > 1, not inverse and P > 1
    if q.dim() != (4 if grouped_in else 3) or P < 1:
        raise ValueError("rope: q is [T, Hq, d], or [P, T, Hq / P, d] for the inverse of a grouped q")
    if grouped_in:
        if q.shape[0] != P:
            raise ValueError("rope: q has another number of head groups than q_groups")
        _, T, hpg, d = q.shape
        Hq = P * hpg
    else:
        T, Hq, d = q.shape
        if Hq % P != 0:
            raise ValueError("rope: q_groups does not divide the heads")
    Hkv = 0
    if k is not None:
        Hkv = k.shape[1] if k.dim() == 3 else -1
        _shape(fn, "k", k, (T, Hkv, d))
    _shape(fn, "positions", positions, (T,))
    if freqs.dim() != 1:
        raise ValueError("rope: freqs is [rot / 2]")
    if positions is None and (cu_seqlens is None or cu_seqlens.dim() != 1 or cu_seqlens.numel() < 2):
        raise ValueError("rope: cu_seqlens [documents + 1] or positions are needed")
    q_shape = (P, T, Hq // P, d) if grouped_out else (T, Hq, d)
    qo_stride = ko_stride = 0                     # (0: packed)
    if qo is None:
        qo = _new(stream, q, q_shape)
    else:
        _shape(fn, "q_out", qo, q_shape)
        if grouped_out:
            _ptr(qo)
        else:
            qo_stride = _token_stride(fn, "q_out", qo)
    one = (_ptr(q) if grouped_in else q.data_ptr(), qo.data_ptr(),
           0 if grouped_in else _token_stride(fn, "q", q), qo_stride, Hq, P)
    if k is None:
        ko, n, arr = None, 1, _Rope1(one)
    else:
        if ko is None:
            ko = _new(stream, k, (T, Hkv, d))
        else:
            _shape(fn, "k_out", ko, (T, Hkv, d))
            ko_stride = _token_stride(fn, "k_out", ko)
        n, arr = 2, _Rope2(one, (k.data_ptr(), ko.data_ptr(), _token_stride(fn, "k", k), ko_stride,
                                 Hkv, 1))
    st = load().nsp_rope(C.addressof(arr), n, _ptr(cu_seqlens),
                         0 if cu_seqlens is None else cu_seqlens.numel() - 1, _ptr(positions),
                         int(start), T, d, 2 * freqs.numel(), _ptr(freqs), layout == "interleaved",
                         mscale, bool(inverse), io, _stream_of(stream, dev))
    _check("nsp_rope", st)
    return qo, ko


def _vectors(fn, q1, k1, q2, k2):
    s = q1.shape
    if len(s) != 2:
        raise ValueError(f"{fn}: the vectors are [n, dl]")
    if k1.shape != s or q2.shape != s or k2.shape != s:
        raise ValueError(f"{fn}: the vectors are of different shapes")
    return s[0], s[1]


def diff_lambda(q1, k1, q2, k2, heads, lambda_init, stream=None):
    """lambda [heads] = exp(<q1, k1>) - exp(<q2, k2>) + lambda_init of vectors
    [n, dl], n = heads, or 1 for one set shared by every head."""
    fn = "diff_lambda"
    io = _io(fn, q1.dtype)
    dev = _on_device(fn, q1.dtype, q1=q1, k1=k1, q2=q2, k2=k2)
    n, dl = _vectors(fn, q1, k1, q2, k2)
    heads = int(heads)
    lam = _new(stream, q1, (heads,))
    st = load().nsp_diff_lambda_fwd(_ptr(q1), _ptr(k1), _ptr(q2), _ptr(k2), n, dl, heads,
                                    lambda_init, io, lam.data_ptr(), _stream_of(stream, dev))
    _check("nsp_diff_lambda_fwd", st)
    return lam


def diff_lambda_bwd(dlam, q1, k1, q2, k2, stream=None):
    """Gradients of q1, k1, q2, k2 from dlam [heads] (or [heads, 1])."""
    fn = "diff_lambda_bwd"
    io = _io(fn, q1.dtype)
    dev = _on_device(fn, q1.dtype, dlam=dlam, q1=q1, k1=k1, q2=q2, k2=k2)
    n, dl = _vectors(fn, q1, k1, q2, k2)
    shape = (n, dl)
    g = (_new(stream, q1, shape), _new(stream, q1, shape), _new(stream, q1, shape),
         _new(stream, q1, shape))             # (less host time than views of one tensor)
    st = load().nsp_diff_lambda_bwd(_ptr(dlam), _ptr(q1), _ptr(k1), _ptr(q2), _ptr(k2), n, dl,
                                    dlam.numel(), io, g[0].data_ptr(), g[1].data_ptr(),
                                    g[2].data_ptr(), g[3].data_ptr(), _stream_of(stream, dev))
    _check("nsp_diff_lambda_bwd", st)
    return g


def _diff_shapes(fn, q, k, v, lam, cu_seqlens, **rows):
    """Checks of differential attention's tensors; `rows`: more of q's shape."""
    io = _io(fn, q.dtype)
    dev = _on_device(fn, q.dtype, q=q, k=k, v=v, lam=lam, **rows)
    _on_device(fn, torch.int32, cu_seqlens=cu_seqlens)
    if q.dim() != 3 or k.dim() != 3 or cu_seqlens.dim() != 1:
        raise ValueError(f"{fn}: q is [T, Hq, d], k and v [T, Hkv, d], cu_seqlens [documents + 1]")
    T, Hq, d = q.shape
    Hkv = k.shape[1]
    _shape(fn, "k", k, (T, Hkv, d))
    _shape(fn, "v", v, (T, Hkv, d))
    n = lam.numel() // Hq if Hq > 0 else 0
    if lam.dim() not in (1, 2) or lam.shape[0] != Hq or n not in (1, T):
        raise ValueError(f"{fn}: lam is [Hq], [Hq, 1] or [Hq, T]")
    for name, t in rows.items():
        _shape(fn, name, t, q.shape)
    return io, dev, T, Hq, Hkv, d, n


def _workspace(fn, stream, like, nbytes, workspace):
    if workspace is None:
        return _new(stream, like, nbytes, torch.uint8)
    _on_device(fn, torch.uint8, workspace=workspace)
    return workspace


def diff_attn_fwd(q, k, v, lam, cu_seqlens, scale=None, causal=True, save=False, workspace=None,
                  stream=None):
    """Differential attention of a packed stream: q [T, Hq, d], k and v
    [T, Hkv, d], map m of a head in columns [m d/2, (m + 1) d/2) of q and k,
    lam [Hq], [Hq, 1] or [Hq, T].  Returns out [T, Hq, d]; with save=True
    (out, out2, lse), what diff_attn_bwd needs.  v has to be finite in every row,
    those of padding documents too (see nsp_diff_attn_fwd)."""
    fn = "diff_attn_fwd"
    io, dev, T, Hq, Hkv, d, n = _diff_shapes(fn, q, k, v, lam, cu_seqlens)
    scale = (d // 2) ** -0.5 if scale is None else scale
    lib = load()
    out = _new(stream, q, (T, Hq, d))
    out2 = lse = None
    if save:
        out2, lse = _new(stream, q, (T, Hq, d)), _new(stream, q, (Hq, 2, T), torch.float32)
    ws = _workspace(fn, stream, q, lib.nsp_diff_attn_fwd_workspace_size(T), workspace)
    st = lib.nsp_diff_attn_fwd(_ptr(q), _ptr(k), _ptr(v), _ptr(lam), n, _ptr(cu_seqlens),
                               cu_seqlens.numel() - 1, T, Hq, Hkv, d, scale, bool(causal), io,
                               _ptr(out), _ptr(out2), _ptr(lse), _ptr(ws), ws.numel(),
                               _stream_of(stream, dev))
    _check("nsp_diff_attn_fwd", st)
    return (out, out2, lse) if save else out


def diff_attn_bwd(q, k, v, lam, out, out2, dout, lse, cu_seqlens, scale=None, causal=True,
                  workspace=None, stream=None):
    """Gradients (dq, dk, dv, dlam) of diff_attn_fwd(save=True); dlam is
    [Hq, 1] or [Hq, T].  q, k, v and dout have to be finite in every row."""
    fn = "diff_attn_bwd"
    io, dev, T, Hq, Hkv, d, n = _diff_shapes(fn, q, k, v, lam, cu_seqlens, out=out, out2=out2,
                                             dout=dout)
    _on_device(fn, torch.float32, lse=lse)
    _shape(fn, "lse", lse, (Hq, 2, T))
    scale = (d // 2) ** -0.5 if scale is None else scale
    lib = load()
    dq, dk, dv = (_new(stream, q, t.shape) for t in (q, k, v))
    dlam = _new(stream, q, (Hq, n))
    ws = _workspace(fn, stream, q, lib.nsp_diff_attn_bwd_workspace_size(T, Hq, Hkv, d, io), workspace)
    st = lib.nsp_diff_attn_bwd(_ptr(q), _ptr(k), _ptr(v), _ptr(lam), n, _ptr(out), _ptr(out2),
                               _ptr(dout), _ptr(lse), _ptr(cu_seqlens), cu_seqlens.numel() - 1, T,
                               Hq, Hkv, d, scale, bool(causal), io, _ptr(dq), _ptr(dk), _ptr(dv),
                               _ptr(dlam), _ptr(ws), ws.numel(), _stream_of(stream, dev))
    _check("nsp_diff_attn_bwd", st)
    return dq, dk, dv, dlam


def _norm_shapes(fn, x, weight, gate, dy=None):
    io = _io(fn, x.dtype)
    dev = _on_device(fn, x.dtype, x=x, weight=weight, gate=gate, dy=dy)
    if x.dim() != 3:
        raise ValueError(f"{fn}: x is [tokens, heads, d]")
    _shape(fn, "weight", weight, x.shape[2:])
    _shape(fn, "gate", gate, x.shape)
    return io, dev, _token_stride(fn, "x", x)


def head_norm(x, weight=None, gate=None, eps=1e-6, scale=1.0, stream=None):
    """scale * weight * x / sqrt(mean(x^2) + eps) [* sigmoid(gate)] of every
    head's row of x [tokens, heads, d] (tokens any stride apart); weight [d]."""
    io, dev, stride = _norm_shapes("head_norm", x, weight, gate)
    T, H, d = x.shape
    y = _new(stream, x, (T, H, d))
    st = load().nsp_head_norm_fwd(x.data_ptr(), stride, _ptr(weight), _ptr(gate), T, H, d, eps,
                                  scale, io, _ptr(y), _stream_of(stream, dev))
    _check("nsp_head_norm_fwd", st)
    return y


def head_norm_bwd(x, dy, weight=None, gate=None, eps=1e-6, scale=1.0, workspace=None, stream=None):
    """Gradients (dx, dweight, dgate) of head_norm; None for a weight or gate
    that is not there."""
    fn = "head_norm_bwd"
    io, dev, stride = _norm_shapes(fn, x, weight, gate, dy)
    T, H, d = x.shape
    _shape(fn, "dy", dy, (T, H, d))
    lib = load()
    dx, dw, dg, ws = _new(stream, x, (T, H, d)), None, None, None
    if gate is not None:
        dg = _new(stream, x, (T, H, d))
    if weight is not None:
        dw = _new(stream, x, (d,))
        ws = _workspace(fn, stream, x, lib.nsp_head_norm_bwd_workspace_size(T, H, d), workspace)
    st = lib.nsp_head_norm_bwd(x.data_ptr(), stride, _ptr(weight), _ptr(gate), _ptr(dy), T, H, d,
                               eps, scale, io, _ptr(dx), _ptr(dg), _ptr(dw), _ptr(ws),
                               0 if ws is None else ws.numel(), _stream_of(stream, dev))
    _check("nsp_head_norm_bwd", st)
    return dx, dw, dg


# ----------------------------------------------------------------------------- packed post-training step


def _at(a) -> int:
    """Address of an array's elements."""
    return a.buffer_info()[0]


def _qk_words(x, weight, y, dy, dx, dweight, x_stride, y_stride, dx_stride, heads, groups):
    """One nsp_qk_tensor_t as 64-bit words (built in a fraction of a structure's time)."""
    return (x, weight or 0, y or 0, dy or 0, dx or 0, dweight or 0, x_stride, y_stride, dx_stride,
            heads | groups << 32)


def _qk_shapes(fn, q, k, cu_seqlens, freqs, wq, wk, layout, positions, q_groups, **more):
    """Checks of q, k and what rotates them; `more`: more tensors of their type."""
    io = _io(fn, q.dtype)
    dev = _on_device(fn, q.dtype, q=q, k=k, wq=wq, wk=wk, **more)
    _on_device(fn, torch.int32, cu_seqlens=cu_seqlens, positions=positions)
    _on_device(fn, torch.float64, freqs=freqs)
    if layout not in ("half", "interleaved"):
        raise ValueError(f"{fn}: unknown layout {layout!r}")
    if q.dim() != 3 or (k is not None and k.dim() != 3):
        raise ValueError(f"{fn}: q is [T, Hq, d], k [T, Hkv, d]")
    T, Hq, d = q.shape
    if k is not None:
        _shape(fn, "k", k, (T, k.shape[1], d))
    elif wk is not None:
        raise ValueError(f"{fn}: wk without k")
    if q_groups < 1 or Hq % q_groups != 0:
        raise ValueError(f"{fn}: q_groups does not divide the heads")
    _shape(fn, "wq", wq, (d,))
    _shape(fn, "wk", wk, (d,))
    _shape(fn, "positions", positions, (T,))
    if freqs.dim() != 1:
        raise ValueError(f"{fn}: freqs is [rot / 2]")
    if positions is None and (cu_seqlens is None or cu_seqlens.dim() != 1 or cu_seqlens.numel() < 2):
        raise ValueError(f"{fn}: cu_seqlens [documents + 1] or positions are needed")
    return io, dev, T, Hq, d


def qk_norm_rope(q, k, cu_seqlens, freqs, wq=None, wk=None, layout="half", mscale=1.0, eps=1e-6,
                 start=0, positions=None, q_groups=1, out=None, stream=None):
    """Norm every head's row of q [T, Hq, d] and k [T, Hkv, d] (k may be None) by
    its root mean square, weight it by wq and wk [d] (None: ones) and rotate it
    by its token's position, in one pass: rope(head_norm(q, wq), head_norm(k,
    wk), ...) without the rounding in between.

    The other arguments are those of `rope`: q and k may have tokens any stride
    apart, q_groups = P > 1 returns q as [P, T, Hq / P, d], out = (q_out, k_out)
    may be q and k themselves, and rows at or past cu_seqlens[-1] are not
    written."""
    fn = "qk_norm_rope"
    P = int(q_groups)
    qo, ko = out if out is not None else (None, None)
    io, dev, T, Hq, d = _qk_shapes(fn, q, k, cu_seqlens, freqs, wq, wk, layout, positions, P,
                                   q_out=qo, k_out=ko)
    q_shape = (P, T, Hq // P, d) if P > 1 else (T, Hq, d)
    qo_stride = ko_stride = 0                     # (0: packed)
    if qo is None:
        qo = _new_like(stream, q) if P == 1 else _new(stream, q, q_shape)
    else:
        _shape(fn, "q_out", qo, q_shape)
        if P > 1:
            _ptr(qo)
        else:
            qo_stride = _token_stride(fn, "q_out", qo)
    words = _qk_words(q.data_ptr(), _ptr(wq), qo.data_ptr(), 0, 0, 0, _token_stride(fn, "q", q),
                      qo_stride, 0, Hq, P)
    n = 1
    if k is None:
        ko = None
    else:
        if ko is None:
            ko = _new_like(stream, k)
        else:
            _shape(fn, "k_out", ko, k.shape)
            ko_stride = _token_stride(fn, "k_out", ko)
        n = 2
        words += _qk_words(k.data_ptr(), _ptr(wk), ko.data_ptr(), 0, 0, 0, _token_stride(fn, "k", k),
                           ko_stride, 0, k.shape[1], 1)
    arr = array.array("q", words)
    st = load().nsp_qk_norm_rope_fwd(_at(arr), n, _ptr(cu_seqlens),
                                     0 if cu_seqlens is None else cu_seqlens.numel() - 1,
                                     _ptr(positions), int(start), T, d, 2 * freqs.numel(), _ptr(freqs),
                                     layout == "interleaved", mscale, eps, io, _stream_of(stream, dev))
    _check("nsp_qk_norm_rope_fwd", st)
    return qo, ko


def qk_norm_rope_bwd(q, k, dqr, dkr, cu_seqlens, freqs, wq=None, wk=None, layout="half", mscale=1.0,
                     eps=1e-6, start=0, positions=None, q_groups=1, out=None, workspace=None,
                     stream=None):
    """Gradients (dq, dk, dwq, dwk) of qk_norm_rope from those of its results, dqr
    ([P, T, Hq / P, d] with q_groups = P > 1) and dkr; q and k as the forward
    took them.  None for a k or a weight that is not there.  out: (dq, dk) to
    write, tokens any stride apart (columns of the fused projection's gradient),
    or q and k, or dqr and dkr themselves.  Rows at or past cu_seqlens[-1] are
    not written and add nothing to the weights' gradients."""
    fn = "qk_norm_rope_bwd"
    P = int(q_groups)
    dq, dk = out if out is not None else (None, None)
    io, dev, T, Hq, d = _qk_shapes(fn, q, k, cu_seqlens, freqs, wq, wk, layout, positions, P, dqr=dqr,
                                   dkr=dkr, dq=dq, dk=dk)
    _shape(fn, "dqr", dqr, (P, T, Hq // P, d) if P > 1 else (T, Hq, d))
    dq_stride = dk_stride = 0
    if dq is None:
        dq = _new_like(stream, q)
    else:
        _shape(fn, "dq", dq, q.shape)
        dq_stride = _token_stride(fn, "dq", dq)
    dwq = None if wq is None else _new_like(stream, wq)
    dwk = None if wk is None else _new_like(stream, wk)
    n = 1
    words = _qk_words(q.data_ptr(), _ptr(wq), 0, _ptr(dqr) if P > 1 else dqr.data_ptr(), dq.data_ptr(),
                      _ptr(dwq), _token_stride(fn, "q", q),
                      0 if P > 1 else _token_stride(fn, "dqr", dqr), dq_stride, Hq, P)
    if k is None:
        if dkr is not None:
            raise ValueError(f"{fn}: dkr without k")
        dk = None
    else:
        if dkr is None:
            raise ValueError(f"{fn}: k without dkr")
        _shape(fn, "dkr", dkr, k.shape)
        if dk is None:
            dk = _new_like(stream, k)
        else:
            _shape(fn, "dk", dk, k.shape)
            dk_stride = _token_stride(fn, "dk", dk)
        n = 2
        words += _qk_words(k.data_ptr(), _ptr(wk), 0, dkr.data_ptr(), dk.data_ptr(), _ptr(dwk),
                           _token_stride(fn, "k", k), _token_stride(fn, "dkr", dkr), dk_stride, k.shape[1], 1)
    arr = array.array("q", words)
    lib, at = load(), _at(arr)
    ws = _workspace(fn, stream, q, lib.nsp_qk_norm_rope_bwd_workspace_size(at, n, T, d), workspace)
    st = lib.nsp_qk_norm_rope_bwd(at, n, _ptr(cu_seqlens),
                                  0 if cu_seqlens is None else cu_seqlens.numel() - 1, _ptr(positions),
                                  int(start), T, d, 2 * freqs.numel(), _ptr(freqs),
                                  layout == "interleaved", mscale, eps, io, _ptr(ws), ws.numel(),
                                  _stream_of(stream, dev))
    _check("nsp_qk_norm_rope_bwd", st)
    return dq, dk, dwq, dwk


def _logit_rows(fn, name, x, shape=None):
    """Row stride of logits [T, V] whose rows are packed."""
    if x.dim() != 2:
        raise ValueError(f"{fn}: {name} is [T, vocabulary]")
    if shape is not None:
        _shape(fn, name, x, shape)
    if x.is_contiguous():
        return x.shape[1]
    if x.shape[1] > 1 and x.stride(1) != 1:
        raise ValueError(f"{fn}: the rows of {name} are not packed")
    if x.shape[0] <= 1:
        return x.shape[1]
    if x.stride(0) < x.shape[1]:
        raise ValueError(f"{fn}: the rows of {name} overlap")
    return x.stride(0)


def token_logp(logits, targets, scale=1.0, workspace=None, stream=None):
    """Log-probabilities of targets (int32 [T]; negative: none, the row is not read
    and gives zeros) under the rows of scale * logits [T, vocabulary] (rows any
    stride apart), and the rows' log sums of exponentials: (logp, lse), float32 [T]."""
    fn = "token_logp"
    io = _io(fn, logits.dtype)
    dev = _on_device(fn, logits.dtype, logits=logits)
    _on_device(fn, torch.int32, targets=targets)
    stride = _logit_rows(fn, "logits", logits)
    T, V = logits.shape
    _shape(fn, "targets", targets, (T,))
    logp, lse = _new(stream, logits, (T,), torch.float32), _new(stream, logits, (T,), torch.float32)
    lib = load()
    ws = _workspace(fn, stream, logits, lib.nsp_token_logp_workspace_size(T), workspace)
    st = lib.nsp_token_logp_fwd(logits.data_ptr(), stride, _ptr(targets), T, V, scale, io, _ptr(logp),
                                _ptr(lse), _ptr(ws), ws.numel(), _stream_of(stream, dev))
    _check("nsp_token_logp_fwd", st)
    return logp, lse


def token_logp_bwd(logits, targets, lse, dlogp, scale=1.0, out=None, stream=None):
    """Gradient of the logits from that of token_logp's logp (dlogp float32 [T]; not
    used where there is no target: such rows get zeros).  out: where to write it,
    logits themselves allowed; default a new packed tensor."""
    fn = "token_logp_bwd"
    io = _io(fn, logits.dtype)
    dev = _on_device(fn, logits.dtype, logits=logits, out=out)
    _on_device(fn, torch.int32, targets=targets)
    _on_device(fn, torch.float32, lse=lse, dlogp=dlogp)
    stride = _logit_rows(fn, "logits", logits)
    T, V = logits.shape
    for name, t in (("targets", targets), ("lse", lse), ("dlogp", dlogp)):
        _shape(fn, name, t, (T,))
    if out is None:
        out = _new(stream, logits, (T, V))
    out_stride = _logit_rows(fn, "out", out, (T, V))
    st = load().nsp_token_logp_bwd(logits.data_ptr(), stride, _ptr(targets), _ptr(lse), _ptr(dlogp), T, V,
                                   scale, io, out.data_ptr(), out_stride, _stream_of(stream, dev))
    _check("nsp_token_logp_bwd", st)
    return out


MEANS = {"tokens": 0, "documents": 1}
PREFERENCES = {"sigmoid": 0, "hinge": 1, "square": 2}


def _policy(fn, T, targets, old_logp, advantages, cu_seqlens, ref, clip_low, clip_high, kl_coef, mean,
            total, per_token):
    """nsp_policy_t of a call, and its number of documents."""
    _on_device(fn, torch.int32, targets=targets, cu_seqlens=cu_seqlens)
    _on_device(fn, torch.float32, old_logp=old_logp, advantages=advantages, ref=ref)
    if mean not in MEANS:
        raise ValueError(f"{fn}: unknown mean {mean!r}")
    if cu_seqlens.dim() != 1 or cu_seqlens.numel() < 2:
        raise ValueError(f"{fn}: cu_seqlens is [documents + 1]")
    docs = cu_seqlens.numel() - 1
    _shape(fn, "targets", targets, (T,))
    _shape(fn, "old_logp", old_logp, (T,))
    _shape(fn, "ref", ref, (T,))
    if per_token is None:
        per_token = advantages.numel() != docs
    _shape(fn, "advantages", advantages, (T if per_token else docs,))
    if ref is None:
        kl_coef = 0.0
    return Policy(_ptr(old_logp), _ptr(ref), _ptr(advantages), bool(per_token), MEANS[mean], clip_low,
                  clip_high, kl_coef, total), docs


def policy_loss(logp, targets, old_logp, advantages, cu_seqlens, ref=None, clip_low=0.2, clip_high=0.2,
                kl_coef=0.0, mean="tokens", total=0.0, per_token=None, workspace=None, stream=None):
    """Clipped policy loss of a packed stream and its gradient: (stats, dlogp).

    logp, old_logp, ref (None: no KL term): float32 [T]; targets int32 [T], negative
    where a row is not scored; advantages float32 [documents] or [T] (told apart by
    their number, documents where both are the same; per_token says which).  mean:
    "tokens" or "documents"; total: the number of scored tokens or of documents
    with one, where the mean is over more than this call.  stats float32 [4]: loss,
    and the means of the surrogate, the KL term and the clipped share; dlogp float32
    [T], zero for rows not scored (see nsp_policy_loss)."""
    fn = "policy_loss"
    dev = _on_device(fn, torch.float32, logp=logp)
    if logp.dim() != 1:
        raise ValueError(f"{fn}: logp is [T]")
    T = logp.shape[0]
    p, docs = _policy(fn, T, targets, old_logp, advantages, cu_seqlens, ref, clip_low, clip_high, kl_coef,
                      mean, total, per_token)
    lib = load()
    stats, dlogp = _new(stream, logp, (4,)), _new(stream, logp, (T,))
    ws = _workspace(fn, stream, logp, lib.nsp_policy_loss_workspace_size(T, docs, 0), workspace)
    st = lib.nsp_policy_loss(_ptr(logp), _ptr(targets), _ptr(cu_seqlens), docs, T, C.addressof(p),
                             _ptr(stats), _ptr(dlogp), _ptr(ws), ws.numel(), _stream_of(stream, dev))
    _check("nsp_policy_loss", st)
    return stats, dlogp


def policy_loss_logits(logits, targets, old_logp, advantages, cu_seqlens, ref=None, clip_low=0.2,
                       clip_high=0.2, kl_coef=0.0, mean="tokens", scale=1.0, total=0.0, per_token=None,
                       out=None, workspace=None, stream=None):
    """token_logp, policy_loss and token_logp_bwd in one pass over logits [T,
    vocabulary]: (stats, logp, dlogits), logp zero for rows not scored.  out: where
    dlogits go, logits themselves allowed; the other arguments are policy_loss's."""
    fn = "policy_loss_logits"
    io = _io(fn, logits.dtype)
    dev = _on_device(fn, logits.dtype, logits=logits, out=out)
    stride = _logit_rows(fn, "logits", logits)
    T, V = logits.shape
    p, docs = _policy(fn, T, targets, old_logp, advantages, cu_seqlens, ref, clip_low, clip_high, kl_coef,
                      mean, total, per_token)
    if out is None:
        out = _new(stream, logits, (T, V))
    out_stride = _logit_rows(fn, "out", out, (T, V))
    lib = load()
    stats, logp = _new(stream, logits, (4,), torch.float32), _new(stream, logits, (T,), torch.float32)
    ws = _workspace(fn, stream, logits, lib.nsp_policy_loss_workspace_size(T, docs, 1), workspace)
    st = lib.nsp_policy_loss_logits(logits.data_ptr(), stride, _ptr(targets), _ptr(cu_seqlens), docs, T, V,
                                    scale, io, C.addressof(p), _ptr(stats), _ptr(logp), out.data_ptr(),
                                    out_stride, _ptr(ws), ws.numel(), _stream_of(stream, dev))
    _check("nsp_policy_loss_logits", st)
    return stats, logp, out


def preference_loss(logp, targets, cu_seqlens, ref=None, kind="sigmoid", beta=0.1, smoothing=0.0,
                    margin=0.0, average=False, workspace=None, stream=None):
    """Preference loss over pairs of documents (2 i chosen, 2 i + 1 rejected) and its
    gradient: (stats, rewards, dlogp).

    logp, ref (None: zeros) float32 [T]; targets int32 [T], negative where a row is
    not scored.  kind: "sigmoid", "hinge" or "square"; average: scores are means over
    a document's scored rows instead of sums.  stats float32 [2]: the loss and the
    share of pairs whose chosen answer has the larger reward; rewards float32
    [documents]; dlogp float32 [T] (see nsp_preference_loss)."""
    fn = "preference_loss"
    dev = _on_device(fn, torch.float32, logp=logp, ref=ref)
    _on_device(fn, torch.int32, targets=targets, cu_seqlens=cu_seqlens)
    if kind not in PREFERENCES:
        raise ValueError(f"{fn}: unknown kind {kind!r}")
    if logp.dim() != 1:
        raise ValueError(f"{fn}: logp is [T]")
    T = logp.shape[0]
    _shape(fn, "targets", targets, (T,))
    _shape(fn, "ref", ref, (T,))
    docs = cu_seqlens.numel() - 1
    if cu_seqlens.dim() != 1 or docs < 2 or docs % 2 != 0:
        raise ValueError(f"{fn}: cu_seqlens is [documents + 1] of an even number of documents")
    lib = load()
    stats, rewards, dlogp = _new(stream, logp, (2,)), _new(stream, logp, (docs,)), _new(stream, logp, (T,))
    ws = _workspace(fn, stream, logp, lib.nsp_preference_loss_workspace_size(docs), workspace)
    st = lib.nsp_preference_loss(_ptr(logp), _ptr(ref), _ptr(targets), _ptr(cu_seqlens), docs, T,
                                 PREFERENCES[kind], beta, smoothing, margin, bool(average), _ptr(stats),
                                 _ptr(rewards), _ptr(dlogp), _ptr(ws), ws.numel(), _stream_of(stream, dev))
    _check("nsp_preference_loss", st)
    return stats, rewards, dlogp


NORMS = {2: 0, 2.0: 0, float("inf"): 1}


# (hundreds of tensors a call: one C loop over them for each thing looked at)
_data_ptr, _numel = torch.Tensor.data_ptr, torch.Tensor.numel
_get_device, _is_contiguous = torch.Tensor.get_device, torch.Tensor.is_contiguous
_get_dtype = operator.attrgetter("dtype")


def _gradients(fn, grads, dev=None):
    """HOST arrays of the gradients' pointers, counts and types, and their device."""
    n = len(grads)
    if n == 0:
        raise ValueError(f"{fn}: no gradients")
    at = set(map(_get_device, grads))
    if dev is None:
        if -1 in at:
            raise ValueError(f"{fn}: a gradient is not on a CUDA device")
        dev = _current_device()
    if at != {dev}:
        raise ValueError(f"{fn}: a gradient is not on the current device {dev}")
    if not all(map(_is_contiguous, grads)):
        raise ValueError(f"{fn}: libnsp takes contiguous tensors only")
    types = list(map(_DTYPES.get, map(_get_dtype, grads)))
    if None in types:
        raise TypeError(f"{fn}: unsupported dtype {grads[types.index(None)].dtype}")
    return (array.array("Q", map(_data_ptr, grads)), array.array("q", map(_numel, grads)),
            array.array("i", types), n, dev)


def grad_norm(grads, norm_type=2, unscale=1.0, workspace=None, stream=None):
    """Norm (norm_type 2 or inf) of all gradients of a list taken together, times
    |unscale|: float32 [1].  Contiguous tensors of both types, any sizes."""
    fn = "grad_norm"
    if norm_type not in NORMS:
        raise ValueError(f"{fn}: unknown norm {norm_type!r}")
    ptrs, counts, types, n, dev = _gradients(fn, grads)
    lib = load()
    norm = _new(stream, grads[0], (1,), torch.float32)
    ws = _workspace(fn, stream, norm, lib.nsp_grad_norm_workspace_size(_at(counts), n), workspace)
    st = lib.nsp_grad_norm(_at(ptrs), _at(counts), _at(types), n, NORMS[norm_type], unscale, norm.data_ptr(), _ptr(ws),
                           ws.numel(), _stream_of(stream, dev))
    _check("nsp_grad_norm", st)
    return norm


def clip_grads(grads, max_norm, norm_type=2, unscale=1.0, eps=1e-6, out=None, workspace=None,
               stream=None):
    """Scale all gradients of a list by unscale * min(1, max_norm / (norm + eps)),
    norm their grad_norm, which is returned (before clipping; float32 [1]).  In
    place, or into `out`: a list of tensors of the same sizes, of either type."""
    fn = "clip_grads"
    if norm_type not in NORMS:
        raise ValueError(f"{fn}: unknown norm {norm_type!r}")
    ptrs, counts, types, n, dev = _gradients(fn, grads)
    out_ptrs, out_types = ptrs, types
    if out is not None:
        out_ptrs, out_counts, out_types, _, _ = _gradients(fn, out, dev)
        if out_counts != counts:
            raise ValueError(f"{fn}: out are as many tensors of the gradients' sizes")
    lib = load()
    norm = _new(stream, grads[0], (1,), torch.float32)
    ws = _workspace(fn, stream, norm, lib.nsp_grad_norm_workspace_size(_at(counts), n), workspace)
    st = lib.nsp_grad_clip(_at(ptrs), _at(out_ptrs), _at(counts), _at(types), _at(out_types), n, NORMS[norm_type], unscale, max_norm,
                           eps, norm.data_ptr(), _ptr(ws), ws.numel(), _stream_of(stream, dev))
    _check("nsp_grad_clip", st)
    return norm
