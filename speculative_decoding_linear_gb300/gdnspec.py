"""Thin Python binding of libgdnspec.so (the C ABI in include/gdnspec.h).

Argument marshalling only: every function here forwards device pointers,
sizes and the current CUDA stream to the entry point of the same name and
turns a negative status into :class:`GdnError`.  All arithmetic runs in the
library's CUDA kernels; there is no CPU fallback -- if the compiled library is
missing, importing it raises.

Tensors are PyTorch CUDA tensors (PyTorch is used for device memory and
streams only); plain integer device addresses are accepted as well.
"""
from __future__ import annotations

import ctypes
import functools
import os
import threading

import torch

from . import build as _build

_lib = None
_lock = threading.Lock()

OK, ERR_ARG, ERR_TREE, ERR_PATH, ERR_TIMEOUT, ERR_CUDA, ERR_DEVICE, ERR_CAPACITY, ERR_INDEX = (
    0, -1, -2, -3, -4, -5, -6, -7, -8)
DTYPE_BF16, DTYPE_F32 = 0, 1

# (name, restype, argtypes) for every extern "C" symbol of include/gdnspec.h
_P, _I, _S = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t
SIGNATURES = {
    "gdn_factors_bytes": (_I, [_I, _I, _I, _I, _I, _I, ctypes.POINTER(_S)]),
    "gdn_workspace_bytes": (_I, [_I, _I, _I, _I, _I, ctypes.POINTER(_S)]),
    "gdn_tree_mask": (_I, [_P, _I, _I, _P, _P, _P]),
    "gdn_tree_verify": (_I, [_P, _P, _P, _I, _P, _P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _P]),
    "gdn_tree_verify_noalloc": (_I, [_P, _P, _P, _I, _P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _P]),
    "gdn_chain_verify": (_I, [_P, _P, _P, _I, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _P]),
    "gdn_commit": (_I, [_P, _P, _P, _I, _P, _I, _I, _I, _I, _I, _I, _P]),
    "gdn_commit_tree_verify": (_I, [_P, _P, _I, _P, _I, _P, _P, _P, _I, _P, _P, _P, _P, _P, _P,
                                    _I, _I, _I, _I, _I, _P]),
    "gdn_commit_chain_verify": (_I, [_P, _P, _I, _P, _I, _P, _P, _P, _I, _P, _P, _P, _P,
                                     _I, _I, _I, _I, _I, _P]),
    "gdn_layer_record_bytes": (_I, [_I, _I, _I, _I, _I, _I, ctypes.POINTER(_S)]),
    "gdn_layer_workspace_bytes": (_I, [_I, _I, _I, _I, _I, _I, ctypes.POINTER(_S)]),
    "gdn_layer_tree_step": (_I, [_P, _P, _P, _P, _P, _P, _P, _P, _I, _P, _I, _P, _P, _P,
                                 _I, _I, _I, _I, _I, _I, _P]),
    "gdn_layer_token_step": (_I, [_P, _P, _P, _P, _P, _P, _P, _P, _I, _P, _P, _P,
                                  _I, _I, _I, _I, _I, _I, _P]),
    "gdn_layer_stage_events": (_I, [_P, _I]),
    "gdn_model_workspace_bytes": (_I, [_I, _I, _I, _I, _I, _I, _I, ctypes.POINTER(_S)]),
    "gdn_model_tree_step": (_I, [_I, _P, _P, _P, _P, _P, _P, _P, _P, _I, _P, _I, _P, _P, _P,
                                 _I, _I, _I, _I, _I, _I, _P]),
    "gdn_prune_tree": (_I, [_P, _P, ctypes.c_float, _I, _P, _P, _P, _I, _I, _P]),
    "gdn_hybrid_workspace_bytes": (_I, [_I, _I, _I, _I, _I, _P]),
    "gdn_hybrid_tree_verify": (_I, [_P, _P, _P, _I, _P, _P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _P]),
    "gdn_replay_tree_verify": (_I, [_P, _P, _P, _I, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _P]),
    "gdn_replay_commit": (_I, [_P, _P, _I, _P, _P, _P, _P, _P, _I, _P, _I, _I, _I, _I, _I, _P]),
    "gdn_snapshot_tree_verify": (_I, [_P, _P, _P, _I, _P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _P]),
    "gdn_snapshot_commit": (_I, [_P, _P, _P, _P, _I, _P, _I, _I, _I, _I, _I, _P]),
    "gdn_linear_tree_verify": (_I, [_P, _P, _P, _I, _P, _P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _P]),
    "gdn_gla_factors_bytes": (_I, [_I, _I, _I, _I, _I, _I, ctypes.POINTER(_S)]),
    "gdn_gla_workspace_bytes": (_I, [_I, _I, _I, _I, _I, ctypes.POINTER(_S)]),
    "gdn_gla_tree_verify": (_I, [_P, _P, _P, _I, _P, _P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _P]),
    "gdn_gla_commit": (_I, [_P, _P, _P, _I, _P, _I, _I, _I, _I, _I, _I, _P]),
    "gdn_seq_workspace_bytes": (_I, [_I] * 7 + [ctypes.POINTER(_S)]),
    "gdn_seq_forward_workspace_bytes": (_I, [_I] * 7 + [ctypes.POINTER(_S)]),
    "gdn_seq_record_bytes": (_I, [_I] * 7 + [ctypes.POINTER(_S)]),
    "gdn_seq_forward": (_I, [_P, _I, _P, _I, _P, _I, _I] + [_P] * 8 + [_I] * 6 + [_P]),
    "gdn_seq_backward": (_I, [_P, _I, _P, _I, _P, _I, _I] + [_P] * 13 + [_I] * 6 + [_P]),
    "gdn_seq_step": (_I, [_P, _P, _P, _I] + [_P] * 5 + [_I] * 6 + [_P]),
    "gdn_linear_seq_workspace_bytes": (_I, [_I] * 7 + [ctypes.POINTER(_S)]),
    "gdn_linear_seq_forward_workspace_bytes": (_I, [_I] * 7 + [ctypes.POINTER(_S)]),
    "gdn_linear_seq_record_bytes": (_I, [_I] * 7 + [ctypes.POINTER(_S)]),
    "gdn_linear_seq_forward": (_I, [_P, _I, _P, _I, _P, _I, _I] + [_P] * 8 + [_I] * 6 + [_P]),
    "gdn_linear_seq_backward": (_I, [_P, _I, _P, _I, _P, _I, _I] + [_P] * 13 + [_I] * 6 + [_P]),
    "gdn_linear_seq_step": (_I, [_P, _P, _P, _I] + [_P] * 5 + [_I] * 6 + [_P]),
    "gdn_rotary_frequencies": (_I, [_I] + [ctypes.c_double] * 5 + [_P]),
    "gdn_rotary": (_I, [_P, _I, _P, _I, _I, _P, _P, ctypes.c_float, _P, _I, _P, _I] + [_I] * 7 + [_P]),
    "gdn_norm_workspace_bytes": (_I, [ctypes.c_longlong, _I, ctypes.POINTER(_S)]),
    "gdn_gated_norm": (_I, [_P, _I, _P, _P, _P, _I, ctypes.c_longlong, _I, ctypes.c_float, _P]),
    "gdn_gated_norm_backward": (_I, [_P, _I] + [_P] * 7 + [_I, ctypes.c_longlong, _I, ctypes.c_float, _P]),
    "gdn_block_norm": (_I, [_P] * 7 + [_I, ctypes.c_longlong, _I, ctypes.c_float, ctypes.c_float, _P]),
    "gdn_block_norm_backward": (_I, [_P] * 13 + [_I, ctypes.c_longlong, _I, ctypes.c_float, ctypes.c_float, _P]),
    "gdn_set_launch_overlap": (_I, [_I]),
    "gdn_set_wait_limit_ns": (_I, [ctypes.c_ulonglong]),
    "gdn_selftest_stuck_wait": (_I, [_P]),
    "gdn_last_error": (_I, [_P]),
    "gdn_strerror": (ctypes.c_char_p, [_I]),
}


class GdnError(RuntimeError):
    def __init__(self, code: int, where: str):
        self.code = code
        super().__init__("%s: %s (status %d)" % (where, strerror(code), code))


def library_path() -> str:
    return _build.LIB


def lib(build_if_missing: bool = True) -> ctypes.CDLL:
    """The loaded libgdnspec.so.  Builds it when absent (nvcc required); raises if it cannot."""
    global _lib
    loaded = _lib              # once loaded, every call returns it without taking the lock
    if loaded is not None:
        return loaded
    with _lock:
        if _lib is None:
            path = _build.LIB
            if build_if_missing and not _build.up_to_date():
                _build.build()
            if not os.path.exists(path):
                raise ImportError("libgdnspec.so not found at %s: the CUDA library is required "
                                  "(there is no CPU fallback)" % path)
            L = ctypes.CDLL(path)
            for name, (res, args) in SIGNATURES.items():
                f = getattr(L, name)
                f.restype = res
                f.argtypes = args
            _lib = L
    return _lib


def strerror(code: int) -> str:
    return lib().gdn_strerror(int(code)).decode()


def _check(rc: int, where: str):
    if rc != OK:
        raise GdnError(rc, where)


def _ptr(x):
    if type(x) is torch.Tensor or isinstance(x, torch.Tensor):
        if x.is_cuda and x.is_contiguous():
            return x.data_ptr()
        raise ValueError("expected a contiguous CUDA tensor")
    if x is None:
        return None
    if isinstance(x, int):
        return x
    raise TypeError(type(x))


# The current stream as a raw handle without building a Stream object (a few
# microseconds per call otherwise, more than a chain verification on the GPU).
_raw_current_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


def _stream(stream):
    if stream is None:
        if _raw_current_stream is not None:
            return _raw_current_stream(_current_device())
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, torch.cuda.Stream):
        return stream.cuda_stream
    return int(stream)


_DTYPE_CODES = {torch.bfloat16: DTYPE_BF16, "bf16": DTYPE_BF16, torch.float32: DTYPE_F32, "f32": DTYPE_F32}


def dtype_code(t) -> int:
    code = _DTYPE_CODES.get(t)
    if code is None:
        raise ValueError("q/k/v must be bf16 or fp32, got %s" % (t,))
    return code


# ---------------------------------------------------------------------------
# sizes
# ---------------------------------------------------------------------------
def gdn_factors_bytes(B, N, H, dk, dv, dtype) -> int:
    out = ctypes.c_size_t(0)
    _check(lib().gdn_factors_bytes(B, N, H, dk, dv, dtype_code(dtype) if not isinstance(dtype, int)
                                   else dtype, ctypes.byref(out)), "gdn_factors_bytes")
    return out.value


def gdn_workspace_bytes(B, N, H, dk, dv) -> int:
    out = ctypes.c_size_t(0)
    _check(lib().gdn_workspace_bytes(B, N, H, dk, dv, ctypes.byref(out)), "gdn_workspace_bytes")
    return out.value


def empty_factors(B, N, H, dk, dv, dtype, device="cuda"):
    """Caller-owned factor buffer (uint8 tensor) of the size the library asks for."""
    return torch.empty(gdn_factors_bytes(B, N, H, dk, dv, dtype), dtype=torch.uint8, device=device)


def empty_workspace(B, N, H, dk, dv, device="cuda"):
    return torch.empty(gdn_workspace_bytes(B, N, H, dk, dv), dtype=torch.uint8, device=device)


# ---------------------------------------------------------------------------
# entry points (same names as the C ABI)
# ---------------------------------------------------------------------------
def _dims(q, v):
    B, N, H, dk = q.shape
    return B, N, H, dk, v.shape[-1]


def gdn_tree_mask(parent_idx, mask, depth, stream=None):
    B, N = parent_idx.shape
    _check(lib().gdn_tree_mask(_ptr(parent_idx), B, N, _ptr(mask), _ptr(depth), _stream(stream)),
           "gdn_tree_mask")


def gdn_tree_verify(q, k, v, alpha, beta, parent_idx, S0, out, factors, workspace, stream=None):
    B, N, H, dk, dv = _dims(q, v)
    _check(lib().gdn_tree_verify(_ptr(q), _ptr(k), _ptr(v), dtype_code(q.dtype), _ptr(alpha),
                                 _ptr(beta), _ptr(parent_idx), _ptr(S0), _ptr(out), _ptr(factors),
                                 _ptr(workspace), B, N, H, dk, dv, _stream(stream)),
           "gdn_tree_verify")


def gdn_tree_verify_noalloc(q, k, v, alpha, beta, parent_idx, S0, out, factors, stream=None):
    """gdn_tree_verify without a workspace argument: for callers that cannot allocate device
    memory (a framework that owns all device memory, or a decode loop that must not allocate).
    The workspace is a fixed 32 MiB scratch array inside the library, shared by all calls on a
    device; calls overlapping on the GPU race on it.  See include/gdnspec.h."""
    B, N, H, dk, dv = _dims(q, v)
    _check(lib().gdn_tree_verify_noalloc(_ptr(q), _ptr(k), _ptr(v), dtype_code(q.dtype), _ptr(alpha),
                                         _ptr(beta), _ptr(parent_idx), _ptr(S0), _ptr(out),
                                         _ptr(factors), B, N, H, dk, dv, _stream(stream)),
           "gdn_tree_verify_noalloc")


def gdn_chain_verify(q, k, v, alpha, beta, S0, out, factors, stream=None):
    B, N, H, dk, dv = _dims(q, v)
    _check(lib().gdn_chain_verify(_ptr(q), _ptr(k), _ptr(v), dtype_code(q.dtype), _ptr(alpha),
                                  _ptr(beta), _ptr(S0), _ptr(out), _ptr(factors), B, N, H, dk, dv,
                                  _stream(stream)), "gdn_chain_verify")


def gdn_commit(S0, factors, accepted_path, S_new, N, dtype, stream=None):
    B, H, dv, dk = S0.shape
    _check(lib().gdn_commit(_ptr(S0), _ptr(factors), _ptr(accepted_path), accepted_path.shape[1],
                            _ptr(S_new), B, N, H, dk, dv, dtype_code(dtype), _stream(stream)),
           "gdn_commit")


def gdn_commit_tree_verify(S, prev_factors, N_prev, prev_path, q, k, v, alpha, beta, parent_idx,
                           out, factors, workspace, stream=None):
    B, N, H, dk, dv = _dims(q, v)
    _check(lib().gdn_commit_tree_verify(_ptr(S), _ptr(prev_factors), N_prev, _ptr(prev_path),
                                        prev_path.shape[1], _ptr(q), _ptr(k), _ptr(v),
                                        dtype_code(q.dtype), _ptr(alpha), _ptr(beta),
                                        _ptr(parent_idx), _ptr(out), _ptr(factors), _ptr(workspace),
                                        B, N, H, dk, dv, _stream(stream)), "gdn_commit_tree_verify")


def gdn_commit_chain_verify(S, prev_factors, N_prev, prev_path, q, k, v, alpha, beta, out, factors,
                            stream=None):
    B, N, H, dk, dv = _dims(q, v)
    _check(lib().gdn_commit_chain_verify(_ptr(S), _ptr(prev_factors), N_prev, _ptr(prev_path),
                                         prev_path.shape[1], _ptr(q), _ptr(k), _ptr(v),
                                         dtype_code(q.dtype), _ptr(alpha), _ptr(beta), _ptr(out),
                                         _ptr(factors), B, N, H, dk, dv, _stream(stream)),
           "gdn_commit_chain_verify")


def gdn_layer_record_bytes(B, N, H, hidden, dk, dv) -> int:
    out = ctypes.c_size_t(0)
    _check(lib().gdn_layer_record_bytes(B, N, H, hidden, dk, dv, ctypes.byref(out)), "gdn_layer_record_bytes")
    return out.value


def gdn_layer_workspace_bytes(B, N, H, hidden, dk, dv) -> int:
    out = ctypes.c_size_t(0)
    _check(lib().gdn_layer_workspace_bytes(B, N, H, hidden, dk, dv, ctypes.byref(out)),
           "gdn_layer_workspace_bytes")
    return out.value


def gdn_layer_tree_step(X, W_in, conv_w, W_o, parent_idx, S, conv_state, prev_record, N_prev, prev_path,
                        out, record, workspace, H, dk, dv, stream=None):
    """One GDN layer decode step over B draft trees (see include/gdnspec.h).  prev_record and
    prev_path are both None when there is no pending commit."""
    B, N, hidden = X.shape
    Lmax = 0 if prev_path is None else prev_path.shape[1]
    _check(lib().gdn_layer_tree_step(_ptr(X), _ptr(W_in), _ptr(conv_w), _ptr(W_o), _ptr(parent_idx), _ptr(S),
                                     _ptr(conv_state), _ptr(prev_record), int(N_prev), _ptr(prev_path), Lmax,
                                     _ptr(out), _ptr(record), _ptr(workspace), B, N, H, hidden, dk, dv,
                                     _stream(stream)), "gdn_layer_tree_step")


def gdn_layer_token_step(X, W_in, conv_w, W_o, parent_idx, S0, conv_state, S_nodes, t, out, record, workspace,
                         H, dk, dv, stream=None):
    """Decode node t of every tree on its own from its parent's materialised state (see
    include/gdnspec.h); S_nodes is [N, B, H, dv, dk] fp32."""
    B, N, hidden = X.shape
    _check(lib().gdn_layer_token_step(_ptr(X), _ptr(W_in), _ptr(conv_w), _ptr(W_o), _ptr(parent_idx), _ptr(S0),
                                      _ptr(conv_state), _ptr(S_nodes), int(t), _ptr(out), _ptr(record),
                                      _ptr(workspace), B, N, H, hidden, dk, dv, _stream(stream)),
           "gdn_layer_token_step")


def gdn_layer_stage_events(events):
    """Turn the layer step's per-kernel timing hook on with 6 torch.cuda.Event objects (timing
    enabled, each recorded at least once so that its CUDA event exists), or off with None (see
    include/gdnspec.h)."""
    if events is None:
        _check(lib().gdn_layer_stage_events(None, 0), "gdn_layer_stage_events")
        return
    arr = (ctypes.c_void_p * len(events))(*[e.cuda_event if hasattr(e, "cuda_event") else int(e) for e in events])
    _check(lib().gdn_layer_stage_events(ctypes.cast(arr, ctypes.c_void_p), len(events)), "gdn_layer_stage_events")


def gdn_model_workspace_bytes(L, B, N, H, hidden, dk, dv) -> int:
    out = ctypes.c_size_t(0)
    _check(lib().gdn_model_workspace_bytes(L, B, N, H, hidden, dk, dv, ctypes.byref(out)),
           "gdn_model_workspace_bytes")
    return out.value


def _ptr_array(xs):
    if xs is None:
        return None
    arr = (ctypes.c_void_p * len(xs))(*[_ptr(x) for x in xs])
    return ctypes.cast(arr, ctypes.c_void_p), arr      # keep the array alive with the call


def gdn_model_tree_step(X, W_in, conv_w, W_o, parent_idx, S, conv_state, prev_records, N_prev, prev_path, out,
                        records, workspace, H, dk, dv, stream=None):
    """L layers back to back (see include/gdnspec.h); the per-layer arguments are lists of L tensors."""
    B, N, hidden = X.shape
    L = len(W_in)
    arrs = [_ptr_array(x) for x in (W_in, conv_w, W_o, S, conv_state, prev_records, records)]
    ptrs = [a[0] if a is not None else None for a in arrs]
    Lmax = 0 if prev_path is None else prev_path.shape[1]
    _check(lib().gdn_model_tree_step(L, _ptr(X), ptrs[0], ptrs[1], ptrs[2], _ptr(parent_idx), ptrs[3], ptrs[4],
                                     ptrs[5], int(N_prev), _ptr(prev_path), Lmax, _ptr(out), ptrs[6],
                                     _ptr(workspace), B, N, H, hidden, dk, dv, _stream(stream)),
           "gdn_model_tree_step")


def gdn_prune_tree(parent_idx, logp, tau, budget, new_index, new_parent, n_kept, stream=None):
    """Confidence-guided pruning of B draft trees (see include/gdnspec.h)."""
    B, N = parent_idx.shape
    _check(lib().gdn_prune_tree(_ptr(parent_idx), _ptr(logp), float(tau), int(budget), _ptr(new_index),
                                _ptr(new_parent), _ptr(n_kept), B, N, _stream(stream)), "gdn_prune_tree")


def gdn_hybrid_workspace_bytes(B, N, H, dk, dv) -> int:
    out = ctypes.c_size_t(0)
    _check(lib().gdn_hybrid_workspace_bytes(B, N, H, dk, dv, ctypes.byref(out)), "gdn_hybrid_workspace_bytes")
    return out.value


def gdn_hybrid_tree_verify(q, k, v, alpha, beta, parent_idx, S0, out, factors, workspace, stream=None):
    """Chain-decomposed tree verification (see include/gdnspec.h); same outputs and factor record as
    gdn_tree_verify.  workspace: gdn_hybrid_workspace_bytes(...) bytes (None when that is 0)."""
    B, N, H, dk, dv = _dims(q, v)
    _check(lib().gdn_hybrid_tree_verify(_ptr(q), _ptr(k), _ptr(v), dtype_code(q.dtype), _ptr(alpha), _ptr(beta),
                                        _ptr(parent_idx), _ptr(S0), _ptr(out), _ptr(factors),
                                        _ptr(workspace), B, N, H, dk, dv,
                                        _stream(stream)), "gdn_hybrid_tree_verify")


def gdn_replay_tree_verify(q, k, v, alpha, beta, parent_idx, S0, out, stream=None):
    """Baseline: replay every root-to-leaf path token by token (see include/gdnspec.h)."""
    B, N, H, dk, dv = _dims(q, v)
    _check(lib().gdn_replay_tree_verify(_ptr(q), _ptr(k), _ptr(v), dtype_code(q.dtype), _ptr(alpha), _ptr(beta),
                                        _ptr(parent_idx), _ptr(S0), _ptr(out), B, N, H, dk, dv, _stream(stream)),
           "gdn_replay_tree_verify")


def gdn_replay_commit(k, v, alpha, beta, parent_idx, S0, accepted_path, S_new, stream=None):
    """Baseline: replay the accepted tokens from S0 into S_new (see include/gdnspec.h)."""
    B, N, H, dk, dv = _dims(k, v)
    _check(lib().gdn_replay_commit(_ptr(k), _ptr(v), dtype_code(k.dtype), _ptr(alpha), _ptr(beta), _ptr(parent_idx),
                                   _ptr(S0), _ptr(accepted_path), accepted_path.shape[1], _ptr(S_new), B, N, H, dk,
                                   dv, _stream(stream)), "gdn_replay_commit")


def gdn_snapshot_tree_verify(q, k, v, alpha, beta, parent_idx, S0, out, S_nodes, stream=None):
    """Baseline: build and store every draft node's state, node by node (see include/gdnspec.h);
    S_nodes is [N, B, H, dv, dk] fp32."""
    B, N, H, dk, dv = _dims(q, v)
    _check(lib().gdn_snapshot_tree_verify(_ptr(q), _ptr(k), _ptr(v), dtype_code(q.dtype), _ptr(alpha), _ptr(beta),
                                          _ptr(parent_idx), _ptr(S0), _ptr(out), _ptr(S_nodes), B, N, H, dk, dv,
                                          _stream(stream)), "gdn_snapshot_tree_verify")


def gdn_snapshot_commit(S_nodes, S0, parent_idx, accepted_path, S_new, stream=None):
    """Baseline: the accepted node's stored state becomes the committed state (see include/gdnspec.h)."""
    N, B, H, dv, dk = S_nodes.shape
    _check(lib().gdn_snapshot_commit(_ptr(S_nodes), _ptr(S0), _ptr(parent_idx), _ptr(accepted_path),
                                     accepted_path.shape[1], _ptr(S_new), B, N, H, dk, dv, _stream(stream)),
           "gdn_snapshot_commit")


def gdn_linear_tree_verify(q, k, v, alpha, beta, parent_idx, S0, out, factors, workspace, stream=None):
    """Decay-gated linear attention (no delta-rule erasure) over a draft tree; see include/gdnspec.h."""
    B, N, H, dk, dv = _dims(q, v)
    _check(lib().gdn_linear_tree_verify(_ptr(q), _ptr(k), _ptr(v), dtype_code(q.dtype), _ptr(alpha), _ptr(beta),
                                        _ptr(parent_idx), _ptr(S0), _ptr(out), _ptr(factors), _ptr(workspace),
                                        B, N, H, dk, dv, _stream(stream)), "gdn_linear_tree_verify")


def gdn_gla_factors_bytes(B, N, H, dk, dv, dtype) -> int:
    out = ctypes.c_size_t(0)
    _check(lib().gdn_gla_factors_bytes(B, N, H, dk, dv, dtype_code(dtype) if not isinstance(dtype, int) else dtype,
                                       ctypes.byref(out)), "gdn_gla_factors_bytes")
    return out.value


def gdn_gla_workspace_bytes(B, N, H, dk, dv) -> int:
    out = ctypes.c_size_t(0)
    _check(lib().gdn_gla_workspace_bytes(B, N, H, dk, dv, ctypes.byref(out)), "gdn_gla_workspace_bytes")
    return out.value


def gdn_gla_tree_verify(q, k, v, alpha, beta, parent_idx, S0, out, factors, workspace, stream=None):
    """Gated linear attention (per-channel gates alpha [B,N,H,dk]) over draft trees; see include/gdnspec.h."""
    B, N, H, dk, dv = _dims(q, v)
    _check(lib().gdn_gla_tree_verify(_ptr(q), _ptr(k), _ptr(v), dtype_code(q.dtype), _ptr(alpha), _ptr(beta),
                                     _ptr(parent_idx), _ptr(S0), _ptr(out), _ptr(factors), _ptr(workspace),
                                     B, N, H, dk, dv, _stream(stream)), "gdn_gla_tree_verify")


def gdn_gla_commit(S0, factors, accepted_path, S_new, N, dtype, stream=None):
    """Accepted-path commit from a GLA factor record (see include/gdnspec.h)."""
    B, H, dv, dk = S0.shape
    _check(lib().gdn_gla_commit(_ptr(S0), _ptr(factors), _ptr(accepted_path), accepted_path.shape[1], _ptr(S_new),
                                B, N, H, dk, dv, dtype_code(dtype), _stream(stream)), "gdn_gla_commit")


def gla_factor_views(buf, B, N, H, dk, dv, dtype):
    """(delta [B,H,N,dv] f32, key [B,H,N,dk], g [B,H,N,dk] f32, parent [B,N] i32) views of a GLA factor buffer."""
    esz = 4 if dtype_code(dtype) == DTYPE_F32 else 2
    BHN = B * H * N
    o_key = _align(BHN * dv * 4)
    o_g = _align(o_key + BHN * dk * esz)
    o_par = _align(o_g + BHN * dk * 4)
    kt = torch.float32 if esz == 4 else torch.bfloat16
    delta = buf[: BHN * dv * 4].view(torch.float32).view(B, H, N, dv)
    key = buf[o_key: o_key + BHN * dk * esz].view(kt).view(B, H, N, dk)
    g = buf[o_g: o_g + BHN * dk * 4].view(torch.float32).view(B, H, N, dk)
    par = buf[o_par: o_par + B * N * 4].view(torch.int32).view(B, N)
    return delta, key, g, par


def gdn_seq_workspace_bytes(nseq, total, H, Hk, dk, dv, dtype) -> int:
    out = ctypes.c_size_t(0)
    _check(lib().gdn_seq_workspace_bytes(nseq, total, H, Hk, dk, dv, dtype_code(dtype), ctypes.byref(out)),
           "gdn_seq_workspace_bytes")
    return out.value


def gdn_seq_forward_workspace_bytes(nseq, total, H, Hk, dk, dv, dtype) -> int:
    out = ctypes.c_size_t(0)
    _check(lib().gdn_seq_forward_workspace_bytes(nseq, total, H, Hk, dk, dv, dtype_code(dtype), ctypes.byref(out)),
           "gdn_seq_forward_workspace_bytes")
    return out.value


def gdn_seq_record_bytes(nseq, total, H, Hk, dk, dv, dtype) -> int:
    out = ctypes.c_size_t(0)
    _check(lib().gdn_seq_record_bytes(nseq, total, H, Hk, dk, dv, dtype_code(dtype), ctypes.byref(out)),
           "gdn_seq_record_bytes")
    return out.value


def empty_seq_workspace(nseq, total, H, Hk, dk, dv, dtype, device="cuda", backward=True):
    """Workspace of the sequence calls; with backward=False what gdn_seq_forward takes, a tenth of it."""
    size = gdn_seq_workspace_bytes if backward else gdn_seq_forward_workspace_bytes
    return torch.empty(max(16, size(nseq, total, H, Hk, dk, dv, dtype)), dtype=torch.uint8, device=device)


def empty_seq_record(nseq, total, H, Hk, dk, dv, dtype, device="cuda"):
    """Caller-owned record that gdn_seq_forward writes for gdn_seq_backward."""
    return torch.empty(max(16, gdn_seq_record_bytes(nseq, total, H, Hk, dk, dv, dtype)), dtype=torch.uint8, device=device)


def _tokens(x, what):
    """(pointer, elements between tokens) of [total, heads, d] or [nseq, T, heads, d]; the tokens may be
    columns of a wider tensor, everything inside a token is dense."""
    if not x.is_cuda:
        raise ValueError("%s: expected a CUDA tensor" % what)
    heads, d = x.shape[-2:]
    ld = x.stride(-3) if x.shape[-3] > 1 else (x.stride(0) if x.dim() == 4 and x.shape[0] > 1 else heads * d)
    dense = (d == 1 or x.stride(-1) == 1) and (heads == 1 or x.stride(-2) == d)
    if x.dim() == 4 and x.shape[0] > 1 and x.shape[1] > 0:
        dense = dense and x.stride(0) == x.shape[1] * ld
    if not dense and x.numel() > 0:
        raise ValueError("%s: heads and channels of a token must be dense, tokens evenly spaced" % what)
    return x.data_ptr() or None, ld


def _seq_dims(q, k, v, log_alpha, beta, offsets):
    """(nseq, total, H, Hk, dk, dv) of a sequence call, its shapes checked against one another."""
    if q.dim() not in (3, 4) or v.dim() != q.dim() or k.shape != q.shape or v.shape[:-2] != q.shape[:-2]:
        raise ValueError("q, k [.., Hk, dk] and v [.., H, dv] must have the same leading dimensions")
    if k.dtype != q.dtype or v.dtype != q.dtype:
        raise ValueError("q, k and v must have one type")
    total = q.shape[0] if q.dim() == 3 else q.shape[0] * q.shape[1]
    for x in (log_alpha, beta):
        if x.dtype != torch.float32 or x.shape != v.shape[:-1]:
            raise ValueError("log_alpha and beta must be fp32 %s" % (tuple(v.shape[:-1]),))
    if offsets is None:
        nseq = q.shape[0] if q.dim() == 4 else 1
    else:
        if offsets.dtype != torch.int32 or offsets.dim() != 1 or offsets.numel() < 2:
            raise ValueError("offsets must be int32 [nseq + 1]")
        nseq = offsets.numel() - 1
    return nseq, total, v.shape[-2], q.shape[-2], q.shape[-1], v.shape[-1]


def _same(x, shape, dtype, what):
    if x is not None and (x.shape != shape or x.dtype is not dtype):
        raise ValueError("%s must be %s %s" % (what, dtype, tuple(shape)))


def _sized(x, nbytes, what):
    if x is not None and x.numel() * x.element_size() < nbytes:
        raise ValueError("%s: %d bytes wanted" % (what, nbytes))


def gdn_seq_forward(q, k, v, log_alpha, beta, S0, out, S_T, workspace, offsets=None, record=None, stream=None):
    """The gated delta rule over packed sequences (see include/gdnspec.h): q, k [total, Hk, dk], v [total, H, dv]
    with offsets int32 [nseq + 1], or [nseq, T, heads, d] without.  S0 and S_T [nseq, H, dv, dk] fp32 may be None."""
    nseq, total, H, Hk, dk, dv = dims = _seq_dims(q, k, v, log_alpha, beta, offsets)
    _same(out, v.shape, v.dtype, "out")
    _same(S0, (nseq, H, dv, dk), torch.float32, "S0")
    _same(S_T, (nseq, H, dv, dk), torch.float32, "S_T")
    _sized(workspace, gdn_seq_forward_workspace_bytes(*dims, q.dtype), "workspace")
    if record is not None:
        _sized(record, gdn_seq_record_bytes(*dims, q.dtype), "record")
    qp, ldq = _tokens(q, "q")
    kp, ldk = _tokens(k, "k")
    vp, ldv = _tokens(v, "v")
    _check(lib().gdn_seq_forward(qp, ldq, kp, ldk, vp, ldv, dtype_code(q.dtype), _ptr(log_alpha), _ptr(beta), _ptr(S0),
                                 _ptr(offsets), _ptr(out), _ptr(S_T), _ptr(record), _ptr(workspace), *dims,
                                 _stream(stream)), "gdn_seq_forward")


def gdn_seq_backward(q, k, v, log_alpha, beta, dout, dS_T, record, dq, dk, dv, dlog_alpha, dbeta, dS0, workspace,
                     offsets=None, stream=None):
    """Gradients of gdn_seq_forward at the record that it wrote (see include/gdnspec.h); dS_T and dS0 may be None."""
    dims = nseq, total, H, Hk, d_k, d_v = _seq_dims(q, k, v, log_alpha, beta, offsets)
    for x, like, what in ((dout, v, "dout"), (dq, q, "dq"), (dk, k, "dk"), (dv, v, "dv"), (dlog_alpha, log_alpha, "dlog_alpha"),
                          (dbeta, beta, "dbeta")):
        _same(x, like.shape, like.dtype, what)
    _same(dS_T, (nseq, H, d_v, d_k), torch.float32, "dS_T")
    _same(dS0, (nseq, H, d_v, d_k), torch.float32, "dS0")
    _sized(workspace, gdn_seq_workspace_bytes(*dims, q.dtype), "workspace")
    _sized(record, gdn_seq_record_bytes(*dims, q.dtype), "record")
    qp, ldq = _tokens(q, "q")
    kp, ldk = _tokens(k, "k")
    vp, ldv = _tokens(v, "v")
    _check(lib().gdn_seq_backward(qp, ldq, kp, ldk, vp, ldv, dtype_code(q.dtype), _ptr(log_alpha), _ptr(beta),
                                  _ptr(offsets), _ptr(dout), _ptr(dS_T), _ptr(record), _ptr(dq), _ptr(dk), _ptr(dv),
                                  _ptr(dlog_alpha), _ptr(dbeta), _ptr(dS0), _ptr(workspace), *dims, _stream(stream)),
           "gdn_seq_backward")


def _step_dims(q, k, v, log_alpha, beta, S, out, state_index):
    """(B, slots, H, Hk, dk, dv) of a single-token call, its shapes checked against one another."""
    qs, vs, ss, t, f32 = q.shape, v.shape, S.shape, q.dtype, torch.float32
    B, Hk, dk = qs
    _, H, dv = vs
    if k.shape != qs or vs[0] != B or k.dtype is not t or v.dtype is not t:
        raise ValueError("q, k [B, Hk, dk] and v [B, H, dv] must agree in B and type")
    gates = vs[:2]
    if log_alpha.shape != gates or beta.shape != gates or log_alpha.dtype is not f32 or beta.dtype is not f32:
        raise ValueError("log_alpha and beta must be fp32 %s" % (tuple(gates),))
    if len(ss) != 4 or ss[1:] != (H, dv, dk) or S.dtype is not f32:
        raise ValueError("S must be fp32 [slots, %d, %d, %d]" % (H, dv, dk))
    if out.shape != vs or out.dtype is not t:
        raise ValueError("out must be %s %s" % (t, tuple(vs)))
    if state_index is not None and (state_index.shape != (B,) or state_index.dtype is not torch.int32):
        raise ValueError("state_index must be int32 [%d]" % B)
    return B, ss[0], H, Hk, dk, dv


def gdn_seq_step(q, k, v, log_alpha, beta, S, out, state_index=None, stream=None):
    """One token for each of B sequences, the states S [slots, H, dv, dk] fp32 updated in place (see
    include/gdnspec.h); state_index int32 [B], -1 for an empty row."""
    B, slots, H, Hk, dk, dv = _step_dims(q, k, v, log_alpha, beta, S, out, state_index)
    rc = lib().gdn_seq_step(_ptr(q), _ptr(k), _ptr(v), dtype_code(q.dtype), _ptr(log_alpha), _ptr(beta), _ptr(S),
                            _ptr(state_index), _ptr(out), B, slots, H, Hk, dk, dv, _stream(stream))
    if rc != OK:
        raise GdnError(rc, "gdn_seq_step")


def _here(*tensors):
    """Every tensor on the current device, whose stream the call goes to: a kernel cannot read another's memory."""
    dev = tensors[0].get_device()
    for x in tensors:
        if x is not None and (x.get_device() != dev or dev < 0):
            raise ValueError("expected CUDA tensors on one device")
    if dev != _current_device():
        raise ValueError("expected tensors on the current device")


def _dense(x):
    """Pointer of a contiguous tensor that _here has seen, or None."""
    if x is None:
        return None
    if not x.is_contiguous():
        raise ValueError("expected a contiguous CUDA tensor")
    return x.data_ptr() or None


def _rows(x, what, width):
    """_tokens of a tensor that _here has seen, at once where it is dense: rows of `width` elements."""
    if x.is_contiguous():
        return x.data_ptr() or None, width
    return _tokens(x, what)


@functools.lru_cache(maxsize=256)
def _linear_seq_bytes(name, nseq, total, H, Hk, dk, dv, dtype):
    out = ctypes.c_size_t(0)
    _check(getattr(lib(), name)(nseq, total, H, Hk, dk, dv, dtype_code(dtype), ctypes.byref(out)), name)
    return out.value


def gdn_linear_seq_workspace_bytes(nseq, total, H, Hk, dk, dv, dtype) -> int:
    return _linear_seq_bytes("gdn_linear_seq_workspace_bytes", nseq, total, H, Hk, dk, dv, dtype)


def gdn_linear_seq_forward_workspace_bytes(nseq, total, H, Hk, dk, dv, dtype) -> int:
    return _linear_seq_bytes("gdn_linear_seq_forward_workspace_bytes", nseq, total, H, Hk, dk, dv, dtype)


def gdn_linear_seq_record_bytes(nseq, total, H, Hk, dk, dv, dtype) -> int:
    return _linear_seq_bytes("gdn_linear_seq_record_bytes", nseq, total, H, Hk, dk, dv, dtype)


def empty_linear_seq_workspace(nseq, total, H, Hk, dk, dv, dtype, device="cuda", backward=True):
    """Workspace of the linear-attention sequence calls; with backward=False what gdn_linear_seq_forward takes."""
    size = gdn_linear_seq_workspace_bytes if backward else gdn_linear_seq_forward_workspace_bytes
    return torch.empty(size(nseq, total, H, Hk, dk, dv, dtype), dtype=torch.uint8, device=device)


def empty_linear_seq_record(nseq, total, H, Hk, dk, dv, dtype, device="cuda"):
    """Caller-owned record that gdn_linear_seq_forward writes for gdn_linear_seq_backward."""
    return torch.empty(gdn_linear_seq_record_bytes(nseq, total, H, Hk, dk, dv, dtype), dtype=torch.uint8, device=device)


def gdn_linear_seq_forward(q, k, v, log_alpha, beta, S0, out, S_T, workspace, offsets=None, record=None, stream=None):
    """Decay-gated linear attention over packed sequences (see include/gdnspec.h): arguments as gdn_seq_forward."""
    nseq, total, H, Hk, dk, dv = dims = _seq_dims(q, k, v, log_alpha, beta, offsets)
    _same(out, v.shape, v.dtype, "out")
    _same(S0, (nseq, H, dv, dk), torch.float32, "S0")
    _same(S_T, (nseq, H, dv, dk), torch.float32, "S_T")
    _sized(workspace, gdn_linear_seq_forward_workspace_bytes(*dims, q.dtype), "workspace")
    if record is not None:
        _sized(record, gdn_linear_seq_record_bytes(*dims, q.dtype), "record")
    _here(q, k, v, log_alpha, beta, S0, out, S_T, workspace, offsets, record)
    qp, ldq = _rows(q, "q", Hk * dk)
    kp, ldk = _rows(k, "k", Hk * dk)
    vp, ldv = _rows(v, "v", H * dv)
    _check(lib().gdn_linear_seq_forward(qp, ldq, kp, ldk, vp, ldv, dtype_code(q.dtype), _dense(log_alpha), _dense(beta), _dense(S0),
                                        _dense(offsets), _dense(out), _dense(S_T), _dense(record), _dense(workspace), *dims,
                                        _stream(stream)), "gdn_linear_seq_forward")


def gdn_linear_seq_backward(q, k, v, log_alpha, beta, dout, dS_T, record, dq, dk, dv, dlog_alpha, dbeta, dS0, workspace,
                            offsets=None, stream=None):
    """Gradients of gdn_linear_seq_forward at the record that it wrote (see include/gdnspec.h); dS_T and dS0 may be None."""
    dims = nseq, total, H, Hk, d_k, d_v = _seq_dims(q, k, v, log_alpha, beta, offsets)
    for x, like, what in ((dout, v, "dout"), (dq, q, "dq"), (dk, k, "dk"), (dv, v, "dv"), (dlog_alpha, log_alpha, "dlog_alpha"),
                          (dbeta, beta, "dbeta")):
        _same(x, like.shape, like.dtype, what)
    _same(dS_T, (nseq, H, d_v, d_k), torch.float32, "dS_T")
    _same(dS0, (nseq, H, d_v, d_k), torch.float32, "dS0")
    _sized(workspace, gdn_linear_seq_workspace_bytes(*dims, q.dtype), "workspace")
    _sized(record, gdn_linear_seq_record_bytes(*dims, q.dtype), "record")
    _here(q, k, v, log_alpha, beta, dout, dS_T, record, dq, dk, dv, dlog_alpha, dbeta, dS0, workspace, offsets)
    qp, ldq = _rows(q, "q", Hk * d_k)
    kp, ldk = _rows(k, "k", Hk * d_k)
    vp, ldv = _rows(v, "v", H * d_v)
    _check(lib().gdn_linear_seq_backward(qp, ldq, kp, ldk, vp, ldv, dtype_code(q.dtype), _dense(log_alpha), _dense(beta),
                                         _dense(offsets), _dense(dout), _dense(dS_T), _dense(record), _dense(dq), _dense(dk), _dense(dv),
                                         _dense(dlog_alpha), _dense(dbeta), _dense(dS0), _dense(workspace), *dims, _stream(stream)),
           "gdn_linear_seq_backward")


def gdn_linear_seq_step(q, k, v, log_alpha, beta, S, out, state_index=None, stream=None):
    """One token of decay-gated linear attention for each of B sequences: arguments as gdn_seq_step."""
    B, slots, H, Hk, dk, dv = _step_dims(q, k, v, log_alpha, beta, S, out, state_index)
    _here(q, k, v, log_alpha, beta, S, out, state_index)
    rc = lib().gdn_linear_seq_step(_dense(q), _dense(k), _dense(v), dtype_code(q.dtype), _dense(log_alpha), _dense(beta), _dense(S),
                                   _dense(state_index), _dense(out), B, slots, H, Hk, dk, dv, _stream(stream))
    if rc != OK:
        raise GdnError(rc, "gdn_linear_seq_step")


def gdn_rotary_frequencies(rot, base=10000.0, factor=1.0, original=0.0, low=1.0, high=32.0, device="cuda"):
    """fp32 [rot / 2] frequencies of gdn_rotary, scaled for contexts `factor` times as long (see include/gdnspec.h)."""
    f = torch.empty(max(0, rot // 2), dtype=torch.float32)
    _check(lib().gdn_rotary_frequencies(rot, base, factor, original, low, high, f.data_ptr() or None), "gdn_rotary_frequencies")
    return f.to(device)


def gdn_rotary(q, k, positions, inv_freq, q_out, k_out, scale=1.0, interleaved=False, inverse=False, stream=None):
    """Rotary positions of q [.., H, d] and k [.., Hk, d] (k and k_out may be None), with positions int32 [..] and
    inv_freq fp32 [rot / 2] (see include/gdnspec.h); q_out and k_out may be q and k."""
    qs, t = q.shape, q.dtype                  # a tensor's shape once: each look at it is some 0.2 us of a call of 10
    lead, n = qs[:-2], len(qs)
    if n not in (3, 4) or positions.shape != lead or positions.dtype is not torch.int32:
        raise ValueError("q must be [.., H, d] and positions int32 of its leading dimensions")
    if (k is None) != (k_out is None):
        raise ValueError("k and k_out go together")
    freqs = inv_freq.shape
    if len(freqs) != 1 or inv_freq.dtype is not torch.float32:
        raise ValueError("inv_freq must be fp32 [rot / 2]")
    _same(q_out, qs, t, "q_out")
    H, d = qs[-2:]
    _here(q, k, positions, inv_freq, q_out, k_out)
    qp, ldq = _rows(q, "q", H * d)
    qo, ldqo = _rows(q_out, "q_out", H * d)
    kp = ko = None
    ldk = ldko = Hk = 0
    if k is not None:
        ks = k.shape
        if len(ks) != n or ks[:-2] != lead or ks[-1] != d or k.dtype is not t:
            raise ValueError("k must be as q but for its heads")
        _same(k_out, ks, t, "k_out")
        Hk = ks[-2]
        kp, ldk = _rows(k, "k", Hk * d)
        ko, ldko = _rows(k_out, "k_out", Hk * d)
    rc = lib().gdn_rotary(qp, ldq, kp, ldk, dtype_code(t), _dense(positions), _dense(inv_freq), scale, qo, ldqo, ko, ldko,
                          positions.numel(), H, Hk, d, 2 * freqs[0], int(interleaved), int(inverse), _stream(stream))
    if rc != OK:
        raise GdnError(rc, "gdn_rotary")


def empty_norm_workspace(rows, width, device="cuda"):
    out = ctypes.c_size_t(0)
    _check(lib().gdn_norm_workspace_bytes(rows, width, ctypes.byref(out)), "gdn_norm_workspace_bytes")
    return torch.empty(out.value, dtype=torch.uint8, device=device)


def _norm_workspace(workspace, rows, width):
    out = ctypes.c_size_t(0)
    _check(lib().gdn_norm_workspace_bytes(rows, width, ctypes.byref(out)), "gdn_norm_workspace_bytes")
    _sized(workspace, out.value, "workspace")


def gdn_gated_norm(o, gate, weight, out, eps=1e-6, stream=None):
    """out = weight * RMSNorm(o) * silu(gate) over the last dimension (see include/gdnspec.h)."""
    d = o.shape[-1]
    _same(gate, o.shape, gate.dtype, "gate")
    _same(weight, (d,), gate.dtype, "weight")
    _same(out, o.shape, gate.dtype, "out")
    _check(lib().gdn_gated_norm(_ptr(o), dtype_code(o.dtype), _ptr(gate), _ptr(weight), _ptr(out), dtype_code(gate.dtype),
                                o.numel() // d, d, eps, _stream(stream)), "gdn_gated_norm")


def gdn_gated_norm_backward(o, gate, weight, dout, d_o, dgate, dweight, workspace, eps=1e-6, stream=None):
    """Gradients of gdn_gated_norm: d_o as o, dgate as gate, dweight fp32 [d] (see include/gdnspec.h)."""
    d = o.shape[-1]
    for x, what in ((gate, "gate"), (dout, "dout"), (dgate, "dgate")):
        _same(x, o.shape, gate.dtype, what)
    _same(weight, (d,), gate.dtype, "weight")
    _same(d_o, o.shape, o.dtype, "d_o")
    _same(dweight, (d,), torch.float32, "dweight")
    _norm_workspace(workspace, o.numel() // d, d)
    _check(lib().gdn_gated_norm_backward(_ptr(o), dtype_code(o.dtype), _ptr(gate), _ptr(weight), _ptr(dout), _ptr(d_o),
                                         _ptr(dgate), _ptr(dweight), _ptr(workspace), dtype_code(gate.dtype),
                                         o.numel() // d, d, eps, _stream(stream)), "gdn_gated_norm_backward")


def gdn_block_norm(x, z, post_weight, gate, weight, x_out, h, eps=1e-6, res_scale=1.0, stream=None):
    """x_out = res_scale x + gate * post_weight * RMSNorm(z); h = weight * RMSNorm(x_out) (see include/gdnspec.h).
    z, post_weight, gate and x_out None: h = weight * RMSNorm(x)."""
    D = x.shape[-1]
    for t, what in ((z, "z"), (x_out, "x_out"), (h, "h")):
        _same(t, x.shape, x.dtype, what)
    for t, what in ((post_weight, "post_weight"), (gate, "gate"), (weight, "weight")):
        _same(t, (D,), x.dtype, what)
    _check(lib().gdn_block_norm(_ptr(x), _ptr(z), _ptr(post_weight), _ptr(gate), _ptr(weight), _ptr(x_out), _ptr(h),
                                dtype_code(x.dtype), x.numel() // D, D, eps, res_scale, _stream(stream)), "gdn_block_norm")


def gdn_block_norm_backward(x_out, z, post_weight, gate, weight, dh, dx_out, dx, dz, dpost_weight, dgate, dweight,
                            workspace, eps=1e-6, res_scale=1.0, stream=None):
    """Gradients of gdn_block_norm at the x_out that it wrote (see include/gdnspec.h); dx_out may be None."""
    D = x_out.shape[-1]
    for t, what in ((z, "z"), (dh, "dh"), (dx_out, "dx_out"), (dx, "dx"), (dz, "dz")):
        _same(t, x_out.shape, x_out.dtype, what)
    for t, what in ((post_weight, "post_weight"), (gate, "gate"), (weight, "weight")):
        _same(t, (D,), x_out.dtype, what)
    for t, what in ((dpost_weight, "dpost_weight"), (dgate, "dgate"), (dweight, "dweight")):
        _same(t, (D,), torch.float32, what)
    _norm_workspace(workspace, x_out.numel() // D, D)
    _check(lib().gdn_block_norm_backward(_ptr(x_out), _ptr(z), _ptr(post_weight), _ptr(gate), _ptr(weight), _ptr(dh),
                                         _ptr(dx_out), _ptr(dx), _ptr(dz), _ptr(dpost_weight), _ptr(dgate), _ptr(dweight),
                                         _ptr(workspace), dtype_code(x_out.dtype), x_out.numel() // D, D, eps, res_scale,
                                         _stream(stream)), "gdn_block_norm_backward")


def gdn_set_launch_overlap(enable: bool) -> bool:
    """Process-wide switch; returns the previous setting (see include/gdnspec.h)."""
    return bool(lib().gdn_set_launch_overlap(1 if enable else 0))


def gdn_set_wait_limit_ns(ns: int):
    """Limit of every bounded device wait on the current device (see include/gdnspec.h)."""
    _check(lib().gdn_set_wait_limit_ns(int(ns)), "gdn_set_wait_limit_ns")


def gdn_selftest_stuck_wait(stream=None):
    """Launch a wait that nothing completes; gdn_last_error then reports GDN_ERR_TIMEOUT."""
    _check(lib().gdn_selftest_stuck_wait(_stream(stream)), "gdn_selftest_stuck_wait")


def gdn_last_error(stream=None) -> int:
    return lib().gdn_last_error(_stream(stream))


# ---------------------------------------------------------------------------
# factor-buffer views (host-side reinterpretation of the documented layout)
# ---------------------------------------------------------------------------
def _align(x, a=256):
    return (x + a - 1) // a * a


def factor_views(buf, B, N, H, dk, dv, dtype):
    """(delta [B,H,N,dv] f32, key [B,H,N,dk], g [B,H,N] f32, parent [B,N] i32) views of a factor buffer."""
    esz = 4 if dtype_code(dtype) == DTYPE_F32 else 2
    BHN = B * H * N
    o_key = _align(BHN * dv * 4)
    o_g = _align(o_key + BHN * dk * esz)
    o_par = _align(o_g + BHN * 4)
    kt = torch.float32 if esz == 4 else torch.bfloat16
    delta = buf[: BHN * dv * 4].view(torch.float32).view(B, H, N, dv)
    key = buf[o_key: o_key + BHN * dk * esz].view(kt).view(B, H, N, dk)
    g = buf[o_g: o_g + BHN * 4].view(torch.float32).view(B, H, N)
    par = buf[o_par: o_par + B * N * 4].view(torch.int32).view(B, N)
    return delta, key, g, par


def layer_record_views(buf, B, N, H, hidden, dk, dv):
    """(Y [B*N, rows] fp32 projections, factor-buffer slice) views of a layer record."""
    rows = 2 * H * dk + 2 * H * dv + 2 * H
    ldy = (rows + 3) // 4 * 4
    y_bytes = B * N * ldy * 4
    Y = buf[:y_bytes].view(torch.float32).view(B * N, ldy)[:, :rows]
    fac = buf[_align(y_bytes):]
    return Y, fac


def layer_workspace_views(buf, B, N, H, hidden, dk, dv):
    """q, k [B,N,H,dk], v, o [B,N,H,dv], alpha, beta [B,N,H] fp32; the bf16 hi/lo terms of q and k
    (qhi, qlo, khi, klo [B,N,H,dk]); y_hi, y_lo [B*N, H*dv] bf16.  When the single-kernel verifier runs
    (d_k = d_v = 256) the fp32 q and k rows are not written: q is carried by its hi/lo terms and the
    keys go straight to the factor record."""
    BN = B * N
    sizes = [("q", BN * H * dk * 4), ("k", BN * H * dk * 4), ("v", BN * H * dv * 4), ("alpha", BN * H * 4),
             ("beta", BN * H * 4), ("o", BN * H * dv * 4), ("qhi", BN * H * dk * 2), ("khi", BN * H * dk * 2),
             ("qlo", BN * H * dk * 2), ("klo", BN * H * dk * 2), ("yhi", BN * H * dv * 2),
             ("ylo", BN * H * dv * 2)]
    out, off = {}, 0
    for name, n in sizes:
        out[name] = buf[off:off + n]
        off = _align(off + n)
    f32 = lambda x, *shape: x.view(torch.float32).view(*shape)
    bf = lambda x: x.view(torch.bfloat16).view(B, N, H, dk)
    return dict(q=f32(out["q"], B, N, H, dk), k=f32(out["k"], B, N, H, dk), v=f32(out["v"], B, N, H, dv),
                qhi=bf(out["qhi"]), qlo=bf(out["qlo"]), khi=bf(out["khi"]), klo=bf(out["klo"]),
                alpha=f32(out["alpha"], B, N, H), beta=f32(out["beta"], B, N, H), o=f32(out["o"], B, N, H, dv),
                yhi=out["yhi"].view(torch.bfloat16).view(BN, H * dv),
                ylo=out["ylo"].view(torch.bfloat16).view(BN, H * dv))
