"""Python binding of libdspark.so — the DSpark draft-head round on one GB300.

Argument marshalling only: every step of the path runs in the library's CUDA
kernels.  PyTorch provides device memory and streams.  There is no fallback: if
the library is missing or a call fails, the call raises.

The functions carry the C-ABI names (see include/dspark.h) and take torch
tensors; `draft`, `schedule`, `verify` and `run_round` compose them.
"""
from __future__ import annotations

import ctypes
import math
import os
from dataclasses import dataclass
from typing import Dict, Optional

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libdspark.so")

DSPARK_OK = 0
SCHED_UNCONSTRAINED = 0
SCHED_BREAK = 1
SCHED_FIXED_K = 2
SCHED_ASYNC = 3

EXPORTS = [
    "dspark_lm_head", "dspark_pack_w2", "dspark_markov_workspace_bytes", "dspark_markov_draft",
    "dspark_draft", "dspark_schedule", "dspark_verify_workspace_bytes", "dspark_verify",
    "dspark_device_status", "dspark_error_string", "dspark_launch_count",
    "dspark_markov_draft_static", "dspark_schedule_async", "dspark_conf_logits",
    "dspark_sts_workspace_bytes", "dspark_sts_fit", "dspark_rnn_workspace_bytes",
    "dspark_rnn_draft", "dspark_selftest_wait_timeout", "dspark_fused_workspace_bytes",
    "dspark_pack_fused", "dspark_fused_draft", "dspark_verify_residual_rows",
    "dspark_kv_plan", "dspark_kv_append", "dspark_tree_attention_workspace_bytes",
    "dspark_tree_attention", "dspark_tree_accept", "dspark_kv_compact", "dspark_rope_append",
    "dspark_chunk_attention_workspace_bytes", "dspark_chunk_attention", "dspark_kv_fork",
    "dspark_kv_release", "dspark_kv_squeeze", "dspark_kv_copy",
]
STATIC_SCRATCH_BYTES = 16 << 20
KV_BF16 = 0
KV_E4M3 = 1
MAX_NODES = 64
ROPE_HALVES = 0
ROPE_PAIRS = 1


class DSparkError(RuntimeError):
    pass


class Dims(ctypes.Structure):
    _fields_ = [("R", ctypes.c_int32), ("gamma", ctypes.c_int32), ("V", ctypes.c_int32),
                ("r", ctypes.c_int32), ("d", ctypes.c_int32)]


class KVCacheStruct(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("k_scale", ctypes.c_void_p),
                ("v_scale", ctypes.c_void_p), ("page_stride", ctypes.c_int64),
                ("token_stride", ctypes.c_int64), ("head_stride", ctypes.c_int64),
                ("n_pages", ctypes.c_int32), ("page_size", ctypes.c_int32),
                ("heads", ctypes.c_int32), ("dim", ctypes.c_int32), ("type", ctypes.c_int32)]


class RopeStruct(ctypes.Structure):
    _fields_ = [("turns", ctypes.c_void_p), ("dims", ctypes.c_int32), ("style", ctypes.c_int32)]


_lib = None


def load_library(path: str = LIB_PATH) -> ctypes.CDLL:
    """Load (once) the CUDA library; raises if it has not been built."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise DSparkError(f"{path} not found: build it with "
                          "`python speculative_decoding_draft_02_gb300/build.py`")
    lib = ctypes.CDLL(path)
    P, I32, U64, SZ, F32 = (ctypes.c_void_p, ctypes.c_int32, ctypes.c_uint64, ctypes.c_size_t,
                            ctypes.c_float)
    DP = ctypes.POINTER(Dims)
    CP, I64 = ctypes.POINTER(KVCacheStruct), ctypes.c_int64
    RP = ctypes.POINTER(RopeStruct)
    sig = {
        "dspark_lm_head": (ctypes.c_int, [DP, P, P, P, P]),
        "dspark_pack_w2": (ctypes.c_int, [DP, P, P, P]),
        "dspark_markov_workspace_bytes": (SZ, [DP]),
        "dspark_markov_draft": (ctypes.c_int, [DP, P, P, P, P, P, P, P, F32, U64, P, P, P, P, P,
                                               SZ, P]),
        "dspark_draft": (ctypes.c_int, [DP, P, P, P, P, P, P, P, F32, U64, P, P, P, P, P, P, SZ,
                                        P]),
        "dspark_schedule": (ctypes.c_int, [P, I32, I32, P, I32, I32, I32, P, P, P, P, P, P]),
        "dspark_schedule_async": (ctypes.c_int, [P, I32, I32, P, I32, P, P, P, P, P, P, P]),
        "dspark_conf_logits": (ctypes.c_int, [DP, P, P, P, P, P, P, P]),
        "dspark_sts_workspace_bytes": (SZ, [I32, I32, I32, I32]),
        "dspark_sts_fit": (ctypes.c_int, [P, P, I32, I32, P, I32, I32, P, P, P, SZ, P]),
        "dspark_rnn_workspace_bytes": (SZ, [DP]),
        "dspark_fused_workspace_bytes": (SZ, [DP]),
        "dspark_pack_fused": (ctypes.c_int, [DP, P, P, P, P]),
        "dspark_fused_draft": (ctypes.c_int, [DP, P, P, P, P, P, P, F32, U64, P, P, P, P, P, SZ,
                                              P]),
        "dspark_selftest_wait_timeout": (ctypes.c_int, [U64, P]),
        "dspark_rnn_draft": (ctypes.c_int, [DP, P, P, P, P, P, P, P, P, P, F32, U64, P, P, P, P,
                                            P, SZ, P]),
        "dspark_verify_workspace_bytes": (SZ, [DP]),
        "dspark_verify": (ctypes.c_int, [DP, P, P, P, P, P, P, P, P, P, F32, U64, P, P, P, SZ,
                                         P]),
        "dspark_markov_draft_static": (ctypes.c_int, [DP, P, P, P, P, P, P, P, F32, U64, P, P, P,
                                                      P, P]),
        "dspark_verify_residual_rows": (ctypes.c_int, [DP, P, SZ, P, P, P]),
        "dspark_kv_plan": (ctypes.c_int, [I32] * 7 + [P] * 13 + [P]),
        "dspark_kv_append": (ctypes.c_int, [CP, I32, P, P, I64, I64, P, P]),
        "dspark_tree_attention_workspace_bytes": (SZ, [CP, I32, I32, I32]),
        "dspark_tree_attention": (ctypes.c_int, [CP, I32, I32, I32, I32, I32, P, I64, I64, P, P, P,
                                                 P, F32, P, I64, I64, P, P, SZ, P]),
        "dspark_tree_accept": (ctypes.c_int, [I32, I32, I32, P, P, P, P, P, P, P, P, P, P]),
        "dspark_kv_compact": (ctypes.c_int, [CP, I32, I32, I32, P, P, P, P, P]),
        "dspark_rope_append": (ctypes.c_int, [CP, I32, I32, P, I64, I64, P, P, I64, I64, P, P, F32,
                                              RP, P, P, P, I64, I64, P]),
        "dspark_chunk_attention_workspace_bytes": (SZ, [CP, I32, I32, I32]),
        "dspark_chunk_attention": (ctypes.c_int, [CP, I32, I32, I32, I32, I32, P, I64, I64, P, P, P,
                                                  F32, P, I64, I64, P, P, SZ, P]),
        "dspark_kv_fork": (ctypes.c_int, [I32, P, P, I32, I32, I32, I32] + [P] * 9 + [P]),
        "dspark_kv_release": (ctypes.c_int, [I32, I32, I32] + [P] * 6 + [P]),
        "dspark_kv_squeeze": (ctypes.c_int, [I32, I32, I32] + [P] * 12 + [P]),
        "dspark_kv_copy": (ctypes.c_int, [CP, I32, P, P, P, P]),
        "dspark_device_status": (ctypes.c_int, [P, ctypes.c_int]),
        "dspark_error_string": (ctypes.c_char_p, [ctypes.c_int]),
        "dspark_launch_count": (U64, []),
    }
    for name, (res, args) in sig.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    _lib = lib
    return lib


def _check(rc: int, what: str):
    if rc != DSPARK_OK:
        msg = load_library().dspark_error_string(rc).decode()
        raise DSparkError(f"{what} failed: {msg} ({rc})")


def _ptr(t: Optional[torch.Tensor], device=None):
    if t is None:
        return None
    if not t.is_cuda or (device is not None and t.get_device() != device):
        raise DSparkError("tensor must live on the GPU" if device is None else
                          f"tensor must live on device {device}, with the call's others")
    if not t.is_contiguous():
        raise DSparkError("tensor must be contiguous")
    return ctypes.c_void_p(t.data_ptr())


# The current stream's handle without making a Stream object (3 us of a 3 us launch).
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
_device = getattr(torch._C, "_cuda_getDevice", None)
_initialized = torch.cuda.is_initialized


def _stream(stream: Optional[torch.cuda.Stream]):
    if stream is not None:
        return stream.cuda_stream
    if _raw_stream is not None and _initialized():
        return _raw_stream(_device())
    return torch.cuda.current_stream().cuda_stream


def _stream_on(what: str, t: torch.Tensor, stream):
    """_stream, once the current device is the tensor's: a launch goes there."""
    if t.get_device() != _device():
        raise DSparkError(f"{what}: the tensors are on device {t.get_device()}, which is not the "
                          "current one")
    return _stream(stream)


def _bf16(t: torch.Tensor) -> torch.Tensor:
    return t if t.dtype == torch.bfloat16 else t.to(torch.bfloat16)


def dims_of(R: int, gamma: int, V: int, r: int, d: int) -> Dims:
    return Dims(R, gamma, V, r, d)


def _u64(seed: int) -> int:
    return int(seed) & 0xFFFFFFFFFFFFFFFF


# --------------------------------------------------------------- raw ABI ----

def dspark_lm_head(dims: Dims, h, W_lm, base_logits, stream=None):
    _check(load_library().dspark_lm_head(ctypes.byref(dims), _ptr(h), _ptr(W_lm),
                                         _ptr(base_logits), _stream(stream)), "dspark_lm_head")


def dspark_pack_w2(dims: Dims, W2, W2t, stream=None):
    _check(load_library().dspark_pack_w2(ctypes.byref(dims), _ptr(W2), _ptr(W2t), _stream(stream)),
           "dspark_pack_w2")


def dspark_markov_workspace_bytes(dims: Dims) -> int:
    return int(load_library().dspark_markov_workspace_bytes(ctypes.byref(dims)))


def dspark_verify_workspace_bytes(dims: Dims) -> int:
    return int(load_library().dspark_verify_workspace_bytes(ctypes.byref(dims)))


def dspark_markov_draft(dims, base_logits, h, anchor, W1, W2t, w_conf, T, tau, seed, tokens,
                        conf, logp_d, lse_d, workspace, stream=None):
    _check(load_library().dspark_markov_draft(
        ctypes.byref(dims), _ptr(base_logits), _ptr(h), _ptr(anchor), _ptr(W1), _ptr(W2t),
        _ptr(w_conf), _ptr(T), float(tau), _u64(seed), _ptr(tokens), _ptr(conf), _ptr(logp_d),
        _ptr(lse_d), _ptr(workspace), workspace.numel(), _stream(stream)), "dspark_markov_draft")


def dspark_markov_draft_static(dims, base_logits, h, anchor, W1, W2t, w_conf, T, tau, seed,
                               tokens, conf, logp_d, lse_d, stream=None):
    """dspark_markov_draft with the scratch kept inside the library (no workspace)."""
    _check(load_library().dspark_markov_draft_static(
        ctypes.byref(dims), _ptr(base_logits), _ptr(h), _ptr(anchor), _ptr(W1), _ptr(W2t),
        _ptr(w_conf), _ptr(T), float(tau), _u64(seed), _ptr(tokens), _ptr(conf), _ptr(logp_d),
        _ptr(lse_d), _stream(stream)), "dspark_markov_draft_static")


def dspark_draft(dims, h, anchor, W_lm, W1, W2t, w_conf, T, tau, seed, base_logits, tokens, conf,
                 logp_d, lse_d, workspace, stream=None):
    _check(load_library().dspark_draft(
        ctypes.byref(dims), _ptr(h), _ptr(anchor), _ptr(W_lm), _ptr(W1), _ptr(W2t), _ptr(w_conf),
        _ptr(T), float(tau), _u64(seed), _ptr(base_logits), _ptr(tokens), _ptr(conf),
        _ptr(logp_d), _ptr(lse_d), _ptr(workspace), workspace.numel(), _stream(stream)),
        "dspark_draft")


def dspark_schedule(conf, R, gamma, sps, mode, k_fixed, length, K_out, theta_out, a_out=None,
                    order_out=None, stream=None):
    _check(load_library().dspark_schedule(
        _ptr(conf), int(R), int(gamma), _ptr(sps), int(sps.numel()), int(mode), int(k_fixed),
        _ptr(length), _ptr(K_out), _ptr(theta_out), _ptr(a_out), _ptr(order_out),
        _stream(stream)), "dspark_schedule")


def dspark_schedule_async(conf, R, gamma, sps, k_ring, length, K_out, theta_out, a_out=None,
                          order_out=None, stream=None):
    _check(load_library().dspark_schedule_async(
        _ptr(conf), int(R), int(gamma), _ptr(sps), int(sps.numel()), _ptr(k_ring), _ptr(length),
        _ptr(K_out), _ptr(theta_out), _ptr(a_out), _ptr(order_out), _stream(stream)),
        "dspark_schedule_async")


def dspark_conf_logits(dims, h, anchor, tokens, W1, w_conf, z, stream=None):
    _check(load_library().dspark_conf_logits(
        ctypes.byref(dims), _ptr(h), _ptr(anchor), _ptr(tokens), _ptr(W1), _ptr(w_conf), _ptr(z),
        _stream(stream)), "dspark_conf_logits")


def dspark_rnn_workspace_bytes(dims) -> int:
    return int(load_library().dspark_rnn_workspace_bytes(ctypes.byref(dims)))


def dspark_rnn_draft(dims, base_logits, h, anchor, W1, W2t, W_rec, W_hid, w_conf, T, tau, seed,
                     tokens, conf, logp_d, lse_d, workspace, stream=None):
    _check(load_library().dspark_rnn_draft(
        ctypes.byref(dims), _ptr(base_logits), _ptr(h), _ptr(anchor), _ptr(W1), _ptr(W2t),
        _ptr(W_rec), _ptr(W_hid), _ptr(w_conf), _ptr(T), float(tau), _u64(seed), _ptr(tokens),
        _ptr(conf), _ptr(logp_d), _ptr(lse_d), _ptr(workspace), workspace.numel(),
        _stream(stream)), "dspark_rnn_draft")


def dspark_fused_workspace_bytes(dims) -> int:
    return int(load_library().dspark_fused_workspace_bytes(ctypes.byref(dims)))


def dspark_pack_fused(dims, W_lm, W2t, W_cat, stream=None):
    _check(load_library().dspark_pack_fused(ctypes.byref(dims), _ptr(W_lm), _ptr(W2t),
                                            _ptr(W_cat), _stream(stream)), "dspark_pack_fused")


def dspark_fused_draft(dims, h, anchor, W_cat, W1, w_conf, T, tau, seed, tokens, conf, logp_d,
                       lse_d, workspace, stream=None):
    _check(load_library().dspark_fused_draft(
        ctypes.byref(dims), _ptr(h), _ptr(anchor), _ptr(W_cat), _ptr(W1), _ptr(w_conf), _ptr(T),
        float(tau), _u64(seed), _ptr(tokens), _ptr(conf), _ptr(logp_d), _ptr(lse_d),
        _ptr(workspace), workspace.numel(), _stream(stream)), "dspark_fused_draft")


def dspark_sts_workspace_bytes(N: int, gamma: int, n_grid: int, n_bins: int) -> int:
    return int(load_library().dspark_sts_workspace_bytes(int(N), int(gamma), int(n_grid),
                                                         int(n_bins)))


def dspark_sts_fit(z, accepted, T_grid, n_bins, T_out, ece_out, workspace=None, stream=None):
    """Fit the per-position temperatures (see include/dspark.h); allocates the
    workspace when none is given."""
    N, G = z.shape
    need = load_library().dspark_sts_workspace_bytes(N, G, T_grid.numel(), int(n_bins))
    if need == 0:
        raise DSparkError("dspark_sts_fit: invalid sizes")
    if workspace is None:
        workspace = torch.empty(need, dtype=torch.uint8, device=z.device)
    _check(load_library().dspark_sts_fit(
        _ptr(z), _ptr(accepted), int(N), int(G), _ptr(T_grid), int(T_grid.numel()), int(n_bins),
        _ptr(T_out), _ptr(ece_out), _ptr(workspace), workspace.numel(), _stream(stream)),
        "dspark_sts_fit")


def async_ring(k_round0: int, k_round1: int, device="cuda") -> torch.Tensor:
    """The device state of dspark_schedule_async: {K for round 0, K for round 1, cursor 0}."""
    return torch.tensor([int(k_round0), int(k_round1), 0], dtype=torch.int32, device=device)


def dspark_verify(dims, anchor, tokens, length, base_logits, W1, W2t, lse_d, logp_d, target, tau,
                  seed, accepted, bonus, workspace, stream=None):
    _check(load_library().dspark_verify(
        ctypes.byref(dims), _ptr(anchor), _ptr(tokens), _ptr(length), _ptr(base_logits),
        _ptr(W1), _ptr(W2t), _ptr(lse_d), _ptr(logp_d), _ptr(target), float(tau), _u64(seed),
        _ptr(accepted), _ptr(bonus), _ptr(workspace), workspace.numel(), _stream(stream)),
        "dspark_verify")


def dspark_verify_residual_rows(dims, workspace, stream=None):
    """(rejected, explicit_rows) of the last sampling dspark_verify on `workspace`."""
    rej, expl = ctypes.c_int32(0), ctypes.c_int32(0)
    _check(load_library().dspark_verify_residual_rows(
        ctypes.byref(dims), _ptr(workspace), workspace.numel(), ctypes.byref(rej),
        ctypes.byref(expl), _stream(stream)), "dspark_verify_residual_rows")
    return int(rej.value), int(expl.value)


# ------------------------------------------- the target's paged KV cache ----

# A call's arguments are checked in the 5 to 8 us that the GPU takes for a small one:
# one expression per tensor, and the message only when it is wanted.

# A call's first tensor says on which device the others have to be (`device` below); that
# it is the current one, _stream_on sees to.

def _want(what: str, name: str, t, dtype, shape, device=None) -> int:
    """The tensor's address, once its type, shape and place are what the call reads."""
    try:
        if (t.dtype is dtype and t.shape == shape and t.is_contiguous()
                and (t.is_cuda if device is None else t.get_device() == device)):
            return t.data_ptr()
    except AttributeError:
        raise DSparkError(f"{what}: {name} must be a tensor") from None
    raise DSparkError(f"{what}: {name} must be a contiguous {dtype} tensor {tuple(shape)} on the "
                      f"{'' if device is None else 'same '}GPU, not {t.dtype} {tuple(t.shape)} on "
                      f"{t.device}")


def _rows_view(what: str, name: str, t, heads, dim):
    """A bf16 [rows, heads, dim] view whose last dimension is dense: (address, rows,
    row stride, head stride)."""
    try:
        shape, stride = t.shape, t.stride()
        if not (t.dtype is torch.bfloat16 and len(shape) == 3 and shape[1] == heads
                and shape[2] == dim and stride[2] == 1 and t.is_cuda):
            raise DSparkError(f"{what}: {name} must be bfloat16 [rows, {heads}, {dim}] on the GPU "
                              "with a dense last dimension")
    except AttributeError:
        raise DSparkError(f"{what}: {name} must be a tensor") from None
    # a dimension of one element may carry any stride: what the call would step by is unused
    head = stride[1] if heads > 1 else dim
    row = stride[0] if shape[0] > 1 else dim
    return t.data_ptr(), shape[0], row, head


def _heads_view(what: str, name: str, t, dim, device=None):
    """_rows_view for any number of heads: (address, rows, heads, row stride, head stride)."""
    try:
        (rows, heads, width), (row, head, one) = t.shape, t.stride()
        if (t.dtype is torch.bfloat16 and width == dim and one == 1
                and (t.is_cuda if device is None else t.get_device() == device)):
            return (t.data_ptr(), rows, heads, row if rows > 1 else dim,
                    head if heads > 1 else dim)
    except AttributeError:
        raise DSparkError(f"{what}: {name} must be a tensor") from None
    except ValueError:
        pass
    raise DSparkError(f"{what}: {name} must be bfloat16 [rows, heads, {dim}] on the "
                      f"{'' if device is None else 'same '}GPU with a dense last dimension")


def _size(what: str, name: str, t, dims: int):
    """A tensor's shape, of so many dimensions."""
    try:
        shape = t.shape
        if len(shape) == dims:
            return shape
    except AttributeError:
        pass
    raise DSparkError(f"{what}: {name} must have {dims} dimensions")


def _masks(what: str, anc, rows: int):
    if anc is None:
        return None
    return _want(what, "anc", anc, torch.int64 if anc.dtype is torch.int64 else torch.uint64,
                 (rows,))


class KVCache:
    """One layer's paged cache: k and v [n_pages, page_size, heads, dim], bfloat16 or
    float8_e4m3fn (then with f32 scales [heads], default 1), in any memory order whose
    last dimension is dense."""

    def __init__(self, k, v, k_scale=None, v_scale=None):
        if k.dim() != 4 or k.shape != v.shape or k.dtype != v.dtype or k.stride() != v.stride():
            raise DSparkError("KVCache: k and v must be alike, [n_pages, page_size, heads, dim]")
        if k.dtype not in (torch.bfloat16, torch.float8_e4m3fn):
            raise DSparkError("KVCache: bfloat16 or float8_e4m3fn")
        if not (k.is_cuda and v.is_cuda):
            raise DSparkError("tensor must live on the GPU")
        if k.get_device() != v.get_device():
            raise DSparkError("KVCache: k and v must be on the same GPU")
        if k.stride(3) != 1:
            raise DSparkError("KVCache: the last dimension must be dense")
        self.k, self.v, self.k_scale, self.v_scale = k, v, k_scale, v_scale
        self.n_pages, self.page_size, self.heads, self.dim = k.shape
        fp8 = k.dtype == torch.float8_e4m3fn
        for name, t in (("k_scale", k_scale), ("v_scale", v_scale)):
            if t is not None and not fp8:
                raise DSparkError("KVCache: a bfloat16 cache has no scales")
            if t is not None:
                _want("KVCache", name, t, torch.float32, (self.heads,), k.get_device())
        # strides over a single page or head are never stepped by
        head = k.stride(2) if self.heads > 1 else self.dim
        page = k.stride(0) if self.n_pages > 1 else self.page_size * self.heads * self.dim
        self.struct = KVCacheStruct(k.data_ptr(), v.data_ptr(),
                                    k_scale.data_ptr() if k_scale is not None else None,
                                    v_scale.data_ptr() if v_scale is not None else None,
                                    page, k.stride(1), head, self.n_pages, self.page_size,
                                    self.heads, self.dim, KV_E4M3 if fp8 else KV_BF16)
        self.ref = ctypes.byref(self.struct)
        self.device = k.get_device()

    def on(self, what, device):
        """The cache for a call, once it is on the device of the call's tensors."""
        if self.device != device:
            raise DSparkError(f"{what}: the cache is on device {self.device}, the tensors on device "
                              f"{device}")
        return self.ref


def dspark_kv_plan(ctx, length, extra, parent, page_size, held, n_free, free_pages, block_table,
                   held_out, n_free_out, row_start, position, slot, anc=None, stream=None):
    """parent [R, gamma] or None (chains); anc int64 (the 64-bit words) or None."""
    what, i32 = "dspark_kv_plan", torch.int32
    R, rows = len(ctx), len(position)
    table = _size(what, "block_table", block_table, 2)
    gamma = _size(what, "parent", parent, 2)[1] if parent is not None else 0
    pages = len(free_pages)
    _check(load_library().dspark_kv_plan(
        R, gamma, extra, rows, page_size, pages, table[1],
        _want(what, "ctx", ctx, i32, (R,)), _want(what, "len", length, i32, (R,)),
        None if parent is None else _want(what, "parent", parent, i32, (R, gamma)),
        _want(what, "held", held, i32, (R,)), _want(what, "n_free", n_free, i32, (1,)),
        _want(what, "free_pages", free_pages, i32, (pages,)),
        _want(what, "block_table", block_table, i32, (R, table[1])),
        _want(what, "held_out", held_out, i32, (R,)),
        _want(what, "n_free_out", n_free_out, i32, (1,)),
        _want(what, "row_start", row_start, i32, (R + 1,)),
        _want(what, "position", position, i32, (rows,)),
        _want(what, "slot", slot, torch.int64, (rows,)), _masks(what, anc, rows),
        _stream(stream)), what)


def dspark_kv_append(cache: KVCache, k, v, slot, stream=None):
    """k, v bf16 [rows, heads, dim] views of equal strides."""
    what = "dspark_kv_append"
    kp, rows, row, head = _rows_view(what, "k", k, cache.heads, cache.dim)
    vp, *rest = _rows_view(what, "v", v, cache.heads, cache.dim)
    if rest != [rows, row, head]:
        raise DSparkError(f"{what}: k and v must have equal shapes and strides")
    _check(load_library().dspark_kv_append(
        cache.ref, rows, kp, vp, row, head, _want(what, "slot", slot, torch.int64, (rows,)),
        _stream(stream)), what)


def dspark_tree_attention_workspace_bytes(cache: KVCache, R, heads_q, max_nodes) -> int:
    return int(load_library().dspark_tree_attention_workspace_bytes(
        ctypes.byref(cache.struct), int(R), int(heads_q), int(max_nodes)))


def dspark_tree_attention(cache: KVCache, q, ctx, row_start, anc, block_table, max_nodes, scale,
                          out, lse, workspace, stream=None):
    """q, out bf16 [rows, heads_q, dim] (views with a dense last dimension); anc or lse may
    be None."""
    what, i32 = "dspark_tree_attention", torch.int32
    R, heads_q = len(ctx), _size(what, "q", q, 3)[1]
    qp, rows, q_row, q_head = _rows_view(what, "q", q, heads_q, cache.dim)
    op, o_rows, o_row, o_head = _rows_view(what, "out", out, heads_q, cache.dim)
    if o_rows != rows:
        raise DSparkError(f"{what}: out must have q's rows")
    pages = _size(what, "block_table", block_table, 2)[1]
    _check(load_library().dspark_tree_attention(
        cache.ref, R, heads_q, max_nodes, rows, pages, qp, q_row, q_head,
        _want(what, "ctx", ctx, i32, (R,)), _want(what, "row_start", row_start, i32, (R + 1,)),
        _masks(what, anc, rows), _want(what, "block_table", block_table, i32, (R, pages)), scale,
        op, o_row, o_head,
        None if lse is None else _want(what, "lse", lse, torch.float32, (rows, heads_q)),
        _ptr(workspace), workspace.numel(), _stream(stream)), what)


def dspark_tree_accept(row_start, parent, tokens, choice, ctx, accepted, bonus, path, ctx_out,
                       stream=None):
    """parent [R, gamma] or None (chains)."""
    what, i32 = "dspark_tree_accept", torch.int32
    R, gamma = shape = _size(what, "tokens", tokens, 2)
    rows = len(choice)
    _check(load_library().dspark_tree_accept(
        R, gamma, rows, _want(what, "row_start", row_start, i32, (R + 1,)),
        None if parent is None else _want(what, "parent", parent, i32, shape),
        _want(what, "tokens", tokens, i32, shape), _want(what, "choice", choice, i32, (rows,)),
        _want(what, "ctx", ctx, i32, (R,)), _want(what, "accepted", accepted, i32, (R,)),
        _want(what, "bonus", bonus, i32, (R,)), _want(what, "path", path, i32, shape),
        _want(what, "ctx_out", ctx_out, i32, (R,)), _stream(stream)), what)


def dspark_kv_compact(cache: KVCache, ctx, accepted, path, block_table, stream=None):
    """ctx as it was before dspark_tree_accept."""
    what, i32 = "dspark_kv_compact", torch.int32
    R, gamma = shape = _size(what, "path", path, 2)
    pages = _size(what, "block_table", block_table, 2)[1]
    _check(load_library().dspark_kv_compact(
        cache.ref, R, gamma, pages, _want(what, "ctx", ctx, i32, (R,)),
        _want(what, "accepted", accepted, i32, (R,)), _want(what, "path", path, i32, shape),
        _want(what, "block_table", block_table, i32, (R, pages)), _stream(stream)), what)


class Rotary:
    """The rotation of a head's first 2 * len(inv_freq) values (a multiple of 16): pair i by
    position * inv_freq[i] radians, f64.  A pair is values i and i + len(inv_freq), or with
    `pairs` values 2 i and 2 i + 1.  It serves calls on its own device."""

    def __init__(self, inv_freq, pairs=False, device="cuda"):
        f = torch.as_tensor(inv_freq, dtype=torch.float64)
        if f.dim() != 1 or f.numel() % 8 or not bool(torch.isfinite(f).all()):
            raise DSparkError("Rotary: inv_freq must be finite, one for each pair of values, a "
                              "multiple of 8 of them")
        # a position's part of a turn, in units of 2^-64
        words = [round(x / (2 * math.pi) % 1.0 * 2.0 ** 64) % 2 ** 64 for x in f.tolist()]
        self.turns = torch.tensor([x - 2 ** 64 if x >= 2 ** 63 else x for x in words],
                                  dtype=torch.int64, device=device)
        self.dims = 2 * len(words)
        self.struct = RopeStruct(self.turns.data_ptr(), self.dims,
                                 ROPE_PAIRS if pairs else ROPE_HALVES)
        self.ref = ctypes.byref(self.struct)

    def on(self, what, device):
        """The rotation for a call, once its table is on the device of the call's tensors."""
        if self.dims and self.turns.get_device() != device:
            raise DSparkError(f"{what}: the rotary's turns are on {self.turns.device}, the tensors "
                              f"on device {device}")
        return self.ref


def dspark_rope_append(cache: KVCache, q, k, v, position, slot, rotary: Rotary, q_out,
                       q_weight=None, k_weight=None, eps=1e-6, stream=None):
    """q, q_out bf16 [rows, heads_q, dim], k, v bf16 [rows, heads, dim] (k and v of equal
    strides); weights bf16 [dim] or None (no norm of that side).  q_out may be q."""
    what, dim = "dspark_rope_append", cache.dim
    qp, rows, heads_q, q_row, q_head = _heads_view(what, "q", q, dim)
    on = q.get_device()
    kp, *rest = _heads_view(what, "k", k, dim, on)
    vp, *also = _heads_view(what, "v", v, dim, on)
    op, o_rows, o_heads, o_row, o_head = _heads_view(what, "q_out", q_out, dim, on)
    if rest != also or rest[0] != rows or o_rows != rows:
        raise DSparkError(f"{what}: q, k, v and q_out must have equal rows, k and v equal strides")
    if rest[1] != cache.heads or o_heads != heads_q:
        raise DSparkError(f"{what}: k and v must have the cache's heads, q_out q's")
    bf16, width = torch.bfloat16, (dim,)
    _check(load_library().dspark_rope_append(
        cache.on(what, on), rows, heads_q, qp, q_row, q_head, kp, vp, rest[2], rest[3],
        None if q_weight is None else _want(what, "q_weight", q_weight, bf16, width, on),
        None if k_weight is None else _want(what, "k_weight", k_weight, bf16, width, on), eps,
        rotary.on(what, on), _want(what, "position", position, torch.int32, (rows,), on),
        _want(what, "slot", slot, torch.int64, (rows,), on), op, o_row, o_head,
        _stream_on(what, q, stream)), what)


def dspark_chunk_attention_workspace_bytes(cache: KVCache, R, heads_q, max_rows) -> int:
    return int(load_library().dspark_chunk_attention_workspace_bytes(
        cache.ref, int(R), int(heads_q), int(max_rows)))


def dspark_chunk_attention(cache: KVCache, q, ctx, row_start, block_table, max_rows, scale, out,
                           lse, workspace, stream=None):
    """q, out bf16 [rows, heads_q, dim] (views with a dense last dimension); lse may be None."""
    what, i32 = "dspark_chunk_attention", torch.int32
    qp, rows, heads_q, q_row, q_head = _heads_view(what, "q", q, cache.dim)
    on = q.get_device()
    op, o_rows, o_heads, o_row, o_head = _heads_view(what, "out", out, cache.dim, on)
    if o_rows != rows or o_heads != heads_q:
        raise DSparkError(f"{what}: out must have q's rows and heads")
    R = _size(what, "ctx", ctx, 1)[0]
    pages = _size(what, "block_table", block_table, 2)[1]
    _check(load_library().dspark_chunk_attention(
        cache.on(what, on), R, heads_q, max_rows, rows, pages, qp, q_row, q_head,
        _want(what, "ctx", ctx, i32, (R,), on),
        _want(what, "row_start", row_start, i32, (R + 1,), on),
        _want(what, "block_table", block_table, i32, (R, pages), on), scale, op, o_row, o_head,
        None if lse is None else _want(what, "lse", lse, torch.float32, (rows, heads_q), on),
        _ptr(workspace, on), workspace.numel(), _stream_on(what, q, stream)), what)


def dspark_kv_fork(source, target, page_size, ctx, held, n_free, free_pages, block_table, refs,
                   copy_from, copy_to, copy_tokens, stream=None):
    """Writes ctx, held, n_free, block_table and refs in place."""
    what, i32 = "dspark_kv_fork", torch.int32
    (n,), (R,) = _size(what, "source", source, 1), _size(what, "ctx", ctx, 1)
    pages = _size(what, "free_pages", free_pages, 1)[0]
    table = _size(what, "block_table", block_table, 2)
    places, on = _want(what, "ctx", ctx, i32, (R,)), ctx.get_device()
    _check(load_library().dspark_kv_fork(
        n, _want(what, "source", source, i32, (n,), on),
        _want(what, "target", target, i32, (n,), on), R, page_size, pages, table[1], places,
        _want(what, "held", held, i32, (R,), on), _want(what, "n_free", n_free, i32, (1,), on),
        _want(what, "free_pages", free_pages, i32, (pages,), on),
        _want(what, "block_table", block_table, i32, (R, table[1]), on),
        _want(what, "refs", refs, i32, (pages,), on),
        _want(what, "copy_from", copy_from, i32, (n,), on),
        _want(what, "copy_to", copy_to, i32, (n,), on),
        _want(what, "copy_tokens", copy_tokens, i32, (n,), on), _stream_on(what, ctx, stream)), what)


def dspark_kv_release(ctx, held, n_free, free_pages, block_table, refs, stream=None):
    """Writes held, n_free, free_pages and refs in place."""
    what, i32 = "dspark_kv_release", torch.int32
    (R,), (pages,) = _size(what, "ctx", ctx, 1), _size(what, "free_pages", free_pages, 1)
    table = _size(what, "block_table", block_table, 2)
    places, on = _want(what, "ctx", ctx, i32, (R,)), ctx.get_device()
    _check(load_library().dspark_kv_release(
        R, pages, table[1], places,
        _want(what, "held", held, i32, (R,), on), _want(what, "n_free", n_free, i32, (1,), on),
        _want(what, "free_pages", free_pages, i32, (pages,), on),
        _want(what, "block_table", block_table, i32, (R, table[1]), on),
        _want(what, "refs", refs, i32, (pages,), on), _stream_on(what, ctx, stream)), what)


def dspark_kv_squeeze(held, n_free, free_pages, block_table, refs, free_pages_out, block_table_out,
                      refs_out, new_page, move_from, move_to, n_moves, stream=None):
    """move_from and move_to have half as many entries as there are pages; the *_out tensors
    may be the inputs."""
    what, i32 = "dspark_kv_squeeze", torch.int32
    (R,), (pages,) = _size(what, "held", held, 1), _size(what, "free_pages", free_pages, 1)
    table = _size(what, "block_table", block_table, 2)
    shape, half = (R, table[1]), (pages // 2,)
    holds, on = _want(what, "held", held, i32, (R,)), held.get_device()
    _check(load_library().dspark_kv_squeeze(
        R, pages, table[1], holds,
        _want(what, "n_free", n_free, i32, (1,), on),
        _want(what, "free_pages", free_pages, i32, (pages,), on),
        _want(what, "block_table", block_table, i32, shape, on),
        _want(what, "refs", refs, i32, (pages,), on),
        _want(what, "free_pages_out", free_pages_out, i32, (pages,), on),
        _want(what, "block_table_out", block_table_out, i32, shape, on),
        _want(what, "refs_out", refs_out, i32, (pages,), on),
        _want(what, "new_page", new_page, i32, (pages,), on),
        _want(what, "move_from", move_from, i32, half, on),
        _want(what, "move_to", move_to, i32, half, on),
        _want(what, "n_moves", n_moves, i32, (1,), on), _stream_on(what, held, stream)), what)


def dspark_kv_copy(cache: KVCache, copy_from, copy_to, copy_tokens=None, stream=None):
    """copy_tokens None: whole pages."""
    what, i32 = "dspark_kv_copy", torch.int32
    n = _size(what, "copy_from", copy_from, 1)[0]
    pages, on = _want(what, "copy_from", copy_from, i32, (n,)), copy_from.get_device()
    _check(load_library().dspark_kv_copy(
        cache.on(what, on), n, pages,
        _want(what, "copy_to", copy_to, i32, (n,), on),
        None if copy_tokens is None else _want(what, "copy_tokens", copy_tokens, i32, (n,), on),
        _stream_on(what, copy_from, stream)), what)


def dspark_device_status(stream=None, clear: bool = True) -> int:
    return int(load_library().dspark_device_status(_stream(stream), 1 if clear else 0))


def dspark_selftest_wait_timeout(limit_ns: int, stream=None):
    _check(load_library().dspark_selftest_wait_timeout(int(limit_ns), _stream(stream)),
           "dspark_selftest_wait_timeout")


def dspark_launch_count() -> int:
    return int(load_library().dspark_launch_count())


def check_device_status(stream=None):
    rc = dspark_device_status(stream)
    _check(rc, "device status")


# ------------------------------------------------------- tensor helpers ----

def workspace(nbytes: int, device="cuda") -> torch.Tensor:
    """A byte buffer for the library's scratch (torch allocations are 256-B aligned)."""
    t = torch.empty(max(int(nbytes), 1), dtype=torch.uint8, device=device)
    assert t.data_ptr() % 256 == 0
    return t


class PagePool:
    """The pages of R requests over any number of layers' caches, on the device: who
    holds which, and one round's rows.  A call makes no tensors but attend's scratch, once
    for each size and stream.  A round's calls go on one stream (or are ordered by events):
    they read and write the pool's tensors.

    `ctx` holds the committed tokens, -1 for a free place; a request enters when its
    prompt's rows are planned with ctx 0, and leaves when its ctx is set to -1 (its
    pages go back with the next plan).

    A `shared` pool's requests may be forked: continuations share a prompt's full pages,
    and a page goes back with the last of its holders (with the next plan, fork or
    squeeze)."""

    def __init__(self, R, n_pages, page_size, max_tokens, n_rows, device="cuda", shared=False):
        new = lambda shape, dtype=torch.int32: torch.empty(shape, dtype=dtype, device=device)  # noqa: E731
        self.page_size, self.n_rows = page_size, n_rows
        max_pages = -(-max_tokens // page_size)
        self.ctx = torch.full((R,), -1, dtype=torch.int32, device=device)
        self.held = torch.zeros((R,), dtype=torch.int32, device=device)
        self.free_pages = torch.arange(n_pages - 1, -1, -1, dtype=torch.int32, device=device)
        self.n_free = torch.tensor([n_pages], dtype=torch.int32, device=device)
        self.block_table = torch.full((R, max_pages), -1, dtype=torch.int32, device=device)
        self.row_start, self.position = new(R + 1), new(n_rows)
        self.slot, self.anc = new(n_rows, torch.int64), new(n_rows, torch.int64)
        self.accepted, self.bonus, self.ctx_before = new(R), new(R), new(R)
        # commit's: who is there, and by how much each goes on
        self._live, self._step = new(R, torch.bool), new(R)
        self._prompts = False  # the rows planned last are prompts': anc is not theirs
        self._ws = {}
        self.shared = shared
        self.refs = None       # holders of a page beyond the first
        if shared:
            self.refs = torch.zeros((n_pages,), dtype=torch.int32, device=device)
            self._copies = [new(R) for _ in range(3)]    # of the last fork: from, to, tokens
            self.copies = [t[:0] for t in self._copies]
            # of the last squeeze: none yet
            self.new_page = new(n_pages)
            self.n_moves = torch.zeros((1,), dtype=torch.int32, device=device)
            self.move_from, self.move_to = (torch.full((n_pages // 2,), -1, dtype=torch.int32,
                                                       device=device) for _ in range(2))

    def plan(self, length, extra=1, parent=None, stream=None):
        """Rows, pages, slots, positions (and masks, in a round) for `length` + extra new
        rows of each request: extra 1 in a round, 0 for prompts."""
        if self.shared:
            self.release(stream)
        dspark_kv_plan(self.ctx, length, extra, parent, self.page_size, self.held, self.n_free,
                       self.free_pages, self.block_table, self.held, self.n_free,
                       self.row_start, self.position, self.slot, self.anc if extra else None,
                       stream)
        self._prompts = not extra

    def append(self, cache: KVCache, k, v, stream=None):
        """One layer's new rows into the planned slots."""
        dspark_kv_append(cache, k, v, self.slot, stream)

    def rope_append(self, cache: KVCache, q, k, v, rotary: Rotary, q_out, q_weight=None,
                    k_weight=None, eps=1e-6, stream=None):
        """append, with the queries' and keys' heads normalised (where they have weights) and
        turned by the planned positions; the queries go to q_out, which may be q."""
        dspark_rope_append(cache, q, k, v, self.position, self.slot, rotary, q_out, q_weight,
                           k_weight, eps, stream)

    def attend(self, cache: KVCache, q, max_nodes, out, lse=None, scale=None, stream=None):
        """One layer's attention of the rows that plan was last called for, over contexts and
        trees; a prompt's (max_nodes rows a request at most, any number) are chains.  Which of
        the two is settled at the call: a graph that holds an attend holds its plan too.

        A prompt's rows go to the tree attention up to MAX_NODES a request, as they always
        did: beside a bf16 cache its weights have 16 bits, the chunk attention's 8.  It is the
        slower one there from about 32 rows x query heads of a KV head on (64 requests over 512
        to 4096 tokens, 32 heads over 8, 16 rows each: 138 and 114 us, 64 rows: 364 and 135,
        in 8 bits 799 and 184); dspark_chunk_attention takes the pool's ctx, row_start and
        block_table as they are."""
        scale = cache.dim ** -0.5 if scale is None else scale
        if self._prompts and max_nodes > MAX_NODES:
            need = dspark_chunk_attention_workspace_bytes(cache, len(self.ctx), q.shape[1],
                                                          max_nodes)
            ws = self._scratch(need, q.device, stream)
            dspark_chunk_attention(cache, q, self.ctx, self.row_start, self.block_table, max_nodes,
                                   scale, out, lse, ws, stream)
            return
        need = dspark_tree_attention_workspace_bytes(cache, len(self.ctx), q.shape[1], max_nodes)
        ws = self._scratch(need, q.device, stream)
        dspark_tree_attention(cache, q, self.ctx, self.row_start,
                              None if self._prompts else self.anc, self.block_table, max_nodes,
                              scale, out, lse, ws, stream)

    def _scratch(self, need, device, stream):
        """An attention's workspace, which no call on another stream may use meanwhile: kept
        for each size and stream.  Under capture it is the graph's own memory, as the graph
        may be replayed beside calls on the stream that it was captured on."""
        key = need, device, _stream(stream)
        with torch.cuda.stream(stream):
            if torch.cuda.is_current_stream_capturing():
                return workspace(need, device)
            ws = self._ws.get(key)
            if ws is None:
                ws = self._ws[key] = workspace(need, device)
        return ws

    def commit(self, rows, stream=None):
        """`rows` of each request's new rows are committed: after dspark_verify the anchor
        and the accepted drafts (accepted + 1), after a prompt its length."""
        with torch.cuda.stream(stream):
            torch.ge(self.ctx, 0, out=self._live)
            torch.mul(self._live, rows, out=self._step)
            self.ctx.add_(self._step)

    def accept(self, tokens, choice, path, parent=None, stream=None):
        """The trees' confirmed paths (into `path` [R, gamma], self.accepted, self.bonus);
        commits them.  Each layer's cache then needs compact()."""
        s = stream if stream is not None else torch.cuda.current_stream()
        with torch.cuda.stream(s):
            self.ctx_before.copy_(self.ctx)
        dspark_tree_accept(self.row_start, parent, tokens, choice, self.ctx, self.accepted,
                           self.bonus, path, self.ctx, stream)

    def compact(self, cache: KVCache, path, stream=None):
        dspark_kv_compact(cache, self.ctx_before, self.accepted, path, self.block_table, stream)

    def _needs_shared(self, what):
        if not self.shared:
            raise DSparkError(f"PagePool.{what}: the pool must be made with shared=True")

    def fork(self, source, target, stream=None):
        """Free places target[i] become continuations of requests source[i] (int32, one for
        each fork; source[i] < 0: none), places that were just left among them: what those
        held is given back first.  Each layer's cache then needs copy(), before the next fork
        or squeeze.  Between rounds only: a commit goes on with every place that is there."""
        self._needs_shared("fork")
        if len(source) > len(self.ctx):
            raise DSparkError("PagePool.fork: more forks than places")
        self.release(stream)
        copies = [t[:len(source)] for t in self._copies]
        dspark_kv_fork(source, target, self.page_size, self.ctx, self.held, self.n_free,
                       self.free_pages, self.block_table, self.refs, *copies, stream)
        self.copies = copies

    def copy(self, cache: KVCache, stream=None):
        """One layer's part of the last fork, once: the last pages' tokens."""
        self._needs_shared("copy")
        dspark_kv_copy(cache, *self.copies, stream)

    def release(self, stream=None):
        """The pages of the requests that left (ctx -1), now rather than with the next plan, fork
        or squeeze."""
        self._needs_shared("release")
        dspark_kv_release(self.ctx, self.held, self.n_free, self.free_pages, self.block_table,
                          self.refs, stream)

    def squeeze(self, stream=None):
        """The pages in use renamed to the lowest numbers (and those of requests that left given
        back).  Each layer's cache then needs move(); a planned round's slots are void."""
        self._needs_shared("squeeze")
        self.release(stream)
        dspark_kv_squeeze(self.held, self.n_free, self.free_pages, self.block_table, self.refs,
                          self.free_pages, self.block_table, self.refs, self.new_page,
                          self.move_from, self.move_to, self.n_moves, stream)

    def move(self, cache: KVCache, stream=None):
        """One layer's part of the last squeeze, once and before its next rows."""
        self._needs_shared("move")
        dspark_kv_copy(cache, self.move_from, self.move_to, None, stream)


@dataclass
class DraftHead:
    """Device-resident draft-head weights in the library's layouts."""
    dims: Dims
    W_lm: torch.Tensor    # bf16 [V, d]
    W1: torch.Tensor      # bf16 [V, r]
    W2t: torch.Tensor     # bf16 [V, r]  (W2 transposed once)
    w_conf: torch.Tensor  # bf16 [d + r]
    T: torch.Tensor       # f32 [gamma]

    @staticmethod
    def from_weights(R, gamma, W_lm, W1, W2, w_conf, T, device="cuda") -> "DraftHead":
        V, d = W_lm.shape
        r = W1.shape[1]
        dims = dims_of(R, gamma, V, r, d)
        W2d = _bf16(W2).to(device).contiguous()
        W2t = torch.empty((V, r), dtype=torch.bfloat16, device=device)
        dspark_pack_w2(dims, W2d, W2t)
        return DraftHead(dims, _bf16(W_lm).to(device).contiguous(), _bf16(W1).to(device).contiguous(),
                         W2t, _bf16(w_conf).to(device).contiguous(),
                         T.to(device=device, dtype=torch.float32).contiguous())


class Round:
    """Pre-allocated outputs and workspaces of one round (no allocation per call)."""

    def __init__(self, head: DraftHead, device="cuda"):
        d = head.dims
        self.head = head
        R, G, V = d.R, d.gamma, d.V
        self.base = torch.empty((R * G, V), dtype=torch.bfloat16, device=device)
        self.tokens = torch.empty((R, G), dtype=torch.int32, device=device)
        self.conf = torch.empty((R, G), dtype=torch.float32, device=device)
        self.logp_d = torch.empty((R, G), dtype=torch.float32, device=device)
        self.lse_d = torch.empty((R, G), dtype=torch.float32, device=device)
        self.len = torch.empty((R,), dtype=torch.int32, device=device)
        self.K = torch.empty((1,), dtype=torch.int32, device=device)
        self.theta = torch.empty((1,), dtype=torch.float64, device=device)
        self.accepted = torch.empty((R,), dtype=torch.int32, device=device)
        self.bonus = torch.empty((R,), dtype=torch.int32, device=device)
        self.ws_draft = workspace(dspark_markov_workspace_bytes(d), device)
        self.ws_verify = workspace(dspark_verify_workspace_bytes(d), device)
        # run_host: the target logits come in on a side stream during the draft
        self._copy_stream = torch.cuda.Stream(device=device)
        self._target_ready = torch.cuda.Event()

    def draft(self, h, anchor, tau, seed, stream=None):
        hd = self.head
        dspark_draft(hd.dims, h, anchor, hd.W_lm, hd.W1, hd.W2t, hd.w_conf, hd.T, tau, seed,
                     self.base, self.tokens, self.conf, self.logp_d, self.lse_d, self.ws_draft,
                     stream)

    def schedule(self, sps, mode=SCHED_UNCONSTRAINED, k_fixed=0, stream=None, k_ring=None):
        """mode SCHED_ASYNC takes the device ring of async_ring() and ignores k_fixed."""
        d = self.head.dims
        if mode == SCHED_ASYNC:
            if k_ring is None:
                raise DSparkError("SCHED_ASYNC needs k_ring (see async_ring)")
            dspark_schedule_async(self.conf, d.R, d.gamma, sps, k_ring, self.len, self.K,
                                  self.theta, stream=stream)
            return
        dspark_schedule(self.conf, d.R, d.gamma, sps, mode, k_fixed, self.len, self.K, self.theta,
                        stream=stream)

    def verify(self, anchor, target, tau, seed, stream=None):
        hd = self.head
        dspark_verify(hd.dims, anchor, self.tokens, self.len, self.base, hd.W1, hd.W2t,
                      self.lse_d, self.logp_d, target, tau, seed, self.accepted, self.bonus,
                      self.ws_verify, stream)

    def run(self, h, anchor, target, sps, tau, draft_seed, verify_seed,
            mode=SCHED_UNCONSTRAINED, k_fixed=0, stream=None, k_ring=None):
        """One whole round on device-resident inputs: draft -> schedule -> verify."""
        self.draft(h, anchor, tau, draft_seed, stream)
        self.schedule(sps, mode, k_fixed, stream, k_ring)
        self.verify(anchor, target, tau, verify_seed, stream)

    def run_host(self, h_host, anchor_host, target_host, sps, tau, draft_seed, verify_seed,
                 dev_in: Dict[str, torch.Tensor], out_host: Dict[str, torch.Tensor],
                 mode=SCHED_UNCONSTRAINED, k_fixed=0, stream=None, k_ring=None) -> None:
        """One round from pinned host inputs to pinned host outputs (copies included).

        h and the anchors are copied on `stream` ahead of the draft.  The target
        logits, read only by verify, are copied on a side stream that starts
        once everything already queued on `stream` (the previous round, whose
        verify reads the same buffer) is done, so the copy runs under the draft
        and the schedule; verify waits for it."""
        s = stream if stream is not None else torch.cuda.current_stream()
        c = self._copy_stream
        with torch.cuda.stream(s):
            dev_in["h"].copy_(h_host, non_blocking=True)
            dev_in["anchor"].copy_(anchor_host, non_blocking=True)
        c.wait_stream(s)
        with torch.cuda.stream(c):
            dev_in["target"].copy_(target_host, non_blocking=True)
        dev_in["target"].record_stream(c)
        self._target_ready.record(c)
        self.draft(dev_in["h"], dev_in["anchor"], tau, draft_seed, s)
        self.schedule(sps, mode, k_fixed, s, k_ring)
        s.wait_event(self._target_ready)
        self.verify(dev_in["anchor"], dev_in["target"], tau, verify_seed, s)
        with torch.cuda.stream(s):
            out_host["tokens"].copy_(self.tokens, non_blocking=True)
            out_host["len"].copy_(self.len, non_blocking=True)
            out_host["accepted"].copy_(self.accepted, non_blocking=True)
            out_host["bonus"].copy_(self.bonus, non_blocking=True)
