"""gemm_conv_chain_amd -- Python binding of libfusedchain (MI355X / gfx950).

Argument marshalling only: every computation runs in the HIP kernels of
``libfusedchain.so`` behind the C ABI in ``include/fusedchain.h``.  PyTorch is
used for device memory and the current stream; there is no CPU or PyTorch
fallback -- if the library is missing, every call raises.

The functions mirror the C entry points:

* ``chain_gemm2(A, W0, b0, W1, b1, act)``      D1 = act(A W0 + b0) W1 + b1
* ``chain_conv_pool(x, w, b, act, pool)``      maxpool2x2(act(conv3x3(x) + b))
* ``chain_conv2(x, w0, b0, w1, b1, act)``      conv1x1(act(conv3x3(x) + b0)) + b1
* ``gemm_bias_act``, ``conv_bias_act``, ``maxpool2x2``   single operators
* ``rope(x, positions, turns)``, ``kv_append(k, v, codes, ...)``,
  ``chain_attn(q, codes, ...)``   rotary positions, appending to a paged cache of
  8-bit codes (``kv_cache``), and attention over it (softmax(q K^T) V as a chain)
* ``tree_plan(parents, ...)``, ``chain_attn(..., tree=...)``, ``sample_tokens(logits,
  u)``, ``tree_accept(...)``, ``kv_keep(...)``   a step that verifies drafted tokens;
  ``kv_copy`` and ``KvPages`` copy, fork, pack and free the cache's pages
* ``pad_channels`` / ``pad_weight_channels``   zero padding of channel counts
"""
from __future__ import annotations

import array
import contextlib
import ctypes
import heapq
import itertools
import math
import os
import re

__all__ = ["DTYPE", "ATTN_VARIANT", "rope_turns", "rope", "kv_cache", "kv_append", "kv_check", "chain_attn", "attn_plan",
           "tree_plan", "tree_accept", "kv_keep", "kv_copy", "KvPages", "sample_tokens",
           "TuneEntry", "tune_chain_gemm2_table", "auto_config", "tune_conv_pool", "conv_auto_config", "CONV_VARIANT", "lib", "FusedChainError", "chain_gemm2", "tune_chain_gemm2", "auto_variant", "tune_clear", "chain_gemmN", "chain_conv_pool", "chain_conv_bn_pool", "chain_conv2", "chain_convN", "convN_auto_variant", "tune_chain_convN",
           "gemm_bias_act", "conv_bias_act", "maxpool2x2", "avgpool2x2", "pad_channels", "pad_weight_channels", "abi_version", "ACT", "VARIANT",
           "LIB_PATH", "POISON_LIB_PATH", "poison_build", "HEADER_PATH", "exported_names"]

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libfusedchain.so")
POISON_LIB_PATH = os.path.join(_HERE, "libfusedchain_poison.so")
HEADER_PATH = os.path.join(os.path.dirname(_HERE), "include", "fusedchain.h")

ACT = {"none": 0, "relu": 1, "gelu_tanh": 2, "hardswish": 3}
POOL = {"none": 0, "max2x2": 1, "avg2x2": 2}
VARIANT = {"auto": 0, "rf": 1, "lds": 2, "stream": 3, "pipe": 4}
ATTN_VARIANT = {"auto": 0, "rows": 1, "tile": 2}
DTYPE = {"float16": 0, "bfloat16": 1}
CONV_VARIANT = {"auto": 0, "lds_weights": 1, "reg_weights": 2}


class FusedChainError(RuntimeError):
    def __init__(self, fn, status, detail):
        self.status = status
        super().__init__("%s failed: %s (%s)" % (fn, _lib_status_str(status), detail))


class ConvShape(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("n", "h", "w", "c", "k", "r", "s", "stride", "pad")]


class TuneEntry(ctypes.Structure):
    """One configuration timed by the profiler: kernel form, tile-owning waves
    per block (0 = the form's own block shape), pipeline stages of the
    register-resident row stream (0 = the default 4, or 2), microseconds per
    launch."""
    _fields_ = [("variant", ctypes.c_int32), ("waves", ctypes.c_int32), ("stages", ctypes.c_int32),
                ("us", ctypes.c_float)]


class KvShape(ctypes.Structure):
    """fc_kv_shape: the batch and the paged cache of kv_append and chain_attn."""
    _fields_ = [(n, ctypes.c_int32) for n in ("dtype", "batch", "hq", "hkv", "d", "page", "pages", "table_stride")] + [
        ("tokens", ctypes.c_int64), ("max_q", ctypes.c_int32), ("max_kv", ctypes.c_int32)]


class RopeTable(ctypes.Structure):
    """fc_rope: turns a position of each pair (device), rotated elements, pairing, factor."""
    _fields_ = [("turns", ctypes.c_void_p), ("rot", ctypes.c_int32), ("interleaved", ctypes.c_int32),
                ("mscale", ctypes.c_float)]


class AttnParams(ctypes.Structure):
    _fields_ = [("scale", ctypes.c_float), ("softcap", ctypes.c_float), ("causal", ctypes.c_int32),
                ("window", ctypes.c_int32), ("variant", ctypes.c_int32), ("splits", ctypes.c_int32)]


class AttnPlan(ctypes.Structure):
    _fields_ = [("variant", ctypes.c_int32), ("splits", ctypes.c_int32), ("chunk", ctypes.c_int32),
                ("workspace", ctypes.c_int64)]


class Tree(ctypes.Structure):
    """fc_tree: what the new tokens of a tree see of each other, and where they sit."""
    _fields_ = [("bits", ctypes.c_void_p), ("positions", ctypes.c_void_p), ("words", ctypes.c_int32)]


class Sampling(ctypes.Structure):
    """fc_sampling: arrays of a row's settings (or NULL), and the values for all rows."""
    _fields_ = [(n, ctypes.c_void_p) for n in ("temperatures", "top_ks", "top_ps", "min_ps")] + [
        ("temperature", ctypes.c_float), ("top_k", ctypes.c_int32), ("top_p", ctypes.c_float), ("min_p", ctypes.c_float)]


_lib = None
_poison_lib = None
_override = None
_vp = ctypes.c_void_p
_i32 = ctypes.c_int32
_i64 = ctypes.c_int64


def lib():
    """The library every call goes through: libfusedchain.so (built by
    ``gemm_conv_chain_amd.build``), or the poison debug build inside a
    ``poison_build()`` block."""
    global _lib
    if _override is not None:
        return _override
    if _lib is None:
        _lib = _load(LIB_PATH)
    return _lib


@contextlib.contextmanager
def poison_build():
    """Route every call inside the with-block through libfusedchain_poison.so,
    the -DFC_DEBUG_POISON build: its kernels overwrite each LDS buffer with a
    poison pattern (fp16 65504) when the barrier that releases it has passed,
    so a read that races its producer changes the results.  Test use only."""
    global _override, _poison_lib
    if _poison_lib is None:
        _poison_lib = _load(POISON_LIB_PATH)
    prev, _override = _override, _poison_lib
    try:
        yield _poison_lib
    finally:
        _override = prev


def _load(path):
    if not os.path.exists(path):
        raise FusedChainError("load", -1, "%s not built: run python -m gemm_conv_chain_amd.build"
                              % os.path.basename(path))
    L = ctypes.CDLL(path)
    L.fc_abi_version.restype = _i32
    L.fc_status_str.restype = ctypes.c_char_p
    L.fc_status_str.argtypes = [ctypes.c_int]
    L.fc_last_error.restype = ctypes.c_char_p
    L.chain_gemm2.argtypes = [_vp, _vp, _vp, ctypes.c_int, _vp, _vp, _vp, _i64, _i32, _i32, _i32, _vp]
    L.chain_gemm2_variant.argtypes = [_vp, _vp, _vp, ctypes.c_int, _vp, _vp, _vp, _i64, _i32, _i32, _i32,
                                      ctypes.c_int, _vp]
    L.chain_gemmN.argtypes = [_vp, _i32, ctypes.POINTER(_vp), ctypes.POINTER(_vp), ctypes.POINTER(ctypes.c_int),
                              ctypes.POINTER(_i32), _vp, _i64, _vp]
    L.chain_conv_pool.argtypes = [_vp, _vp, _vp, ctypes.c_int, ctypes.c_int, _vp, ctypes.POINTER(ConvShape),
                                  _vp, _vp]
    L.chain_conv2.argtypes = [_vp, _vp, _vp, ctypes.c_int, _vp, _vp, _i32, _vp, ctypes.POINTER(ConvShape), _vp]
    L.gemm_bias_act.argtypes = [_vp, _vp, _vp, ctypes.c_int, _vp, _i64, _i32, _i32, _vp]
    L.conv_bias_act.argtypes = [_vp, _vp, _vp, ctypes.c_int, _vp, ctypes.POINTER(ConvShape), _vp]
    L.maxpool2x2.argtypes = [_vp, _vp, _vp, _i32, _i32, _i32, _i32, _vp]
    L.avgpool2x2.argtypes = [_vp, _vp, _i32, _i32, _i32, _i32, _vp]
    L.pad_channels.argtypes = [_vp, _vp, _i64, _i32, _i32, _i32, _vp]
    L.chain_gemm2_tune.argtypes = [_vp, _vp, _vp, ctypes.c_int, _vp, _vp, _vp, _i64, _i32, _i32, _i32, _i32,
                                   ctypes.POINTER(ctypes.c_int), ctypes.POINTER(ctypes.c_float), _vp]
    L.chain_gemm2_auto_variant.argtypes = [_i64, _i32, _i32, _i32, ctypes.c_int, ctypes.POINTER(ctypes.c_int)]
    L.chain_convN.argtypes = [_vp, ctypes.POINTER(ConvShape), _i32, ctypes.POINTER(_vp), ctypes.POINTER(_vp),
                              ctypes.POINTER(ctypes.c_int), ctypes.POINTER(_i32), _vp, _vp]
    L.chain_convN_variant.argtypes = [_vp, ctypes.POINTER(ConvShape), _i32, ctypes.POINTER(_vp), ctypes.POINTER(_vp),
                                      ctypes.POINTER(ctypes.c_int), ctypes.POINTER(_i32), _vp, ctypes.c_int, _vp]
    L.chain_convN_auto_variant.argtypes = [ctypes.POINTER(ConvShape), _i32, ctypes.POINTER(_i32),
                                           ctypes.POINTER(ctypes.c_int)]
    L.chain_convN_tune.argtypes = [_vp, ctypes.POINTER(ConvShape), _i32, ctypes.POINTER(_vp), ctypes.POINTER(_vp),
                                   ctypes.POINTER(ctypes.c_int), ctypes.POINTER(_i32), _vp, _i32,
                                   ctypes.POINTER(TuneEntry), _i32, ctypes.POINTER(_i32), ctypes.POINTER(TuneEntry), _vp]
    L.chain_conv_bn_pool.argtypes = [_vp, _vp, _vp, _vp, ctypes.c_int, ctypes.c_int, _vp,
                                     ctypes.POINTER(ConvShape), _vp, _vp]
    L.chain_conv_pool_ex.argtypes = [_vp, _vp, _vp, _vp, ctypes.c_int, ctypes.c_int, _vp,
                                     ctypes.POINTER(ConvShape), _vp, ctypes.c_int, _i32, _vp]
    L.chain_gemm2_ex.argtypes = [_vp, _vp, _vp, ctypes.c_int, _vp, _vp, _vp, _i64, _i32, _i32, _i32,
                                 ctypes.c_int, _i32, _i32, _vp]
    L.fc_probe_mfma.argtypes = [_i32, _i32, _vp, _vp, _i32, ctypes.POINTER(_i32), _vp]
    L.fc_probe_read.argtypes = [_vp, _i64, _vp, _i32, ctypes.POINTER(_i32), _vp]
    L.chain_gemm2_tune_ex.argtypes = [_vp, _vp, _vp, ctypes.c_int, _vp, _vp, _vp, _i64, _i32, _i32, _i32, _i32,
                                      ctypes.POINTER(TuneEntry), _i32, ctypes.POINTER(_i32),
                                      ctypes.POINTER(TuneEntry), _vp]
    L.chain_gemm2_auto_config.argtypes = [_i64, _i32, _i32, _i32, ctypes.c_int, ctypes.POINTER(TuneEntry)]
    L.chain_conv_pool_tune.argtypes = [_vp, _vp, _vp, _vp, ctypes.c_int, ctypes.c_int, _vp,
                                       ctypes.POINTER(ConvShape), _vp, _i32, ctypes.POINTER(TuneEntry), _i32,
                                       ctypes.POINTER(_i32), ctypes.POINTER(TuneEntry), _vp]
    L.chain_conv_pool_auto_config.argtypes = [ctypes.POINTER(ConvShape), ctypes.c_int, ctypes.c_int, _i32,
                                              ctypes.POINTER(TuneEntry)]
    L.chain_conv2_ex.argtypes = [_vp, _vp, _vp, ctypes.c_int, _vp, _vp, _i32, _vp, ctypes.POINTER(ConvShape),
                                 _i32, _i32, _vp]
    L.chain_conv2_variant.argtypes = [_vp, _vp, _vp, ctypes.c_int, _vp, _vp, _i32, _vp, ctypes.POINTER(ConvShape),
                                      ctypes.c_int, _i32, _i32, _vp]
    L.chain_conv2_tune.argtypes = [_vp, _vp, _vp, ctypes.c_int, _vp, _vp, _i32, _vp, ctypes.POINTER(ConvShape),
                                   _i32, ctypes.POINTER(TuneEntry), _i32, ctypes.POINTER(_i32),
                                   ctypes.POINTER(TuneEntry), _vp]
    L.chain_conv2_auto_config.argtypes = [ctypes.POINTER(ConvShape), _i32, ctypes.c_int, ctypes.POINTER(TuneEntry)]
    L.winograd_weights.argtypes = [_vp, _vp, _i32, _i32, _vp]
    L.chain_conv_pool_winograd.argtypes = [_vp, _vp, _vp, ctypes.c_int, ctypes.c_int, _vp,
                                           ctypes.POINTER(ConvShape), _vp, _vp]
    L.rope_apply.argtypes = [_vp, _vp, ctypes.POINTER(_i64), _vp, ctypes.POINTER(RopeTable), _i32, ctypes.c_int, _i64,
                             _i32, _i32, _vp]
    L.kv_append.argtypes = [_vp, _vp, _vp, _vp, ctypes.POINTER(_i64), _vp, _vp, _vp, _vp, _vp, _vp,
                            ctypes.POINTER(RopeTable), ctypes.POINTER(KvShape), _vp]
    L.chain_attn_plan.argtypes = [ctypes.POINTER(KvShape), ctypes.POINTER(AttnParams), ctypes.POINTER(AttnPlan)]
    L.chain_attn.argtypes = [_vp, ctypes.POINTER(_i64), _vp, _vp, _vp, _vp, _vp, _vp, ctypes.POINTER(AttnParams), _vp,
                             _vp, ctypes.POINTER(KvShape), _vp, _i64, _vp]
    L.kv_check.argtypes = [_vp, _vp, _vp, ctypes.POINTER(KvShape), _i32]
    L.chain_attn_tree.argtypes = [_vp, ctypes.POINTER(_i64), _vp, _vp, _vp, _vp, _vp, ctypes.POINTER(Tree), _vp,
                                  ctypes.POINTER(AttnParams), _vp, _vp, ctypes.POINTER(KvShape), _vp, _i64, _vp]
    L.chain_attn_tree_plan.argtypes = L.chain_attn_plan.argtypes
    L.tree_plan.argtypes = [_vp, _vp, _vp, _i32, _i64, _i32, _vp, _vp, _vp]
    L.tree_accept.argtypes = [_vp, _vp, _vp, _vp, _vp, _i32, _i64, _i32, _vp, _vp, _vp, _vp, _vp]
    L.kv_keep.argtypes = [_vp, _vp, _i32, _vp, _vp, _vp, _vp, _vp, _i32, ctypes.POINTER(KvShape), _vp]
    L.kv_copy.argtypes = [_vp, _vp, _i32, _i32, _i32, _i32, _i32, _vp, _i64, _vp]
    L.sample_workspace.argtypes = [_i32, _i64, _i32, ctypes.POINTER(_i64)]
    L.sample_tokens.argtypes = [_vp, _i32, _i64, _i32, _i64, _vp, ctypes.POINTER(Sampling), _vp, _vp, _i64, _vp]
    L.fc_tune_clear.restype = None
    L.fc_tune_clear.argtypes = []
    for name in ("chain_attn_tree", "chain_attn_tree_plan", "tree_plan", "tree_accept", "kv_keep", "kv_copy", "sample_workspace", "sample_tokens",
                 "rope_apply", "kv_append", "chain_attn_plan", "chain_attn", "kv_check", "chain_conv2_auto_config", "chain_conv2_ex", "chain_conv2_variant", "chain_conv2_tune", "winograd_weights", "chain_conv_pool_winograd", "chain_gemm2_ex", "chain_gemm2_tune_ex", "chain_gemm2_auto_config", "chain_conv_pool_tune",
                 "chain_conv_pool_auto_config", "chain_conv_pool_ex", "avgpool2x2", "fc_probe_mfma", "fc_probe_read", "chain_conv_bn_pool", "chain_convN", "chain_convN_variant", "chain_convN_auto_variant", "chain_convN_tune", "chain_gemm2_tune", "chain_gemm2_auto_variant", "chain_gemm2", "chain_gemm2_variant", "chain_gemmN", "chain_conv_pool", "chain_conv2", "gemm_bias_act",
                 "conv_bias_act", "maxpool2x2", "pad_channels"):
        getattr(L, name).restype = ctypes.c_int
    return L


def _lib_status_str(s):
    try:
        return lib().fc_status_str(int(s)).decode()
    except Exception:
        return str(s)


def abi_version() -> int:
    return int(lib().fc_abi_version())


def exported_names():
    """Function names declared in include/fusedchain.h."""
    with open(HEADER_PATH) as f:
        text = f.read()
    return sorted(set(re.findall(r"^\s*(?:const\s+)?[a-z_0-9]+\s*\*?\s*([A-Za-z_0-9]+)\s*\(", text, re.M)))


def _check(fn, status):
    if status != 0:
        raise FusedChainError(fn, status, lib().fc_last_error().decode())


# ------------------------------------------------------------ tensor helpers
# The C ABI sees pointers only, so every size the kernels rely on is checked
# here, against the sizes the inputs imply, before the library is called:
# shapes, dtypes and contiguity first (ValueError / TypeError, testable with
# host tensors), then that every tensor is a device tensor on one device.
def _torch():
    import torch
    return torch


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _ndim(t, name, ndim):
    """t (may be None) is a tensor with ndim dimensions; returns its shape."""
    torch = _torch()
    if t is None:
        return None
    if not isinstance(t, torch.Tensor):
        raise TypeError("%s must be a torch tensor, got %s" % (name, type(t).__name__))
    if ndim is not None and t.dim() != ndim:
        raise ValueError("%s must have %d dims, got shape %s" % (name, ndim, tuple(t.shape)))
    return tuple(t.shape)


def _validate(items):
    """items: (tensor or None, name, shape, dtype) with shape a tuple of ints
    or None (any shape) and dtype None for float16.  Checks every shape,
    dtype and contiguity, then that all tensors sit on one CUDA device."""
    torch = _torch()
    live = []
    for t, name, shape, dtype in items:
        if t is None:
            continue
        if not isinstance(t, torch.Tensor):
            raise TypeError("%s must be a torch tensor, got %s" % (name, type(t).__name__))
        want = torch.float16 if dtype is None else dtype
        if t.dtype != want:
            raise TypeError("%s must be %s, got %s" % (name, want, t.dtype))
        if shape is not None and tuple(t.shape) != tuple(shape):
            raise ValueError("%s must have shape %s, got %s" % (name, tuple(shape), tuple(t.shape)))
        if not t.is_contiguous():
            raise ValueError("%s must be contiguous" % name)
        live.append((t, name))
    dev = None
    for t, name in live:
        if not t.is_cuda:
            raise TypeError("%s must be a device tensor" % name)
        if dev is None:
            dev = t.device
        elif t.device != dev:
            raise ValueError("%s is on %s, the other tensors on %s" % (name, t.device, dev))


def _stream(t):
    torch = _torch()
    return ctypes.c_void_p(torch.cuda.current_stream(t.device).cuda_stream)


def _act(a):
    return ACT[a] if isinstance(a, str) else int(a)


def _empty(shape, like, dtype=None):
    torch = _torch()
    return torch.empty(shape, dtype=like.dtype if dtype is None else dtype, device=like.device)


def _gemm2_shapes(A, W0, b0, W1, b1, out):
    M, K0 = _ndim(A, "A", 2)
    K0w, N0 = _ndim(W0, "W0", 2)
    N0w, N1 = _ndim(W1, "W1", 2)
    if K0w != K0 or N0w != N0:
        raise ValueError("shape mismatch A%s W0%s W1%s" % (tuple(A.shape), tuple(W0.shape), tuple(W1.shape)))
    if out is None:
        _validate([(A, "A", None, None), (W0, "W0", None, None), (b0, "b0", (N0,), None), (W1, "W1", None, None),
                   (b1, "b1", (N1,), None)])
        out = _empty((M, N1), A)
    _validate([(A, "A", None, None), (W0, "W0", None, None), (b0, "b0", (N0,), None), (W1, "W1", None, None),
               (b1, "b1", (N1,), None), (out, "out", (M, N1), None)])
    return M, K0, N0, N1, out


# ------------------------------------------------------------ entry points
def chain_gemm2(A, W0, b0, W1, b1, act="relu", out=None, variant="auto", waves=None, stages=0):
    """D1 [M, N1] = act(A [M,K0] @ W0 [K0,N0] + b0) @ W1 [N0,N1] + b1 (fp16).
    ``waves`` / ``stages`` (explicit variant only, chain_gemm2_ex): tile-owning
    waves per block and row-stream pipeline stages (4 or 2; 0 = 4) of the
    register-resident form."""
    M, K0, N0, N1, out = _gemm2_shapes(A, W0, b0, W1, b1, out)
    v = VARIANT[variant] if isinstance(variant, str) else int(variant)
    if waves is None and not stages:
        _check("chain_gemm2", lib().chain_gemm2_variant(_ptr(A), _ptr(W0), _ptr(b0), _act(act), _ptr(W1), _ptr(b1),
                                                        _ptr(out), M, K0, N0, N1, v, _stream(A)))
    else:
        _check("chain_gemm2_ex", lib().chain_gemm2_ex(_ptr(A), _ptr(W0), _ptr(b0), _act(act), _ptr(W1), _ptr(b1),
                                                      _ptr(out), M, K0, N0, N1, v, int(waves or 0), int(stages),
                                                      _stream(A)))
    return out


_VARIANT_NAME = {v: k for k, v in VARIANT.items()}


def tune_chain_gemm2(A, W0, b0, W1, b1, act="relu", out=None, reps=20):
    """Time every applicable variant of chain_gemm2 on these tensors (blocking),
    cache the fastest for this shape (later variant='auto' calls use it).
    Returns (best variant name, {variant name: us per launch}, out)."""
    M, K0, N0, N1, out = _gemm2_shapes(A, W0, b0, W1, b1, out)
    best = ctypes.c_int(-1)
    us = (ctypes.c_float * 4)()
    _check("chain_gemm2_tune", lib().chain_gemm2_tune(_ptr(A), _ptr(W0), _ptr(b0), _act(act), _ptr(W1), _ptr(b1),
                                                      _ptr(out), M, K0, N0, N1, int(reps), ctypes.byref(best), us,
                                                      _stream(A)))
    times = {_VARIANT_NAME[v]: float(us[v]) for v in (1, 2, 3) if us[v] >= 0}
    return _VARIANT_NAME[best.value], times, out


def tune_chain_gemm2_table(A, W0, b0, W1, b1, act="relu", out=None, reps=20):
    """Time every configuration of chain_gemm2 for these tensors (blocking) and
    cache the fastest.  Returns (best, table, out) where best and the table rows
    are dicts {variant, waves, us}."""
    M, K0, N0, N1, out = _gemm2_shapes(A, W0, b0, W1, b1, out)
    table = (TuneEntry * 16)()
    best = TuneEntry()
    n = _i32(0)
    _check("chain_gemm2_tune_ex", lib().chain_gemm2_tune_ex(_ptr(A), _ptr(W0), _ptr(b0), _act(act), _ptr(W1), _ptr(b1),
                                                            _ptr(out), M, K0, N0, N1, int(reps), table, 16,
                                                            ctypes.byref(n), ctypes.byref(best), _stream(A)))
    return _entry(best, _VARIANT_NAME), [_entry(table[i], _VARIANT_NAME) for i in range(min(n.value, 16))], out


def _entry(e, names):
    return {"variant": names[e.variant], "waves": int(e.waves), "stages": int(e.stages), "us": float(e.us)}


def auto_config(M, K0, N0, N1, act="relu"):
    """{variant, waves, stages} that chain_gemm2(variant='auto') runs for this shape."""
    e = TuneEntry()
    _check("chain_gemm2_auto_config", lib().chain_gemm2_auto_config(int(M), int(K0), int(N0), int(N1), _act(act),
                                                                    ctypes.byref(e)))
    d = _entry(e, _VARIANT_NAME)
    d.pop("us")
    return d


_CONV_VARIANT_NAME = {v: k for k, v in CONV_VARIANT.items()}


def tune_conv_pool(x, w, b, act="relu", pool="max2x2", scale=None, out=None, argmax=None, reps=20):
    """Time every configuration of the pooled conv chain for these tensors
    (blocking) and cache the fastest (chain_conv_pool_tune).  b is the bias,
    or the shift when scale is given.  Returns (best, table, out) with
    dict rows {variant, waves, us}."""
    sh = _conv_shape(x, w)
    P, Q = _conv_out_hw(sh)
    p = POOL[pool] if isinstance(pool, str) else int(pool)
    oshape = (sh.n, P // 2, Q // 2, sh.k)
    am = _argmax_tensor(argmax, oshape, x) if argmax is not True else None
    items = [(x, "x", None, None), (w, "w", None, None), (b, "b" if scale is None else "shift", (sh.k,), None),
             (scale, "scale", (sh.k,), None), (am, "argmax", oshape, _torch().uint8)]
    if out is None:
        _validate(items)
        out = _empty(oshape, x)
    _validate(items + [(out, "out", oshape, None)])
    if argmax is True:
        am = _argmax_tensor(True, oshape, x)
    table = (TuneEntry * 16)()
    best = TuneEntry()
    n = _i32(0)
    _check("chain_conv_pool_tune", lib().chain_conv_pool_tune(_ptr(x), _ptr(w), _ptr(scale), _ptr(b), _act(act), p,
                                                              _ptr(out), ctypes.byref(sh), _ptr(am), int(reps), table,
                                                              16, ctypes.byref(n), ctypes.byref(best), _stream(x)))
    return (_entry(best, _CONV_VARIANT_NAME), [_entry(table[i], _CONV_VARIANT_NAME) for i in range(min(n.value, 16))],
            out)


def conv_auto_config(n, h, w, c, k, act="relu", pool="max2x2", argmax=False):
    """{variant, waves, stages} that the pooled conv chain runs under variant='auto' (stages 0)."""
    e = TuneEntry()
    sh = ConvShape(n, h, w, c, k, 3, 3, 1, 1)
    p = POOL[pool] if isinstance(pool, str) else int(pool)
    _check("chain_conv_pool_auto_config", lib().chain_conv_pool_auto_config(ctypes.byref(sh), _act(act), p,
                                                                            1 if argmax else 0, ctypes.byref(e)))
    d = _entry(e, _CONV_VARIANT_NAME)
    d.pop("us")
    return d


def auto_variant(M, K0, N0, N1, act="relu"):
    """Name of the variant chain_gemm2(variant='auto') runs for this shape."""
    v = ctypes.c_int(-1)
    _check("chain_gemm2_auto_variant", lib().chain_gemm2_auto_variant(int(M), int(K0), int(N0), int(N1), _act(act),
                                                                      ctypes.byref(v)))
    return _VARIANT_NAME[v.value]


def probe_mfma(stamps, sink, waves_per_simd=2, iters=2048):
    """Enqueue the matrix-core rate probe (fc_probe_mfma) on the current
    stream; stamps: int64 [4 * n], sink: float32 [n] with n >= the CU count
    (checked by the library before launching).  Returns the grid
    size (blocks); FLOPs per launch = blocks * 4 * waves_per_simd * iters * 8 * 32768."""
    torch = _torch()
    _validate([(stamps, "stamps", None, torch.int64), (sink, "sink", None, torch.float32)])
    blocks = _i32(0)
    capacity = min(stamps.numel() // 4, sink.numel())
    _check("fc_probe_mfma", lib().fc_probe_mfma(int(waves_per_simd), int(iters), _ptr(stamps), _ptr(sink),
                                                int(capacity), ctypes.byref(blocks), _stream(stamps)))
    return blocks.value


def probe_read(buf, sink):
    """Enqueue the memory read-rate probe (fc_probe_read) over the bytes of the
    contiguous device tensor buf on the current stream; sink: int32 [n] with n
    >= the grid (2 x the CU count for large buffers).  Returns the grid size."""
    torch = _torch()
    _validate([(buf, "buf", None, getattr(buf, "dtype", None)), (sink, "sink", None, torch.int32)])
    blocks = _i32(0)
    _check("fc_probe_read", lib().fc_probe_read(_ptr(buf), buf.numel() * buf.element_size(), _ptr(sink),
                                                int(sink.numel()), ctypes.byref(blocks), _stream(buf)))
    return blocks.value


def tune_clear():
    """Forget every tuned variant choice."""
    lib().fc_tune_clear()


def chain_gemmN(A, Ws, bs, acts, out=None):
    """D = act[n-1](... act[0](A @ Ws[0] + bs[0]) ... @ Ws[n-1] + bs[n-1]) (fp16; n = 3 or 4),
    every intermediate rounded once to fp16 and kept on chip."""
    n = len(Ws)
    if len(bs) != n or len(acts) != n:
        raise ValueError("Ws, bs and acts must have the same length")
    M, K = _ndim(A, "A", 2)
    widths = [K]
    for i, W in enumerate(Ws):
        r, c = _ndim(W, "W%d" % i, 2)
        if r != widths[i]:
            raise ValueError("W%d has %d rows, the previous width is %d" % (i, r, widths[i]))
        widths.append(c)
    items = [(A, "A", None, None)]
    for i in range(n):
        items += [(Ws[i], "W%d" % i, None, None), (bs[i], "b%d" % i, (widths[i + 1],), None)]
    if out is None:
        _validate(items)
        out = _empty((M, widths[-1]), A)
    _validate(items + [(out, "out", (M, widths[-1]), None)])
    Wp = (_vp * n)(*[W.data_ptr() for W in Ws])
    bp = (_vp * n)(*[None if b is None else b.data_ptr() for b in bs])
    ap = (ctypes.c_int * n)(*[_act(a) for a in acts])
    wp = (_i32 * (n + 1))(*widths)
    _check("chain_gemmN", lib().chain_gemmN(_ptr(A), n, Wp, bp, ap, wp, _ptr(out), M, _stream(A)))
    return out


def gemm_bias_act(A, W, b, act="none", out=None):
    """C [M, N] = act(A [M,K] @ W [K,N] + b) (fp16)."""
    M, K = _ndim(A, "A", 2)
    Kw, N = _ndim(W, "W", 2)
    if Kw != K:
        raise ValueError("shape mismatch A%s W%s" % (tuple(A.shape), tuple(W.shape)))
    items = [(A, "A", None, None), (W, "W", None, None), (b, "b", (N,), None)]
    if out is None:
        _validate(items)
        out = _empty((M, N), A)
    _validate(items + [(out, "out", (M, N), None)])
    _check("gemm_bias_act", lib().gemm_bias_act(_ptr(A), _ptr(W), _ptr(b), _act(act), _ptr(out), M, K, N,
                                                _stream(A)))
    return out


def _conv_shape(x, w, stride=1, pad=1):
    n, h, wd, c = _ndim(x, "x", 4)
    r, s, c2, k = _ndim(w, "w", 4)
    if c2 != c:
        raise ValueError("x has %d channels, w expects %d" % (c, c2))
    return ConvShape(n, h, wd, c, k, r, s, stride, pad)


def _conv_out_hw(sh):
    P = (sh.h + 2 * sh.pad - sh.r) // sh.stride + 1
    Q = (sh.w + 2 * sh.pad - sh.s) // sh.stride + 1
    return max(P, 0), max(Q, 0)


def _argmax_tensor(argmax, oshape, like):
    """None/False: no argmax; True: allocate one; else the caller's uint8 tensor."""
    if argmax is True:
        return _empty(oshape, like, _torch().uint8)
    if argmax is None or argmax is False:
        return None
    return argmax


def chain_conv_pool(x, w, b, act="relu", pool="max2x2", out=None, argmax=None, variant="auto", waves=0):
    """y = maxpool2x2(act(conv3x3(x, w) + b)) (or act(conv+b) with pool='none').
    ``argmax``: None, True (allocate) or a uint8 tensor; returns y or (y, argmax).
    ``variant``: kernel form ("auto", "lds_weights", "reg_weights"); ``waves``:
    tile-owning waves per block of the pooled "lds_weights" form (0 = 8)."""
    return _conv_pool("chain_conv_pool", x, w, None, b, act, pool, out, argmax, variant, waves)


def chain_conv_bn_pool(x, w, scale, shift, act="relu", pool="max2x2", out=None, argmax=None, variant="auto",
                       waves=0):
    """y = maxpool2x2(act(conv3x3(x, w) * scale + shift)) per output channel (batch
    norm at inference as a scale and a shift); pool='none' stores act(...)."""
    if scale is None:
        raise ValueError("scale is required")
    return _conv_pool("chain_conv_bn_pool", x, w, scale, shift, act, pool, out, argmax, variant, waves)


def _conv_pool(fn, x, w, scale, b, act, pool, out, argmax, variant="auto", waves=0):
    sh = _conv_shape(x, w)
    P, Q = _conv_out_hw(sh)
    p = POOL[pool] if isinstance(pool, str) else int(pool)
    v = CONV_VARIANT[variant] if isinstance(variant, str) else int(variant)
    oshape = (sh.n, P // 2, Q // 2, sh.k) if p else (sh.n, P, Q, sh.k)
    am = _argmax_tensor(argmax, oshape, x) if argmax is not True else None   # the caller's, checked below
    items = [(x, "x", None, None), (w, "w", None, None), (b, "b" if scale is None else "shift", (sh.k,), None),
             (scale, "scale", (sh.k,), None), (am, "argmax", oshape, _torch().uint8)]
    if out is None:
        _validate(items)
        out = _empty(oshape, x)
    _validate(items + [(out, "out", oshape, None)])
    if argmax is True:
        am = _argmax_tensor(True, oshape, x)
    st = lib().chain_conv_pool_ex(_ptr(x), _ptr(w), _ptr(scale), _ptr(b), _act(act), p, _ptr(out), ctypes.byref(sh),
                                  _ptr(am), v, int(waves), _stream(x))
    _check(fn, st)
    return (out, am) if am is not None else out


def winograd_weights(w, out=None):
    """U = G g G^T of a 3x3 HWIO weight w [3, 3, c, k] for chain_conv_pool_winograd,
    in the library's operand layout, returned as a [16, c/8, k, 8] fp16 tensor."""
    r, s, c, k = _ndim(w, "w", 4)
    if (r, s) != (3, 3):
        raise ValueError("w must be [3, 3, c, k], got %s" % ((r, s, c, k),))
    if c % 8 or k % 8:
        raise ValueError("c=%d and k=%d must be multiples of 8" % (c, k))
    oshape = (16, c // 8, k, 8)
    if out is None:
        _validate([(w, "w", None, None)])
        out = _empty(oshape, w)
    _validate([(w, "w", None, None), (out, "out", oshape, None)])
    _check("winograd_weights", lib().winograd_weights(_ptr(w), _ptr(out), c, k, _stream(w)))
    return out


def chain_conv_pool_winograd(x, U, b, act="relu", pool="max2x2", out=None, argmax=None):
    """y = pool2x2(act(conv3x3(x, w) + b)) with the conv by Winograd F(2x2, 3x3)
    from U = winograd_weights(w).  ``argmax`` as for chain_conv_pool (max pool)."""
    n, h, wd, c = _ndim(x, "x", 4)
    ushape = _ndim(U, "U", 4)
    if ushape[0] != 16 or ushape[1] != c // 8 or ushape[3] != 8 or c % 8:
        raise ValueError("U must be [16, %d, k, 8] (winograd_weights of a [3, 3, %d, k] weight), got %s"
                         % (c // 8, c, ushape))
    k = ushape[2]
    sh = ConvShape(n, h, wd, c, k, 3, 3, 1, 1)
    p = POOL[pool] if isinstance(pool, str) else int(pool)
    oshape = (n, h // 2, wd // 2, k)
    am = _argmax_tensor(argmax, oshape, x) if argmax is not True else None
    items = [(x, "x", None, None), (U, "U", None, None), (b, "b", (k,), None),
             (am, "argmax", oshape, _torch().uint8)]
    if out is None:
        _validate(items)
        out = _empty(oshape, x)
    _validate(items + [(out, "out", oshape, None)])
    if argmax is True:
        am = _argmax_tensor(True, oshape, x)
    st = lib().chain_conv_pool_winograd(_ptr(x), _ptr(U), _ptr(b), _act(act), p, _ptr(out), ctypes.byref(sh),
                                        _ptr(am), _stream(x))
    _check("chain_conv_pool_winograd", st)
    return (out, am) if am is not None else out


def conv_bias_act(x, w, b, act="relu", out=None):
    """y NHWC = act(conv3x3(x, w) + b)."""
    sh = _conv_shape(x, w)
    P, Q = _conv_out_hw(sh)
    items = [(x, "x", None, None), (w, "w", None, None), (b, "b", (sh.k,), None)]
    if out is None:
        _validate(items)
        out = _empty((sh.n, P, Q, sh.k), x)
    _validate(items + [(out, "out", (sh.n, P, Q, sh.k), None)])
    _check("conv_bias_act", lib().conv_bias_act(_ptr(x), _ptr(w), _ptr(b), _act(act), _ptr(out), ctypes.byref(sh),
                                                _stream(x)))
    return out


def _w1x1(t, name, kin):
    """A 1x1 conv weight: [kin, kout] or [1, 1, kin, kout]; returns kout."""
    shp = _ndim(t, name, None)
    if len(shp) == 2 and shp[0] == kin:
        return shp[1]
    if len(shp) == 4 and shp[:3] == (1, 1, kin):
        return shp[3]
    raise ValueError("%s must be [%d, k] or [1, 1, %d, k], got %s" % (name, kin, kin, shp))


def _conv2_prep(x, w0, b0, w1, b1, out):
    sh = _conv_shape(x, w0)
    P, Q = _conv_out_hw(sh)
    k1 = _w1x1(w1, "w1", sh.k)
    items = [(x, "x", None, None), (w0, "w0", None, None), (b0, "b0", (sh.k,), None), (w1, "w1", None, None),
             (b1, "b1", (k1,), None)]
    if out is None:
        _validate(items)
        out = _empty((sh.n, P, Q, k1), x)
    _validate(items + [(out, "out", (sh.n, P, Q, k1), None)])
    return sh, k1, out


def chain_conv2(x, w0, b0, w1, b1, act="relu", out=None, waves=0, stages=0, variant="auto"):
    """y = conv1x1(act(conv3x3(x, w0) + b0), w1) + b1; w1 is [k0, k1] or [1,1,k0,k1].
    ``variant``: kernel form ("auto", "rf" or "pipe"); for "rf", ``waves``:
    tile-owning waves per block (1..8) and ``stages``: row-stream pipeline
    stages (4 or 2; 0 = 4).  waves > 0 with variant "auto" means "rf"."""
    sh, k1, out = _conv2_prep(x, w0, b0, w1, b1, out)
    v = VARIANT[variant] if isinstance(variant, str) else int(variant)
    if v == 0 and waves:
        v = VARIANT["rf"]
    _check("chain_conv2", lib().chain_conv2_variant(_ptr(x), _ptr(w0), _ptr(b0), _act(act), _ptr(w1), _ptr(b1), k1,
                                                    _ptr(out), ctypes.byref(sh), v, int(waves), int(stages),
                                                    _stream(x)))
    return out


def tune_chain_conv2(x, w0, b0, w1, b1, act="relu", out=None, reps=20):
    """Time every block shape of the conv3x3 -> conv1x1 chain for these tensors
    (blocking) and cache the fastest (chain_conv2_tune).  Returns (best, table,
    out) with dict rows {variant, waves, us}."""
    sh, k1, out = _conv2_prep(x, w0, b0, w1, b1, out)
    table = (TuneEntry * 16)()
    best = TuneEntry()
    n = _i32(0)
    _check("chain_conv2_tune", lib().chain_conv2_tune(_ptr(x), _ptr(w0), _ptr(b0), _act(act), _ptr(w1), _ptr(b1), k1,
                                                      _ptr(out), ctypes.byref(sh), int(reps), table, 16,
                                                      ctypes.byref(n), ctypes.byref(best), _stream(x)))
    return _entry(best, _VARIANT_NAME), [_entry(table[i], _VARIANT_NAME) for i in range(min(n.value, 16))], out


def conv2_auto_config(n, h, w, c, k0, k1, act="relu"):
    """{variant, waves, stages} that chain_conv2 runs for this shape (waves=0)."""
    e = TuneEntry()
    sh = ConvShape(n, h, w, c, k0, 3, 3, 1, 1)
    _check("chain_conv2_auto_config", lib().chain_conv2_auto_config(ctypes.byref(sh), int(k1), _act(act),
                                                                    ctypes.byref(e)))
    d = _entry(e, _VARIANT_NAME)
    d.pop("us")
    return d


def convN_auto_variant(n, h, w, c, ks):
    """The kernel form ("pipe" or "rf") chain_convN runs for x [n,h,w,c] and
    stage widths ks (host only)."""
    sh = ConvShape(n, h, w, c, ks[0], 3, 3, 1, 1)
    kp = (_i32 * len(ks))(*ks)
    v = ctypes.c_int(-1)
    _check("chain_convN_auto_variant", lib().chain_convN_auto_variant(ctypes.byref(sh), len(ks), kp, ctypes.byref(v)))
    return _VARIANT_NAME[v.value]


def _convN_prep(x, ws, bs, acts, out):
    n = len(ws)
    if len(bs) != n or len(acts) != n:
        raise ValueError("ws, bs and acts must have the same length")
    sh = _conv_shape(x, ws[0])
    P, Q = _conv_out_hw(sh)
    ks = [sh.k]
    for i in range(1, n):
        ks.append(_w1x1(ws[i], "w%d" % i, ks[-1]))
    items = [(x, "x", None, None)]
    for i in range(n):
        items += [(ws[i], "w%d" % i, None, None), (bs[i], "b%d" % i, (ks[i],), None)]
    if out is None:
        _validate(items)
        out = _empty((sh.n, P, Q, ks[-1]), x)
    _validate(items + [(out, "out", (sh.n, P, Q, ks[-1]), None)])
    wp = (_vp * n)(*[w.data_ptr() for w in ws])
    bp = (_vp * n)(*[None if b is None else b.data_ptr() for b in bs])
    ap = (ctypes.c_int * n)(*[_act(a) for a in acts])
    kp = (_i32 * n)(*ks)
    return sh, n, wp, bp, ap, kp, out


def chain_convN(x, ws, bs, acts, out=None, variant="auto"):
    """y = stage_{n-1}(... stage_0(x)): stage 0 = act[0](conv3x3(x, ws[0]) + bs[0]),
    stage i > 0 = act[i](1x1 conv with ws[i] [k_{i-1}, k_i] (or [1,1,k_{i-1},k_i]) + bs[i]);
    n = 3 or 4, every intermediate rounded once to fp16 and kept on chip.
    ``variant``: kernel form ("auto", "rf" or "pipe")."""
    sh, n, wp, bp, ap, kp, out = _convN_prep(x, ws, bs, acts, out)
    v = VARIANT[variant] if isinstance(variant, str) else int(variant)
    _check("chain_convN", lib().chain_convN_variant(_ptr(x), ctypes.byref(sh), n, wp, bp, ap, kp, _ptr(out), v,
                                                    _stream(x)))
    return out


def tune_chain_convN(x, ws, bs, acts, out=None, reps=20):
    """Time each kernel form of the N-stage conv chain for these tensors
    (blocking) and cache the fastest (chain_convN_tune).  Returns (best,
    table, out) with dict rows {variant, waves, stages, us}."""
    sh, n, wp, bp, ap, kp, out = _convN_prep(x, ws, bs, acts, out)
    table = (TuneEntry * 4)()
    best = TuneEntry()
    cnt = _i32(0)
    _check("chain_convN_tune", lib().chain_convN_tune(_ptr(x), ctypes.byref(sh), n, wp, bp, ap, kp, _ptr(out),
                                                      int(reps), table, 4, ctypes.byref(cnt), ctypes.byref(best),
                                                      _stream(x)))
    return _entry(best, _VARIANT_NAME), [_entry(table[i], _VARIANT_NAME) for i in range(min(cnt.value, 4))], out


def avgpool2x2(x, out=None):
    """y [n, h/2, w/2, c] = 2x2/2 average pool of NHWC x (fp16 mean of each window)."""
    n, h, w, c = _ndim(x, "x", 4)
    oshape = (n, h // 2, w // 2, c)
    if out is None:
        _validate([(x, "x", None, None)])
        out = _empty(oshape, x)
    _validate([(x, "x", None, None), (out, "out", oshape, None)])
    _check("avgpool2x2", lib().avgpool2x2(_ptr(x), _ptr(out), n, h, w, c, _stream(x)))
    return out


def maxpool2x2(x, out=None, argmax=None):
    """y [n, h/2, w/2, c] = 2x2/2 max pool of NHWC x (+ optional argmax)."""
    n, h, w, c = _ndim(x, "x", 4)
    oshape = (n, h // 2, w // 2, c)
    am = _argmax_tensor(argmax, oshape, x) if argmax is not True else None   # the caller's, checked below
    items = [(x, "x", None, None), (am, "argmax", oshape, _torch().uint8)]
    if out is None:
        _validate(items)
        out = _empty(oshape, x)
    _validate(items + [(out, "out", oshape, None)])
    if argmax is True:
        am = _argmax_tensor(True, oshape, x)
    _check("maxpool2x2", lib().maxpool2x2(_ptr(x), _ptr(out), _ptr(am), n, h, w, c, _stream(x)))
    return (out, am) if am is not None else out


def pad_channels(x, c_out):
    """Zero-pad the channels (last dim) of NHWC x to c_out."""
    _ndim(x, "x", None)
    _validate([(x, "x", None, None)])
    c_in = x.shape[-1]
    out = _torch().empty(tuple(x.shape[:-1]) + (c_out,), dtype=x.dtype, device=x.device)
    _check("pad_channels", lib().pad_channels(_ptr(x), _ptr(out), x.numel() // max(c_in, 1), c_in, c_out, 1,
                                              _stream(x)))
    return out


def pad_weight_channels(w, c_out):
    """Zero-pad the input channels of HWIO w [r,s,c,k] to c_out."""
    _ndim(w, "w", 4)
    _validate([(w, "w", None, None)])
    r, s, c_in, k = w.shape
    out = _torch().empty((r, s, c_out, k), dtype=w.dtype, device=w.device)
    _check("pad_channels", lib().pad_channels(_ptr(w), _ptr(out), r * s, c_in, c_out, k, _stream(w)))
    return out


# ---------------------------------------- attention over a paged 8-bit cache
# These calls are made for every layer of every step, so their checks are few
# and plain: a launch of 3 us should not wait for 10 us of checking.
_STRIDES = {n: _i64 * n for n in (2, 4, 6)}


_CODES = {}   # torch dtype -> fc_dtype


def _rows(t, name, dtype=None):
    """t [tokens, heads, d] of a 16-bit float type, elements of a head adjacent;
    token and head strides are free.  Returns its fc_dtype."""
    if not _CODES:
        torch = _torch()
        _CODES.update({torch.float16: 0, torch.bfloat16: 1})
    code = _CODES.get(getattr(t, "dtype", None))
    if code is None:
        raise TypeError("%s must be a torch tensor of float16 or bfloat16, got %s"
                        % (name, getattr(t, "dtype", type(t).__name__)))
    if dtype is not None and code != dtype:
        raise TypeError("%s is %s, unlike the other activations" % (name, t.dtype))
    if t.dim() != 3:
        raise ValueError("%s must be [tokens, heads, d], got shape %s" % (name, tuple(t.shape)))
    if t.stride(2) != 1 and t.shape[2] > 1:
        raise ValueError("the elements of a head of %s must be adjacent" % name)
    return code


def _exact(t, name, shape, dtype):
    """t is a contiguous torch tensor of this shape and type."""
    if getattr(t, "dtype", None) is not dtype:
        raise TypeError("%s must be a torch tensor of %s, got %s" % (name, dtype, getattr(t, "dtype", type(t).__name__)))
    if t.shape != shape or not t.is_contiguous():
        raise ValueError("%s must be contiguous with shape %s, got %s" % (name, tuple(shape), tuple(t.shape)))


def _dense(table):
    """table, or a copy of it if it is a slice of a wider one: a row ends where the
    slice ends, which the C entry points cannot be told apart from a row's stride."""
    if isinstance(table, _torch().Tensor) and not table.is_contiguous():
        return table.contiguous()
    return table


def _one_device(dev, tensors):
    """Every tensor (None: absent) sits on device `dev`."""
    if dev < 0:
        raise TypeError("the activations must be device tensors")
    for t in tensors:
        if t is not None and t.get_device() != dev:
            if t.is_cuda:
                raise ValueError("a tensor of shape %s is on %s, the activations on device %d" % (tuple(t.shape), t.device, dev))
            raise TypeError("a tensor of shape %s is no device tensor, the activations are" % (tuple(t.shape),))


def _raw_stream(dev):
    """torch's current stream of device `dev`."""
    return _torch()._C._cuda_getCurrentRawStream(dev)


def _call(dev, f, *args):
    """f(*args) with device `dev`, whose stream the call names, as the current one."""
    torch = _torch()
    if torch._C._cuda_getDevice() == dev:
        return f(*args)
    with torch.cuda.device(dev):
        return f(*args)


def _addr(t):
    return None if t is None else t.data_ptr()


def rope_turns(rot, base=10000.0, scaling=None, factor=1.0, original=None, low=1.0, high=None, device=None):
    """(turns, mscale) of a rotary table: turns int64 [rot / 2], pair i's turns a
    position as 64-bit fractions (2^64 = one turn).  Without scaling pair i's
    frequency is f_i = base^(-2 i / rot) radians a position.  scaling, for
    contexts ``factor`` times as long as trained on:

    * "linear"       f_i / factor;
    * "base"         base raised to base * factor^(rot / (rot - 2)), which leaves the
                     first pair as it is and stretches the last by factor;
    * "wavelength"   pairs that turn at least ``high`` (4 by default) times within
                     ``original`` positions stay, those that turn at most ``low``
                     times are divided by factor, those between blend linearly in
                     their number of turns;
    * "ramp"         the same with the blend linear in the pair's index (between
                     the indices where ``high``, 32 by default, and ``low`` turns
                     are reached), and mscale = 0.1 ln(factor) + 1.

    The last two are the by-parts interpolation of Peng et al., "YaRN: efficient
    context window extension of large language models" (2023), in the forms that
    models are trained with.
    """
    torch = _torch()
    if rot <= 0 or rot % 16:
        raise ValueError("rot must be a positive multiple of 16, got %r" % (rot,))
    if not base > 1.0 or not factor >= 1.0:
        raise ValueError("base > 1 and factor >= 1 required")
    i = torch.arange(rot // 2, dtype=torch.float64)
    mscale = 1.0
    if scaling == "base":
        base = base * factor ** (rot / (rot - 2))
    f = base ** (-2.0 * i / rot)
    if scaling == "linear":
        f = f / factor
    elif scaling in ("wavelength", "ramp"):
        high = (32.0 if scaling == "ramp" else 4.0) if high is None else high
        if not original or original <= 0 or not high > low:
            raise ValueError("scaling %r needs original > 0 and high > low" % scaling)
        if scaling == "wavelength":
            keep = ((original * f / (2 * math.pi) - low) / (high - low)).clamp(0.0, 1.0)
        else:
            def index(turns):
                return rot * math.log(original / (turns * 2 * math.pi)) / (2 * math.log(base))
            first = max(math.floor(index(high)), 0)
            last = min(math.ceil(index(low)), rot - 1)
            keep = 1.0 - ((i - first) / max(last - first, 1e-3)).clamp(0.0, 1.0)
            mscale = 0.1 * math.log(factor) + 1.0
        f = f * keep + f / factor * (1.0 - keep)
    elif scaling not in (None, "base"):
        raise ValueError("unknown scaling %r" % (scaling,))
    turns = torch.round(f / (2 * math.pi) * 2.0 ** 64).to(torch.int64)
    return (turns if device is None else turns.to(device)), mscale


def _table(turns, interleaved, mscale):
    torch = _torch()
    if turns is None:
        return None
    if not isinstance(turns, torch.Tensor) or turns.dtype is not torch.int64:
        raise TypeError("turns must be a tensor of torch.int64")
    if turns.dim() != 1 or not turns.is_contiguous():
        raise ValueError("turns must be contiguous with one dim, got shape %s" % (tuple(turns.shape),))
    return RopeTable(turns.data_ptr(), 2 * turns.shape[0], 1 if interleaved else 0, mscale)


def rope(x, positions, turns, interleaved=False, mscale=1.0, inverse=False, out=None):
    """x [tokens, heads, d] with the first 2 * len(turns) elements of each head
    turned by its token's position (``positions`` int32 [tokens]): the pairs (i, i +
    rot / 2), or (2 i, 2 i + 1) if ``interleaved``.  ``inverse`` turns back, which is
    also the gradient.  ``out`` may be x itself."""
    dt = _rows(x, "x")
    T, H, D = shape = x.shape
    table = _table(turns, interleaved, mscale)
    if table is None:
        raise ValueError("turns is required")
    _exact(positions, "positions", (T,), _torch().int32)
    if out is not None:
        _rows(out, "out", dt)
        if out.shape != shape:
            raise ValueError("out must have shape %s, got %s" % (tuple(shape), tuple(out.shape)))
    dev = x.get_device()
    _one_device(dev, (positions, turns, out))
    if out is None:
        out = x.new_empty(shape)
    st = _STRIDES[4](x.stride(0), x.stride(1), out.stride(0), out.stride(1))
    s = lib().rope_apply(x.data_ptr(), out.data_ptr(), st, positions.data_ptr(), table, 1 if inverse else 0, dt, T, H, D,
                         _raw_stream(dev))
    if s:
        _check("rope", s)
    return out


def kv_cache(pages, hkv, page, d, device="cuda"):
    """An empty pool: (codes uint8 [pages, hkv, 2, page / 16, 16 d], scales float32
    [pages, hkv, 2]).  Its pages need no clearing between sequences."""
    torch = _torch()
    if page % 16:
        raise ValueError("page must be a multiple of 16, got %d" % page)
    return (torch.zeros((pages, hkv, 2, page // 16, 16 * d), dtype=torch.uint8, device=device),
            torch.ones((pages, hkv, 2), dtype=torch.float32, device=device))


def _kv_shape(dt, tokens, hq, hkv, d, codes, scales, table, cu_q, kv_lens, max_q, max_kv):
    """Checks the cache's and the batch's tensors against each other."""
    torch = _torch()
    if len(_ndim(codes, "codes", 5)) == 5:
        _exact(codes, "codes", codes.shape, torch.uint8)
    P, H, two, n, w = codes.shape
    if H != hkv or two != 2 or w != 16 * d:
        raise ValueError("codes must have shape (pages, %d, 2, page / 16, %d), got %s" % (hkv, 16 * d, tuple(codes.shape)))
    B, stride = shape = _ndim(table, "table", 2)
    i32 = torch.int32
    _exact(scales, "scales", (P, H, 2), torch.float32)
    _exact(table, "table", shape, i32)
    _exact(cu_q, "cu_q", (B + 1,), i32)
    _exact(kv_lens, "kv_lens", (B,), i32)
    page = 16 * n
    return KvShape(dt, B, hq, hkv, d, page, P, stride, tokens, tokens if max_q is None else int(max_q),
                   min(stride * page, 0x7fffffff) if max_kv is None else int(max_kv))


def kv_append(k, v, codes, scales, table, cu_q, kv_lens, turns=None, interleaved=False, mscale=1.0, positions=None,
              q=None, q_out=None, max_q=None):
    """Append k, v [tokens, hkv, d] to the paged cache (codes, scales), k turned by
    the rotary table ``turns`` on the way (None: as it is).  Sequence b's new tokens
    are rows cu_q[b]:cu_q[b+1] and the last of its kv_lens[b] tokens; slot s is in
    page table[b, s // page] (a table that is a slice of a wider one is copied, one
    small launch).  ``positions`` (int32 [tokens]) turn instead of the slots.
    With ``q`` [tokens, hq, d] the same launch returns q turned alike (``q_out``).
    ``max_q``: a bound of the new tokens of a sequence; it sizes the launch."""
    dt = _rows(k, "k")
    _rows(v, "v", dt)
    T, hkv, d = k.shape
    if v.shape != k.shape:
        raise ValueError("v must have k's shape %s, got %s" % (tuple(k.shape), tuple(v.shape)))
    hq, qs = hkv, (0, 0)
    if q is not None:
        _rows(q, "q", dt)
        Tq, hq, dq = q.shape
        if Tq != T or dq != d:
            raise ValueError("q must have shape (%d, hq, %d), got %s" % (T, d, tuple(q.shape)))
        qs = q.stride()
        if q_out is not None:
            _exact(q_out, "q_out", q.shape, q.dtype)
    elif q_out is not None:
        raise ValueError("q_out needs q")
    table = _dense(table)
    sh = _kv_shape(dt, T, hq, hkv, d, codes, scales, table, cu_q, kv_lens, max_q, None)
    rt = _table(turns, interleaved, mscale)
    if positions is not None:
        _exact(positions, "positions", (T,), _torch().int32)
    dev = k.get_device()
    _one_device(dev, (v, q, q_out, codes, scales, table, cu_q, kv_lens, positions, turns))
    if q is not None and q_out is None:
        q_out = q.new_empty(q.shape)
    st = _STRIDES[6](k.stride(0), k.stride(1), v.stride(0), v.stride(1), qs[0], qs[1])
    s = lib().kv_append(k.data_ptr(), v.data_ptr(), _addr(q), _addr(q_out), st, codes.data_ptr(), scales.data_ptr(),
                        table.data_ptr(), cu_q.data_ptr(), kv_lens.data_ptr(), _addr(positions), rt, sh, _raw_stream(dev))
    if s:
        _check("kv_append", s)
    return q_out


def kv_check(table, cu_q, kv_lens, pages, page, tokens=None, writes=False):
    """Look HOST copies (int32 tensors) of a batch's table, cu_q and kv_lens over:
    raises FusedChainError at the first fault (an id outside the pool, a length the
    table cannot hold, ...; with ``writes`` also a page to be written that two
    sequences name).  On the device such faults give NaN rows."""
    torch = _torch()
    B, stride = _ndim(table, "table", 2)
    table = _dense(table)
    for t, name, shape in ((table, "table", (B, stride)), (cu_q, "cu_q", (B + 1,)), (kv_lens, "kv_lens", (B,))):
        if not isinstance(t, torch.Tensor) or t.dtype is not torch.int32 or t.is_cuda:
            raise TypeError("%s must be a host tensor of torch.int32" % name)
        if tuple(t.shape) != shape or not t.is_contiguous():
            raise ValueError("%s must be contiguous with shape %s, got %s" % (name, shape, tuple(t.shape)))
    n = int(cu_q[-1]) if tokens is None else int(tokens)
    sh = KvShape(0, B, 1, 1, 64, int(page), int(pages), stride, max(n, 0), 0, 0)
    _check("kv_check", lib().kv_check(_ptr(table), _ptr(cu_q), _ptr(kv_lens), sh, 1 if writes else 0))


def _attn_params(d, scale, causal, softcap, window, variant, splits):
    v = ATTN_VARIANT[variant] if isinstance(variant, str) else int(variant)
    window = max(-1, min(int(window), 0x7fffffff))   # (ctypes would keep the low 32 bits)
    return AttnParams(d ** -0.5 if scale is None else scale, softcap, 1 if causal else 0, window, v, int(splits))


_ATTN_VARIANT_NAME = {v: k for k, v in ATTN_VARIANT.items()}


def attn_plan(tokens, batch, hq, hkv, d, page, table_stride, max_q, max_kv, dtype="bfloat16", causal=True, window=0,
              variant="auto", splits=0, tree=False):
    """{variant, splits, chunk, workspace}: the kernel form chain_attn runs, the blocks
    a sequence's keys are split over, keys a block, workspace bytes (host only);
    ``tree``: of a call with a tree."""
    sh = KvShape(DTYPE[dtype], batch, hq, hkv, d, page, 1, table_stride, tokens, max_q, max_kv)
    plan = AttnPlan()
    f = lib().chain_attn_tree_plan if tree else lib().chain_attn_plan
    _check("chain_attn_plan", f(sh, _attn_params(d, None, causal, 0.0, window, variant, splits), plan))
    return {"variant": _ATTN_VARIANT_NAME[plan.variant], "splits": int(plan.splits), "chunk": int(plan.chunk),
            "workspace": int(plan.workspace)}


def _tree(tree, tokens):
    """(fc_tree, bits, positions) of the pair that ``tree_plan`` returns."""
    torch = _torch()
    if tree is None:
        return None, None, None
    if not isinstance(tree, (tuple, list)) or len(tree) != 2:
        raise TypeError("tree must be the pair (bits, positions), got %s" % type(tree).__name__)
    bits, positions = tree
    words = _ndim(bits, "the tree's bits", 2)[1]
    _exact(bits, "the tree's bits", (tokens, words), torch.int64)
    _exact(positions, "the tree's positions", (tokens,), torch.int32)
    return Tree(bits.data_ptr(), positions.data_ptr(), words), bits, positions


def chain_attn(q, codes, scales, table, cu_q, kv_lens, scale=None, causal=True, softcap=0.0, window=0, slopes=None,
               max_q=None, max_kv=None, out=None, lse=None, workspace=None, variant="auto", splits=0, tree=None):
    """out [tokens, hq, d] = softmax(scale * q K^T) V over the paged cache: queries
    cu_q[b]:cu_q[b+1] are the last of sequence b's kv_lens[b] tokens and, if ``causal``,
    see the slots up to their own (the last ``window`` of them if window > 0).
    ``scale``: 1 / sqrt(d) by default; ``softcap`` > 0: scores become softcap *
    tanh(score / softcap); ``slopes`` (float32 [hq]): minus slope * distance.  A row that
    sees no key is 0.  ``lse``: None, True (allocate) or a float32 [tokens, hq] tensor;
    returns out or (out, lse).  ``max_q``, ``max_kv``: bounds of the new tokens and lengths
    (they size the launch; give ``max_q`` for steps: None takes all the tokens for one
    sequence's, and 64 single queries over 8192 keys take 290 us rather than 127);
    ``workspace``: uint8 device memory of attn_plan's size
    (allocated if None); ``variant``, ``splits``: kernel form and split, by rule if not given.
    ``tree``: the new tokens are nodes of a tree of drafts, (bits, positions) as ``tree_plan``
    returns them: a node sees every slot before its sequence's first node and the nodes of
    its bits; ``window`` and ``slopes`` go by the positions."""
    torch = _torch()
    dt = _rows(q, "q")
    T, hq, d = shape = q.shape
    hkv = _ndim(codes, "codes", 5)[1]
    table = _dense(table)
    sh = _kv_shape(dt, T, hq, hkv, d, codes, scales, table, cu_q, kv_lens, max_q, max_kv)
    pa = _attn_params(d, scale, causal, softcap, window, variant, splits)
    tr, bits, positions = _tree(tree, T)
    if slopes is not None:
        _exact(slopes, "slopes", (hq,), torch.float32)
    if out is not None:
        _exact(out, "out", shape, q.dtype)
    le = None if lse is True or lse is False else lse
    if le is not None:
        _exact(le, "lse", (T, hq), torch.float32)
    if workspace is not None and (workspace.dtype is not torch.uint8 or not workspace.is_contiguous()):
        raise TypeError("workspace must be contiguous torch.uint8")
    dev = q.get_device()
    _one_device(dev, (codes, scales, table, cu_q, kv_lens, slopes, out, le, workspace, bits, positions))
    L = lib()
    plan = AttnPlan()
    s = (L.chain_attn_plan if tr is None else L.chain_attn_tree_plan)(sh, pa, plan)
    if s:
        _check("chain_attn", s)
    if out is None:
        out = q.new_empty(shape)
    if lse is True:
        le = torch.empty((T, hq), dtype=torch.float32, device=q.device)
    room = plan.workspace
    if workspace is not None:
        room = workspace.numel()
    elif room:
        workspace = torch.empty(room, dtype=torch.uint8, device=q.device)
    st = _STRIDES[2](q.stride(0), q.stride(1))
    if tr is None:
        s = _call(dev, L.chain_attn, q.data_ptr(), st, codes.data_ptr(), scales.data_ptr(), table.data_ptr(), cu_q.data_ptr(),
                  kv_lens.data_ptr(), _addr(slopes), pa, out.data_ptr(), _addr(le), sh, _addr(workspace), room,
                  _raw_stream(dev))
    else:
        s = _call(dev, L.chain_attn_tree, q.data_ptr(), st, codes.data_ptr(), scales.data_ptr(), table.data_ptr(),
                  cu_q.data_ptr(), kv_lens.data_ptr(), tr, _addr(slopes), pa, out.data_ptr(), _addr(le), sh,
                  _addr(workspace), room, _raw_stream(dev))
    if s:
        _check("chain_attn", s)
    return (out, le) if le is not None else out


# -------------------------------------------------- trees of drafted tokens
def _indices(tensors, shape):
    for t, name in tensors:
        _exact(t, name, shape, _torch().int32)


def _bound(max_q, tokens):
    """A bound of the nodes of a tree that a row of bits or of kept nodes holds."""
    n = tokens if max_q is None else int(max_q)
    if n > 4096:
        if max_q is not None:
            raise ValueError("max_q must be at most 4096, got %d" % n)
        n = 4096
    return max(n, 1)


def tree_plan(parents, cu_q, kv_lens, max_q=None):
    """(bits int64 [tokens, ceil(max_q / 64)], positions int32 [tokens]) of trees of new
    tokens, for ``chain_attn(tree=...)`` and ``kv_append(positions=...)``: once a step, for all
    layers.  ``parents`` (int32 [tokens]): each token's parent among its sequence's new ones,
    an earlier one, or -1.  A token sees its ancestors and itself, and sits its depth past
    what the sequence held before.  ``max_q``: a bound of the new tokens of a sequence, at
    most 4096 (sequences past it get NaN rows)."""
    torch = _torch()
    T, = _ndim(parents, "parents", 1)
    B, = _ndim(kv_lens, "kv_lens", 1)
    _indices(((parents, "parents"),), (T,))
    _indices(((kv_lens, "kv_lens"),), (B,))
    _indices(((cu_q, "cu_q"),), (B + 1,))
    words = -(-_bound(max_q, T) // 64)
    dev = parents.get_device()
    _one_device(dev, (cu_q, kv_lens))
    bits = parents.new_empty((T, words), dtype=torch.int64)
    positions = torch.empty_like(parents)
    s = _call(dev, lib().tree_plan, parents.data_ptr(), cu_q.data_ptr(), kv_lens.data_ptr(), B, T, words, bits.data_ptr(),
              positions.data_ptr(), _raw_stream(dev))
    if s:
        _check("tree_plan", s)
    return bits, positions


def tree_accept(parents, drafted, targets, cu_q, kv_lens, max_q=None):
    """(keep [batch, max_q], kept [batch], next [batch], lens [batch]), all int32: each tree
    walked from node 0, the token that the last step decided, to the first child whose
    ``drafted`` token is the one that ``targets`` holds for the present node (the model's own
    choice there, of ``sample_tokens``), until there is none or that target is under 0 (its mark
    of a row it cannot draw from).  ``keep``: the nodes passed, rising,
    -1 behind them; ``kept``: how many; ``next``: the target of the last; ``lens``: the
    sequence's length with them."""
    T, = _ndim(parents, "parents", 1)
    B, = _ndim(kv_lens, "kv_lens", 1)
    _indices(((parents, "parents"), (drafted, "drafted"), (targets, "targets")), (T,))
    _indices(((kv_lens, "kv_lens"),), (B,))
    _indices(((cu_q, "cu_q"),), (B + 1,))
    most = _bound(max_q, T)
    dev = parents.get_device()
    _one_device(dev, (drafted, targets, cu_q, kv_lens))
    keep = parents.new_empty((B, most))
    kept, nxt, lens = parents.new_empty((3, B)).unbind()
    s = _call(dev, lib().tree_accept, parents.data_ptr(), drafted.data_ptr(), targets.data_ptr(), cu_q.data_ptr(),
              kv_lens.data_ptr(), B, T, most, keep.data_ptr(), kept.data_ptr(), nxt.data_ptr(), lens.data_ptr(),
              _raw_stream(dev))
    if s:
        _check("tree_accept", s)
    return keep, kept, nxt, lens


def _pool(codes, scales):
    """(layers, pages, hkv, page, d) of a pool, one layer's or [layers, ...] of several."""
    torch = _torch()
    shape = _ndim(codes, "codes", None)
    if len(shape) not in (5, 6):
        raise ValueError("codes must have 5 dims, or 6 with layers, got shape %s" % (shape,))
    _exact(codes, "codes", codes.shape, torch.uint8)
    L = shape[0] if len(shape) == 6 else 1
    P, H, two, n, w = shape[-5:]
    if two != 2 or w % 16:
        raise ValueError("codes must have shape ([layers,] pages, hkv, 2, page / 16, 16 d), got %s" % (shape,))
    _exact(scales, "scales", codes.shape[:-2], torch.float32)
    return L, P, H, 16 * n, w // 16


def kv_keep(codes, scales, table, cu_q, kv_lens, keep, kept):
    """Of each sequence's new tokens in the cache (the last cu_q[b + 1] - cu_q[b] of kv_lens[b]),
    those that ``keep`` (int32 [batch, n], rising) names, ``kept`` (int32 [batch]) of them, move to
    the front: slots kv_lens[b] - new + i.  ``codes`` and ``scales`` may be one layer's or
    [layers, ...] of all that share the table.  A page's scale becomes the largest of its own
    and its tokens' pages'.  A sequence whose list is not rising stays as it is.  The lengths
    do not change: ``tree_accept`` returns the new ones."""
    torch = _torch()
    L, P, H, page, d = _pool(codes, scales)
    table = _dense(table)
    B, stride = shape = _ndim(table, "table", 2)
    _indices(((table, "table"),), shape)
    _indices(((cu_q, "cu_q"),), (B + 1,))
    _indices(((kv_lens, "kv_lens"), (kept, "kept")), (B,))
    most = _ndim(keep, "keep", 2)[1]
    _indices(((keep, "keep"),), (B, most))
    dev = codes.get_device()
    _one_device(dev, (scales, table, cu_q, kv_lens, keep, kept))
    sh = KvShape(0, B, H, H, d, page, P, stride, 0x3fffffff // max(H, 1), 0, 0)
    s = _call(dev, lib().kv_keep, codes.data_ptr(), scales.data_ptr(), L, table.data_ptr(), cu_q.data_ptr(),
              kv_lens.data_ptr(), keep.data_ptr(), kept.data_ptr(), most, sh, _raw_stream(dev))
    if s:
        _check("kv_keep", s)


def kv_copy(codes, scales, pairs):
    """Pages of the pool to others, codes and scales: ``pairs`` is a list of (from, to) or a host
    tensor int32 [n, 2], checked before anything is copied: ids inside the pool, no page the
    destination of two, none a source and a destination.  ``codes`` and ``scales`` may be one
    layer's or [layers, ...]."""
    torch = _torch()
    L, P, H, page, d = _pool(codes, scales)
    if isinstance(pairs, torch.Tensor):
        n = _ndim(pairs, "pairs", 2)[0]
        if pairs.is_cuda:
            raise TypeError("pairs must be on the host")
        _exact(pairs, "pairs", (n, 2), torch.int32)
        at = pairs.data_ptr()
    else:
        pairs = list(pairs)
        n = len(pairs)
        if any(len(p) != 2 for p in pairs):
            raise ValueError("pairs must be of two pages each")
        pairs = array.array("i", itertools.chain.from_iterable(pairs))
        at = pairs.buffer_info()[0]
    dev = codes.get_device()
    _one_device(dev, (scales,))
    s = _call(dev, lib().kv_copy, codes.data_ptr(), scales.data_ptr(), L, P, H, page, d, at, n, _raw_stream(dev))
    if s:
        _check("kv_copy", s)


# ------------------------------------------------------------ drawing tokens
_LOGITS = {}   # torch dtype -> C code


def _setting(v, name, rows, dtype):
    """(address or None, value, tensor or None) of a row's setting."""
    torch = _torch()
    if isinstance(v, torch.Tensor):
        _exact(v, name, (rows,), dtype)
        return v.data_ptr(), 0, v
    return None, v, None


def sample_tokens(logits, u, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0, out=None, workspace=None):
    """One token (int32 [rows]) drawn from each row of ``logits`` [rows, vocab] (float16,
    bfloat16 or float32, a row's logits adjacent) by the random numbers ``u`` (float32
    [rows], in [0, 1)).  Weights are exp((x - max) / temperature).  In falling order, equal
    logits by index, a token stays if it is among the first ``top_k`` (0: all), the weights
    before it are under ``top_p`` of what top_k left, and its own is at least ``min_p`` of the
    largest; the first always stays.  Of these the first token in order of index is drawn at
    which the running sum of weights exceeds u times their sum.  Temperature 0 takes the
    first of the falling order.  Each setting is a number or a device tensor [rows] (float32,
    top_k int32).  A row with a NaN or +inf, or of -inf alone, gives -1.  ``workspace``: uint8
    device memory (allocated if None)."""
    torch = _torch()
    if not _LOGITS:
        _LOGITS.update({torch.float16: 0, torch.bfloat16: 1, torch.float32: 2})
    dt = _LOGITS.get(getattr(logits, "dtype", None))
    if dt is None:
        raise TypeError("logits must be a torch tensor of float16, bfloat16 or float32, got %s"
                        % (getattr(logits, "dtype", type(logits).__name__),))
    R, V = _ndim(logits, "logits", 2)
    if logits.stride(1) != 1 and V > 1:
        raise ValueError("the logits of a row must be adjacent")
    f32 = torch.float32
    _exact(u, "u", (R,), f32)
    ta, t, tt = _setting(temperature, "temperature", R, f32)
    ka, k, kt = _setting(top_k, "top_k", R, torch.int32)
    pa, p, pt = _setting(top_p, "top_p", R, f32)
    ma, m, mt = _setting(min_p, "min_p", R, f32)
    if not -1 <= k <= 0x7fffffff:      # (ctypes would keep the low 32 bits)
        k = 0x7fffffff if k > 0 else -1
    if out is not None:
        _exact(out, "out", (R,), torch.int32)
    if workspace is not None and (workspace.dtype is not torch.uint8 or not workspace.is_contiguous()):
        raise TypeError("workspace must be contiguous torch.uint8")
    dev = logits.get_device()
    _one_device(dev, (u, tt, kt, pt, mt, out, workspace))
    L = lib()
    need = _i64()
    s = L.sample_workspace(dt, R, V, need)
    if s:
        _check("sample_tokens", s)
    room = need.value
    if workspace is not None:
        room = workspace.numel()
    elif room:
        workspace = torch.empty(room, dtype=torch.uint8, device=logits.device)
    if out is None:
        out = torch.empty(R, dtype=torch.int32, device=logits.device)
    s = _call(dev, L.sample_tokens, logits.data_ptr(), dt, R, V, logits.stride(0), u.data_ptr(),
              Sampling(ta, ka, pa, ma, t, k, p, m), out.data_ptr(), _addr(workspace), room, _raw_stream(dev))
    if s:
        _check("sample_tokens", s)
    return out


# ------------------------------------------------------------- pages (host)
class KvPages:
    """Hands out a pool's pages on the host: which sequence (any hashable name) holds which
    page, and how many hold it.  Pages that a fork shares are copied before the one that
    writes gets them.  Nothing here touches the device: what has to be copied there is
    returned as pairs for ``kv_copy``, to be run before the next call here and before what
    the pages are grown for is written.

        pages.fork("a", "b")                                  # b continues a: its pages are shared
        kv_copy(codes, scales, pages.grow("b", new_length))   # room for b's next tokens
        table = pages.table(["a", "b"])                       # host int32, a row a sequence
    """

    def __init__(self, pages, page):
        if pages < 0 or page < 16 or page % 16:
            raise ValueError("pages >= 0 and a page of a multiple of 16 tokens required")
        self.page = int(page)
        self.refs = [0] * int(pages)
        self._free = list(range(int(pages)))   # a heap: the lowest page first
        self._rows = {}
        self._lens = {}

    @property
    def available(self):
        """Pages that nobody holds."""
        return len(self._free)

    def length(self, seq):
        return self._lens[seq]

    def held(self, seq):
        """The pages of a sequence, in order of its tokens."""
        return list(self._rows[seq])

    def add(self, seq):
        """A sequence without tokens."""
        if seq in self._rows:
            raise ValueError("sequence %r is there already" % (seq,))
        self._rows[seq], self._lens[seq] = [], 0

    def _take(self, n):
        if n > len(self._free):
            raise MemoryError("%d pages are needed, %d are free" % (n, len(self._free)))
        got = [heapq.heappop(self._free) for _ in range(n)]
        for p in got:
            self.refs[p] = 1
        return got

    def _drop(self, p):
        self.refs[p] -= 1
        if self.refs[p] == 0:
            heapq.heappush(self._free, p)

    def grow(self, seq, length):
        """Room for the tokens up to ``length``; the pages that they are written to become the
        sequence's own.  Returns the pairs to copy.  All or nothing: without enough free
        pages MemoryError, and nothing has changed."""
        row, now = self._rows[seq], self._lens[seq]
        if length < now:
            raise ValueError("sequence %r has %d tokens, cannot grow to %d" % (seq, now, length))
        if length == now:
            return []
        first = now // self.page                          # the first page that is written
        shared = [i for i in range(first, min(len(row), -(-length // self.page))) if self.refs[row[i]] > 1]
        more = max(0, -(-length // self.page) - len(row))
        got = self._take(len(shared) + more)
        pairs = []
        for i in shared:
            to = got.pop(0)
            if i * self.page < now:                       # it holds tokens
                pairs.append((row[i], to))
            self._drop(row[i])
            row[i] = to
        row += got
        self._lens[seq] = length
        return pairs

    def cut(self, seq, length):
        """Forgets the tokens past ``length`` and frees the pages that only they needed."""
        row = self._rows[seq]
        if not 0 <= length <= self._lens[seq]:
            raise ValueError("sequence %r has %d tokens, cannot be cut to %d" % (seq, self._lens[seq], length))
        keep = -(-length // self.page)
        for p in row[keep:]:
            self._drop(p)
        del row[keep:]
        self._lens[seq] = length

    def fork(self, seq, new):
        """``new`` continues ``seq``: every page is shared, and a partly filled last one copied by
        the ``grow`` of whoever writes to it first."""
        if new in self._rows:
            raise ValueError("sequence %r is there already" % (new,))
        row = self._rows[seq]
        for p in row:
            self.refs[p] += 1
        self._rows[new], self._lens[new] = list(row), self._lens[seq]

    def free(self, seq):
        """Forgets a sequence; pages that nobody else holds are free again."""
        for p in self._rows.pop(seq):
            self._drop(p)
        del self._lens[seq]

    def pack(self):
        """Moves the pages in use to the front of the pool.  Returns the pairs to copy; tables made
        before name the old places."""
        used = [p for p, n in enumerate(self.refs) if n]
        to = {}
        holes = [p for p in range(len(used)) if not self.refs[p]]
        for p in reversed(used):
            if p < len(used):
                break
            to[p] = holes[len(to)]
        for a, b in to.items():
            self.refs[b], self.refs[a] = self.refs[a], 0
        for row in self._rows.values():
            row[:] = [to.get(p, p) for p in row]
        self._free = list(range(len(used), len(self.refs)))
        return list(to.items())

    def table(self, seqs, width=None):
        """Host int32 [len(seqs), width]: each sequence's pages, 0 behind them."""
        torch = _torch()
        rows = [self._rows[s] for s in seqs]
        most = max([len(r) for r in rows], default=0)
        width = max(most, 1) if width is None else int(width)
        if most > width:
            raise ValueError("a sequence has %d pages, the table %d" % (most, width))
        return torch.tensor([r + [0] * (width - len(r)) for r in rows], dtype=torch.int32).view(len(rows), width)
