"""Thin ctypes binding of libkvc (the C ABI declared in ``include/kvc.h``).

Argument marshalling only: every function takes torch tensors (device
memory), checks dtype / device / contiguity, passes raw pointers to the
library function of the same name and raises :class:`KvcError` on a non-OK
status.  All arithmetic runs in the CUDA kernels of libkvc; there is no
fallback.  If the library cannot be built or loaded, importing the binding
fails loudly.
"""
from __future__ import annotations

import ctypes
import os

import torch

from . import _build

KVC_OK = 0
STATUS_NAMES = {0: "KVC_OK", 1: "KVC_ERR_INVALID_ARG", 2: "KVC_ERR_SHAPE",
                3: "KVC_ERR_CUDA", 4: "KVC_ERR_TIMEOUT", 5: "KVC_ERR_UNSUPPORTED",
                6: "KVC_ERR_WORKSPACE"}
RULE_SINGLE, RULE_CUMULATIVE, RULE_EMA, RULE_MI, RULE_EMA_CHAINED = 0, 1, 2, 3, 4
CORR_OFF, CORR_ZERO_ORDER, CORR_FIRST_ORDER = 0, 1, 2
ALLOC_GLOBAL, ALLOC_LAYER, ALLOC_HEAD = 0, 1, 2
TREE_MAX = 64      # most drafted tokens per tree, most victims per commit

EXPORTED = (
    "kvc_version", "kvc_last_error", "kvc_status_string",
    "kvc_decode_workspace_size", "kvc_decode_workspace_init", "kvc_get_device_status",
    "kvc_decode_attend", "kvc_aggregate_evict", "kvc_moment_update", "kvc_correct",
    "kvc_compact", "kvc_zip_merge", "kvc_mi_scores", "kvc_mi_evict", "kvc_decode_step", "kvc_decode_attend_noalloc", "kvc_prefill_prepare",
    "kvc_prefill_workspace_size", "kvc_prefill_score", "kvc_prefill_window_attention",
    "kvc_prefill_snapkv", "kvc_prefill_handoff_workspace_size", "kvc_prefill_handoff",
    "kvc_tree_workspace_size", "kvc_tree_attend", "kvc_tree_weights", "kvc_tree_commit",
    "kvc_tree_weights_f64", "kvc_tree_commit_f64",
)


class KvcError(RuntimeError):
    def __init__(self, status: int, msg: str):
        super().__init__(f"{STATUS_NAMES.get(status, status)}: {msg}")
        self.status = status


class kvc_params(ctypes.Structure):
    _fields_ = [("U", ctypes.c_int32), ("G", ctypes.c_int32), ("d", ctypes.c_int32),
                ("cap", ctypes.c_int32), ("L", ctypes.c_int32), ("rule", ctypes.c_int32),
                ("alpha", ctypes.c_float), ("refresh_period", ctypes.c_int32),
                ("correction", ctypes.c_int32), ("merge", ctypes.c_int32),
                ("merge_recent", ctypes.c_int32), ("budget", ctypes.c_void_p),
                ("chain_layers", ctypes.c_int32), ("chain_heads", ctypes.c_int32)]


class kvc_cache(ctypes.Structure):
    _fields_ = [("K", ctypes.c_void_p), ("V", ctypes.c_void_p), ("votes", ctypes.c_void_p),
                ("pos", ctypes.c_void_p), ("util", ctypes.c_void_p), ("len", ctypes.c_void_p)]


class kvc_moments(ctypes.Structure):
    _fields_ = [("n", ctypes.c_void_p), ("mu_k", ctypes.c_void_p),
                ("mu_v", ctypes.c_void_p), ("C", ctypes.c_void_p)]


class kvc_tree(ctypes.Structure):
    _fields_ = [("T", ctypes.c_int32), ("units", ctypes.c_int32), ("mask", ctypes.c_void_p),
                ("n", ctypes.c_void_p)]


class kvc_path(ctypes.Structure):
    _fields_ = [("A", ctypes.c_int32), ("token", ctypes.c_void_p), ("n", ctypes.c_void_p),
                ("pos", ctypes.c_void_p)]


_lib = None


def library_path() -> str:
    return _build.LIB


def load(build: bool = True):
    """Load libkvc (building it first when sources changed)."""
    global _lib
    if _lib is not None:
        return _lib
    path = _build.build() if build else _build.LIB
    if not os.path.exists(path):
        raise ImportError(f"libkvc not built at {path}")
    lib = ctypes.CDLL(path)
    P, I32, I64, SZ = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t
    PP = ctypes.POINTER(kvc_params)
    PC = ctypes.POINTER(kvc_cache)
    PM = ctypes.POINTER(kvc_moments)
    PT, PA = ctypes.POINTER(kvc_tree), ctypes.POINTER(kvc_path)
    sigs = {
        "kvc_version": (I32, []),
        "kvc_last_error": (ctypes.c_char_p, []),
        "kvc_status_string": (ctypes.c_char_p, [I32]),
        "kvc_decode_workspace_size": (SZ, [PP]),
        "kvc_decode_workspace_init": (I32, [PP, P, SZ, P]),
        "kvc_get_device_status": (I32, [P, SZ, P, ctypes.POINTER(I32)]),
        "kvc_decode_attend": (I32, [PP, I32, I32, I32, P, P, P, PC, P, P, P, P, SZ, P]),
        "kvc_aggregate_evict": (I32, [PP, I32, P, PC, I32, P, P, P, P, SZ, P]),
        "kvc_moment_update": (I32, [PP, PC, I32, P, P, PM, P, SZ, P]),
        "kvc_correct": (I32, [PP, P, PC, I32, P, P, P, P, PM, P, P, P, P, SZ, P]),
        "kvc_compact": (I32, [PP, PC, I32, P, P, P, SZ, P]),
        "kvc_zip_merge": (I32, [PP, I32, P, PC, I32, P, P, P, P, SZ, P]),
        "kvc_mi_scores": (I32, [PP, PC, PM, I32, P, P, P]),
        "kvc_mi_evict": (I32, [PP, I32, PC, PM, P, I32, P, P, P, P, SZ, P]),
        "kvc_decode_step": (I32, [PP, I32, I32, I32, P, P, P, PC, PM, P, P, I32, P, P, P, P, SZ, P]),
        "kvc_decode_attend_noalloc": (I32, [PP, I32, I32, I32, P, P, P, PC, P, P, P, P, P]),
        "kvc_prefill_prepare": (I32, [I32, I32, I32, I32, I32, P, P, P]),
        "kvc_prefill_workspace_size": (SZ, [I32, I32, I32, I64]),
        "kvc_prefill_score": (I32, [I32, I32, I32, I32, I32, I32, I64, I32, I32, P, P, P, P, P,
                                    P, P, P, P, SZ, P]),
        "kvc_prefill_window_attention": (I32, [I32, I32, I32, I32, I32, I32, P, P, P, P, P, SZ,
                                               P]),
        "kvc_prefill_handoff_workspace_size": (SZ, [I32, I32]),
        "kvc_prefill_handoff": (I32, [PP, I32, P, P, P, P, P, PC, PM, P, P, SZ, P]),
        "kvc_prefill_snapkv": (I32, [I32, I32, I32, I32, I32, I32, I64, I32, I32, P, P, P, P, P,
                                     P, P, SZ, P]),
        "kvc_tree_workspace_size": (SZ, [PP, I32]),
        "kvc_tree_attend": (I32, [PP, I32, PT, P, P, P, PC, PM, P, P, P, SZ, P]),
        "kvc_tree_weights": (I32, [PP, I32, PT, PA, P, P, P, P, PC, P, P, SZ, P]),
        "kvc_tree_commit": (I32, [PP, I32, PT, PA, P, P, P, PC, PM, I32, P, P, P, P, SZ, P]),
    }
    for name in ("kvc_tree_weights", "kvc_tree_commit"):
        sigs[name + "_f64"] = sigs[name]
    for name, (res, args) in sigs.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    _lib = lib
    return lib


def _check(status: int):
    if status != KVC_OK:
        raise KvcError(status, load().kvc_last_error().decode())


def _ptr(t, dtype=None, name="tensor", optional=False):
    if t is None:
        if optional:
            return None
        raise ValueError(f"{name} is required")
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_cuda:
        raise ValueError(f"{name} must live on a CUDA device")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream))


def make_params(U, G, cap, L, rule=RULE_EMA, alpha=0.9, refresh_period=1,
                correction=CORR_FIRST_ORDER, d=128, merge_recent=None, budget=None,
                chain=None) -> kvc_params:
    """merge_recent = R (not None) turns on KeepKV ZIP-merging with the last R
    positions excluded from the partner search; budget (a device int32 [U]
    tensor, kept alive by the caller) gives every unit its own budget;
    chain = (NL, Hkv) groups the units by sequence for the layer-chained EMA."""
    merge = 0 if merge_recent is None else 1
    NL, Hkv = (0, 0) if chain is None else (int(chain[0]), int(chain[1]))
    return kvc_params(U, G, d, cap, L, rule, alpha, refresh_period, correction, merge,
                      0 if merge_recent is None else int(merge_recent),
                      _ptr(budget, torch.int32, "budget", optional=True), NL, Hkv)


def make_cache(K, V, votes, pos, util, length) -> kvc_cache:
    return kvc_cache(_ptr(K, torch.bfloat16, "K"), _ptr(V, torch.bfloat16, "V"),
                     _ptr(votes, torch.int32, "votes", optional=True),
                     _ptr(pos, torch.int32, "pos"), _ptr(util, torch.float64, "util"),
                     _ptr(length, torch.int32, "len"))


def make_moments(n, mu_k, mu_v, C) -> kvc_moments:
    return kvc_moments(_ptr(n, torch.float32, "n"), _ptr(mu_k, torch.float32, "mu_k"),
                       _ptr(mu_v, torch.float32, "mu_v"), _ptr(C, torch.float32, "C"))


# ------------------------------------------------------------------ library

def kvc_version() -> int:
    return int(load().kvc_version())


def kvc_last_error() -> str:
    return load().kvc_last_error().decode()


def kvc_status_string(status: int) -> str:
    return load().kvc_status_string(int(status)).decode()


# ------------------------------------------------------------------ decode

def kvc_decode_workspace_size(p: kvc_params) -> int:
    return int(load().kvc_decode_workspace_size(ctypes.byref(p)))


def kvc_decode_workspace_init(p: kvc_params, ws: torch.Tensor, stream=None):
    _check(load().kvc_decode_workspace_init(ctypes.byref(p), _ptr(ws, torch.uint8, "ws"),
                                            ws.numel(), _stream(stream)))


def kvc_get_device_status(ws: torch.Tensor, stream=None) -> int:
    out = ctypes.c_int32(0)
    _check(load().kvc_get_device_status(_ptr(ws, torch.uint8, "ws"), ws.numel(),
                                        _stream(stream), ctypes.byref(out)))
    return int(out.value)


def kvc_decode_attend(p, t, new_pos, max_len, q, k_new, v_new, cache: kvc_cache, lse, f_all,
                      probs, ws, stream=None):
    bf = torch.bfloat16
    _check(load().kvc_decode_attend(
        ctypes.byref(p), int(t), int(new_pos), int(max_len), _ptr(q, bf, "q"),
        _ptr(k_new, bf, "k_new"), _ptr(v_new, bf, "v_new"), ctypes.byref(cache),
        _ptr(lse, torch.float32, "lse"), _ptr(f_all, torch.float32, "f_all"),
        _ptr(probs, torch.float64, "probs", optional=True), _ptr(ws, torch.uint8, "ws"),
        ws.numel(), _stream(stream)))


def kvc_aggregate_evict(p, t, probs, cache: kvc_cache, kmax, evict_idx, evict_pos, n_evict, ws,
                        stream=None):
    i32 = torch.int32
    _check(load().kvc_aggregate_evict(
        ctypes.byref(p), int(t), _ptr(probs, torch.float64, "probs", optional=True),
        ctypes.byref(cache), int(kmax), _ptr(evict_idx, i32, "evict_idx"),
        _ptr(evict_pos, i32, "evict_pos", optional=True), _ptr(n_evict, i32, "n_evict"),
        _ptr(ws, torch.uint8, "ws"), ws.numel(), _stream(stream)))


def kvc_moment_update(p, cache: kvc_cache, kmax, evict_idx, n_evict, mom: kvc_moments, ws,
                      stream=None):
    i32 = torch.int32
    _check(load().kvc_moment_update(
        ctypes.byref(p), ctypes.byref(cache), int(kmax), _ptr(evict_idx, i32, "evict_idx"),
        _ptr(n_evict, i32, "n_evict"), ctypes.byref(mom), _ptr(ws, torch.uint8, "ws"),
        ws.numel(), _stream(stream)))


def kvc_correct(p, q, cache: kvc_cache, kmax, evict_idx, n_evict, lse, f_all, mom: kvc_moments,
                o, f_R, logZ_R, ws, stream=None):
    i32, f32 = torch.int32, torch.float32
    _check(load().kvc_correct(
        ctypes.byref(p), _ptr(q, torch.bfloat16, "q"), ctypes.byref(cache), int(kmax),
        _ptr(evict_idx, i32, "evict_idx"), _ptr(n_evict, i32, "n_evict"),
        _ptr(lse, f32, "lse"), _ptr(f_all, f32, "f_all"), ctypes.byref(mom),
        _ptr(o, f32, "o"), _ptr(f_R, f32, "f_R", optional=True),
        _ptr(logZ_R, f32, "logZ_R", optional=True), _ptr(ws, torch.uint8, "ws"), ws.numel(),
        _stream(stream)))


def kvc_compact(p, cache: kvc_cache, kmax, evict_idx, n_evict, ws, stream=None):
    i32 = torch.int32
    _check(load().kvc_compact(
        ctypes.byref(p), ctypes.byref(cache), int(kmax), _ptr(evict_idx, i32, "evict_idx"),
        _ptr(n_evict, i32, "n_evict"), _ptr(ws, torch.uint8, "ws"), ws.numel(),
        _stream(stream)))


def kvc_mi_scores(p, cache: kvc_cache, mom: kvc_moments, max_len, probs, scores, stream=None):
    f64 = torch.float64
    _check(load().kvc_mi_scores(
        ctypes.byref(p), ctypes.byref(cache), ctypes.byref(mom), int(max_len),
        _ptr(probs, f64, "probs"), _ptr(scores, f64, "scores"), _stream(stream)))


def kvc_mi_evict(p, max_len, cache: kvc_cache, mom: kvc_moments, lse, kmax, evict_idx, evict_pos,
                 n_evict, ws, stream=None):
    i32 = torch.int32
    _check(load().kvc_mi_evict(
        ctypes.byref(p), int(max_len), ctypes.byref(cache), ctypes.byref(mom),
        _ptr(lse, torch.float32, "lse"), int(kmax), _ptr(evict_idx, i32, "evict_idx"),
        _ptr(evict_pos, i32, "evict_pos", optional=True), _ptr(n_evict, i32, "n_evict"),
        _ptr(ws, torch.uint8, "ws"), ws.numel(), _stream(stream)))


def kvc_zip_merge(p, new_pos, q, cache: kvc_cache, kmax, evict_idx, n_evict, partner_pos, ws,
                  stream=None):
    i32 = torch.int32
    _check(load().kvc_zip_merge(
        ctypes.byref(p), int(new_pos), _ptr(q, torch.bfloat16, "q"), ctypes.byref(cache),
        int(kmax), _ptr(evict_idx, i32, "evict_idx"), _ptr(n_evict, i32, "n_evict"),
        _ptr(partner_pos, i32, "partner_pos", optional=True), _ptr(ws, torch.uint8, "ws"),
        ws.numel(), _stream(stream)))


def kvc_decode_step(p, t, new_pos, max_len, q, k_new, v_new, cache: kvc_cache,
                    mom: kvc_moments, o, probs, kmax, evict_idx, evict_pos, n_evict, ws,
                    stream=None):
    bf, i32 = torch.bfloat16, torch.int32
    _check(load().kvc_decode_step(
        ctypes.byref(p), int(t), int(new_pos), int(max_len), _ptr(q, bf, "q"),
        _ptr(k_new, bf, "k_new"), _ptr(v_new, bf, "v_new"), ctypes.byref(cache),
        ctypes.byref(mom), _ptr(o, torch.float32, "o"),
        _ptr(probs, torch.float64, "probs", optional=True), int(kmax),
        _ptr(evict_idx, i32, "evict_idx", optional=True),
        _ptr(evict_pos, i32, "evict_pos", optional=True), _ptr(n_evict, i32, "n_evict"),
        _ptr(ws, torch.uint8, "ws"), ws.numel(), _stream(stream)))


def kvc_decode_attend_noalloc(p, t, new_pos, max_len, q, k_new, v_new, cache: kvc_cache, lse,
                              f_all, probs, device_status=None, stream=None):
    """kvc_decode_attend without a workspace, for callers that cannot allocate
    device memory: the scratch is a 32 MiB static array inside the library."""
    bf = torch.bfloat16
    _check(load().kvc_decode_attend_noalloc(
        ctypes.byref(p), int(t), int(new_pos), int(max_len), _ptr(q, bf, "q"),
        _ptr(k_new, bf, "k_new"), _ptr(v_new, bf, "v_new"), ctypes.byref(cache),
        _ptr(lse, torch.float32, "lse"), _ptr(f_all, torch.float32, "f_all"),
        _ptr(probs, torch.float64, "probs", optional=True),
        _ptr(device_status, torch.int32, "device_status", optional=True), _stream(stream)))


# ------------------------------------------------------------------ drafted tokens

_BF16, _F32, _F64, _I32, _U8, _Tensor = (torch.bfloat16, torch.float32, torch.float64, torch.int32,
                                          torch.uint8, torch.Tensor)


def _sized(t, dtype, name, numel, device, optional=False):
    """The address of a tensor, as _ptr, with the element count and the device
    checked too: a row stride or a unit count that does not fit the tensor is
    an error here, not a read out of range on the device."""
    if (type(t) is _Tensor and t.dtype is dtype and t.get_device() == device
            and t.is_contiguous() and t.numel() >= numel):
        return t.data_ptr()
    ptr = _ptr(t, dtype, name, optional)
    if t is not None:
        if t.numel() < numel:
            raise ValueError(f"{name} has {t.numel()} elements, needs {numel}")
        if t.device.index != device:
            raise ValueError(f"{name} must live on the current device cuda:{device}, not {t.device}")
    return ptr


# the current device and stream without what torch.cuda's functions do around them
_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream_on(stream, device):
    """_stream, without building a Stream object where torch gives the handle."""
    if stream is None and _raw_stream is not None:
        return _raw_stream(device)
    return _stream(stream)


_ref = ctypes.byref


def make_tree(T, units, mask, n=None) -> kvc_tree:
    """A tree of T drafted tokens per sequence, shared by `units` consecutive
    units.  mask: int64 [trees][T], bit j of row i set when token i attends
    drafted token j; n: int32 [trees] live tokens or None (= T).  The tensors
    are kept alive with the structure."""
    T, units = int(T), int(units)
    if mask is None or mask.dim() != 2 or mask.shape[1] != T:
        raise ValueError(f"mask must be [trees][T = {T}]")
    trees, dev = mask.shape[0], mask.device.index
    tr = kvc_tree(T, units, _sized(mask, torch.int64, "mask", trees * T, dev),
                  _sized(n, torch.int32, "n", trees, dev, optional=True))
    tr.trees, tr.keep = trees, (mask, n)
    return tr


def make_path(A, token, n, pos) -> kvc_path:
    """The accepted tokens of every tree: token int32 [trees][A] (root first),
    n int32 [trees] how many of them, pos int32 [trees] the position of the
    first.  The tensors are kept alive with the structure."""
    A = int(A)
    if token is None or token.dim() != 2 or token.shape[1] != A:
        raise ValueError(f"token must be [trees][A = {A}]")
    trees, dev, i32 = token.shape[0], token.device.index, torch.int32
    pa = kvc_path(A, _sized(token, i32, "token", trees * A, dev),
                  _sized(n, i32, "n", trees, dev), _sized(pos, i32, "pos", trees, dev))
    pa.trees, pa.keep = trees, (token, n, pos)
    return pa


def _tree_device(U, tree, path=None):
    """The current device; the tree (and path) must live there and cover the units."""
    dev = _device()
    if tree.keep[0].get_device() != dev or (path is not None and path.keep[0].get_device() != dev):
        raise ValueError(f"the tree and path must live on the current device cuda:{dev}")
    units = tree.units
    if units < 1 or tree.trees * units < U or (path is not None and path.trees * units < U):
        raise ValueError(f"the trees of {units} units do not cover U = {U}")
    return dev


def kvc_tree_workspace_size(p: kvc_params, T: int) -> int:
    return int(load().kvc_tree_workspace_size(ctypes.byref(p), int(T)))


def kvc_tree_attend(p, max_len, tree: kvc_tree, q, k_tree, v_tree, cache: kvc_cache, mom, o, lse,
                    ws, stream=None):
    """mom: kvc_moments or None (no correction)."""
    U, G, d = p.U, p.G, p.d
    dev = _tree_device(U, tree)
    rows = U * tree.T
    n, heads = rows * d, rows * G
    _check(load().kvc_tree_attend(
        _ref(p), int(max_len), _ref(tree),
        _sized(q, _BF16, "q", heads * d, dev), _sized(k_tree, _BF16, "k_tree", n, dev),
        _sized(v_tree, _BF16, "v_tree", n, dev), _ref(cache),
        None if mom is None else _ref(mom), _sized(o, _BF16, "o", heads * d, dev),
        _sized(lse, _F32, "lse", heads, dev), _sized(ws, _U8, "ws", 0, dev),
        ws.numel(), _stream_on(stream, dev)))


def kvc_tree_weights(p, max_len, tree: kvc_tree, path: kvc_path, row_weight, q, k_tree, lse,
                     cache: kvc_cache, S, ws, stream=None):
    """row_weight: fp32 [trees][A] or None (all 1).  S: fp64 [U][cap], or fp32
    (weights below its range are 0)."""
    U, G, d = p.U, p.G, p.d
    dev = _tree_device(U, tree, path)
    rows = U * tree.T
    weights = None
    if row_weight is not None:
        weights = _sized(row_weight, _F32, "row_weight", U // tree.units * path.A, dev)
    lib, wide = load(), getattr(S, "dtype", None) is _F64
    _check((lib.kvc_tree_weights_f64 if wide else lib.kvc_tree_weights)(
        _ref(p), int(max_len), _ref(tree), _ref(path), weights,
        _sized(q, _BF16, "q", rows * G * d, dev), _sized(k_tree, _BF16, "k_tree", rows * d, dev),
        _sized(lse, _F32, "lse", rows * G, dev), _ref(cache),
        _sized(S, _F64 if wide else _F32, "S", U * p.cap, dev), _sized(ws, _U8, "ws", 0, dev), ws.numel(),
        _stream_on(stream, dev)))


def kvc_tree_commit(p, max_len, tree: kvc_tree, path: kvc_path, k_tree, v_tree, S,
                    cache: kvc_cache, mom, kmax, evict_idx, evict_pos, n_evict, ws, stream=None):
    """S: [U][cap] from kvc_tree_weights (fp64 or fp32) or None (no refresh); mom:
    kvc_moments or None; evict_idx, evict_pos: int32 [U][kmax] or None."""
    U, kmax = p.U, int(kmax)
    dev = _tree_device(U, tree, path)
    n = U * tree.T * p.d
    lib, wide = load(), getattr(S, "dtype", None) is _F64
    _check((lib.kvc_tree_commit_f64 if wide else lib.kvc_tree_commit)(
        _ref(p), int(max_len), _ref(tree), _ref(path),
        _sized(k_tree, _BF16, "k_tree", n, dev), _sized(v_tree, _BF16, "v_tree", n, dev),
        None if S is None else _sized(S, _F64 if wide else _F32, "S", U * p.cap, dev), _ref(cache),
        None if mom is None else _ref(mom), kmax,
        None if evict_idx is None else _sized(evict_idx, _I32, "evict_idx", U * kmax, dev),
        None if evict_pos is None else _sized(evict_pos, _I32, "evict_pos", U * kmax, dev),
        _sized(n_evict, _I32, "n_evict", U, dev), _sized(ws, _U8, "ws", 0, dev),
        ws.numel(), _stream_on(stream, dev)))


# ------------------------------------------------------------------ prefill

def kvc_prefill_prepare(NL, Hq, Hkv, d, D, W_O, R, stream=None):
    _check(load().kvc_prefill_prepare(int(NL), int(Hq), int(Hkv), int(d), int(D),
                                      _ptr(W_O, torch.bfloat16, "W_O"),
                                      _ptr(R, torch.float32, "R"), _stream(stream)))


def kvc_prefill_workspace_size(NL, Hkv, N, B_total) -> int:
    return int(load().kvc_prefill_workspace_size(int(NL), int(Hkv), int(N), int(B_total)))


def kvc_prefill_score(NL, Hq, Hkv, d, N, w, B_total, normalize, q_win, K, V, R, scores, keep,
                      counts, idx, ws, stream=None, alloc=ALLOC_GLOBAL):
    bf = torch.bfloat16
    _check(load().kvc_prefill_score(
        int(NL), int(Hq), int(Hkv), int(d), int(N), int(w), int(B_total), int(normalize),
        int(alloc),
        _ptr(q_win, bf, "q_win"), _ptr(K, bf, "K"), _ptr(V, bf, "V"),
        _ptr(R, torch.float32, "R"), _ptr(scores, torch.float32, "scores", optional=True),
        _ptr(keep, torch.uint8, "keep"), _ptr(counts, torch.int32, "counts", optional=True),
        _ptr(idx, torch.int64, "idx", optional=True), _ptr(ws, torch.uint8, "ws", optional=True),
        0 if ws is None else ws.numel(), _stream(stream)))


def kvc_prefill_window_attention(NL, Hq, Hkv, d, N, w, row_weight, q_win, K, S, ws, stream=None):
    """row_weight: w host floats (a sequence); S: [NL][Hkv][N] fp32 output."""
    rw = (ctypes.c_float * max(1, len(row_weight)))(*[float(x) for x in row_weight])
    bf = torch.bfloat16
    _check(load().kvc_prefill_window_attention(
        int(NL), int(Hq), int(Hkv), int(d), int(N), int(w), ctypes.cast(rw, ctypes.c_void_p),
        _ptr(q_win, bf, "q_win"), _ptr(K, bf, "K"), _ptr(S, torch.float32, "S"),
        _ptr(ws, torch.uint8, "ws"), ws.numel(), _stream(stream)))


def kvc_prefill_snapkv(NL, Hq, Hkv, d, N, w, B_total, pool, sink, q_win, K, scores, keep, counts,
                       idx, ws, stream=None):
    bf = torch.bfloat16
    _check(load().kvc_prefill_snapkv(
        int(NL), int(Hq), int(Hkv), int(d), int(N), int(w), int(B_total), int(pool), int(sink),
        _ptr(q_win, bf, "q_win"), _ptr(K, bf, "K"),
        _ptr(scores, torch.float32, "scores", optional=True), _ptr(keep, torch.uint8, "keep"),
        _ptr(counts, torch.int32, "counts", optional=True),
        _ptr(idx, torch.int64, "idx", optional=True), _ptr(ws, torch.uint8, "ws"), ws.numel(),
        _stream(stream)))


def kvc_prefill_handoff_workspace_size(U, N) -> int:
    return int(load().kvc_prefill_handoff_workspace_size(int(U), int(N)))


def kvc_prefill_handoff(p, N, keep, K_src, V_src, votes_src, util_init, cache: kvc_cache,
                        mom: kvc_moments, budget, ws, stream=None):
    bf = torch.bfloat16
    _check(load().kvc_prefill_handoff(
        ctypes.byref(p), int(N), _ptr(keep, torch.uint8, "keep"), _ptr(K_src, bf, "K_src"),
        _ptr(V_src, bf, "V_src"), _ptr(votes_src, torch.int32, "votes_src", optional=True),
        _ptr(util_init, torch.float64, "util_init", optional=True), ctypes.byref(cache),
        ctypes.byref(mom), _ptr(budget, torch.int32, "budget", optional=True),
        _ptr(ws, torch.uint8, "ws"), ws.numel(), _stream(stream)))
