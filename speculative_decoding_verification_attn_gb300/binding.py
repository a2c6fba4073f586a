"""Thin ctypes binding of ``libspecverify.so`` (see ``include/spec_verify.h``).

Argument marshalling only: torch tensors supply device pointers, shapes,
dtypes and the current CUDA stream; every step of the computation runs in
the library's kernels.  There is no fallback: if the library has not been
built (``python -c "import __graft_entry__ as g; g.build()"``) or fails to
load, every call raises.
"""
from __future__ import annotations

import ctypes
import os
from typing import Optional

import numpy as np
import torch

LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libspecverify.so")

SPEC_DTYPE_F32, SPEC_DTYPE_BF16, SPEC_DTYPE_F16, SPEC_DTYPE_I8, SPEC_DTYPE_I32 = 0, 1, 2, 3, 4
SPEC_DTYPE_E4M3 = 5
SPEC_OK, SPEC_ERR_INVALID, SPEC_ERR_UNSUPPORTED, SPEC_ERR_CUDA = 0, -1, -2, -3
SPEC_OPT_ATTN_PATH, SPEC_OPT_NUM_CTAS, SPEC_OPT_VALIDATE, SPEC_OPT_SIMT_CHUNK = 0, 1, 2, 3
SPEC_OPT_SPLIT_WEIGHT = 4
SPEC_OPT_SMALL_CLUSTER = 5
NUM_OPTIONS = 6
SPEC_DEVERR_PAGE, SPEC_DEVERR_CTX, SPEC_DEVERR_TIMEOUT, SPEC_DEVERR_TOKEN = 1, 2, 4, 8
SPEC_DEVERR_TREE = 16
SPEC_DEVERR_CODEC = 32
SPEC_ROPE_PLAIN, SPEC_ROPE_LINEAR, SPEC_ROPE_NTK, SPEC_ROPE_YARN = 0, 1, 2, 3
SPEC_ROPE_RAMP_BY_INDEX = 16

# every symbol the public header declares
EXPORTED = ["spec_version", "spec_last_error", "spec_set_option", "spec_verify_attn",
            "spec_accept_greedy", "spec_verify_attn_tensors", "spec_accept_greedy_tensors",
            "spec_accept_greedy_noalloc", "spec_accept_rejection",
            "spec_kv_append", "spec_commit", "spec_verify_attn_tree", "spec_accept_tree",
            "spec_verify_attn_window", "spec_rope_append", "spec_rope_table", "spec_kv_gather",
            "spec_codec_encode", "spec_codec_decode", "spec_device_error", "spec_release"]
SPEC_NOALLOC_MAX_PARTIALS, SPEC_NOALLOC_MAX_BATCH = 65536, 4096

_TORCH_DT = {torch.float32: SPEC_DTYPE_F32, torch.bfloat16: SPEC_DTYPE_BF16,
             torch.float16: SPEC_DTYPE_F16, torch.int8: SPEC_DTYPE_I8,
             torch.int32: SPEC_DTYPE_I32, torch.float8_e4m3fn: SPEC_DTYPE_E4M3}


class SpecTensor(ctypes.Structure):
    """spec_tensor_t: data pointer, element type, rank, shape, strides (elements)."""
    _fields_ = [("data", ctypes.c_void_p), ("dtype", ctypes.c_int32), ("ndim", ctypes.c_int32),
                ("shape", ctypes.c_int64 * 4), ("stride", ctypes.c_int64 * 4)]


def tensor_desc(t: Optional[torch.Tensor]):
    """The spec_tensor_t of a torch tensor (any strides; None stays None)."""
    if t is None:
        return None
    if t.dim() > 4:
        raise ValueError("descriptors hold at most 4 dimensions")
    d = SpecTensor()
    d.data = t.data_ptr()
    d.dtype = _TORCH_DT[t.dtype]
    d.ndim = t.dim()
    for i, (n, st) in enumerate(zip(t.shape, t.stride())):
        d.shape[i] = n
        d.stride[i] = st
    return d

_lib = None


class SpecError(RuntimeError):
    def __init__(self, code: int, msg: str):
        super().__init__("spec call failed (%d): %s" % (code, msg))
        self.code = code


def load():
    """Load the in-tree library (once).  Raises if it is missing."""
    global _lib
    if _lib is None:
        _lib = _open(LIB_PATH)
    return _lib


def _open(path: str):
    if not os.path.exists(path):
        raise RuntimeError("libspecverify.so not built at %s; run __graft_entry__.build()" % path)
    lib = ctypes.CDLL(path)
    P, i32, i64 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64
    lib.spec_version.restype = ctypes.c_int
    lib.spec_last_error.restype = ctypes.c_char_p
    lib.spec_set_option.argtypes = [i32, i64]
    lib.spec_set_option.restype = ctypes.c_int
    lib.spec_verify_attn.argtypes = [P, P, P, P, P, P, P, i32, i32, i32, i32, i32, i32, i32, i32,
                                     i32, i32, ctypes.c_float, P, P, P]
    lib.spec_verify_attn.restype = ctypes.c_int
    lib.spec_accept_greedy.argtypes = [P, i32, P, i32, i32, i64, P, P, P]
    lib.spec_accept_greedy.restype = ctypes.c_int
    lib.spec_accept_greedy_noalloc.argtypes = [P, i32, P, i32, i32, i64, P, P, P]
    lib.spec_accept_greedy_noalloc.restype = ctypes.c_int
    lib.spec_accept_rejection.argtypes = [P, P, i32, P, i32, i32, i64, ctypes.c_float,
                                          ctypes.c_uint64, P, P, P]
    lib.spec_accept_rejection.restype = ctypes.c_int
    lib.spec_kv_append.argtypes = [P, P, i32, P, P, P, P, i32, P, P, i32, i32, i32, i32, i32, i32,
                                   i32, P]
    lib.spec_kv_append.restype = ctypes.c_int
    lib.spec_commit.argtypes = [P, P, i32, i32, P]
    lib.spec_commit.restype = ctypes.c_int
    lib.spec_codec_encode.argtypes = [P, ctypes.c_int64, i32, i32, P, P, P]
    lib.spec_codec_encode.restype = ctypes.c_int
    lib.spec_codec_decode.argtypes = [P, P, ctypes.c_int64, i32, i32, P, P]
    lib.spec_codec_decode.restype = ctypes.c_int
    lib.spec_verify_attn_tree.argtypes = [P, P, P, P, P, P, P, P, i32, i32, i32, i32, i32, i32, i32,
                                          i32, i32, i32, ctypes.c_float, P, P, P]
    lib.spec_verify_attn_tree.restype = ctypes.c_int
    lib.spec_verify_attn_window.argtypes = [P, P, P, P, P, P, P, P, i32, i32, i32, i32, i32, i32,
                                            i32, i32, i32, i32, ctypes.c_float, i32, i32, P, P, P]
    lib.spec_verify_attn_window.restype = ctypes.c_int
    lib.spec_rope_append.argtypes = ([P] * 4 + [i64] * 4 + [i32] + [P] * 4 + [i32] + [P] * 5 +
                                     [i32, i32, ctypes.c_float] + [i32] * 8 + [P])
    lib.spec_rope_append.restype = ctypes.c_int
    f64 = ctypes.c_double
    lib.spec_rope_table.argtypes = [i32, f64, i32, f64, f64, f64, f64, P, P]
    lib.spec_rope_table.restype = ctypes.c_int
    lib.spec_kv_gather.argtypes = [P, P, P, P, i32, P, P, P] + [i32] * 8 + [P, P, P]
    lib.spec_kv_gather.restype = ctypes.c_int
    lib.spec_accept_tree.argtypes = [P, i32, P, P, i32, i32, i64, P, P, P, P]
    lib.spec_accept_tree.restype = ctypes.c_int
    T = ctypes.POINTER(SpecTensor)
    lib.spec_verify_attn_tensors.argtypes = [T, T, T, T, T, T, T, i32, ctypes.c_float, T, T, P]
    lib.spec_verify_attn_tensors.restype = ctypes.c_int
    lib.spec_accept_greedy_tensors.argtypes = [T, T, i32, T, T, P]
    lib.spec_accept_greedy_tensors.restype = ctypes.c_int
    lib.spec_device_error.argtypes = [ctypes.POINTER(ctypes.c_int32)]
    lib.spec_device_error.restype = ctypes.c_int
    lib.spec_release.restype = ctypes.c_int
    return lib


def _check(rc: int):
    if rc != SPEC_OK:
        raise SpecError(rc, load().spec_last_error().decode())


def _ptr(t: Optional[torch.Tensor]):
    if t is None:
        return None
    if not t.is_contiguous():
        raise ValueError("tensors must be contiguous")
    return t.data_ptr()  # the entry points' argtypes turn it into a pointer


# The current stream's handle without building a Stream object (0.1 us against
# 2.9 of a call that takes 4 to 9 in the library).
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
_get_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device


def _stream(stream) -> int:
    if stream is None:
        if _raw_stream is not None:
            return _raw_stream(_get_device())
        stream = torch.cuda.current_stream()
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def spec_version() -> int:
    return load().spec_version()


def spec_last_error() -> str:
    return load().spec_last_error().decode()


def spec_set_option(option: int, value: int) -> None:
    _check(load().spec_set_option(option, int(value)))


_E4M3, _F32, _F16 = torch.float8_e4m3fn, torch.float32, torch.float16
_I32, _I8 = torch.int32, torch.int8


def _check_scales(k_cache, v_cache, k_scale, v_scale) -> None:
    """The scales of an int8 cache (float16 [num_pages, Hkv, P]) or a float8_e4m3fn
    one (float32 [num_pages, Hkv]): the library takes a bare pointer and cannot
    tell."""
    kind = k_cache.dtype
    if kind is _E4M3:
        dt, want, what = _F32, k_cache.shape[:2], "an e4m3 cache must be float32 [num_pages, Hkv]"
    elif kind is _I8:
        dt, want, what = _F16, k_cache.shape[:3], "an int8 cache must be float16 [num_pages, Hkv, P]"
    else:
        return
    if (k_scale is not None and (k_scale.dtype is not dt or k_scale.shape != want)
            or v_scale is not None and (v_scale.dtype is not dt or v_scale.shape != want)):
        raise ValueError("scales of " + what)


def _device_of(first) -> int:
    """The current device, on which ``first`` has to lie (kernels launch there)."""
    dev = first.get_device()  # -1: not on a GPU
    if dev < 0 or dev != _get_device():
        raise ValueError("tensors must lie on the current CUDA device")
    return dev


def _ptrs(dev: int, *tensors):
    """Pointers of dense tensors of device ``dev`` (None stays None), in one
    pass: a call's checks cost the host as much as its launch."""
    for t in tensors:
        if t is not None and (t.get_device() != dev or not t.is_contiguous()):
            raise ValueError("tensors must be contiguous and lie on the current CUDA device")
    return [None if t is None else t.data_ptr() for t in tensors]


_gpus = 0  # of this process, once known


def _reach(tensors):
    """Pointers of dense tensors that the current device reaches: its own memory or
    the host's, but no other GPU's (None stays None).  With one GPU there is no
    other, and a call's nine tensors are not asked (0.6 us of a call of 7)."""
    global _gpus
    if _gpus != 1:
        _gpus = _gpus or torch.cuda.device_count()
        here = (_get_device(), -1)  # (-1: host memory)
        for t in tensors:
            if t is not None and t.get_device() not in here:
                raise ValueError("tensors must not lie on another GPU than the current device")
    for t in tensors:
        if t is not None and not t.is_contiguous():
            raise ValueError("tensors must be contiguous")
    return [None if t is None else t.data_ptr() for t in tensors]


def _check_attn(q, k_cache, v_cache, k_scale, v_scale, block_table, ctx_lens, out, lse) -> None:
    """What the library cannot see behind the pointers of an attention call."""
    kind, dt = k_cache.dtype, q.dtype
    if v_cache.dtype is not kind or v_cache.numel() != k_cache.numel():
        raise ValueError("k_cache and v_cache must share a dtype and a shape")
    if kind is not dt:  # (scales come with a cache of codes)
        _check_scales(k_cache, v_cache, k_scale, v_scale)
    if block_table.dtype is not _I32 or ctx_lens.dtype is not _I32:
        raise ValueError("block_table and ctx_lens must be int32")
    if out.dtype is not dt or out.numel() < q.numel():
        raise ValueError("out must have q's dtype and size")
    if lse is not None and lse.dtype is not _F32:
        raise ValueError("lse must be float32")


def _stream_on(stream, dev: int) -> int:
    if stream is None and _raw_stream is not None:
        return _raw_stream(dev)
    return _stream(stream)


def spec_verify_attn(q, k_cache, v_cache, block_table, ctx_lens, num_draft: int, scale: float,
                     out, lse=None, k_scale=None, v_scale=None, stream=None) -> None:
    """Verification attention; writes ``out`` (and ``lse`` if given).

    q [B, k, Hq, D]; k_cache / v_cache [NP, Hkv, P, D]; block_table
    [B, max_pages] int32; ctx_lens [B] int32; out like q; lse [B, k, Hq] f32;
    k_scale / v_scale [NP, Hkv, P] fp16 for an int8 cache, [NP, Hkv] float32
    for a float8_e4m3fn cache.
    """
    B, k, Hq, D = q.shape
    NP, Hkv, P, D2 = k_cache.shape
    if k != num_draft or D2 != D:
        raise ValueError("shape mismatch between q, num_draft and the cache")
    tensors = (q, k_cache, v_cache, k_scale, v_scale, block_table, ctx_lens, out, lse)
    _check_attn(*tensors)
    qp, kp, vp, ksp, vsp, tp, cp, op, lp = _reach(tensors)
    _check(load().spec_verify_attn(
        qp, kp, vp, ksp, vsp, tp, cp, B, k, Hq, Hkv, D, P, NP, block_table.shape[1],
        _TORCH_DT[q.dtype], _TORCH_DT[k_cache.dtype], float(scale), op, lp, _stream(stream)))


def _ref(d):
    return None if d is None else ctypes.byref(d)


def spec_verify_attn_tensors(q, k_cache, v_cache, block_table, ctx_lens, num_draft: int,
                             scale: float, out, lse=None, k_scale=None, v_scale=None,
                             stream=None) -> None:
    """spec_verify_attn through the descriptor form (sizes and strides are
    read from the tensors; the library checks them)."""
    descs = [tensor_desc(t) for t in (q, k_cache, v_cache, k_scale, v_scale, block_table,
                                      ctx_lens, out, lse)]
    _check(load().spec_verify_attn_tensors(*[_ref(d) for d in descs[:7]], int(num_draft),
                                           float(scale), _ref(descs[7]), _ref(descs[8]),
                                           _stream(stream)))


def spec_accept_greedy_tensors(logits, draft_tokens, num_draft: int, accepted_len, next_token,
                               stream=None) -> None:
    """spec_accept_greedy through the descriptor form."""
    descs = [tensor_desc(t) for t in (logits, draft_tokens, accepted_len, next_token)]
    _check(load().spec_accept_greedy_tensors(_ref(descs[0]), _ref(descs[1]), int(num_draft),
                                             _ref(descs[2]), _ref(descs[3]), _stream(stream)))


def spec_verify_attn_tree(q, k_cache, v_cache, block_table, ctx_lens, tree_mask, num_draft: int,
                          scale: float, out, lse=None, k_scale=None, v_scale=None,
                          stream=None) -> None:
    """spec_verify_attn with draft visibility from ``tree_mask`` (64-bit [B, k],
    bit t of row i: query i sees draft t; int64 or uint64 tensor)."""
    B, k, Hq, D = q.shape
    NP, Hkv, P, D2 = k_cache.shape
    if k != num_draft or D2 != D or tree_mask.shape != (B, k):
        raise ValueError("q must be [B, num_draft, Hq, D], tree_mask [B, num_draft]")
    if tree_mask.element_size() != 8:
        raise ValueError("tree_mask must hold 64-bit words")
    tensors = (q, k_cache, v_cache, k_scale, v_scale, block_table, ctx_lens, out, lse)
    _check_attn(*tensors)
    qp, kp, vp, ksp, vsp, tp, cp, op, lp, mp = _reach(tensors + (tree_mask,))
    _check(load().spec_verify_attn_tree(
        qp, kp, vp, ksp, vsp, tp, cp, mp, B, k, Hq, Hkv, D, P, NP, block_table.shape[1],
        _TORCH_DT[q.dtype], _TORCH_DT[k_cache.dtype], float(scale), op, lp, _stream(stream)))


def _span(n) -> int:
    """A number of positions as int32: one past its range stands for as many as
    there are (ctypes would drop its upper bits)."""
    return max(-1, min(int(n), 2 ** 31 - 1))


def spec_verify_attn_window(q, k_cache, v_cache, block_table, ctx_lens, num_draft: int,
                            scale: float, window: int, num_sinks: int, out, lse=None,
                            k_scale=None, v_scale=None, tree_mask=None, stream=None) -> None:
    """spec_verify_attn (or, with ``tree_mask``, spec_verify_attn_tree) with a
    sliding window: a query sees the first ``num_sinks`` keys and those less
    than ``window`` positions before it (its own counts)."""
    B, k, Hq, D = q.shape
    NP, Hkv, P, D2 = k_cache.shape
    if k != num_draft or D2 != D or v_cache.shape != k_cache.shape:
        raise ValueError("shape mismatch between q, num_draft and the caches")
    if v_cache.dtype != k_cache.dtype or out.dtype != q.dtype or out.shape != q.shape:
        raise ValueError("v_cache must have k_cache's dtype, out q's dtype and shape")
    if block_table.dtype is not _I32 or ctx_lens.dtype is not _I32:
        raise ValueError("block_table and ctx_lens must be int32")
    if block_table.shape[0] != B or ctx_lens.shape != (B,):
        raise ValueError("block_table must be [B, max_pages] and ctx_lens [B]")
    if lse is not None and (lse.dtype is not _F32 or lse.shape != (B, k, Hq)):
        raise ValueError("lse must be float32 [B, k, Hq]")
    if tree_mask is not None and (tree_mask.shape != (B, k) or tree_mask.element_size() != 8):
        raise ValueError("tree_mask must hold 64-bit words [B, num_draft]")
    _check_scales(k_cache, v_cache, k_scale, v_scale)
    dev = _device_of(q)
    qp, kp, vp, ksp, vsp, tp, cp, mp, op, lp = _ptrs(
        dev, q, k_cache, v_cache, k_scale, v_scale, block_table, ctx_lens, tree_mask, out, lse)
    _check(load().spec_verify_attn_window(
        qp, kp, vp, ksp, vsp, tp, cp, mp, B, k, Hq, Hkv, D, P, NP, block_table.shape[1],
        _TORCH_DT[q.dtype], _TORCH_DT[k_cache.dtype], float(scale), _span(window), _span(num_sinks),
        op, lp, _stream_on(stream, dev)))


def spec_accept_tree(logits, draft_tokens, parents, num_draft: int, accepted_len, next_token,
                     path=None, stream=None) -> None:
    """Greedy acceptance over a tree of drafts (parents int32 [B, k] in [-1, i))."""
    B, k1, V = logits.shape
    if (k1 != num_draft + 1 or tuple(draft_tokens.shape) != (B, num_draft)
            or tuple(parents.shape) != (B, num_draft)):
        raise ValueError("logits [B, k+1, V], drafts and parents [B, k]")
    _check(load().spec_accept_tree(_ptr(logits), _TORCH_DT[logits.dtype], _ptr(draft_tokens),
                                   _ptr(parents), B, num_draft, V, _ptr(accepted_len),
                                   _ptr(next_token), _ptr(path), _stream(stream)))


def spec_accept_greedy(logits, draft_tokens, num_draft: int, accepted_len, next_token,
                       stream=None) -> None:
    """Greedy acceptance; writes ``accepted_len`` and ``next_token`` (int32 [B])."""
    B, k1, V = logits.shape
    if k1 != num_draft + 1 or tuple(draft_tokens.shape) != (B, num_draft):
        raise ValueError("logits must be [B, num_draft+1, V] and drafts [B, num_draft]")
    _check(load().spec_accept_greedy(_ptr(logits), _TORCH_DT[logits.dtype], _ptr(draft_tokens), B,
                                     num_draft, V, _ptr(accepted_len), _ptr(next_token),
                                     _stream(stream)))


def spec_accept_greedy_noalloc(logits, draft_tokens, num_draft: int, accepted_len, next_token,
                               stream=None) -> None:
    """spec_accept_greedy without any device allocation (fixed library scratch).

    For callers that cannot allocate device memory, e.g. a serving loop whose
    GPU memory is reserved up front by its own allocator.  Sizes are limited
    (see include/spec_verify.h); calls that overlap on the GPU share the
    scratch and race.
    """
    B, k1, V = logits.shape
    if k1 != num_draft + 1 or tuple(draft_tokens.shape) != (B, num_draft):
        raise ValueError("logits must be [B, num_draft+1, V] and drafts [B, num_draft]")
    _check(load().spec_accept_greedy_noalloc(_ptr(logits), _TORCH_DT[logits.dtype],
                                             _ptr(draft_tokens), B, num_draft, V,
                                             _ptr(accepted_len), _ptr(next_token),
                                             _stream(stream)))


def spec_accept_rejection(target_logits, draft_logits, draft_tokens, num_draft: int,
                          temperature: float, seed: int, accepted_len, next_token,
                          stream=None) -> None:
    """Rejection-sampling acceptance; writes ``accepted_len`` and ``next_token``.

    target_logits [B, k+1, V], draft_logits [B, k, V] (same dtype), drafts
    int32 [B, k]; draws from SplitMix64 keyed by ``seed``.
    """
    B, k1, V = target_logits.shape
    if (k1 != num_draft + 1 or tuple(draft_logits.shape) != (B, num_draft, V)
            or tuple(draft_tokens.shape) != (B, num_draft)):
        raise ValueError("target_logits must be [B, k+1, V], draft_logits [B, k, V], drafts [B, k]")
    if draft_logits.dtype != target_logits.dtype:
        raise ValueError("target and draft logits must share a dtype")
    _check(load().spec_accept_rejection(_ptr(target_logits), _ptr(draft_logits),
                                        _TORCH_DT[target_logits.dtype], _ptr(draft_tokens), B,
                                        num_draft, V, float(temperature),
                                        int(seed) & (2**64 - 1), _ptr(accepted_len),
                                        _ptr(next_token), _stream(stream)))


def spec_kv_append(k_new, v_new, k_cache, v_cache, block_table, ctx_lens, k_scale=None,
                   v_scale=None, stream=None) -> None:
    """Write k_new / v_new [B, n, Hkv, D] at positions ctx_b .. ctx_b + n - 1 of
    the paged caches (INT8 caches are quantised into k_scale / v_scale)."""
    B, n, Hkv, D = k_new.shape
    NP, Hkv2, P, D2 = k_cache.shape
    if (Hkv2, D2) != (Hkv, D) or v_new.shape != k_new.shape:
        raise ValueError("k_new / v_new must be [B, n, Hkv, D] matching the cache")
    if v_new.dtype is not k_new.dtype:
        raise ValueError("k_new and v_new must share a dtype")
    if v_cache.dtype is not k_cache.dtype or v_cache.numel() != k_cache.numel():
        raise ValueError("k_cache and v_cache must share a dtype and a shape")
    if block_table.dtype is not _I32 or ctx_lens.dtype is not _I32:
        raise ValueError("block_table and ctx_lens must be int32")
    _check_scales(k_cache, v_cache, k_scale, v_scale)
    kp, vp, kcp, vcp, ksp, vsp, tp, cp = _reach(
        (k_new, v_new, k_cache, v_cache, k_scale, v_scale, block_table, ctx_lens))
    _check(load().spec_kv_append(kp, vp, _TORCH_DT[k_new.dtype], kcp, vcp, ksp, vsp,
                                 _TORCH_DT[k_cache.dtype], tp, cp, B, n, Hkv, D, P, NP,
                                 block_table.shape[1], _stream(stream)))


_ROPE_SCALING = {"none": SPEC_ROPE_PLAIN, "linear": SPEC_ROPE_LINEAR, "ntk": SPEC_ROPE_NTK,
                 "yarn": SPEC_ROPE_YARN, "yarn-index": SPEC_ROPE_YARN | SPEC_ROPE_RAMP_BY_INDEX}


def spec_rope_table(rotary_dim: int, theta: float = 10000.0, scaling: str = "none",
                    factor: float = 1.0, original_len: float = 0.0, fast_turns: float = 32.0,
                    slow_turns: float = 1.0, device="cuda"):
    """The frequency table of spec_rope_append (int64 [rotary_dim / 2] on
    ``device``, the bits of uint64 fractions of a turn) and its amplitude.

    ``scaling``: "none", "linear", "ntk", or with ``original_len`` "yarn" (its ramp
    linear in a pair's number of turns, as the method is written down) or
    "yarn-index" (linear in the pair's index, as checkpoints that were extended
    with its published code have it).
    """
    if scaling not in _ROPE_SCALING:
        raise ValueError("scaling must be one of %s" % ", ".join(sorted(_ROPE_SCALING)))
    table = np.zeros(max(1, int(rotary_dim) // 2), np.uint64)
    amplitude = ctypes.c_float(0.0)
    _check(load().spec_rope_table(int(rotary_dim), float(theta), _ROPE_SCALING[scaling],
                                  float(factor), float(original_len), float(fast_turns),
                                  float(slow_turns), table.ctypes.data_as(ctypes.c_void_p),
                                  ctypes.byref(amplitude)))
    return torch.from_numpy(table.view(np.int64)).to(device), amplitude.value


def _token_rows(t, dev: int, name: str, B: int, n: int, H: int, D: int):
    """Pointer and token stride (elements) of [B, n, H, D] whose rows are dense
    and whose tokens are evenly spaced (a slice of a wider projection is)."""
    if t.get_device() != dev:
        raise ValueError("tensors must lie on the current CUDA device")
    if t.is_contiguous():
        return t.data_ptr(), H * D
    sb, sn, sh, sd = t.stride()
    if n == 1:
        sn = sb
    if B * n == 1:  # one token: its stride is never taken
        sn = H * D
    if sd != 1 or (H > 1 and sh != D) or (B > 1 and n > 1 and sb != n * sn):
        raise ValueError("%s: heads must be dense and tokens evenly spaced" % name)
    return t.data_ptr(), sn


def spec_rope_append(q, k_new, v_new, q_out, k_cache, v_cache, block_table, ctx_lens, rope_table,
                     interleaved: bool = False, amplitude: float = 1.0, positions=None,
                     new_lens=None, k_scale=None, v_scale=None, stream=None) -> None:
    """Rotate q [B, n, Hq, D] into ``q_out`` and append the rotated k_new and
    v_new [B, n, Hkv, D] at positions ctx_b .. of the paged caches.

    ``rope_table`` (spec_rope_table) rotates the first 2 * len(table) elements
    of a head; None rotates nothing.  q, k_new, v_new and q_out may be slices
    of wider rows; q_out may be q; q and q_out may be None.  ``positions``
    [B, n] int32 replaces ctx_b + t in the angles; ``new_lens`` [B] int32
    limits each sequence's tokens.  An e4m3 cache takes float32 scales
    [num_pages, Hkv], an int8 cache fp16 [num_pages, Hkv, P].
    """
    B, n, Hkv, D = rows = k_new.shape
    NP, Hkv2, P, D2 = pool = k_cache.shape
    src, kind = k_new.dtype, k_cache.dtype
    if (Hkv2, D2) != (Hkv, D) or v_new.shape != rows or v_cache.shape != pool:
        raise ValueError("k_new / v_new must be [B, n, Hkv, D] matching the caches")
    if (q is None) != (q_out is None):
        raise ValueError("q and q_out go together")
    Hq = 0
    if q is not None:
        Bq, nq, Hq, Dq = heads = q.shape
        if (Bq, nq, Dq) != (B, n, D) or q_out.shape != heads:
            raise ValueError("q and q_out must be [B, n, Hq, D]")
        if q.dtype != src or q_out.dtype != src:
            raise ValueError("q, q_out, k_new and v_new must share a dtype")
    if v_new.dtype != src or v_cache.dtype != kind:
        raise ValueError("k and v must share a dtype")
    if (block_table.dtype is not _I32 or ctx_lens.dtype is not _I32
            or block_table.shape[0] != B or ctx_lens.shape != (B,)):
        raise ValueError("block_table must be int32 [B, max_pages] and ctx_lens int32 [B]")
    if positions is not None and (positions.dtype is not _I32
                                  or positions.shape != (B, n)):
        raise ValueError("positions must be int32 [B, n]")
    if new_lens is not None and (new_lens.dtype is not _I32 or new_lens.shape != (B,)):
        raise ValueError("new_lens must be int32 [B]")
    if rope_table is not None and (rope_table.element_size() != 8 or rope_table.dim() != 1):
        raise ValueError("rope_table must be a row of 64-bit words")
    _check_scales(k_cache, v_cache, k_scale, v_scale)
    dev = k_new.get_device()  # (a CPU tensor's layout is still checked first)
    qp, qs, op, os_ = None, 0, None, 0
    if q is not None:
        qp, qs = _token_rows(q, dev, "q", B, n, Hq, D)
        op, os_ = _token_rows(q_out, dev, "q_out", B, n, Hq, D)
    kp, ks = _token_rows(k_new, dev, "k_new", B, n, Hkv, D)
    vp, vs = _token_rows(v_new, dev, "v_new", B, n, Hkv, D)
    _device_of(k_new)
    kcp, vcp, ksp, vsp, tp, cp, pp, lp, rp = _ptrs(
        dev, k_cache, v_cache, k_scale, v_scale, block_table, ctx_lens, positions, new_lens,
        rope_table)
    _check(load().spec_rope_append(
        qp, kp, vp, op, qs, ks, vs, os_, _TORCH_DT[src], kcp, vcp, ksp, vsp, _TORCH_DT[kind], tp,
        cp, pp, lp, rp, 0 if rope_table is None else 2 * rope_table.shape[0], bool(interleaved),
        float(amplitude), B, n, Hq, Hkv, D, P, NP, block_table.shape[1], _stream_on(stream, dev)))


def spec_kv_gather(k_cache, v_cache, block_table, lens, k_out, v_out, starts=None, k_scale=None,
                   v_scale=None, stream=None) -> None:
    """Rows of positions starts_b .. starts_b + lens_b - 1 of the paged caches
    into k_out / v_out [B, max_len, Hkv, D] (float32 or bfloat16); rows from
    lens_b on are left as they were."""
    B, n, Hkv, D = k_out.shape
    NP, Hkv2, P, D2 = k_cache.shape
    if (Hkv2, D2) != (Hkv, D) or v_out.shape != k_out.shape or v_cache.shape != k_cache.shape:
        raise ValueError("k_out / v_out must be [B, max_len, Hkv, D] matching the caches")
    if v_out.dtype != k_out.dtype or v_cache.dtype != k_cache.dtype:
        raise ValueError("k and v must share a dtype")
    if (block_table.dtype is not _I32 or lens.dtype is not _I32
            or block_table.shape[0] != B or lens.shape != (B,)):
        raise ValueError("block_table must be int32 [B, max_pages] and lens int32 [B]")
    if starts is not None and (starts.dtype is not _I32 or starts.shape != (B,)):
        raise ValueError("starts must be int32 [B]")
    _check_scales(k_cache, v_cache, k_scale, v_scale)
    dev = _device_of(k_cache)
    kp, vp, ksp, vsp, tp, sp, lp, kop, vop = _ptrs(
        dev, k_cache, v_cache, k_scale, v_scale, block_table, starts, lens, k_out, v_out)
    _check(load().spec_kv_gather(
        kp, vp, ksp, vsp, _TORCH_DT[k_cache.dtype], tp, sp, lp, B, n, Hkv, D, P, NP,
        block_table.shape[1], _TORCH_DT[k_out.dtype], kop, vop, _stream_on(stream, dev)))


def spec_codec_encode(codes, pairs, num_pairs, stream=None) -> None:
    """codes int8 [num_blocks, P, D] -> pairs uint8 [num_blocks, 2*P*D], num_pairs int32."""
    nblk, P, D = codes.shape
    _check(load().spec_codec_encode(_ptr(codes), nblk, P, D, _ptr(pairs), _ptr(num_pairs),
                                    _stream(stream)))


def spec_codec_decode(pairs, num_pairs, codes, stream=None) -> None:
    """pairs uint8 [num_blocks, 2*P*D], num_pairs int32 -> codes int8 [num_blocks, P, D]."""
    nblk, P, D = codes.shape
    _check(load().spec_codec_decode(_ptr(pairs), _ptr(num_pairs), nblk, P, D, _ptr(codes),
                                    _stream(stream)))


def spec_commit(ctx_lens, accepted_len, extra: int = 1, stream=None) -> None:
    """ctx_lens[b] += accepted_len[b] + extra, on the device."""
    _check(load().spec_commit(_ptr(ctx_lens), _ptr(accepted_len), ctx_lens.shape[0], int(extra),
                              _stream(stream)))


def spec_device_error() -> int:
    v = ctypes.c_int32(0)
    _check(load().spec_device_error(ctypes.byref(v)))
    return v.value


def spec_release() -> None:
    _check(load().spec_release())


# ---------------------------------------------------------------- plumbing

def _np_to_torch(a: np.ndarray, kind: str) -> torch.Tensor:
    if kind == "bf16":
        return torch.from_numpy(np.ascontiguousarray(a).view(np.int16)).view(torch.bfloat16)
    if kind == "f16":
        return torch.from_numpy(np.ascontiguousarray(a).view(np.int16)).view(torch.float16)
    return torch.from_numpy(np.ascontiguousarray(a))


def inputs_to_torch(inp, device="cuda", pin: bool = False) -> dict:
    """Generator output (numpy) -> torch tensors on `device` (or pinned host)."""
    s = inp.spec
    t = {
        "q": _np_to_torch(inp.q, s.q_dtype),
        "k_cache": _np_to_torch(inp.k_cache, s.kv_dtype),
        "v_cache": _np_to_torch(inp.v_cache, s.kv_dtype),
        "block_table": torch.from_numpy(inp.block_table),
        "ctx_lens": torch.from_numpy(inp.ctx_lens),
        "logits": _np_to_torch(inp.logits, s.logits_dtype),
        "draft_tokens": torch.from_numpy(inp.draft_tokens),
    }
    if inp.k_scale is not None:
        t["k_scale"] = _np_to_torch(inp.k_scale, "f16")
        t["v_scale"] = _np_to_torch(inp.v_scale, "f16")
    if pin:
        return {n: v.pin_memory() for n, v in t.items()}
    return {n: v.to(device) for n, v in t.items()}


def alloc_outputs(inp, device="cuda") -> dict:
    s = inp.spec
    qdt = torch.float32 if s.q_dtype == "f32" else torch.bfloat16
    B, k = s.batch, s.num_draft
    return {
        "out": torch.empty((B, k, s.num_q_heads, s.head_dim), dtype=qdt, device=device),
        "lse": torch.empty((B, k, s.num_q_heads), dtype=torch.float32, device=device),
        "accepted_len": torch.empty((B,), dtype=torch.int32, device=device),
        "next_token": torch.empty((B,), dtype=torch.int32, device=device),
    }


def run_verify(t: dict, o: dict, num_draft: int, scale: float, stream=None) -> None:
    """One verification step: attention, then acceptance, on one stream."""
    spec_verify_attn(t["q"], t["k_cache"], t["v_cache"], t["block_table"], t["ctx_lens"],
                     num_draft, scale, o["out"], o["lse"], t.get("k_scale"), t.get("v_scale"),
                     stream=stream)
    spec_accept_greedy(t["logits"], t["draft_tokens"], num_draft, o["accepted_len"],
                       o["next_token"], stream=stream)
