"""Python binding of libwq (the weight-format GEMM/GEMV library for sm_103a).

Argument marshalling only: every function forwards to the C entry point of the
same name in ``_build/libwq.so`` (declared in ``include/wq.h``), through ctypes or, for
the calls of a decode step, the C module ``_build/_wq_calls.*.so`` where it was built; all the
work runs in the library's CUDA kernels.  There is no CPU fallback: if the library is not
built, or no CUDA device is present, the calls raise.

Tensor arguments may be ``torch.Tensor`` (device memory) or raw integer device
pointers; ``stream`` may be a ``torch.cuda.Stream``, a raw ``cudaStream_t``
integer, or ``None`` for torch's current stream on the current device.
"""
from __future__ import annotations

import ctypes
import importlib.machinery
import importlib.util
import operator
import os
import threading
import types

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "_build", "libwq.so")
CALLS_PATH = os.path.join(HERE, "_build",
                          "_wq_calls" + importlib.machinery.EXTENSION_SUFFIXES[0])

WQ_BF16, WQ_Q8_0, WQ_Q4_0, WQ_F16, WQ_F32 = 0, 1, 2, 3, 4
WQ_BIAS, WQ_GELU, WQ_RESIDUAL, WQ_TC_BF16 = 1, 2, 4, 256
WQ_SILU, WQ_RELU, WQ_TANH = 8, 16, 32
WQ_OK, WQ_ERR_INVALID_ARG, WQ_ERR_UNSUPPORTED, WQ_ERR_CUDA = 0, 1, 2, 3
WQ_ERR_DEVICE_TIMEOUT, WQ_ERR_BAD_EXPERT, WQ_ERR_TOO_LARGE, WQ_ERR_BAD_INDEX = 4, 5, 6, 7
WQ_GEMM_NOALLOC_SCRATCH_BYTES = 16 << 20
WQ_GEMV_MAX_N = 16
WQ_MOE_WINDOW_SLOTS = 256
WQ_ROPE_INTERLEAVED, WQ_ROPE_TRANSPOSE = 1, 2
WQ_ROPE_PLAIN, WQ_ROPE_LINEAR, WQ_ROPE_NTK, WQ_ROPE_YARN, WQ_ROPE_BANDS = 0, 1, 2, 3, 4

WQ_AXES_DEALT, WQ_AXES_RESTART = 4, 8
WQ_HEAD_NONE, WQ_HEAD_RMS, WQ_HEAD_LAYER = 0, 1, 2

EXPORTS = ("wq_gemm", "wq_gemm_ws", "wq_gemm_alpha", "wq_gemm_dual", "wq_gemm_workspace_bytes",
           "wq_gemm_noalloc",
           "wq_gemm_ln_ws", "wq_gemm_ln_workspace_bytes", "wq_gemv",
           "wq_moe_gemv", "wq_weight_bytes", "wq_dequantize", "wq_embed", "wq_get_device_status",
           "wq_status_string", "wq_set_wait_limit",
           "wq_rope_table", "wq_rope", "wq_kv_append", "wq_attn_paged",
           "wq_attn_paged_workspace_bytes", "wq_kv_evict", "wq_kv_evict_workspace_bytes",
           "wq_norm_rope", "wq_norm_rope_grad", "wq_norm_rope_grad_workspace_bytes",
           "wq_kv_append_norm", "wq_attn_tokens", "wq_attn_tokens_workspace_bytes",
           "wq_kv_accept", "wq_kv_accept_slots")

_lock = threading.Lock()
_lib = None


class RopeScaling(ctypes.Structure):
    """wq_rope_scaling."""
    _fields_ = [("kind", ctypes.c_int32), ("original", ctypes.c_int32),
                ("factor", ctypes.c_double), ("low", ctypes.c_double), ("high", ctypes.c_double),
                ("magnitude", ctypes.c_double)]


class KvCache(ctypes.Structure):
    """wq_kv_cache."""
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("dtype", ctypes.c_int32),
                ("n_pages", ctypes.c_int32), ("page_size", ctypes.c_int32),
                ("n_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32),
                ("reserved", ctypes.c_int32), ("page_stride", ctypes.c_int64),
                ("head_stride", ctypes.c_int64), ("token_stride", ctypes.c_int64)]


class HeadNorm(ctypes.Structure):
    """wq_head_norm."""
    _fields_ = [("kind", ctypes.c_int32), ("eps", ctypes.c_float), ("weight", ctypes.c_void_p),
                ("bias", ctypes.c_void_p)]


class RopeAxes(ctypes.Structure):
    """wq_rope_axes."""
    _fields_ = [("rot", ctypes.c_int32), ("flags", ctypes.c_uint32), ("axes", ctypes.c_int32),
                ("pairs", ctypes.c_int32 * 4), ("table_rows", ctypes.c_int32),
                ("table_pairs", ctypes.c_int32), ("reserved", ctypes.c_int32),
                ("pos", ctypes.c_void_p), ("pos_stride", ctypes.c_int64),
                ("table", ctypes.c_void_p)]


class AttnForm(ctypes.Structure):
    """wq_attn_form."""
    _fields_ = [("softcap", ctypes.c_float), ("window", ctypes.c_int32),
                ("slopes", ctypes.c_void_p), ("first", ctypes.c_void_p),
                ("prefix", ctypes.c_void_p), ("tree", ctypes.c_void_p),
                ("tree_stride", ctypes.c_int64), ("pos", ctypes.c_void_p)]


class SlotArrays(ctypes.Structure):
    """wq_slot_arrays."""
    _fields_ = [("acc", ctypes.c_void_p), ("slot_pos", ctypes.c_void_p)]


def head_norm(kind, eps=1e-6, weight=None, bias=None) -> HeadNorm:
    """The descriptor of a norm of heads.  Like the others it keeps addresses, not the tensors."""
    return HeadNorm(kind, eps, _p(weight), _p(bias))


def rope_axes(rot, flags, pairs, pos, table) -> RopeAxes:
    """The descriptor of a rotation: `pairs` of each axis, pos int32 [axes][tokens] (or [tokens])
    and table f32 [rows][pairs of the table][2], tensors with contiguous last dimensions."""
    if not 1 <= len(pairs) <= 4:
        raise ValueError("one to four axes")
    step = pos.stride(0) if pos.dim() == 2 else 0
    return RopeAxes(rot, flags, len(pairs), (ctypes.c_int32 * 4)(*pairs), table.shape[0],
                    table.shape[1], 0, pos.data_ptr(), step, table.data_ptr())


def attn_form(softcap=0.0, window=0, slopes=None, first=None, prefix=None, tree=None,
              pos=None) -> AttnForm:
    """The descriptor of what wq_attn_tokens' tokens see; tree: int32 [tokens][words]."""
    return AttnForm(softcap, window, _p(slopes), _p(first), _p(prefix), _p(tree),
                    0 if tree is None else tree.stride(0), _p(pos))


def kv_caches(ks, vs):
    """The descriptors of several layers' pools, for wq_kv_accept."""
    caches = [kv_cache(k, v) for k, v in zip(ks, vs, strict=True)]
    return (KvCache * len(caches))(*caches)


def slot_arrays(accs, positions):
    """The slots' weights and positions of several layers ([sequence][kv head][slot], or None), for
    wq_kv_accept_slots."""
    arrays = [SlotArrays(_p(a), _p(b)) for a, b in zip(accs, positions, strict=True)]
    return (SlotArrays * len(arrays))(*arrays)


def kv_cache(k, v) -> KvCache:
    """The descriptor of two pools seen as [page][head][row][dim] (a view with any strides
    but a last one of 1).  It keeps addresses, not the tensors: the caller keeps those."""
    import torch
    if k.dim() != 4 or k.shape != v.shape or k.dtype != v.dtype or k.stride() != v.stride():
        raise ValueError("k and v: two 4-D tensors of one shape, type and layout")
    kinds = {torch.bfloat16: WQ_BF16, torch.float16: WQ_F16, torch.float32: WQ_F32}
    if k.dtype not in kinds or k.stride(3) != 1:
        raise ValueError("a cache holds bf16, f16 or f32 with contiguous dims")
    pages, heads, rows, dims = k.shape
    # A stride of an extent of 1 is never used; torch may give any value there.
    step = [k.stride(i) if k.shape[i] > 1 else pages * heads * rows * dims for i in range(3)]
    return KvCache(k.data_ptr(), v.data_ptr(), kinds[k.dtype], pages, rows, heads, dims, 0,
                   step[0], step[1], step[2])


class WqError(RuntimeError):
    def __init__(self, status: int, what: str = ""):
        self.status = status
        super().__init__(f"{what}: {wq_status_string(status)} ({status})" if what
                         else f"{wq_status_string(status)} ({status})")


def _open(path: str):
    """Open a libwq build and declare its signatures (raises if the file is missing)."""
    if not os.path.exists(path):
        raise RuntimeError(f"libwq is not built ({path} missing): run "
                           "gemv_transformer_gb300.build.build()")
    lib = ctypes.CDLL(path)
    ci, cu, vp, sz = ctypes.c_int, ctypes.c_uint, ctypes.c_void_p, ctypes.c_size_t
    gemm_args = [ci, ci, ci, ci, cu, vp, vp, vp, vp, vp, vp]
    lib.wq_gemm.argtypes = gemm_args
    lib.wq_gemm.restype = ci
    lib.wq_gemv.argtypes = gemm_args
    lib.wq_gemv.restype = ci
    lib.wq_gemm_ln_ws.argtypes = gemm_args[:6] + [vp] + gemm_args[6:-1] + [vp, sz, vp]
    lib.wq_gemm_ln_ws.restype = ci
    lib.wq_gemm_ln_workspace_bytes.argtypes = [ci, ci, ci, ci, cu]
    lib.wq_gemm_ln_workspace_bytes.restype = sz
    lib.wq_gemm_noalloc.argtypes = gemm_args
    lib.wq_gemm_noalloc.restype = ci
    lib.wq_gemm_ws.argtypes = gemm_args[:-1] + [vp, sz, vp]
    lib.wq_gemm_ws.restype = ci
    lib.wq_gemm_workspace_bytes.argtypes = [ci, ci, ci, ci, cu]
    lib.wq_gemm_workspace_bytes.restype = sz
    lib.wq_moe_gemv.argtypes = [ci, ci, ci, ci, ci, ci, cu, vp, vp, vp, vp, vp, vp, vp]
    lib.wq_moe_gemv.restype = ci
    lib.wq_weight_bytes.argtypes = [ci, ci, ci]
    lib.wq_weight_bytes.restype = sz
    lib.wq_dequantize.argtypes = [ci, ci, ci, vp, vp, vp]
    lib.wq_dequantize.restype = ci
    lib.wq_gemm_alpha.argtypes = [ci, ci, ci, ci, ctypes.c_uint, ctypes.c_float, vp, vp, vp, vp,
                                  vp, vp, sz, vp]
    lib.wq_gemm_alpha.restype = ci
    lib.wq_gemm_dual.argtypes = [ci, ci, ci, ci, ci, ctypes.c_uint, ctypes.c_float, vp, vp, vp, vp,
                                 vp, vp, vp, sz, vp]
    lib.wq_gemm_dual.restype = ci
    lib.wq_embed.argtypes = [ci, ci, ci, ci, vp, vp, vp, vp, vp, vp]
    lib.wq_embed.restype = ci
    cp = ctypes.POINTER(KvCache)
    lib.wq_rope_table.argtypes = [ci, ci, ctypes.c_double, ctypes.POINTER(RopeScaling), vp, vp]
    lib.wq_rope_table.restype = ci
    i64, cf = ctypes.c_int64, ctypes.c_float
    lib.wq_rope.argtypes = [ci, ci, ci, ci, cu, vp, i64, vp, vp, ci, vp, i64, vp]
    lib.wq_rope.restype = ci
    lib.wq_kv_append.argtypes = [cp, ci, ci, ci, cu, vp, i64, vp, i64, vp, i64, vp, vp, ci, ci, vp,
                                 vp, vp, ci, vp, i64, vp, vp, i64, vp]
    lib.wq_kv_append.restype = ci
    lib.wq_attn_paged.argtypes = [cp, ci, ci, cf, ci, vp, i64, vp, ci, vp, vp, i64, vp, i64, vp, vp,
                                  vp, i64, vp, sz, vp]
    lib.wq_attn_paged.restype = ci
    lib.wq_kv_evict.argtypes = [cp, ci, vp, ci, vp, vp, ci, ci, ci, vp, vp, vp, vp, i64, vp, vp, sz,
                                vp]
    lib.wq_kv_evict.restype = ci
    lib.wq_attn_paged_workspace_bytes.argtypes = [cp, ci, ci, ci, ci]
    lib.wq_attn_paged_workspace_bytes.restype = sz
    lib.wq_kv_evict_workspace_bytes.argtypes = [cp, ci, ci, ci]
    lib.wq_kv_evict_workspace_bytes.restype = sz
    np_, xp, fp = (ctypes.POINTER(t) for t in (HeadNorm, RopeAxes, AttnForm))
    lib.wq_norm_rope.argtypes = [ci, ci, ci, np_, xp, vp, i64, ci, vp, i64, vp]
    lib.wq_norm_rope.restype = ci
    lib.wq_norm_rope_grad.argtypes = [ci, ci, ci, np_, xp, vp, i64, vp, i64, vp, i64, vp, vp, vp,
                                      sz, vp]
    lib.wq_norm_rope_grad.restype = ci
    lib.wq_norm_rope_grad_workspace_bytes.argtypes = [ci, ci, ci]
    lib.wq_norm_rope_grad_workspace_bytes.restype = sz
    lib.wq_kv_append_norm.argtypes = [cp, ci, ci, np_, np_, xp, vp, i64, vp, i64, vp, i64, ci, vp,
                                      vp, vp, ci, ci, vp, i64, vp, vp, i64, vp]
    lib.wq_kv_append_norm.restype = ci
    lib.wq_attn_tokens.argtypes = [cp, ci, ci, ci, cf, fp, ci, vp, i64, vp, vp, ci, vp, ci, vp,
                                   i64, vp, vp, sz, vp]
    lib.wq_attn_tokens.restype = ci
    lib.wq_attn_tokens_workspace_bytes.argtypes = [cp, ci, ci, ci, ci]
    lib.wq_attn_tokens_workspace_bytes.restype = sz
    lib.wq_kv_accept.argtypes = [cp, ci, ci, ci, vp, ci, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp]
    lib.wq_kv_accept.restype = ci
    lib.wq_kv_accept_slots.argtypes = lib.wq_kv_accept.argtypes[:-1] + [
        ctypes.POINTER(SlotArrays), i64, vp]
    lib.wq_kv_accept_slots.restype = ci
    lib.wq_get_device_status.argtypes = [vp]
    lib.wq_get_device_status.restype = ci
    lib.wq_status_string.argtypes = [ci]
    lib.wq_status_string.restype = ctypes.c_char_p
    lib.wq_set_wait_limit.argtypes = [ctypes.c_uint64]
    lib.wq_set_wait_limit.restype = None
    return lib


def load():
    """The process-wide libwq handle (raises if the library has not been built)."""
    global _lib
    if _lib is not None:  # set once, under the lock
        return _lib
    with _lock:
        if _lib is None:
            _lib = _open(LIB_PATH)
        return _lib


_calls = None


_CALLS = ("wq_rope", "wq_kv_append", "wq_attn_paged", "wq_kv_evict")
_TOKEN_CALLS = ("wq_norm_rope", "wq_norm_rope_grad", "wq_kv_append_norm", "wq_attn_tokens",
                "wq_kv_accept")


def _through_ctypes(f):
    kinds = f.argtypes[:-1]

    def call(*args):
        if len(args) != len(f.argtypes):
            raise TypeError(f"{len(f.argtypes)} arguments are wanted, got {len(args)}")
        return f(*(_p(x) if t is ctypes.c_void_p else
                   operator.index(x) if t in (ctypes.c_int, ctypes.c_uint, ctypes.c_int64,
                                              ctypes.c_size_t) else x
                   for x, t in zip(args, kinds)), _s(args[-1]))
    return call


def _load_calls():
    """The marshalling module of the decode-step calls, bound to the process-wide libwq; the
    same calls through ctypes (some microseconds slower) where it was not built."""
    global _calls
    lib = load()
    with _lock:
        if _calls is None and not os.path.exists(CALLS_PATH):
            _calls = types.SimpleNamespace(**{f: _through_ctypes(getattr(lib, f))
                                              for f in _CALLS + _TOKEN_CALLS})
        if _calls is None:
            spec = importlib.util.spec_from_file_location("_wq_calls", CALLS_PATH)
            mod = importlib.util.module_from_spec(spec)
            spec.loader.exec_module(mod)
            mod.bind(*(ctypes.cast(getattr(lib, f), ctypes.c_void_p).value
                       for f in _CALLS),
                     _current_stream, KvCache)
            mod.bind_tokens(*(ctypes.cast(getattr(lib, f), ctypes.c_void_p).value
                              for f in _TOKEN_CALLS),
                            HeadNorm, RopeAxes, AttnForm)
            _calls = mod
        return _calls


def _p(x):
    if x is None:
        return None
    if isinstance(x, int):
        return x
    return x.data_ptr()


_raw_stream = None


def _current_stream():
    """torch's current stream of the current device as a cudaStream_t."""
    global _raw_stream
    if _raw_stream is None:
        import torch
        torch.cuda.init()
        get, device = (getattr(torch._C, name, None)
                       for name in ("_cuda_getCurrentRawStream", "_cuda_getDevice"))
        # The raw getter takes 0.1 us where a Stream object takes 2.8 us on the host.
        _raw_stream = (lambda: get(device())) if get and device else \
            (lambda: torch.cuda.current_stream().cuda_stream)
    return _raw_stream()


def _s(stream):
    if stream is None:
        return _current_stream()
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def wq_gemm(n, m, k, wtype, flags, X, W, bias=None, residual=None, Y=None, stream=None) -> int:
    return load().wq_gemm(n, m, k, wtype, flags, _p(X), _p(W), _p(bias), _p(residual), _p(Y),
                          _s(stream))


def wq_gemm_ws(n, m, k, wtype, flags, X, W, bias=None, residual=None, Y=None, workspace=None,
               workspace_bytes=0, stream=None) -> int:
    return load().wq_gemm_ws(n, m, k, wtype, flags, _p(X), _p(W), _p(bias), _p(residual), _p(Y),
                             _p(workspace), int(workspace_bytes), _s(stream))


def wq_gemm_noalloc(n, m, k, wtype, flags, X, W, bias=None, residual=None, Y=None,
                    stream=None) -> int:
    return load().wq_gemm_noalloc(n, m, k, wtype, flags, _p(X), _p(W), _p(bias), _p(residual),
                                  _p(Y), _s(stream))


def wq_gemm_ln_ws(n, m, k, wtype, flags, X, ln_gb, W, bias=None, residual=None, Y=None,
                  workspace=None, workspace_bytes=0, stream=None) -> int:
    return load().wq_gemm_ln_ws(n, m, k, wtype, flags, _p(X), _p(ln_gb), _p(W), _p(bias),
                                _p(residual), _p(Y), _p(workspace), int(workspace_bytes),
                                _s(stream))


def wq_gemm_ln_workspace_bytes(n, m, k, wtype, flags) -> int:
    return int(load().wq_gemm_ln_workspace_bytes(n, m, k, wtype, flags))


def wq_gemm_workspace_bytes(n, m, k, wtype, flags) -> int:
    return int(load().wq_gemm_workspace_bytes(n, m, k, wtype, flags))


def wq_gemv(n, m, k, wtype, flags, X, W, bias=None, residual=None, Y=None, stream=None) -> int:
    return load().wq_gemv(n, m, k, wtype, flags, _p(X), _p(W), _p(bias), _p(residual), _p(Y),
                          _s(stream))


def wq_moe_gemv(n_tok, topk, n_experts, m, k, wtype, flags, X, Wbank, ids, bias=None,
                residual=None, Y=None, stream=None) -> int:
    return load().wq_moe_gemv(n_tok, topk, n_experts, m, k, wtype, flags, _p(X), _p(Wbank),
                              _p(ids), _p(bias), _p(residual), _p(Y), _s(stream))


def wq_weight_bytes(wtype, m, k) -> int:
    return int(load().wq_weight_bytes(wtype, m, k))


def wq_dequantize(wtype, m, k, W, out, stream=None) -> int:
    return load().wq_dequantize(wtype, m, k, _p(W), _p(out), _s(stream))


def wq_gemm_alpha(n, m, k, wtype, flags, alpha, X, W, bias=None, residual=None, Y=None,
                  workspace=None, workspace_bytes=0, stream=None) -> int:
    return load().wq_gemm_alpha(n, m, k, wtype, flags, float(alpha), _p(X), _p(W), _p(bias),
                                _p(residual), _p(Y), _p(workspace), int(workspace_bytes),
                                _s(stream))


def wq_gemm_dual(n, m, k, dual, wtype, flags, alpha, X, W, bias=None, bias2=None, residual=None,
                 Y=None, workspace=None, workspace_bytes=0, stream=None) -> int:
    return load().wq_gemm_dual(n, m, k, dual, wtype, flags, float(alpha), _p(X), _p(W), _p(bias),
                               _p(bias2), _p(residual), _p(Y), _p(workspace), int(workspace_bytes),
                               _s(stream))


def wq_embed(n_ids, rows, k, wtype, W, ids, pos=None, bias=None, out=None, stream=None) -> int:
    return load().wq_embed(n_ids, rows, k, wtype, _p(W), _p(ids), _p(pos), _p(bias), _p(out),
                           _s(stream))


def wq_rope_table(rows, rot, base, scaling, table, stream=None) -> int:
    return load().wq_rope_table(rows, rot, base, scaling, _p(table), _s(stream))


def wq_rope(n, n_heads, head_dim, rot, flags, x, x_stride, pos, table, table_rows, out,
            out_stride, stream=None) -> int:
    return (_calls or _load_calls()).wq_rope(n, n_heads, head_dim, rot, flags, x, x_stride, pos,
                                             table, table_rows, out, out_stride, stream)


def wq_kv_append(cache, n_tok, h_q, rot, flags, q, q_stride, k, k_stride, v, v_stride, pos, table,
                 table_rows, n_seq, seq, slot, page_table, max_pages, q_out=None, q_out_stride=0,
                 acc=None, slot_pos=None, acc_stride=0, stream=None) -> int:
    return (_calls or _load_calls()).wq_kv_append(
        cache, n_tok, h_q, rot, flags, q, q_stride, k, k_stride, v, v_stride, pos, table,
        table_rows, n_seq, seq, slot, page_table, max_pages, q_out, q_out_stride, acc, slot_pos,
        acc_stride, stream)


def wq_attn_paged(cache, n_seq, h_q, scale, window, q, q_stride, page_table, max_pages, lens,
                  mask=None, mask_stride=0, out=None, out_stride=0, lse=None, acc_in=None,
                  acc_out=None, acc_stride=0, workspace=None, workspace_bytes=0,
                  stream=None) -> int:
    return (_calls or _load_calls()).wq_attn_paged(
        cache, n_seq, h_q, scale, window, q, q_stride, page_table, max_pages, lens, mask,
        mask_stride, out, out_stride, lse, acc_in, acc_out, acc_stride, workspace,
        workspace_bytes, stream)


def wq_attn_paged_workspace_bytes(cache, n_seq, h_q, max_pages, with_acc) -> int:
    return load().wq_attn_paged_workspace_bytes(cache, n_seq, h_q, max_pages, int(with_acc))


def wq_kv_evict(cache, n_seq, page_table, max_pages, lens, seen, keep, sinks, recent, acc,
                slot_pos, acc_out, pos_out, acc_stride, lens_out, workspace=None,
                workspace_bytes=0, stream=None) -> int:
    return (_calls or _load_calls()).wq_kv_evict(
        cache, n_seq, page_table, max_pages, lens, seen, keep, sinks, recent, acc, slot_pos,
        acc_out, pos_out, acc_stride, lens_out, workspace, workspace_bytes, stream)


def wq_kv_evict_workspace_bytes(cache, n_seq, max_pages, keep) -> int:
    return load().wq_kv_evict_workspace_bytes(cache, n_seq, max_pages, keep)


def wq_norm_rope(n, n_heads, head_dim, norm, rope, x, x_stride, out_type, out, out_stride,
                 stream=None) -> int:
    return (_calls or _load_calls()).wq_norm_rope(n, n_heads, head_dim, norm, rope, x, x_stride,
                                                  out_type, out, out_stride, stream)


def wq_norm_rope_grad(n, n_heads, head_dim, norm, rope, x, x_stride, grad_out, grad_out_stride,
                      grad_x, grad_x_stride, grad_weight=None, grad_bias=None, workspace=None,
                      workspace_bytes=0, stream=None) -> int:
    return (_calls or _load_calls()).wq_norm_rope_grad(
        n, n_heads, head_dim, norm, rope, x, x_stride, grad_out, grad_out_stride, grad_x,
        grad_x_stride, grad_weight, grad_bias, workspace, workspace_bytes, stream)


def wq_norm_rope_grad_workspace_bytes(n, n_heads, head_dim) -> int:
    return load().wq_norm_rope_grad_workspace_bytes(n, n_heads, head_dim)


def wq_kv_append_norm(cache, n_tok, h_q, q_norm, k_norm, rope, q, q_stride, k, k_stride, v,
                      v_stride, n_seq, seq, slot, page_table, max_pages, q_type=WQ_F32,
                      q_out=None, q_out_stride=0, acc=None, slot_pos=None, acc_stride=0,
                      stream=None) -> int:
    return (_calls or _load_calls()).wq_kv_append_norm(
        cache, n_tok, h_q, q_norm, k_norm, rope, q, q_stride, k, k_stride, v, v_stride, n_seq, seq,
        slot, page_table, max_pages, q_type, q_out, q_out_stride, acc, slot_pos, acc_stride, stream)


def wq_attn_tokens(cache, n_seq, n_tok, h_q, scale, form, q_type, q, q_stride, starts, page_table,
                   max_pages, lens, out_type, out, out_stride, lse=None, workspace=None,
                   workspace_bytes=0, stream=None) -> int:
    return (_calls or _load_calls()).wq_attn_tokens(
        cache, n_seq, n_tok, h_q, scale, form, q_type, q, q_stride, starts, page_table, max_pages,
        lens, out_type, out, out_stride, lse, workspace, workspace_bytes, stream)


def wq_attn_tokens_workspace_bytes(cache, n_seq, n_tok, h_q, q_type) -> int:
    return load().wq_attn_tokens_workspace_bytes(cache, n_seq, n_tok, h_q, q_type)


def wq_kv_accept(caches, n_seq, n_tok, page_table, max_pages, starts, parent, tokens, choice, lens,
                 path, accepted, next, lens_out, stream=None) -> int:
    """caches: kv_caches(...), or one KvCache."""
    if isinstance(caches, KvCache):
        caches = (KvCache * 1)(caches)
    return (_calls or _load_calls()).wq_kv_accept(
        caches, len(caches), n_seq, n_tok, page_table, max_pages, starts, parent, tokens, choice,
        lens, path, accepted, next, lens_out, stream)


def wq_kv_accept_slots(caches, n_seq, n_tok, page_table, max_pages, starts, parent, tokens, choice,
                       lens, path, accepted, next, lens_out, slots, acc_stride,
                       stream=None) -> int:
    """caches as wq_kv_accept's; slots: slot_arrays(...), one for each cache, or one SlotArrays."""
    if isinstance(caches, KvCache):
        caches = (KvCache * 1)(caches)
    if isinstance(slots, SlotArrays):
        slots = (SlotArrays * 1)(slots)
    if slots is not None and len(slots) != len(caches):
        raise TypeError("slots: not as many as the caches")
    return load().wq_kv_accept_slots(
        caches, len(caches), n_seq, n_tok, _p(page_table), max_pages, _p(starts), _p(parent),
        _p(tokens), _p(choice), _p(lens), _p(path), _p(accepted), _p(next), _p(lens_out), slots,
        acc_stride, _s(stream))


def wq_get_device_status(stream=None) -> int:
    return load().wq_get_device_status(_s(stream))


def wq_status_string(status) -> str:
    return load().wq_status_string(int(status)).decode()


def wq_set_wait_limit(polls: int) -> None:
    load().wq_set_wait_limit(int(polls))


def check(status: int, what: str = "") -> None:
    """Raise WqError unless ``status`` is WQ_OK."""
    if status != WQ_OK:
        raise WqError(status, what)
