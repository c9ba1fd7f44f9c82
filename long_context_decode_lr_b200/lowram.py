"""Python binding of liblowram.so: the C entry points of include/lowram.h under the same
names, with torch CUDA tensors in place of device pointers.

This layer only marshals arguments: every step of the compressed-cache path runs
in the library's CUDA kernels. A missing library raises at import of the first
call; there is no other implementation to fall back to.
"""
from __future__ import annotations

import ctypes
import os
from typing import Optional

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "liblowram.so")

LR_OK, LR_ERR_INVALID_ARG, LR_ERR_UNSUPPORTED, LR_ERR_WORKSPACE, LR_ERR_CUDA, LR_ERR_DEVICE_CHECK = range(6)
LR_F32, LR_BF16 = 0, 1
LR_BLOCK_TOKENS = 64
LR_MAX_TAIL = 4096
LR_DEVERR_BLOCK_RANGE, LR_DEVERR_BLOCK_ORDER, LR_DEVERR_RES_RANGE, LR_DEVERR_RES_ORDER, LR_DEVERR_PTR = 1, 2, 4, 8, 16
LR_DEVERR_TIMEOUT, LR_DEVERR_LAUNCH, LR_DEVERR_PAGE, LR_DEVERR_LEN = 32, 64, 128, 256

_DT = {torch.float32: LR_F32, torch.bfloat16: LR_BF16}


class LowRAMError(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__(f"{message} (status {status})")
        self.status = status


class lr_cache_shape(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int32), ("T", ctypes.c_int32), ("n_layers", ctypes.c_int32),
                ("n_kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32), ("rank", ctypes.c_int32),
                ("hidden", ctypes.c_int32), ("dtype", ctypes.c_int32)]


class lr_predictor(ctypes.Structure):
    _fields_ = [("W_lin", ctypes.c_void_p), ("W1", ctypes.c_void_p), ("b1", ctypes.c_void_p),
                ("W2", ctypes.c_void_p), ("b2", ctypes.c_void_p), ("per_sequence", ctypes.c_int32)]


class lr_predictor_f32(ctypes.Structure):
    _fields_ = [("W_lin", ctypes.c_void_p), ("W1", ctypes.c_void_p), ("b1", ctypes.c_void_p),
                ("W2", ctypes.c_void_p), ("b2", ctypes.c_void_p), ("per_sequence", ctypes.c_int32)]


class lr_predictor_out(ctypes.Structure):
    _fields_ = [("W_lin", ctypes.c_void_p), ("W1", ctypes.c_void_p), ("b1", ctypes.c_void_p),
                ("W2", ctypes.c_void_p), ("b2", ctypes.c_void_p)]


class lr_kv8_pages(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int32), ("n_kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32),
                ("n_pages", ctypes.c_int32), ("max_pages", ctypes.c_int32), ("dtype", ctypes.c_int32),
                ("page_stride", ctypes.c_int64), ("k_codes", ctypes.c_void_p), ("v_codes", ctypes.c_void_p),
                ("k_scale", ctypes.c_void_p), ("v_scale", ctypes.c_void_p), ("page_table", ctypes.c_void_p),
                ("lens", ctypes.c_void_p)]


class lr_rope(ctypes.Structure):
    _fields_ = [("inv_freq", ctypes.c_void_p), ("rot_dim", ctypes.c_int32), ("interleaved", ctypes.c_int32)]


_lib = None
_P = ctypes.c_void_p
_I = ctypes.c_int32
_Z = ctypes.c_size_t


def library() -> ctypes.CDLL:
    """Load liblowram.so (built in-tree); raises if it is missing."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build it with "
                               "`python -m long_context_decode_lr_b200.build`")
        lib = ctypes.CDLL(LIB_PATH)
        S, Pr = ctypes.POINTER(lr_cache_shape), ctypes.POINTER(lr_predictor)
        K8, L = ctypes.POINTER(lr_kv8_pages), ctypes.c_int64
        sig = {
            "lr_pack_workspace_bytes": (_Z, [S, _I]),
            "lr_pack_prefill": (_I, [S, _P, _P, _P, Pr, _I, _P, _P, _P, _P, _P, _P, _Z, _P]),
            "lr_decode_workspace_bytes": (_Z, [S, _I, _I]),
            "lr_decode_attn": (_I, [S, _I, _I, _P, _P, _P, Pr, _P, _P, _P, _I, _P, _I, ctypes.c_float,
                                    _P, _P, _Z, _P]),
            "lr_decode_attn_noalloc": (_I, [S, _I, _I, _P, _P, _P, Pr, _P, _P, _P, _I, _P, _I, ctypes.c_float,
                                            _P, _P]),
            "lr_decode_attn_tail": (_I, [S, _I, _I, _P, _P, _P, Pr, _P, _P, _P, _I, _P, _I, _P, _P, _I,
                                         ctypes.c_float, _P, _P, _Z, _P]),
            "lr_select_workspace_bytes": (_Z, [S, _I]),
            "lr_block_means": (_I, [S, _P, _P, _P]),
            "lr_fit_workspace_bytes": (_Z, [S, _I]),
            "lr_fit_predictor": (_I, [S, _P, _P, _P, ctypes.POINTER(lr_predictor_f32), _I, ctypes.c_float,
                                      ctypes.POINTER(lr_predictor_out), _P, _Z, _P]),
            "lr_quantize_residuals": (_I, [S, ctypes.c_int64, _P, _P, _P, _P, _P]),
            "lr_decode_attn_q2": (_I, [S, _I, _I, _P, _P, _P, Pr, _P, _P, _P, _P, _P, _I, _P, _I, ctypes.c_float,
                                       _P, _P, _Z, _P]),
            "lr_select_blocks": (_I, [S, _I, _I, _P, _P, _P, _I, ctypes.c_float, _P, _P, _P, _Z, _P]),
            "lr_topk_workspace_bytes": (_Z, [_I, _I, _I]),
            "lr_topk_tokens": (_I, [_P, _I, _I, _I, _P, _P, _Z, _P]),
            "lr_residual_block_ptr": (_I, [_P, _I, _I, _I, _P, _P]),
            "lr_decode_attn_lse": (_I, [S, _I, _I, _P, _P, _P, Pr, _P, _P, _P, _I, _P, _I, ctypes.c_float,
                                        _P, _P, _P, _Z, _P]),
            "lr_kv8_append_workspace_bytes": (_Z, [K8]),
            "lr_kv8_append": (_I, [K8, _I, _I, _P, ctypes.POINTER(lr_rope), _P, L, _P, L, _P, L, _P, _P, _Z, _P]),
            "lr_kv8_attn_workspace_bytes": (_Z, [K8, _I]),
            "lr_decode_attn_kv8": (_I, [K8, _I, _P, _I, ctypes.c_float, _P, _P, _P, _P, _P, _Z, _P]),
            "lr_get_device_error": (_I, [_P, _P, ctypes.POINTER(_I)]),
            "lr_status_string": (ctypes.c_char_p, [_I]),
            "lr_last_error": (ctypes.c_char_p, []),
            "lr_abi_version": (_I, []),
        }
        for name, (res, args) in sig.items():
            f = getattr(lib, name)
            f.restype, f.argtypes = res, args
        _lib = lib
    return _lib


def _ptr(t: Optional[torch.Tensor]) -> Optional[int]:
    if t is None:
        return None
    if not isinstance(t, torch.Tensor):
        raise TypeError("expected a torch.Tensor or None")
    if not t.is_cuda:
        raise ValueError("tensor must live on a CUDA device")
    if not t.is_contiguous():
        raise ValueError("tensor must be contiguous")
    return t.data_ptr() or None


def _stream(stream) -> Optional[int]:
    if stream is None:
        stream = torch.cuda.current_stream()
    return getattr(stream, "cuda_stream", stream) or None


def _check(status: int) -> None:
    if status != LR_OK:
        lib = library()
        raise LowRAMError(status, lib.lr_last_error().decode() or lib.lr_status_string(status).decode())


def cache_shape(batch: int, T: int, n_layers: int, n_kv_heads: int, head_dim: int, rank: int,
                hidden: int, dtype) -> lr_cache_shape:
    dt = _DT[dtype] if isinstance(dtype, torch.dtype) else int(dtype)
    return lr_cache_shape(batch, T, n_layers, n_kv_heads, head_dim, rank, hidden, dt)


class Predictor:
    """Holds the predictor tensors alive and exposes the C struct."""

    def __init__(self, W_lin, W1, b1, W2, b2=None, per_sequence: bool = True):
        self.tensors = (W_lin, W1, b1, W2, b2)
        self.c = lr_predictor(_ptr(W_lin), _ptr(W1), _ptr(b1), _ptr(W2), _ptr(b2), int(per_sequence))


def lr_abi_version() -> int:
    return library().lr_abi_version()


def lr_pack_workspace_bytes(shape: lr_cache_shape, k: int) -> int:
    return library().lr_pack_workspace_bytes(ctypes.byref(shape), k)


def lr_pack_prefill(shape, K_group, V, Bt, predictor: Predictor, k, A, res_idx, res_val,
                    res_blk_ptr=None, err_out=None, ws=None, stream=None) -> None:
    _check(library().lr_pack_prefill(
        ctypes.byref(shape), _ptr(K_group), _ptr(V), _ptr(Bt), ctypes.byref(predictor.c), k, _ptr(A),
        _ptr(res_idx), _ptr(res_val), _ptr(res_blk_ptr), _ptr(err_out), _ptr(ws),
        0 if ws is None else ws.numel() * ws.element_size(), _stream(stream)))


def lr_decode_workspace_bytes(shape: lr_cache_shape, n_q_heads: int, n_sel: int = 0) -> int:
    return library().lr_decode_workspace_bytes(ctypes.byref(shape), n_q_heads, n_sel)


def lr_decode_attn(shape, layer, n_q_heads, q, A, Bt, predictor: Predictor, res_idx, res_val,
                   res_blk_ptr, k, block_list, n_sel, scale, o, ws, stream=None) -> None:
    _check(library().lr_decode_attn(
        ctypes.byref(shape), layer, n_q_heads, _ptr(q), _ptr(A), _ptr(Bt), ctypes.byref(predictor.c),
        _ptr(res_idx), _ptr(res_val), _ptr(res_blk_ptr), k, _ptr(block_list), n_sel, float(scale),
        _ptr(o), _ptr(ws), 0 if ws is None else ws.numel() * ws.element_size(), _stream(stream)))


def lr_fit_workspace_bytes(shape: lr_cache_shape, per_sequence: bool = True) -> int:
    return library().lr_fit_workspace_bytes(ctypes.byref(shape), int(per_sequence))


def lr_fit_predictor(shape, A, Bt, V, params, n_steps, lr, ws, out=None, per_sequence=True, stream=None) -> None:
    """Fit the predictor to the context: params = (W_lin, W1, b1, W2, b2 or None), fp32 tensors
    updated in place; out = the same five in the cache dtype (written after the last step) or None."""
    p = lr_predictor_f32(*[_ptr(t) for t in params], int(per_sequence))
    o = None if out is None else ctypes.byref(lr_predictor_out(*[_ptr(t) for t in out]))
    _check(library().lr_fit_predictor(ctypes.byref(shape), _ptr(A), _ptr(Bt), _ptr(V), ctypes.byref(p), int(n_steps),
                                      float(lr), o, _ptr(ws), 0 if ws is None else ws.numel() * ws.element_size(),
                                      _stream(stream)))


def lr_quantize_residuals(shape, n_rows, res_val, res_codes, res_lo, res_step, stream=None) -> None:
    """2-bit codes [n_rows, hd / 4] uint8 plus row minimum and step (fp32) of residual rows."""
    _check(library().lr_quantize_residuals(ctypes.byref(shape), int(n_rows), _ptr(res_val), _ptr(res_codes),
                                           _ptr(res_lo), _ptr(res_step), _stream(stream)))


def lr_decode_attn_q2(shape, layer, n_q_heads, q, A, Bt, predictor: Predictor, res_idx, res_codes, res_lo,
                      res_step, res_blk_ptr, k, block_list, n_sel, scale, o, ws, stream=None) -> None:
    """lr_decode_attn with 2-bit residual rows (codes, row minimum, step)."""
    _check(library().lr_decode_attn_q2(
        ctypes.byref(shape), layer, n_q_heads, _ptr(q), _ptr(A), _ptr(Bt), ctypes.byref(predictor.c),
        _ptr(res_idx), _ptr(res_codes), _ptr(res_lo), _ptr(res_step), _ptr(res_blk_ptr), k, _ptr(block_list),
        n_sel, float(scale), _ptr(o), _ptr(ws), 0 if ws is None else ws.numel() * ws.element_size(),
        _stream(stream)))


def lr_decode_attn_noalloc(shape, layer, n_q_heads, q, A, Bt, predictor: Predictor, res_idx, res_val,
                           res_blk_ptr, k, block_list, n_sel, scale, o, stream=None) -> None:
    """lr_decode_attn on the library's static scratch area (no workspace, no allocation)."""
    _check(library().lr_decode_attn_noalloc(
        ctypes.byref(shape), layer, n_q_heads, _ptr(q), _ptr(A), _ptr(Bt), ctypes.byref(predictor.c),
        _ptr(res_idx), _ptr(res_val), _ptr(res_blk_ptr), k, _ptr(block_list), n_sel, float(scale),
        _ptr(o), _stream(stream)))


def lr_decode_attn_lse(shape, layer, n_q_heads, q, A, Bt, predictor: Predictor, res_idx, res_val,
                       res_blk_ptr, k, block_list, n_sel, scale, o, lse, ws, stream=None) -> None:
    """lr_decode_attn that also returns the log-sum-exp of every query head, lse [B, Hq] fp32."""
    _check(library().lr_decode_attn_lse(
        ctypes.byref(shape), layer, n_q_heads, _ptr(q), _ptr(A), _ptr(Bt), ctypes.byref(predictor.c),
        _ptr(res_idx), _ptr(res_val), _ptr(res_blk_ptr), k, _ptr(block_list), n_sel, float(scale),
        _ptr(o), _ptr(lse), _ptr(ws), 0 if ws is None else ws.numel() * ws.element_size(), _stream(stream)))


def lr_decode_attn_tail(shape, layer, n_q_heads, q, A, Bt, predictor: Predictor, res_idx, res_val,
                        res_blk_ptr, k, block_list, n_sel, tail_K, tail_V, n_tail, scale, o, ws,
                        stream=None) -> None:
    """lr_decode_attn plus an exact recent-token tail tail_K / tail_V [B, Hkv, n_tail, hd]."""
    _check(library().lr_decode_attn_tail(
        ctypes.byref(shape), layer, n_q_heads, _ptr(q), _ptr(A), _ptr(Bt), ctypes.byref(predictor.c),
        _ptr(res_idx), _ptr(res_val), _ptr(res_blk_ptr), k, _ptr(block_list), n_sel, _ptr(tail_K),
        _ptr(tail_V), n_tail, float(scale), _ptr(o), _ptr(ws), 0 if ws is None else ws.numel() * ws.element_size(),
        _stream(stream)))


def lr_select_workspace_bytes(shape: lr_cache_shape, n_q_heads: int) -> int:
    return library().lr_select_workspace_bytes(ctypes.byref(shape), n_q_heads)


def lr_block_means(shape, A, Abar, stream=None) -> None:
    """Abar [B, nblk, r] fp32: the mean A row of every 64-token block (query-independent)."""
    _check(library().lr_block_means(ctypes.byref(shape), _ptr(A), _ptr(Abar), _stream(stream)))


def lr_select_blocks(shape, layer, n_q_heads, q, Abar, Bt, n_sel, scale, block_list, ws, scores_out=None,
                     stream=None) -> None:
    """The n_sel blocks per (sequence, KV head) whose mean rebuilt key best matches the query;
    scores_out [B, Hkv, nblk] fp32 (optional) receives the scores the list was taken from."""
    _check(library().lr_select_blocks(
        ctypes.byref(shape), layer, n_q_heads, _ptr(q), _ptr(Abar), _ptr(Bt), n_sel, float(scale),
        _ptr(block_list), _ptr(scores_out), _ptr(ws), 0 if ws is None else ws.numel() * ws.element_size(),
        _stream(stream)))


def lr_topk_workspace_bytes(n_segments: int, T: int, k: int) -> int:
    return library().lr_topk_workspace_bytes(n_segments, T, k)


def lr_topk_tokens(err, n_segments, T, k, idx_out, ws, stream=None) -> None:
    _check(library().lr_topk_tokens(_ptr(err), n_segments, T, k, _ptr(idx_out), _ptr(ws),
                                    0 if ws is None else ws.numel() * ws.element_size(), _stream(stream)))


def lr_residual_block_ptr(idx, n_segments, k, T, ptr_out, stream=None) -> None:
    _check(library().lr_residual_block_ptr(_ptr(idx), n_segments, k, T, _ptr(ptr_out), _stream(stream)))


# ---- 8-bit paged cache


class Kv8Pages:
    """An 8-bit paged cache of one layer: holds the tensors alive and exposes the C struct.

    k_codes, v_codes [n_pages, Hkv, 64, hd] uint8 (e4m3 codes; pages dense inside, any equal distance
    between pages), k_scale, v_scale [n_pages, Hkv] fp32, page_table [B, max_pages] int32, lens [B]
    int32; dtype is that of q, k, v and o beside the cache."""

    def __init__(self, k_codes, v_codes, k_scale, v_scale, page_table, lens, dtype):
        self.tensors = (k_codes, v_codes, k_scale, v_scale, page_table, lens)
        if k_codes.dim() != 4 or k_codes.shape != v_codes.shape or k_codes.shape[2] != LR_BLOCK_TOKENS:
            raise ValueError("k_codes and v_codes must both be [n_pages, Hkv, 64, hd]")
        n_pages, hkv, _, hd = k_codes.shape
        if page_table.dim() != 2 or tuple(lens.shape) != (page_table.shape[0],):
            raise ValueError("page_table must be [B, max_pages] and lens [B]")
        if tuple(k_scale.shape) != (n_pages, hkv) or tuple(v_scale.shape) != (n_pages, hkv):
            raise ValueError("k_scale and v_scale must be [n_pages, Hkv]")
        want = (torch.uint8, torch.uint8, torch.float32, torch.float32, torch.int32, torch.int32)
        if tuple(t.dtype for t in self.tensors) != want:
            raise ValueError("codes must be uint8, scales float32, page_table and lens int32")
        if any(t.device != k_codes.device for t in self.tensors):
            raise ValueError("the cache's tensors must live on one device")
        codes = []
        for t in (k_codes, v_codes):
            if not t.is_cuda:
                raise ValueError("tensor must live on a CUDA device")
            if n_pages and not t[0].is_contiguous():
                raise ValueError("a page must be contiguous")
            codes.append(t.data_ptr() or None)
        stride = k_codes.stride(0) if n_pages > 1 else 0
        if n_pages > 1 and v_codes.stride(0) != stride:
            raise ValueError("k_codes and v_codes must have the same distance between pages")
        self.device, self.dtype = k_codes.device, dtype
        self._index = k_codes.get_device()
        self.batch, self.n_kv_heads, self.head_dim = page_table.shape[0], hkv, hd
        self.c = lr_kv8_pages(self.batch, hkv, hd, n_pages, page_table.shape[1], _DT[dtype], stride, *codes,
                              _ptr(k_scale), _ptr(v_scale), _ptr(page_table), _ptr(lens))
        self.ref = ctypes.byref(self.c)

    # These run on every call of a decode step: plain comparisons of a tensor's type, device index, shape and strides.
    def _dense_rows(self, t, n_rows, n_heads, name):
        """Address of a dense [n_rows, n_heads, hd] tensor of the cache's dtype and device."""
        if t.dtype is not self.dtype or t.get_device() != self._index or t.shape != (n_rows, n_heads, self.head_dim):
            raise self._wrong_rows(n_rows, n_heads, name)
        if not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous")
        return t.data_ptr() or None

    def _token_rows(self, t, n_rows, n_heads, name):
        """(address, elements from one token to the next, 0 for one token): the rows of a token are dense."""
        hd = self.head_dim
        if t.dtype is not self.dtype or t.get_device() != self._index or t.shape != (n_rows, n_heads, hd):
            raise self._wrong_rows(n_rows, n_heads, name)
        token, head, dim = t.stride()
        if hd > 1 and dim != 1 or n_heads > 1 and head != hd:
            raise ValueError(f"{name}: the heads of a token must be contiguous")
        if n_rows < 2:
            token = 0
        elif token < n_heads * hd:
            raise ValueError(f"{name}: the rows of two tokens must not overlap")
        return t.data_ptr() or None, token

    def _wrong_rows(self, n_rows, n_heads, name):
        return ValueError(f"{name} must be a {self.dtype} tensor [{n_rows}, {n_heads}, {self.head_dim}] on {self.device}")

    def _beside(self, t, dtype, shape, name):
        if t.dtype is not dtype or t.get_device() != self._index or t.shape != shape or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous {dtype} tensor {list(shape)} on {self.device}")
        return t.data_ptr() or None

    def _call(self, entry, args, ws, stream):
        """Run an entry point on the cache's device, on its current stream unless one is given."""
        ptr = size = None
        if ws is not None:
            if ws.get_device() != self._index or not ws.is_contiguous():
                raise ValueError(f"the workspace must be contiguous and live on {self.device}")
            ptr, size = ws.data_ptr() or None, ws.nbytes
        if stream is None:
            stream = torch._C._cuda_getCurrentRawStream(self._index) or None
        else:
            stream = getattr(stream, "cuda_stream", stream) or None
        if torch.cuda.current_device() == self._index:
            status = entry(*args, ptr, size or 0, stream)
        else:
            with torch.cuda.device(self.device):
                status = entry(*args, ptr, size or 0, stream)
        if status:
            _check(status)


class Rope:
    """Rotary embedding of the first rot_dim dims: inv_freq [rot_dim / 2] fp32, radians per token."""

    def __init__(self, inv_freq, rot_dim: int, interleaved: bool = False):
        if inv_freq.dtype != torch.float32 or inv_freq.numel() != rot_dim // 2:
            raise ValueError("inv_freq must be float32 with rot_dim / 2 entries")
        self.inv_freq = inv_freq
        self.c = lr_rope(_ptr(inv_freq), int(rot_dim), int(interleaved))
        self.ref = ctypes.byref(self.c)
        self.index = inv_freq.get_device()


def lr_kv8_append_workspace_bytes(kv: Kv8Pages) -> int:
    return library().lr_kv8_append_workspace_bytes(kv.ref)


def lr_kv8_append(kv: Kv8Pages, k, v, ws, cu_tokens=None, rope: Optional[Rope] = None, q=None, q_out=None,
                  stream=None) -> None:
    """New keys and values k, v [n, Hkv, hd] into their pages (kv.lens counts them already), keys and the
    queries q [n, Hq, hd] -> q_out rotated by position. k, v and q may be slices of one fused tensor.
    cu_tokens [B + 1] int32 gives each sequence's rows; without it every sequence has one."""
    n = k.shape[0]
    k_ptr, k_stride = kv._token_rows(k, n, kv.n_kv_heads, "k")
    v_ptr, v_stride = kv._token_rows(v, n, kv.n_kv_heads, "v")
    hq, q_ptr, q_stride, out_ptr = 0, None, 0, None
    if (q is None) != (q_out is None):
        raise ValueError("q and q_out go together")
    if q is not None:
        hq = q.shape[1]
        q_ptr, q_stride = kv._token_rows(q, n, hq, "q")
        out_ptr = kv._dense_rows(q_out, n, hq, "q_out")
    if rope is not None and rope.index != kv._index:
        raise ValueError(f"inv_freq must live on {kv.device}")
    cu = None if cu_tokens is None else kv._beside(cu_tokens, torch.int32, (kv.batch + 1,), "cu_tokens")
    kv._call(library().lr_kv8_append,
             (kv.ref, hq, n, cu, None if rope is None else rope.ref, q_ptr, q_stride, k_ptr, k_stride, v_ptr, v_stride,
              out_ptr), ws, stream)


def lr_kv8_attn_workspace_bytes(kv: Kv8Pages, n_q_heads: int) -> int:
    if torch.cuda.is_available() and torch.cuda.current_device() != kv.device.index:
        with torch.cuda.device(kv.device):
            return library().lr_kv8_attn_workspace_bytes(kv.ref, n_q_heads)
    return library().lr_kv8_attn_workspace_bytes(kv.ref, n_q_heads)


def lr_decode_attn_kv8(kv: Kv8Pages, n_q_heads, q, o, ws, lse=None, window=0, scale=0.0, o_prev=None, lse_prev=None,
                       stream=None) -> None:
    """One decode step over the 8-bit paged cache: q, o [B, Hq, hd]; lse [B, Hq] fp32 (optional);
    o_prev, lse_prev: an earlier partial result over other tokens, joined to the same softmax."""
    b, shape = kv.batch, (kv.batch, n_q_heads)
    args = (kv.ref, n_q_heads, kv._dense_rows(q, b, n_q_heads, "q"), min(int(window), 0x7fffffff), float(scale),
            None if o_prev is None else kv._dense_rows(o_prev, b, n_q_heads, "o_prev"),
            None if lse_prev is None else kv._beside(lse_prev, torch.float32, shape, "lse_prev"),
            kv._dense_rows(o, b, n_q_heads, "o"), None if lse is None else kv._beside(lse, torch.float32, shape, "lse"))
    kv._call(library().lr_decode_attn_kv8, args, ws, stream)


def lr_get_device_error(ws, stream=None) -> int:
    code = ctypes.c_int32(0)
    st = library().lr_get_device_error(_ptr(ws), _stream(stream), ctypes.byref(code))
    if st not in (LR_OK, LR_ERR_DEVICE_CHECK):
        _check(st)
    return code.value


def workspace(nbytes: int, device=None) -> torch.Tensor:
    """A caller-owned workspace tensor (256-byte aligned by the caching allocator)."""
    return torch.empty(max(int(nbytes), 256), dtype=torch.uint8, device=device or "cuda")
