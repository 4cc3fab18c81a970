"""ctypes binding of libmla_decode.so (include/mla_decode.h).

Argument marshalling only: tensors are passed as raw device pointers with their strides,
and every step of the decode path runs in the library's CUDA kernels. torch is used for
device memory and streams. Loading fails loudly if the library has not been built.
"""

from __future__ import annotations

import ctypes
import os
import struct
from typing import Optional, Tuple

import torch

LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libmla_decode.so")

MLA_OK = 0
MLA_ERR_INVALID_ARG = -1
MLA_ERR_UNSUPPORTED = -2
MLA_ERR_CUDA = -3
MLA_ERR_OOM = -4
MLA_ERR_DEVICE_CHECK = -5

ERR_BAD_PAGE = 1 << 0
ERR_TIMEOUT = 1 << 1
ERR_BAD_KV_LEN = 1 << 2

ROW = 576
D_LATENT = 512

ROW_TYPES = {torch.bfloat16: 0, torch.float32: 1}   # MLA_BF16, MLA_F32
_INT8 = (torch.int8,)


class MlaConfig(ctypes.Structure):
    _fields_ = [
        ("n_heads", ctypes.c_int32),
        ("d_head", ctypes.c_int32),
        ("d_latent", ctypes.c_int32),
        ("d_rope", ctypes.c_int32),
        ("page_size", ctypes.c_int32),
        ("max_batch", ctypes.c_int32),
        ("max_kv_len", ctypes.c_int64),
        ("softmax_scale", ctypes.c_float),
        ("rope_base", ctypes.c_float),
        ("max_splits", ctypes.c_int32),
        ("yarn_factor", ctypes.c_float),
        ("yarn_original_len", ctypes.c_int32),
        ("yarn_alpha", ctypes.c_float),
        ("yarn_beta", ctypes.c_float),
        ("yarn_mscale_coef", ctypes.c_float),
        ("q_len", ctypes.c_int32),
    ]


_P = ctypes.c_void_p
_I32 = ctypes.c_int32
_I64 = ctypes.c_int64

# name -> (restype, argtypes); every function include/mla_decode.h declares
SIGNATURES = {
    "mla_check_config": (ctypes.c_int, [ctypes.POINTER(MlaConfig)]),
    "mla_decode_create": (ctypes.c_int, [ctypes.POINTER(MlaConfig), ctypes.c_int, ctypes.POINTER(_P)]),
    "mla_destroy": (ctypes.c_int, [_P]),
    "mla_absorb_q": (ctypes.c_int, [_P, _I32, _P, _P, _P, _P, _P, _P]),
    "mla_decode_attn": (ctypes.c_int, [_P, _I32, _P, _P, _P, _I64, _I64, _P, _P, _I32, _I32, _P, _P, _P]),
    "mla_apply_wuv": (ctypes.c_int, [_P, _I32, _P, _P, _P, _P]),
    "mla_decode_step": (ctypes.c_int, [_P, _I32, _P, _P, _P, _P, _P, _P, _I64, _I64, _P, _P, _I32, _I32,
                                       _P, _P, _P, _P]),
    "mla_prefill_attn": (ctypes.c_int, [_P, _I32, _P, _P, _P, _I64, _I64, _P, _P, _I32, _I32, _P, _P, _P]),
    "mla_absorb_q_fp8": (ctypes.c_int, [_P, _I32, _P, _P, _P, _P, _P, _P, _P]),
    "mla_apply_wuv_fp8": (ctypes.c_int, [_P, _I32, _P, _P, _P, _P, _P]),
    "mla_append_kv_fp8": (ctypes.c_int, [_P, _I32, _I32, _P, _P, _P, _P, ctypes.c_float, _P, _P,
                                         _I64, _I64, _P, _P, _I32, _I32, _P]),
    "mla_decode_attn_fp8": (ctypes.c_int, [_P, _I32, _P, _P, _P, _I64, _I64, _P, _P, _I32, _I32, _P, _P, _P]),
    "mla_decode_attn_partial": (ctypes.c_int, [_P, _I32, _P, _P, _P, _I64, _I64, _P, _P, _I32, _I32,
                                               _P, _P, _P]),
    "mla_merge_partials": (ctypes.c_int, [_P, _I32, _I32, _P, _P, _P, _P, _P]),
    "mla_append_kv": (ctypes.c_int, [_P, _I32, _I32, _P, _P, _P, _P, ctypes.c_float, _P, _P,
                                     _I64, _I64, _P, _P, _I32, _I32, _P]),
    **{name: (ctypes.c_int, [_P, ctypes.c_char_p, _P]) for name in (
        "mla_add_norm_q8", "mla_quantize_rows", "mla_linear_q8", "mla_append_rows", "mla_append_rows_fp8")},
    "mla_decode_attn_noalloc": (ctypes.c_int, [_I32, ctypes.c_float, _I32, _I64, _I32, _P, _P, _P,
                                               _I64, _I64, _P, _P, _I32, _I32, _P, _P, _P, _P]),
    "mla_check_device_errors": (ctypes.c_int, [_P, _P, ctypes.POINTER(ctypes.c_uint32)]),
    "mla_workspace_bytes": (ctypes.c_int64, [_P]),
    "mla_status_string": (ctypes.c_char_p, [ctypes.c_int]),
}

# The argument structs of the calls around the decode step (mla_add_norm_q8_t and so on), packed into
# bytes: a fraction of what passing each argument by itself takes.
NORM_ARGS = struct.Struct("qiiQqQqQqQQqQqQif")
QUANTIZE_ARGS = struct.Struct("qiiQqQqQ")
LINEAR_ARGS = struct.Struct("iiiiQqQQqQQq")
ROWS_ARGS = struct.Struct("iiifQqQQQQqqQQQii")

_lib = None


def load_library(path: str = LIB_PATH) -> ctypes.CDLL:
    """Load libmla_decode.so once and declare its functions."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise RuntimeError(
            f"{path} is missing: build the CUDA library first "
            "(python -m mla_latent_kv_28_b200.build, or __graft_entry__.build())")
    lib = ctypes.CDLL(path)
    for name, (res, args) in SIGNATURES.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    _lib = lib
    return lib


class MlaError(RuntimeError):
    def __init__(self, status: int, what: str, detail: int = 0):
        name = load_library().mla_status_string(status).decode()
        super().__init__(f"{what}: {name} ({status})" + (f", device error word {detail:#x}" if detail else ""))
        self.status = status
        self.detail = detail


def _check(status: int, what: str) -> None:
    if status != MLA_OK:
        raise MlaError(status, what)


def make_config(n_heads: int, max_batch: int, max_kv_len: int, page_size: int = 0,
                softmax_scale: float = 0.0, rope_base: float = 10000.0,
                max_splits: int = 0, yarn_factor: float = 0.0, yarn_original_len: int = 4096,
                yarn_alpha: float = 1.0, yarn_beta: float = 32.0,
                yarn_mscale_coef: float = 0.0707, q_len: int = 1) -> MlaConfig:
    """yarn_factor > 1 turns on YaRN (DeepSeek-V2 uses 40 with the other defaults); q_len > 1
    makes every call take q_len new tokens per sequence (a token axis after the batch axis)."""
    return MlaConfig(n_heads, 128, 512, 64, page_size, max_batch, max_kv_len,
                     softmax_scale, rope_base, max_splits, yarn_factor, yarn_original_len,
                     yarn_alpha, yarn_beta, yarn_mscale_coef, q_len)


def check_config(cfg: MlaConfig) -> int:
    return load_library().mla_check_config(ctypes.byref(cfg))


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream) -> ctypes.c_void_p:
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def _need(t: torch.Tensor, dtype, name: str) -> None:
    if not t.is_cuda or t.dtype != dtype or not t.is_contiguous():
        raise ValueError(f"{name}: expected a contiguous CUDA {dtype} tensor, got "
                         f"{t.dtype} on {t.device} (contiguous={t.is_contiguous()})")


def _shape(t: torch.Tensor) -> str:
    return f"{t.dtype} {tuple(t.shape)} with strides {tuple(t.stride())} on {t.device}"


class MlaDecode:
    """One handle of the library: its configuration plus its device workspace."""

    def __init__(self, n_heads: int, max_batch: int, max_kv_len: int, page_size: int = 0,
                 softmax_scale: float = 0.0, rope_base: float = 10000.0, max_splits: int = 0,
                 device: Optional[int] = None, q_len: int = 1, **yarn):
        """`yarn`: yarn_factor, yarn_original_len, yarn_alpha, yarn_beta, yarn_mscale_coef
        (make_config). With q_len > 1 the per-sequence tensors carry a token axis:
        q_c [B, q_len, n_h, 128], q_abs [B, q_len, n_h, 576], latent [B, q_len, n_h, 512], ..."""
        self._lib = load_library()
        self.q_len = max(1, int(q_len))
        self.cfg = make_config(n_heads, max_batch, max_kv_len, page_size, softmax_scale,
                               rope_base, max_splits, q_len=q_len, **yarn)
        self.device = torch.cuda.current_device() if device is None else int(device)
        h = ctypes.c_void_p()
        _check(self._lib.mla_decode_create(ctypes.byref(self.cfg), self.device, ctypes.byref(h)),
               "mla_decode_create")
        self._h = h

    # -- lifetime ----------------------------------------------------------------------
    def close(self) -> None:
        if getattr(self, "_h", None) is not None and self._h.value is not None:
            _check(self._lib.mla_destroy(self._h), "mla_destroy")
            self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def __enter__(self):
        return self

    def __exit__(self, *exc):
        self.close()

    @property
    def workspace_bytes(self) -> int:
        return int(self._lib.mla_workspace_bytes(self._h))

    # -- the three steps ---------------------------------------------------------------
    def absorb_q(self, q_c: torch.Tensor, q_r: torch.Tensor, w_uk: torch.Tensor,
                 kv_lens: torch.Tensor, q_abs: Optional[torch.Tensor] = None,
                 stream=None) -> torch.Tensor:
        B = q_c.shape[0]
        for t, n in ((q_c, "q_c"), (q_r, "q_r"), (w_uk, "w_uk")):
            _need(t, torch.bfloat16, n)
        _need(kv_lens, torch.int32, "kv_lens")
        if q_abs is None:
            q_abs = torch.empty(tuple(q_c.shape[:-1]) + (ROW,), dtype=torch.bfloat16, device=q_c.device)
        _need(q_abs, torch.bfloat16, "q_abs")
        _check(self._lib.mla_absorb_q(self._h, B, _ptr(q_c), _ptr(q_r), _ptr(w_uk), _ptr(kv_lens),
                                      _ptr(q_abs), _stream(stream)), "mla_absorb_q")
        return q_abs

    def append_kv(self, hidden: torch.Tensor, w_dkv: torch.Tensor, w_kr: torch.Tensor,
                  gamma: torch.Tensor, cache: torch.Tensor, kv_lens: torch.Tensor,
                  page_table: Optional[torch.Tensor] = None, eps: float = 1e-6,
                  stream=None) -> torch.Tensor:
        """Write the new token's cache row [RMSNorm(W_DKV h)*gamma ; RoPE(W_KR h)] as token
        kv_lens[b]-1 of every sequence b. hidden [B, d] bf16; w_dkv [512, d]; w_kr [64, d];
        gamma [512]; cache as for decode_attn. Returns the cache."""
        B, d = hidden.shape[0], hidden.shape[-1]
        for t, n in ((hidden, "hidden"), (w_dkv, "w_dkv"), (w_kr, "w_kr"), (gamma, "gamma")):
            _need(t, torch.bfloat16, n)
        _need(kv_lens, torch.int32, "kv_lens")
        row_stride, seq_stride, c_kv, k_r, max_pages, num_pages = self._cache_view(cache, page_table)
        _check(self._lib.mla_append_kv(
            self._h, B, d, _ptr(hidden), _ptr(w_dkv), _ptr(w_kr), _ptr(gamma), float(eps),
            ctypes.c_void_p(c_kv), ctypes.c_void_p(k_r), row_stride, seq_stride, _ptr(kv_lens),
            _ptr(page_table), max_pages, num_pages, _stream(stream)), "mla_append_kv")
        return cache

    def append_kv_fp8(self, hidden: torch.Tensor, w_dkv: torch.Tensor, w_kr: torch.Tensor,
                      gamma: torch.Tensor, codes: torch.Tensor, exps: torch.Tensor,
                      kv_lens: torch.Tensor, page_table: Optional[torch.Tensor] = None,
                      eps: float = 1e-6, stream=None):
        """append_kv into a quantised cache: codes uint8 [B, Lmax, 576] or [P, 64, 576], exps
        int8 shaped like codes[..., 0] (the layout of decode_attn_fp8)."""
        B, d = hidden.shape[0], hidden.shape[-1]
        for t, n in ((hidden, "hidden"), (w_dkv, "w_dkv"), (w_kr, "w_kr"), (gamma, "gamma")):
            _need(t, torch.bfloat16, n)
        _need(kv_lens, torch.int32, "kv_lens")
        if not codes.is_cuda or codes.dtype != torch.uint8 or codes.dim() != 3 or codes.stride(-1) != 1:
            raise ValueError("codes: expected a CUDA uint8 [*, *, 576] tensor with unit inner stride")
        _need(exps, torch.int8, "exps")
        row_stride = codes.stride(1)
        seq_stride = codes.stride(0) // row_stride
        if exps.shape != codes.shape[:2] or exps.stride(0) != seq_stride:
            raise ValueError("exps must index rows as codes does")
        max_pages = num_pages = 0
        if page_table is not None:
            _need(page_table, torch.int32, "page_table")
            max_pages, num_pages, seq_stride = page_table.shape[1], codes.shape[0], 0
        _check(self._lib.mla_append_kv_fp8(
            self._h, B, d, _ptr(hidden), _ptr(w_dkv), _ptr(w_kr), _ptr(gamma), float(eps),
            _ptr(codes), _ptr(exps), row_stride, seq_stride, _ptr(kv_lens), _ptr(page_table),
            max_pages, num_pages, _stream(stream)), "mla_append_kv_fp8")
        return codes, exps

    @staticmethod
    def _cache_view(cache: torch.Tensor, page_table: Optional[torch.Tensor]):
        if not cache.is_cuda or cache.dtype != torch.bfloat16 or cache.dim() != 3 or cache.stride(-1) != 1:
            raise ValueError("cache: expected a CUDA bf16 [*, *, 576] tensor with unit inner stride")
        row_stride = cache.stride(1)
        seq_stride = cache.stride(0) // row_stride
        c_kv = cache.data_ptr()
        k_r = c_kv + D_LATENT * cache.element_size()
        max_pages = num_pages = 0
        if page_table is not None:
            _need(page_table, torch.int32, "page_table")
            max_pages = page_table.shape[1]
            num_pages = cache.shape[0]
            seq_stride = 0
        return row_stride, seq_stride, c_kv, k_r, max_pages, num_pages

    def decode_attn(self, q_abs: torch.Tensor, cache: torch.Tensor, kv_lens: torch.Tensor,
                    page_table: Optional[torch.Tensor] = None,
                    out_latent: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None,
                    want_lse: bool = True, stream=None) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
        """cache: contiguous [B, Lmax, 576] or paged [num_pages, page_size, 576] bf16 rows
        [c^KV ; k^R]. Returns (out_latent [B, n_h, 512] bf16, lse [B, n_h] fp32 or None)."""
        B = q_abs.shape[0]
        _need(q_abs, torch.bfloat16, "q_abs")
        _need(kv_lens, torch.int32, "kv_lens")
        row_stride, seq_stride, c_kv, k_r, max_pages, num_pages = self._cache_view(cache, page_table)
        if out_latent is None:
            out_latent = torch.empty(tuple(q_abs.shape[:-1]) + (D_LATENT,), dtype=torch.bfloat16,
                                     device=q_abs.device)
        if lse is None and want_lse:
            lse = torch.empty(tuple(q_abs.shape[:-1]), dtype=torch.float32, device=q_abs.device)
        _check(self._lib.mla_decode_attn(
            self._h, B, _ptr(q_abs), ctypes.c_void_p(c_kv), ctypes.c_void_p(k_r), row_stride,
            seq_stride, _ptr(kv_lens), _ptr(page_table), max_pages, num_pages, _ptr(out_latent),
            _ptr(lse), _stream(stream)), "mla_decode_attn")
        return out_latent, lse

    def prefill_attn(self, q_abs: torch.Tensor, cache: torch.Tensor, kv_lens: torch.Tensor,
                     page_table: Optional[torch.Tensor] = None,
                     out_latent: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None,
                     want_lse: bool = True, stream=None) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
        """Prefill: the handle's q_len new tokens of every sequence, q_abs [B, T, n_h, 576], over
        the cache (as decode_attn), in one kernel. Returns (out_latent [B, T, n_h, 512] bf16,
        lse [B, T, n_h] fp32 or None); the same results as decode_attn with this handle."""
        B = q_abs.shape[0]
        _need(q_abs, torch.bfloat16, "q_abs")
        _need(kv_lens, torch.int32, "kv_lens")
        row_stride, seq_stride, c_kv, k_r, max_pages, num_pages = self._cache_view(cache, page_table)
        if out_latent is None:
            out_latent = torch.empty(tuple(q_abs.shape[:-1]) + (D_LATENT,), dtype=torch.bfloat16,
                                     device=q_abs.device)
        if lse is None and want_lse:
            lse = torch.empty(tuple(q_abs.shape[:-1]), dtype=torch.float32, device=q_abs.device)
        _check(self._lib.mla_prefill_attn(
            self._h, B, _ptr(q_abs), ctypes.c_void_p(c_kv), ctypes.c_void_p(k_r), row_stride,
            seq_stride, _ptr(kv_lens), _ptr(page_table), max_pages, num_pages, _ptr(out_latent),
            _ptr(lse), _stream(stream)), "mla_prefill_attn")
        return out_latent, lse

    def decode_attn_fp8(self, q_abs: torch.Tensor, codes: torch.Tensor, exps: torch.Tensor,
                        kv_lens: torch.Tensor, page_table: Optional[torch.Tensor] = None,
                        out_latent: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None,
                        want_lse: bool = True, stream=None):
        """Attention over a quantised cache: codes uint8 [B, Lmax, 576] or [P, 64, 576] (E4M3),
        exps int8 [B, Lmax] or [P, 64] (row r is 2^exps[r] times its codes' values)."""
        B = q_abs.shape[0]
        _need(q_abs, torch.bfloat16, "q_abs")
        _need(kv_lens, torch.int32, "kv_lens")
        if not codes.is_cuda or codes.dtype != torch.uint8 or codes.dim() != 3 or codes.stride(-1) != 1:
            raise ValueError("codes: expected a CUDA uint8 [*, *, 576] tensor with unit inner stride")
        _need(exps, torch.int8, "exps")
        if exps.stride(-1) != 1 or exps.shape != codes.shape[:2]:
            raise ValueError("exps: one int8 per cached row, shaped like codes[..., 0]")
        row_stride = codes.stride(1)
        seq_stride = codes.stride(0) // row_stride
        if exps.stride(0) != seq_stride:
            raise ValueError("exps must index rows as codes does")
        max_pages = num_pages = 0
        if page_table is not None:
            _need(page_table, torch.int32, "page_table")
            max_pages, num_pages, seq_stride = page_table.shape[1], codes.shape[0], 0
        if out_latent is None:
            out_latent = torch.empty(tuple(q_abs.shape[:-1]) + (D_LATENT,), dtype=torch.bfloat16,
                                     device=q_abs.device)
        if lse is None and want_lse:
            lse = torch.empty(tuple(q_abs.shape[:-1]), dtype=torch.float32, device=q_abs.device)
        _check(self._lib.mla_decode_attn_fp8(
            self._h, B, _ptr(q_abs), _ptr(codes), _ptr(exps), row_stride, seq_stride, _ptr(kv_lens),
            _ptr(page_table), max_pages, num_pages, _ptr(out_latent), _ptr(lse), _stream(stream)),
            "mla_decode_attn_fp8")
        return out_latent, lse

    def decode_attn_partial(self, q_abs: torch.Tensor, cache: torch.Tensor, kv_lens: torch.Tensor,
                            page_table: Optional[torch.Tensor] = None,
                            out_latent: Optional[torch.Tensor] = None,
                            lse: Optional[torch.Tensor] = None,
                            stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
        """Attention over the cache rows this caller holds (one shard of each sequence):
        (latent fp32 [B, (T,) n_h, 512], lse fp32 [B, (T,) n_h]), to be merged across shards
        with merge_partials. q_abs is rotated at the request's global positions."""
        B = q_abs.shape[0]
        _need(q_abs, torch.bfloat16, "q_abs")
        _need(kv_lens, torch.int32, "kv_lens")
        row_stride, seq_stride, c_kv, k_r, max_pages, num_pages = self._cache_view(cache, page_table)
        if out_latent is None:
            out_latent = torch.empty(tuple(q_abs.shape[:-1]) + (D_LATENT,), dtype=torch.float32,
                                     device=q_abs.device)
        if lse is None:
            lse = torch.empty(tuple(q_abs.shape[:-1]), dtype=torch.float32, device=q_abs.device)
        _need(out_latent, torch.float32, "out_latent")
        _need(lse, torch.float32, "lse")
        _check(self._lib.mla_decode_attn_partial(
            self._h, B, _ptr(q_abs), ctypes.c_void_p(c_kv), ctypes.c_void_p(k_r), row_stride,
            seq_stride, _ptr(kv_lens), _ptr(page_table), max_pages, num_pages, _ptr(out_latent),
            _ptr(lse), _stream(stream)), "mla_decode_attn_partial")
        return out_latent, lse

    def merge_partials(self, latent_parts: torch.Tensor, lse_parts: torch.Tensor,
                       out_latent: Optional[torch.Tensor] = None,
                       lse: Optional[torch.Tensor] = None, want_lse: bool = True,
                       stream=None) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
        """latent_parts fp32 [P, B, (T,) n_h, 512], lse_parts fp32 [P, B, (T,) n_h] ->
        (latent bf16 [B, (T,) n_h, 512], lse fp32 or None)."""
        _need(latent_parts, torch.float32, "latent_parts")
        _need(lse_parts, torch.float32, "lse_parts")
        P, B = latent_parts.shape[0], latent_parts.shape[1]
        if out_latent is None:
            out_latent = torch.empty(tuple(latent_parts.shape[1:]), dtype=torch.bfloat16,
                                     device=latent_parts.device)
        if lse is None and want_lse:
            lse = torch.empty(tuple(lse_parts.shape[1:]), dtype=torch.float32, device=lse_parts.device)
        _check(self._lib.mla_merge_partials(self._h, B, P, _ptr(latent_parts), _ptr(lse_parts),
                                            _ptr(out_latent), _ptr(lse), _stream(stream)),
               "mla_merge_partials")
        return out_latent, lse

    def apply_wuv(self, latent: torch.Tensor, w_uv: torch.Tensor,
                  out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
        B = latent.shape[0]
        _need(latent, torch.bfloat16, "latent")
        _need(w_uv, torch.bfloat16, "w_uv")
        if out is None:
            out = torch.empty(tuple(latent.shape[:-1]) + (128,), dtype=torch.bfloat16, device=latent.device)
        _need(out, torch.bfloat16, "out")
        _check(self._lib.mla_apply_wuv(self._h, B, _ptr(latent), _ptr(w_uv), _ptr(out),
                                       _stream(stream)), "mla_apply_wuv")
        return out

    @staticmethod
    def _fp8_weight(codes: torch.Tensor, exps: torch.Tensor, n_heads: int, what: str):
        if not codes.is_cuda or codes.dtype != torch.uint8 or not codes.is_contiguous() or \
                codes.numel() != n_heads * 128 * D_LATENT:
            raise ValueError(f"{what} codes: expected a contiguous CUDA uint8 [n_h * 128, 512] tensor")
        if not exps.is_cuda or exps.dtype != torch.int8 or not exps.is_contiguous() or \
                exps.numel() != n_heads * 128 * (D_LATENT // 128):
            raise ValueError(f"{what} exponents: expected a contiguous CUDA int8 [n_h * 128, 4] tensor")

    def absorb_q_fp8(self, q_c: torch.Tensor, q_r: torch.Tensor, w_uk_codes: torch.Tensor,
                     w_uk_exp: torch.Tensor, kv_lens: torch.Tensor,
                     q_abs: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
        """absorb_q with W_UK as E4M3 codes [n_h * 128, 512] and one int8 exponent per 1 x 128
        tile [n_h * 128, 4] (W = value(code) * 2^exp)."""
        B = q_c.shape[0]
        for t, n in ((q_c, "q_c"), (q_r, "q_r")):
            _need(t, torch.bfloat16, n)
        _need(kv_lens, torch.int32, "kv_lens")
        self._fp8_weight(w_uk_codes, w_uk_exp, self.cfg.n_heads, "w_uk")
        if q_abs is None:
            q_abs = torch.empty(tuple(q_c.shape[:-1]) + (ROW,), dtype=torch.bfloat16, device=q_c.device)
        _need(q_abs, torch.bfloat16, "q_abs")
        _check(self._lib.mla_absorb_q_fp8(self._h, B, _ptr(q_c), _ptr(q_r), _ptr(w_uk_codes),
                                          _ptr(w_uk_exp), _ptr(kv_lens), _ptr(q_abs), _stream(stream)),
               "mla_absorb_q_fp8")
        return q_abs

    def apply_wuv_fp8(self, latent: torch.Tensor, w_uv_codes: torch.Tensor, w_uv_exp: torch.Tensor,
                      out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
        """apply_wuv with W_UV as E4M3 codes and per-tile exponents (as absorb_q_fp8)."""
        B = latent.shape[0]
        _need(latent, torch.bfloat16, "latent")
        self._fp8_weight(w_uv_codes, w_uv_exp, self.cfg.n_heads, "w_uv")
        if out is None:
            out = torch.empty(tuple(latent.shape[:-1]) + (128,), dtype=torch.bfloat16, device=latent.device)
        _need(out, torch.bfloat16, "out")
        _check(self._lib.mla_apply_wuv_fp8(self._h, B, _ptr(latent), _ptr(w_uv_codes), _ptr(w_uv_exp),
                                           _ptr(out), _stream(stream)), "mla_apply_wuv_fp8")
        return out

    # -- around the decode step: int8 rows, the int8 projection, projected rows ----------
    def _here(self, stream):
        """The stream to launch on: the current one of the handle's device unless given."""
        return torch._C._cuda_getCurrentRawStream(self.device) if stream is None else stream.cuda_stream

    def _own_stream(self, stream) -> None:
        if stream is not None and stream.device.index != self.device:
            raise ValueError(f"stream: expected one of cuda:{self.device}, got one of {stream.device}")

    def _outputs_on(self, stream):
        """For a call on a stream that need not be the current one: tensors that the call makes belong to
        the stream that writes them (memory freed on the current one may still be in use there)."""
        self._own_stream(stream)
        return torch.cuda.stream(stream)

    def _rows(self, t: torch.Tensor, name: str, dtypes, shape=None) -> Tuple[int, int, int]:
        """Rows, width and the stride between the rows of a [rows, d] tensor on the handle's device."""
        sizes = t.shape
        if len(sizes) == 2 and t.dtype in dtypes and t.get_device() == self.device and \
                (shape is None or sizes == shape):
            rows, d = sizes
            stride, inner = t.stride()
            if inner == 1 or d <= 1:
                if rows <= 1:
                    return rows, d, d
                if stride >= d:
                    return rows, d, stride
        raise ValueError(f"{name}: expected {' or '.join(str(d) for d in dtypes)} "
                         f"{'[rows, d]' if shape is None else tuple(shape)} with unit inner stride and rows "
                         f"apart on cuda:{self.device}, got {_shape(t)}")

    def _flat(self, t: torch.Tensor, name: str, dtype, n: int) -> None:
        if t.dtype != dtype or t.get_device() != self.device or t.shape != (n,) or not t.is_contiguous():
            raise ValueError(f"{name}: expected a contiguous {dtype} [{n}] tensor on cuda:{self.device}, "
                             f"got {_shape(t)}")

    def _new_codes(self, rows: int, d: int, codes, scales, device):
        """Codes and scales to write (rows of new codes are a multiple of 16 bytes apart)."""
        if codes is None:
            stride = (d + 15) // 16 * 16
            codes = torch.empty_strided((rows, d), (stride, 1), dtype=torch.int8, device=device)
        else:
            _, _, stride = self._rows(codes, "codes", _INT8, (rows, d))
        if scales is None:
            scales = torch.empty_strided((rows,), (1,), dtype=torch.float32, device=device)
        else:
            self._flat(scales, "scales", torch.float32, rows)
        return codes, stride, scales

    def add_norm_q8(self, x: torch.Tensor, gamma: torch.Tensor, residual: Optional[torch.Tensor] = None,
                    eps: float = 1e-6, want_y: bool = False, residual_out: Optional[torch.Tensor] = None,
                    codes: Optional[torch.Tensor] = None, scales: Optional[torch.Tensor] = None,
                    y: Optional[torch.Tensor] = None, stream=None):
        """r = x + residual; RMSNorm of r with weight gamma; its int8 codes with a scale per row.
        x [rows, d] bf16 or fp32 (rows may lie apart), residual likewise (its own type), gamma [d]
        bf16. Returns (codes int8 [rows, d], scales fp32 [rows], residual_out, y): residual_out is
        r in the residual's type (a new tensor unless given; `residual` itself is allowed), None
        without a residual; y is the normalised row in bf16, None unless wanted or given."""
        if stream is not None:
            with self._outputs_on(stream):
                return self.add_norm_q8(x, gamma, residual, eps, want_y, residual_out, codes, scales, y)
        rows, d, x_stride = self._rows(x, "x", ROW_TYPES)
        shape, device = (rows, d), x.device
        self._flat(gamma, "gamma", torch.bfloat16, d)
        res_stride = out_stride = y_stride = res_type = 0
        if residual is not None:
            _, _, res_stride = self._rows(residual, "residual", ROW_TYPES, shape)
            if residual_out is None:
                residual_out = torch.empty_strided(shape, (d, 1), dtype=residual.dtype, device=device)
                out_stride = d
            else:
                _, _, out_stride = self._rows(residual_out, "residual_out", (residual.dtype,), shape)
            res_type = ROW_TYPES[residual.dtype]
        elif residual_out is not None:
            raise ValueError("residual_out without a residual")
        codes, codes_stride, scales = self._new_codes(rows, d, codes, scales, device)
        if y is not None:
            _, _, y_stride = self._rows(y, "y", (torch.bfloat16,), shape)
        elif want_y:
            y, y_stride = torch.empty_strided(shape, (d, 1), dtype=torch.bfloat16, device=device), d
        if rows > 0:
            args = NORM_ARGS.pack(
                rows, d, ROW_TYPES[x.dtype], x.data_ptr(), x_stride, 0 if residual is None else residual.data_ptr(),
                res_stride, 0 if residual is None else residual_out.data_ptr(), out_stride, gamma.data_ptr(),
                0 if y is None else y.data_ptr(), y_stride, codes.data_ptr(), codes_stride, scales.data_ptr(),
                res_type, eps)
            _check(self._lib.mla_add_norm_q8(self._h, args, self._here(None)), "mla_add_norm_q8")
        return codes, scales, residual_out, y

    def quantize_rows(self, x: torch.Tensor, codes: Optional[torch.Tensor] = None,
                      scales: Optional[torch.Tensor] = None, stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
        """int8 codes of the rows of x [rows, d] (bf16 or fp32) and a scale for each: the input of
        linear_q8, or its weight (x [n, k], a scale per output channel)."""
        if stream is not None:
            with self._outputs_on(stream):
                return self.quantize_rows(x, codes, scales)
        rows, d, x_stride = self._rows(x, "x", ROW_TYPES)
        codes, codes_stride, scales = self._new_codes(rows, d, codes, scales, x.device)
        if rows > 0:
            args = QUANTIZE_ARGS.pack(rows, d, ROW_TYPES[x.dtype], x.data_ptr(), x_stride, codes.data_ptr(),
                                      codes_stride, scales.data_ptr())
            _check(self._lib.mla_quantize_rows(self._h, args, self._here(None)), "mla_quantize_rows")
        return codes, scales

    def linear_q8(self, codes: torch.Tensor, scales: torch.Tensor, w_codes: torch.Tensor, w_scales: torch.Tensor,
                  out: Optional[torch.Tensor] = None, out_dtype=torch.bfloat16, stream=None) -> torch.Tensor:
        """out[i, j] = (codes[i] . w_codes[j]) * w_scales[j] * scales[i]: codes [rows, k] and
        w_codes [n, k] int8, rows 16-byte aligned; scales [rows], w_scales [n] fp32. out [rows, n]
        bf16 or fp32 (out_dtype unless given)."""
        if stream is not None:
            with self._outputs_on(stream):
                return self.linear_q8(codes, scales, w_codes, w_scales, out, out_dtype)
        rows, k, a_stride = self._rows(codes, "codes", _INT8)
        n, w_k, w_stride = self._rows(w_codes, "w_codes", _INT8)
        if w_k != k:
            raise ValueError(f"w_codes: expected [n, {k}], got {_shape(w_codes)}")
        self._flat(scales, "scales", torch.float32, rows)
        self._flat(w_scales, "w_scales", torch.float32, n)
        if out is not None:
            out_dtype = out.dtype
            _, _, out_stride = self._rows(out, "out", ROW_TYPES, (rows, n))
        else:
            if out_dtype not in ROW_TYPES:
                raise ValueError(f"out_dtype: expected torch.bfloat16 or torch.float32, got {out_dtype}")
            out, out_stride = torch.empty_strided((rows, n), (n, 1), dtype=out_dtype, device=codes.device), n
        # one row has no stride of its own: any multiple of 16 will do
        if rows == 1:
            a_stride = (k + 15) // 16 * 16
        if n == 1:
            w_stride = (k + 15) // 16 * 16
        if rows > 0:
            args = LINEAR_ARGS.pack(rows, k, n, ROW_TYPES[out_dtype], codes.data_ptr(), a_stride, scales.data_ptr(),
                                    w_codes.data_ptr(), w_stride, w_scales.data_ptr(), out.data_ptr(), out_stride)
            _check(self._lib.mla_linear_q8(self._h, args, self._here(None)), "mla_linear_q8")
        return out

    def _append_rows(self, call, x, gamma, cache, cache_type, exps, kv_lens, row_starts, page_table, eps, stream):
        """The checks and the call that append_rows and append_rows_fp8 share (exps: a quantised cache)."""
        self._own_stream(stream)
        rows, d, x_stride = self._rows(x, "x", ROW_TYPES)
        if d != ROW:
            raise ValueError(f"x: expected [rows, {ROW}], got {_shape(x)}")
        self._flat(gamma, "gamma", torch.bfloat16, D_LATENT)
        B = kv_lens.shape[0] if kv_lens.dim() == 1 else -1
        self._flat(kv_lens, "kv_lens", torch.int32, B)
        if row_starts is not None:
            self._flat(row_starts, "row_starts", torch.int32, B + 1)
        sizes, strides = cache.shape, cache.stride()
        if cache.get_device() != self.device or cache.dtype != cache_type or len(sizes) != 3 or \
                sizes[2] != ROW or strides[2] != 1 or strides[1] < ROW:
            raise ValueError(f"cache: expected {cache_type} [*, *, {ROW}] with unit inner stride on "
                             f"cuda:{self.device}, got {_shape(cache)}")
        row_stride = strides[1]
        if page_table is None:
            seq_stride, rest = divmod(strides[0], row_stride)
            if sizes[0] < B or (sizes[0] > 1 and (rest != 0 or seq_stride < sizes[1])) or \
                    sizes[1] < self.cfg.max_kv_len:
                raise ValueError(f"cache: expected [>= {B}, >= {self.cfg.max_kv_len}, {ROW}] with a whole number of "
                                 f"rows between sequences, got {_shape(cache)}")
            seq_stride, max_pages, num_pages = max(seq_stride, sizes[1]), 0, 0
        elif page_table.get_device() != self.device or page_table.dtype != torch.int32 or page_table.dim() != 2 or \
                page_table.shape[0] < B or not page_table.is_contiguous():
            raise ValueError(f"page_table: expected a contiguous int32 [>= {B}, pages] tensor on "
                             f"cuda:{self.device}, got {_shape(page_table)}")
        elif sizes[1] != self.cfg.page_size or (sizes[0] > 1 and strides[0] != sizes[1] * row_stride):
            raise ValueError(f"cache: expected pages of {self.cfg.page_size} rows end to end, got {_shape(cache)}")
        else:
            seq_stride, max_pages, num_pages = 0, page_table.shape[1], sizes[0]
        c_kv = cache.data_ptr()
        if exps is None:
            k_r, kv_exp = c_kv + 2 * D_LATENT, 0
        else:
            if exps.get_device() != self.device or exps.dtype != torch.int8 or exps.shape != sizes[:2] or \
                    not exps.is_contiguous() or (page_table is None and seq_stride != sizes[1]):
                raise ValueError(f"exps: expected a contiguous int8 {tuple(sizes[:2])} tensor indexed as codes is, "
                                 f"got {_shape(exps)}")
            k_r, kv_exp = 0, exps.data_ptr()
        if rows > 0:
            args = ROWS_ARGS.pack(B, rows, ROW_TYPES[x.dtype], eps, x.data_ptr(), x_stride, gamma.data_ptr(), c_kv, k_r,
                                  kv_exp, row_stride, seq_stride, kv_lens.data_ptr(),
                                  0 if row_starts is None else row_starts.data_ptr(),
                                  0 if page_table is None else page_table.data_ptr(), max_pages, num_pages)
            _check(getattr(self._lib, call)(self._h, args, self._here(stream)), call)

    def append_rows(self, x: torch.Tensor, gamma: torch.Tensor, cache: torch.Tensor, kv_lens: torch.Tensor,
                    row_starts: Optional[torch.Tensor] = None, page_table: Optional[torch.Tensor] = None,
                    eps: float = 1e-6, stream=None) -> torch.Tensor:
        """Write the cache rows [RMSNorm(x[:, :512])*gamma ; RoPE(x[:, 512:])] of projected rows x
        [rows, 576] (bf16 or fp32; rows may lie apart): rows row_starts[b] .. row_starts[b+1]-1 are
        the last of sequence b's kv_lens[b] tokens; without row_starts every sequence has q_len.
        Rows outside every sequence write nothing. cache as for decode_attn; returned."""
        self._append_rows("mla_append_rows", x, gamma, cache, torch.bfloat16, None, kv_lens, row_starts, page_table,
                          eps, stream)
        return cache

    def append_rows_fp8(self, x: torch.Tensor, gamma: torch.Tensor, codes: torch.Tensor, exps: torch.Tensor,
                        kv_lens: torch.Tensor, row_starts: Optional[torch.Tensor] = None,
                        page_table: Optional[torch.Tensor] = None, eps: float = 1e-6, stream=None):
        """append_rows into a quantised cache: codes uint8 and exps int8 as for decode_attn_fp8."""
        self._append_rows("mla_append_rows_fp8", x, gamma, codes, torch.uint8, exps, kv_lens, row_starts, page_table,
                          eps, stream)
        return codes, exps

    def step(self, q_c, q_r, w_uk, w_uv, cache, kv_lens, page_table=None, stream=None,
             bufs: Optional[dict] = None):
        """One decode step in one C call (mla_decode_step): absorb -> split-KV attention -> W_UV,
        the same results as the three calls, with the work plan built beside the absorption.
        Returns the head outputs [B, (T,) n_h, 128] bf16. `bufs` may hold preallocated q_abs /
        latent / out; q_abs and latent are left holding the intermediate results."""
        bufs = bufs or {}
        B = q_c.shape[0]
        for t, n in ((q_c, "q_c"), (q_r, "q_r"), (w_uk, "w_uk"), (w_uv, "w_uv")):
            _need(t, torch.bfloat16, n)
        _need(kv_lens, torch.int32, "kv_lens")
        row_stride, seq_stride, c_kv, k_r, max_pages, num_pages = self._cache_view(cache, page_table)
        lead = tuple(q_c.shape[:-1])
        q_abs, latent, out = bufs.get("q_abs"), bufs.get("latent"), bufs.get("out")
        if q_abs is None:
            q_abs = torch.empty(lead + (ROW,), dtype=torch.bfloat16, device=q_c.device)
        if latent is None:
            latent = torch.empty(lead + (D_LATENT,), dtype=torch.bfloat16, device=q_c.device)
        if out is None:
            out = torch.empty(lead + (128,), dtype=torch.bfloat16, device=q_c.device)
        for t, n in ((q_abs, "q_abs"), (latent, "latent"), (out, "out")):
            _need(t, torch.bfloat16, n)
        _check(self._lib.mla_decode_step(
            self._h, B, _ptr(q_c), _ptr(q_r), _ptr(w_uk), _ptr(w_uv), ctypes.c_void_p(c_kv),
            ctypes.c_void_p(k_r), row_stride, seq_stride, _ptr(kv_lens), _ptr(page_table), max_pages,
            num_pages, _ptr(q_abs), _ptr(latent), _ptr(out), _stream(stream)), "mla_decode_step")
        return out

    def check_device_errors(self, stream=None) -> int:
        """Synchronise the stream; raise MlaError if a kernel set the device error word."""
        word = ctypes.c_uint32(0)
        st = self._lib.mla_check_device_errors(self._h, _stream(stream), ctypes.byref(word))
        if st != MLA_OK:
            raise MlaError(st, "device check", int(word.value))
        return 0
