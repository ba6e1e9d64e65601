"""KronQ per-sublayer quantization path on AMD Instinct MI355X (gfx950).

Thin ctypes binding over libkronq.so (the C ABI declared in include/kronq.h):
argument marshalling only -- every step of the path runs in the library's HIP
kernels.  PyTorch provides device memory (tensors, workspaces) and the
current HIP stream.  The library must be built first
(``python -m post_quantization_02_amd.build``); importing this module without
it raises, there is no fallback.
"""
from __future__ import annotations

import contextlib
import ctypes
import functools
import math
import os

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libkronq.so")

(KRONQ_OK, KRONQ_EINVAL, KRONQ_ENOTPD, KRONQ_EHIP, KRONQ_EWORKSPACE, KRONQ_EUNSUPPORTED,
 KRONQ_ENUMERIC, KRONQ_ENOMEM) = range(8)
KRONQ_F32, KRONQ_BF16, KRONQ_F16 = 0, 1, 2

# every entry point declared in include/kronq.h
EXPORTS = ("kronq_status_string", "kronq_last_error", "kronq_version", "kronq_gram_ws",
           "kronq_gram", "kronq_biip_ws", "kronq_biip_rotate", "kronq_chol_inv_ws",
           "kronq_chol_inv", "kronq_gptq_ws", "kronq_gptq_quantize", "kronq_sensitivity",
           "kronq_allocate_bits", "kronq_biip_unrotate_ws", "kronq_biip_unrotate",
           "kronq_packed_row_bytes", "kronq_pack_codes", "kronq_unpack_codes", "kronq_decode_ws",
           "kronq_decode_matvec", "kronq_allocate_bits_passwise", "kronq_allocate_bits_marginal",
           "kronq_allocate_types", "kronq_weight_cv_ws", "kronq_weight_cv", "kronq_signs",
           "kronq_check_finite", "kronq_decode_matvec_noalloc", "kronq_decode_noalloc_max_bytes",
           "kronq_gram_cross_ws", "kronq_gram_cross", "kronq_drift_cross_ws", "kronq_drift_cross",
           "kronq_gptaq_correction_ws",
           "kronq_gptaq_correction", "kronq_gptaq_ws", "kronq_gptaq_quantize", "kronq_biip_sx_ws",
           "kronq_biip_rotate_sx", "kronq_biip_unrotate_sx_ws", "kronq_biip_unrotate_sx",
           "kronq_incoherence_ws", "kronq_incoherence", "kronq_kv_append", "kronq_kv_read",
           "kronq_kv_attention_ws", "kronq_kv_attention", "kronq_rope_tables", "kronq_rotate",
           "kronq_token_logprobs_ws", "kronq_token_logprobs", "kronq_token_logprobs_grad",
           "kronq_prompt_attention", "kronq_prompt_attention_grad_ws", "kronq_prompt_attention_grad")


class KronqError(RuntimeError):
    def __init__(self, status: int, where: str, detail: str):
        super().__init__("%s: status %d (%s)" % (where, status, detail))
        self.status = status


class Had(ctypes.Structure):
    _fields_ = [("dim", ctypes.c_int64), ("block", ctypes.c_int64), ("signs", ctypes.c_void_p)]


class QCfg(ctypes.Structure):
    _fields_ = [("bits", ctypes.c_int32), ("group", ctypes.c_int32)]


class _Cache(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("k_codes", "v_codes", "k_grid", "v_grid")] + \
               [(n, ctypes.c_int64) for n in ("k_codes_stride", "v_codes_stride", "k_grid_stride",
                                              "v_grid_stride", "pages")] + \
               [(n, ctypes.c_int32) for n in ("heads", "page", "dim")]


class _Batch(ctypes.Structure):
    _fields_ = [("table", ctypes.c_void_p), ("ctx", ctypes.c_void_p), ("cu", ctypes.c_void_p),
                ("ld_table", ctypes.c_int64), ("seqs", ctypes.c_int32), ("columns", ctypes.c_int32)]


class _Rope(ctypes.Structure):
    _fields_ = [("cos", ctypes.c_void_p), ("sin", ctypes.c_void_p), ("ld", ctypes.c_int64),
                ("positions", ctypes.c_int64), ("dim", ctypes.c_int32), ("neighbours", ctypes.c_int32)]


class _RopeScaling(ctypes.Structure):
    _fields_ = [(n, ctypes.c_double) for n in ("base", "factor", "original", "low", "high", "magnitude")] + \
               [("scaling", ctypes.c_int32)]


class _Heads(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("row_stride", ctypes.c_int64), ("head_stride", ctypes.c_int64)]


_lib = None


def load(path: str = LIB_PATH):
    """Load libkronq.so (raises OSError when it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise OSError("libkronq.so not built: run `python -m post_quantization_02_amd.build` (%s)" % path)
    lib = ctypes.CDLL(path)
    i32, i64, f32, vp, sz = ctypes.c_int32, ctypes.c_int64, ctypes.c_float, ctypes.c_void_p, ctypes.c_size_t
    lib.kronq_status_string.argtypes = [i32]
    lib.kronq_status_string.restype = ctypes.c_char_p
    lib.kronq_last_error.argtypes = []
    lib.kronq_last_error.restype = ctypes.c_char_p
    lib.kronq_version.restype = i32
    lib.kronq_gram_ws.argtypes = [i64, i64, i32]
    lib.kronq_gram_ws.restype = sz
    lib.kronq_gram.argtypes = [vp, i32, i64, i64, i64, vp, i64, f32, f32, vp, sz, vp]
    lib.kronq_gram.restype = i32
    lib.kronq_biip_ws.argtypes = [i64, i64]
    lib.kronq_biip_ws.restype = sz
    lib.kronq_biip_rotate.argtypes = [vp, i64, i64, i64, vp, i64, vp, i64, ctypes.POINTER(Had),
                                      ctypes.POINTER(Had), f32, vp, vp, sz, vp]
    lib.kronq_biip_rotate.restype = i32
    lib.kronq_chol_inv_ws.argtypes = [i64]
    lib.kronq_chol_inv_ws.restype = sz
    lib.kronq_chol_inv.argtypes = [vp, i64, i64, f32, i32, vp, vp, i64, ctypes.POINTER(i64), vp, sz, vp]
    lib.kronq_chol_inv.restype = i32
    lib.kronq_gptq_ws.argtypes = [i64, i64]
    lib.kronq_gptq_ws.restype = sz
    lib.kronq_gptq_quantize.argtypes = [vp, i64, i64, i64, vp, i64, vp, ctypes.POINTER(QCfg), vp, vp,
                                        vp, vp, vp, vp, vp, sz, vp]
    lib.kronq_gptq_quantize.restype = i32
    lib.kronq_sensitivity.argtypes = [vp, i64, i64, vp, i64, i64, vp, vp]
    lib.kronq_sensitivity.restype = i32
    lib.kronq_allocate_bits.argtypes = [i32, vp, vp, i32, i32, i64, vp]
    lib.kronq_allocate_bits.restype = i32
    lib.kronq_biip_unrotate_ws.argtypes = [i64, i64]
    lib.kronq_biip_unrotate_ws.restype = sz
    lib.kronq_biip_unrotate.argtypes = [vp, i64, i64, i64, ctypes.POINTER(Had), ctypes.POINTER(Had),
                                        vp, vp, sz, vp]
    lib.kronq_biip_unrotate.restype = i32
    lib.kronq_packed_row_bytes.argtypes = [i64, i32]
    lib.kronq_packed_row_bytes.restype = i64
    lib.kronq_pack_codes.argtypes = [vp, i64, i64, i64, i32, vp, vp, i64, vp]
    lib.kronq_pack_codes.restype = i32
    lib.kronq_unpack_codes.argtypes = [vp, i64, i64, i64, i32, vp, i64, vp]
    lib.kronq_unpack_codes.restype = i32
    lib.kronq_decode_ws.argtypes = [i64, i64, i32]
    lib.kronq_decode_ws.restype = sz
    lib.kronq_decode_matvec.argtypes = [vp, i64, i64, i64, ctypes.POINTER(QCfg), vp, vp, vp,
                                        ctypes.POINTER(Had), ctypes.POINTER(Had), vp, vp, vp, vp,
                                        sz, vp]
    lib.kronq_decode_matvec.restype = i32
    for nm in ("kronq_allocate_bits_passwise", "kronq_allocate_bits_marginal"):
        getattr(lib, nm).argtypes = [i32, vp, vp, i32, i32, i64, vp]
        getattr(lib, nm).restype = i32
    lib.kronq_allocate_types.argtypes = [i32, vp, vp, i32, i32, i32, vp]
    lib.kronq_allocate_types.restype = i32
    lib.kronq_weight_cv_ws.argtypes = [i64, i64]
    lib.kronq_weight_cv_ws.restype = sz
    lib.kronq_weight_cv.argtypes = [vp, i64, i64, i64, vp, vp, vp, vp, sz, vp]
    lib.kronq_weight_cv.restype = i32
    lib.kronq_signs.argtypes = [ctypes.c_uint64, i64, vp]
    lib.kronq_signs.restype = i32
    lib.kronq_check_finite.argtypes = [vp, i64, i64, i64, vp, vp]
    lib.kronq_check_finite.restype = i32
    lib.kronq_decode_matvec_noalloc.argtypes = [vp, i64, i64, i64, ctypes.POINTER(QCfg), vp, vp, vp,
                                                ctypes.POINTER(Had), ctypes.POINTER(Had), vp, vp, vp,
                                                vp]
    lib.kronq_decode_matvec_noalloc.restype = i32
    lib.kronq_decode_noalloc_max_bytes.argtypes = []
    lib.kronq_decode_noalloc_max_bytes.restype = sz
    lib.kronq_gram_cross_ws.argtypes = [i64, i64]
    lib.kronq_gram_cross_ws.restype = sz
    lib.kronq_gram_cross.argtypes = [vp, vp, i64, i64, i64, vp, i64, f32, vp, i64, vp, sz, vp]
    lib.kronq_gram_cross.restype = i32
    lib.kronq_drift_cross_ws.argtypes = [i64, i64]
    lib.kronq_drift_cross_ws.restype = sz
    lib.kronq_drift_cross.argtypes = [vp, vp, i64, i64, i64, vp, i64, vp, sz, vp]
    lib.kronq_drift_cross.restype = i32
    lib.kronq_gptaq_correction_ws.argtypes = [i64]
    lib.kronq_gptaq_correction_ws.restype = sz
    lib.kronq_gptaq_correction.argtypes = [vp, i64, i64, vp, i64, vp, f32, vp, i64, vp, sz, vp]
    lib.kronq_gptaq_correction.restype = i32
    lib.kronq_gptaq_ws.argtypes = [i64, i64]
    lib.kronq_gptaq_ws.restype = sz
    lib.kronq_gptaq_quantize.argtypes = [vp, i64, i64, i64, vp, i64, vp, ctypes.POINTER(QCfg), vp, i64,
                                         vp, vp, vp, vp, vp, vp, vp, sz, vp]
    lib.kronq_gptaq_quantize.restype = i32
    lib.kronq_biip_sx_ws.argtypes = [i64, i64]
    lib.kronq_biip_sx_ws.restype = sz
    lib.kronq_biip_rotate_sx.argtypes = [vp, i64, i64, i64, vp, i64, vp, i64, ctypes.POINTER(Had),
                                         ctypes.POINTER(Had), f32, f32, vp, vp, i32, vp, sz, vp]
    lib.kronq_biip_rotate_sx.restype = i32
    lib.kronq_biip_unrotate_sx_ws.argtypes = [i64, i64]
    lib.kronq_biip_unrotate_sx_ws.restype = sz
    lib.kronq_biip_unrotate_sx.argtypes = [vp, i64, i64, i64, ctypes.POINTER(Had), ctypes.POINTER(Had),
                                           vp, vp, vp, sz, vp]
    lib.kronq_biip_unrotate_sx.restype = i32
    lib.kronq_incoherence_ws.argtypes = [i64]
    lib.kronq_incoherence_ws.restype = sz
    lib.kronq_incoherence.argtypes = [vp, i64, i64, ctypes.c_double, i32, ctypes.POINTER(ctypes.c_double),
                                      vp, vp, i64, ctypes.POINTER(i32), vp, sz, vp]
    lib.kronq_incoherence.restype = i32
    kvh, kvc, kvb, kvr = (ctypes.POINTER(s) for s in (_Heads, _Cache, _Batch, _Rope))
    lib.kronq_kv_append.argtypes = [kvh, kvh, i32, i64, kvc, kvb, kvr, vp]
    lib.kronq_kv_append.restype = i32
    lib.kronq_kv_read.argtypes = [kvh, kvh, i32, i64, kvc, kvb, vp]
    lib.kronq_kv_read.restype = i32
    lib.kronq_kv_attention_ws.argtypes = [i64, i64, i32, i32, i32]
    lib.kronq_kv_attention_ws.restype = sz
    lib.kronq_kv_attention.argtypes = [kvh, i32, i64, i32, kvc, kvb, kvr, f32, i64, i64, kvh, vp, vp, sz, vp]
    lib.kronq_kv_attention.restype = i32
    lib.kronq_rope_tables.argtypes = [vp, vp, i64, i64, i64, i32, ctypes.POINTER(_RopeScaling), vp]
    lib.kronq_rope_tables.restype = i32
    lib.kronq_rotate.argtypes = [kvh, i32, kvh, i32, i32, i64, i32, vp, kvr, i32, kvh, kvh, vp]
    lib.kronq_rotate.restype = i32
    lib.kronq_token_logprobs_ws.argtypes = [i64, i64, i32]
    lib.kronq_token_logprobs_ws.restype = sz
    lib.kronq_token_logprobs.argtypes = [vp, i32, i64, i64, i64, vp, vp, vp, vp, i32, vp, vp, vp, sz, vp]
    lib.kronq_token_logprobs.restype = i32
    lib.kronq_token_logprobs_grad.argtypes = [vp, i32, i64, i64, i64, vp, vp, vp, vp, vp, i32, vp, vp, vp, i64, vp]
    lib.kronq_token_logprobs_grad.restype = i32
    lib.kronq_prompt_attention.argtypes = [kvh, kvh, kvh, i32, i64, i32, i32, i32, vp, i32, f32, i64, kvh, vp, vp]
    lib.kronq_prompt_attention.restype = i32
    lib.kronq_prompt_attention_grad_ws.argtypes = [i64, i32]
    lib.kronq_prompt_attention_grad_ws.restype = sz
    lib.kronq_prompt_attention_grad.argtypes = [kvh, kvh, kvh, kvh, kvh, vp, i32, i64, i32, i32, i32, vp, i32, f32,
                                                i64, kvh, kvh, kvh, vp, sz, vp]
    lib.kronq_prompt_attention_grad.restype = i32
    _lib = lib
    return lib


def _check(st: int, where: str):
    if st != KRONQ_OK:
        lib = load()
        raise KronqError(st, where, lib.kronq_last_error().decode(errors="replace"))


def _ptr(t):
    return None if t is None else t.data_ptr()


def _stream(stream):
    if stream is None:
        stream = torch.cuda.current_stream()
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _ws(nbytes: int, device):
    if nbytes == 0:
        return None
    return torch.empty(int(nbytes), dtype=torch.uint8, device=device)


def _dev(t: torch.Tensor, name: str, dtype=None):
    if not t.is_cuda:
        raise ValueError("%s must be a device tensor" % name)
    if dtype is not None and t.dtype != dtype:
        raise ValueError("%s must be %s" % (name, dtype))
    if t.dim() == 2 and t.stride(1) != 1:
        raise ValueError("%s must be row-major (unit column stride)" % name)


def _ld(t: torch.Tensor) -> int:
    return t.stride(0) if t.dim() == 2 else t.shape[-1]


# ---------------------------------------------------------------- calls

def kronq_gram(A: torch.Tensor, H: torch.Tensor | None = None, scale: float | None = None,
               beta: float = 0.0, stream=None, ws: torch.Tensor | None = None) -> torch.Tensor:
    """H <- scale * A^T A + beta * H (A: N x d bf16 or fp32; H: d x d fp32)."""
    lib = load()
    _dev(A, "A")
    if A.dtype == torch.bfloat16:
        dt = KRONQ_BF16
    elif A.dtype == torch.float32:
        dt = KRONQ_F32
    else:
        raise ValueError("A must be bfloat16 or float32")
    N, d = A.shape
    if H is None:
        H = torch.empty((d, d), dtype=torch.float32, device=A.device)
    _dev(H, "H", torch.float32)
    scale = 1.0 / N if scale is None else scale
    need = lib.kronq_gram_ws(N, d, dt)
    if ws is None or ws.numel() < need:
        ws = _ws(need, A.device)
    _check(lib.kronq_gram(_ptr(A), dt, N, d, _ld(A), _ptr(H), _ld(H), scale, beta, _ptr(ws),
                          need, _stream(stream)), "kronq_gram")
    return H


def kronq_biip_rotate(W: torch.Tensor, HX: torch.Tensor | None, HG: torch.Tensor | None,
                      in_signs: torch.Tensor, in_block: int, out_signs: torch.Tensor,
                      out_block: int, alpha: float, sg: torch.Tensor | None = None,
                      stream=None, ws: torch.Tensor | None = None) -> torch.Tensor:
    """In place: W <- U S_G W V^T, HX <- V HX V^T, HG <- U S_G^-1 HG S_G^-1 U^T.
    Returns s_g = diag(H_G)^alpha (allocated when `sg` is None)."""
    lib = load()
    _dev(W, "W", torch.float32)
    m, n = W.shape
    if sg is None:
        sg = torch.empty(m, dtype=torch.float32, device=W.device)
    for t, nm in ((HX, "HX"), (HG, "HG"), (sg, "sg"), (in_signs, "in_signs"), (out_signs, "out_signs")):
        if t is not None:
            _dev(t, nm, torch.float32)
    hin = Had(n, in_block, _ptr(in_signs))     # signs None with block 1: identity side
    hout = Had(m, out_block, _ptr(out_signs))
    need = lib.kronq_biip_ws(m, n)
    if ws is None or ws.numel() < need:
        ws = _ws(need, W.device)
    _check(lib.kronq_biip_rotate(_ptr(W), m, n, _ld(W), _ptr(HX), _ld(HX) if HX is not None else n,
                                 _ptr(HG), _ld(HG) if HG is not None else m, ctypes.byref(hin),
                                 ctypes.byref(hout), alpha, _ptr(sg), _ptr(ws), need,
                                 _stream(stream)), "kronq_biip_rotate")
    return sg


def kronq_biip_rotate_sx(W: torch.Tensor | None, HX: torch.Tensor | None, HG: torch.Tensor | None,
                         in_signs: torch.Tensor | None, in_block: int, out_signs: torch.Tensor | None,
                         out_block: int, alpha: float, alpha_x: float, sg: torch.Tensor | None = None,
                         sx: torch.Tensor | None = None, sx_given: bool = False, m: int | None = None,
                         n: int | None = None, stream=None, ws: torch.Tensor | None = None):
    """In place, with the input rescale: W <- U S_G W S_X V^T,
    HX <- V S_X^-1 HX S_X^-1 V^T, HG <- U S_G^-1 HG S_G^-1 U^T.  Returns (sg, sx);
    sx is computed as diag(HX)^alpha_x unless sx_given (then it is read).  With
    W None, m and n come from HG / HX or the arguments."""
    lib = load()
    if W is not None:
        _dev(W, "W", torch.float32)
        m, n = W.shape
    else:
        m = m if m is not None else (HG.shape[0] if HG is not None else 1)
        n = n if n is not None else HX.shape[0]
    dev = next(t.device for t in (W, HX, HG, sx) if t is not None)
    if sg is None:
        sg = torch.empty(m, dtype=torch.float32, device=dev)
    if sx is None and not sx_given:
        sx = torch.empty(n, dtype=torch.float32, device=dev)
    for t, nm in ((HX, "HX"), (HG, "HG"), (sg, "sg"), (sx, "sx"), (in_signs, "in_signs"),
                  (out_signs, "out_signs")):
        if t is not None:
            _dev(t, nm, torch.float32)
    hin = Had(n, in_block, _ptr(in_signs))
    hout = Had(m, out_block, _ptr(out_signs))
    need = lib.kronq_biip_sx_ws(m, n)
    if ws is None or ws.numel() < need:
        ws = _ws(need, dev)
    _check(lib.kronq_biip_rotate_sx(_ptr(W), m, n, _ld(W) if W is not None else n, _ptr(HX),
                                    _ld(HX) if HX is not None else n, _ptr(HG),
                                    _ld(HG) if HG is not None else m, ctypes.byref(hin),
                                    ctypes.byref(hout), alpha, alpha_x, _ptr(sg), _ptr(sx),
                                    1 if sx_given else 0, _ptr(ws), need, _stream(stream)),
           "kronq_biip_rotate_sx")
    return sg, sx


def kronq_chol_inv(H: torch.Tensor, lam: float, act_order: bool = False,
                   perm: torch.Tensor | None = None, R: torch.Tensor | None = None, stream=None,
                   ws: torch.Tensor | None = None):
    """Returns (R, perm, info): R upper with R^T R = (P(H + lam mean(diag) I)P^T)^-1.
    Raises KronqError (status KRONQ_ENOTPD, .info set) when not positive definite."""
    lib = load()
    _dev(H, "H", torch.float32)
    n = H.shape[0]
    if perm is None:
        perm = torch.empty(n, dtype=torch.int32, device=H.device)
    if R is None:
        R = torch.empty((n, n), dtype=torch.float32, device=H.device)
    need = lib.kronq_chol_inv_ws(n)
    if ws is None or ws.numel() < need:
        ws = _ws(need, H.device)
    info = ctypes.c_int64(-1)
    st = lib.kronq_chol_inv(_ptr(H), n, _ld(H), lam, 1 if act_order else 0, _ptr(perm), _ptr(R),
                            _ld(R), ctypes.byref(info), _ptr(ws), need, _stream(stream))
    if st != KRONQ_OK:
        err = KronqError(st, "kronq_chol_inv", lib.kronq_last_error().decode(errors="replace"))
        err.info = info.value
        raise err
    return R, perm, info.value


def kronq_gptq_quantize(W: torch.Tensor, R: torch.Tensor, perm: torch.Tensor | None, bits: int,
                        group: int, What: torch.Tensor | None = None, want_pre: bool = False,
                        stream=None, ws: torch.Tensor | None = None, codes=None, scales=None,
                        zeros=None, want_row_loss: bool = False, row_loss=None):
    """Column-wise OBS loop.  Returns dict(codes, scales, zeros, What, pre,
    row_loss); pre and row_loss are None unless asked for."""
    lib = load()
    _dev(W, "W", torch.float32)
    _dev(R, "R", torch.float32)
    m, n = W.shape
    ng = 1 if group <= 0 else n // group
    dev = W.device
    if codes is None:
        codes = torch.empty((m, n), dtype=torch.uint8, device=dev)
    if scales is None:
        scales = torch.empty((m, ng), dtype=torch.float32, device=dev)
    if zeros is None:
        zeros = torch.empty((m, ng), dtype=torch.float32, device=dev)
    if What is None:
        What = torch.empty((m, n), dtype=torch.float32, device=dev)
    pre = torch.empty((m, n), dtype=torch.float32, device=dev) if want_pre else None
    if row_loss is None and want_row_loss:
        row_loss = torch.empty(m, dtype=torch.float64, device=dev)
    q = QCfg(bits, group)
    need = lib.kronq_gptq_ws(m, n)
    if ws is None or ws.numel() < need:
        ws = _ws(need, dev)
    _check(lib.kronq_gptq_quantize(_ptr(W), m, n, _ld(W), _ptr(R), _ld(R), _ptr(perm),
                                   ctypes.byref(q), _ptr(codes), _ptr(scales), _ptr(zeros),
                                   _ptr(What), _ptr(pre), _ptr(row_loss), _ptr(ws), need,
                                   _stream(stream)),
           "kronq_gptq_quantize")
    return dict(codes=codes, scales=scales, zeros=zeros, What=What, pre=pre, row_loss=row_loss)


def kronq_sensitivity(HX: torch.Tensor, HG: torch.Tensor, out: torch.Tensor | None = None,
                      stream=None) -> torch.Tensor:
    """Device tensor of 3 doubles: tr(HX), tr(HG), product."""
    lib = load()
    _dev(HX, "HX", torch.float32)
    _dev(HG, "HG", torch.float32)
    if out is None:
        out = torch.empty(3, dtype=torch.float64, device=HX.device)
    _check(lib.kronq_sensitivity(_ptr(HX), HX.shape[0], _ld(HX), _ptr(HG), HG.shape[0], _ld(HG),
                                 _ptr(out), _stream(stream)), "kronq_sensitivity")
    return out


def _allocate(name, scores, n_params, bmin, bmax, budget_bits):
    import numpy as np
    lib = load()
    sc = np.ascontiguousarray(scores, dtype=np.float64)
    npar = np.ascontiguousarray(n_params, dtype=np.int64)
    out = np.zeros(len(sc), dtype=np.int32)
    _check(getattr(lib, name)(len(sc), sc.ctypes.data, npar.ctypes.data, bmin, bmax,
                              int(budget_bits), out.ctypes.data), name)
    return [int(x) for x in out]


def kronq_allocate_bits(scores, n_params, bmin: int, bmax: int, budget_bits: int) -> list:
    """Host-only greedy allocation (see include/kronq.h)."""
    return _allocate("kronq_allocate_bits", scores, n_params, bmin, bmax, budget_bits)


def kronq_allocate_bits_passwise(scores, n_params, bmin: int, bmax: int, budget_bits: int) -> list:
    return _allocate("kronq_allocate_bits_passwise", scores, n_params, bmin, bmax, budget_bits)


def kronq_allocate_bits_marginal(scores, n_params, bmin: int, bmax: int, budget_bits: int) -> list:
    return _allocate("kronq_allocate_bits_marginal", scores, n_params, bmin, bmax, budget_bits)


def kronq_allocate_types(scores, type_of, n_types: int, base_bits: int, n_upgrade: int) -> list:
    import numpy as np
    lib = load()
    sc = np.ascontiguousarray(scores, dtype=np.float64)
    ty = np.ascontiguousarray(type_of, dtype=np.int32)
    out = np.zeros(len(sc), dtype=np.int32)
    _check(lib.kronq_allocate_types(len(sc), sc.ctypes.data, ty.ctypes.data, n_types, base_bits,
                                    n_upgrade, out.ctypes.data), "kronq_allocate_types")
    return [int(x) for x in out]


def kronq_biip_unrotate(W: torch.Tensor, in_signs: torch.Tensor, in_block: int,
                        out_signs: torch.Tensor, out_block: int, sg: torch.Tensor | None = None,
                        stream=None, ws: torch.Tensor | None = None) -> torch.Tensor:
    """In place: W <- diag(sg)^-1 U^T W V (the inverse of the weight side of BiIP)."""
    lib = load()
    _dev(W, "W", torch.float32)
    m, n = W.shape
    for t, nm in ((sg, "sg"), (in_signs, "in_signs"), (out_signs, "out_signs")):
        if t is not None:
            _dev(t, nm, torch.float32)
    hin = Had(n, in_block, _ptr(in_signs))
    hout = Had(m, out_block, _ptr(out_signs))
    need = lib.kronq_biip_unrotate_ws(m, n)
    if ws is None or ws.numel() < need:
        ws = _ws(need, W.device)
    _check(lib.kronq_biip_unrotate(_ptr(W), m, n, _ld(W), ctypes.byref(hin), ctypes.byref(hout),
                                   _ptr(sg), _ptr(ws), need, _stream(stream)), "kronq_biip_unrotate")
    return W


def kronq_biip_unrotate_sx(W: torch.Tensor, in_signs: torch.Tensor | None, in_block: int,
                           out_signs: torch.Tensor | None, out_block: int, sg: torch.Tensor | None,
                           sx: torch.Tensor, stream=None, ws: torch.Tensor | None = None) -> torch.Tensor:
    """In place: W <- diag(sg)^-1 U^T W V diag(sx)^-1."""
    lib = load()
    _dev(W, "W", torch.float32)
    m, n = W.shape
    for t, nm in ((sg, "sg"), (sx, "sx"), (in_signs, "in_signs"), (out_signs, "out_signs")):
        if t is not None:
            _dev(t, nm, torch.float32)
    hin = Had(n, in_block, _ptr(in_signs))
    hout = Had(m, out_block, _ptr(out_signs))
    need = lib.kronq_biip_unrotate_sx_ws(m, n)
    if ws is None or ws.numel() < need:
        ws = _ws(need, W.device)
    _check(lib.kronq_biip_unrotate_sx(_ptr(W), m, n, _ld(W), ctypes.byref(hin), ctypes.byref(hout),
                                      _ptr(sg), _ptr(sx), _ptr(ws), need, _stream(stream)),
           "kronq_biip_unrotate_sx")
    return W


def kronq_incoherence(H: torch.Tensor, tol: float = 1e-13, max_sweeps: int = 40,
                      want_evals: bool = False, want_q: bool = False, stream=None,
                      ws: torch.Tensor | None = None) -> dict:
    """mu(H)/sqrt(n) = max_ij |Q_ij| of H = Q Lambda Q^T (fp64 block Jacobi).
    Returns {"mu", "sweeps"} and, when asked, "evals" (n doubles) and "Q"."""
    lib = load()
    _dev(H, "H", torch.float32)
    n = H.shape[0]
    evals = torch.empty(n, dtype=torch.float64, device=H.device) if want_evals else None
    Q = torch.empty((n, n), dtype=torch.float64, device=H.device) if want_q else None
    need = lib.kronq_incoherence_ws(n)
    if ws is None or ws.numel() < need:
        ws = _ws(need, H.device)
    mu = ctypes.c_double(0.0)
    sw = ctypes.c_int32(0)
    _check(lib.kronq_incoherence(_ptr(H), n, _ld(H), tol, max_sweeps, ctypes.byref(mu), _ptr(evals),
                                 _ptr(Q), n, ctypes.byref(sw), _ptr(ws), need, _stream(stream)),
           "kronq_incoherence")
    out = {"mu": mu.value, "sweeps": sw.value}
    if want_evals:
        out["evals"] = evals
    if want_q:
        out["Q"] = Q
    return out


def kronq_packed_row_bytes(n: int, bits: int) -> int:
    return int(load().kronq_packed_row_bytes(n, bits))


def kronq_pack_codes(codes: torch.Tensor, bits: int, packed: torch.Tensor | None = None,
                     stream=None, perm: torch.Tensor | None = None) -> torch.Tensor:
    """m x n uint8 codes -> m x ldp packed bytes (ldp = row bytes unless `packed` is given);
    with `perm`, stored column j holds code column perm[j] (processing order)."""
    lib = load()
    _dev(codes, "codes", torch.uint8)
    m, n = codes.shape
    if packed is None:
        packed = torch.zeros((m, lib.kronq_packed_row_bytes(n, bits)), dtype=torch.uint8,
                             device=codes.device)
    _dev(packed, "packed", torch.uint8)
    _check(lib.kronq_pack_codes(_ptr(codes), m, n, _ld(codes), bits, _ptr(perm), _ptr(packed),
                                _ld(packed), _stream(stream)), "kronq_pack_codes")
    return packed


def kronq_unpack_codes(packed: torch.Tensor, bits: int, n: int, codes: torch.Tensor | None = None,
                       stream=None) -> torch.Tensor:
    lib = load()
    _dev(packed, "packed", torch.uint8)
    m = packed.shape[0]
    if codes is None:
        codes = torch.empty((m, n), dtype=torch.uint8, device=packed.device)
    _dev(codes, "codes", torch.uint8)
    _check(lib.kronq_unpack_codes(_ptr(packed), m, n, _ld(packed), bits, _ptr(codes), _ld(codes),
                                  _stream(stream)), "kronq_unpack_codes")
    return codes


def kronq_decode_matvec(codes: torch.Tensor, n: int, bits: int, group: int, scales: torch.Tensor,
                        zeros: torch.Tensor, in_signs: torch.Tensor, in_block: int,
                        out_signs: torch.Tensor, out_block: int, sg: torch.Tensor | None,
                        x: torch.Tensor, y: torch.Tensor | None = None,
                        perm: torch.Tensor | None = None, stream=None,
                        ws: torch.Tensor | None = None) -> torch.Tensor:
    """y = diag(sg)^-1 U^T W'^ V x for stored codes (m rows of ldp bytes)."""
    lib = load()
    _dev(codes, "codes", torch.uint8)
    for t, nm in ((scales, "scales"), (zeros, "zeros"), (in_signs, "in_signs"),
                  (out_signs, "out_signs"), (sg, "sg"), (x, "x")):
        if t is not None:
            _dev(t, nm, torch.float32)
    m = codes.shape[0]
    if y is None:
        y = torch.empty(m, dtype=torch.float32, device=codes.device)
    q = QCfg(bits, group)
    hin = Had(n, in_block, _ptr(in_signs))
    hout = Had(m, out_block, _ptr(out_signs))
    need = lib.kronq_decode_ws(m, n, bits)
    if ws is None or ws.numel() < need:
        ws = _ws(need, codes.device)
    _check(lib.kronq_decode_matvec(_ptr(codes), m, n, _ld(codes), ctypes.byref(q), _ptr(scales),
                                   _ptr(zeros), _ptr(perm), ctypes.byref(hin), ctypes.byref(hout),
                                   _ptr(sg), _ptr(x), _ptr(y), _ptr(ws), need, _stream(stream)),
           "kronq_decode_matvec")
    return y


def kronq_decode_matvec_noalloc(codes: torch.Tensor, n: int, bits: int, group: int,
                                scales: torch.Tensor, zeros: torch.Tensor, in_signs: torch.Tensor,
                                in_block: int, out_signs: torch.Tensor, out_block: int,
                                sg: torch.Tensor | None, x: torch.Tensor, y: torch.Tensor,
                                perm: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """kronq_decode_matvec without a workspace (the library's fixed per-GPU
    buffer); y must be given, so the call allocates nothing."""
    lib = load()
    m = codes.shape[0]
    q = QCfg(bits, group)
    hin = Had(n, in_block, _ptr(in_signs))
    hout = Had(m, out_block, _ptr(out_signs))
    _check(lib.kronq_decode_matvec_noalloc(_ptr(codes), m, n, _ld(codes), ctypes.byref(q),
                                           _ptr(scales), _ptr(zeros), _ptr(perm), ctypes.byref(hin),
                                           ctypes.byref(hout), _ptr(sg), _ptr(x), _ptr(y),
                                           _stream(stream)),
           "kronq_decode_matvec_noalloc")
    return y


INCOH_MODES = ("full", "no_rescale", "su_only", "sv_only")


def kronq_biip_rotate_mode(W, HX, HG, in_signs, in_block, out_signs, out_block, alpha, mode="full",
                           sg=None, stream=None, ws=None):
    """kronq_biip_rotate for an incoherence mode: full (S_G, U, V), no_rescale
    (U, V), su_only (S_G and U; V = I), sv_only (V; U = I, no S_G).  An unused
    side is passed as the identity (block 1, no signs)."""
    if mode not in INCOH_MODES:
        raise ValueError("unknown incoherence mode %r" % (mode,))
    if mode == "no_rescale":
        alpha = 0.0
    if mode == "su_only":
        in_signs, in_block = None, 1
    if mode == "sv_only":
        out_signs, out_block, alpha = None, 1, 0.0
    return kronq_biip_rotate(W, HX, HG, in_signs, in_block, out_signs, out_block, alpha, sg=sg,
                             stream=stream, ws=ws)


def kronq_weight_cv(W: torch.Tensor, col_norms=None, row_norms=None, out=None, stream=None,
                    ws=None) -> torch.Tensor:
    """Device tensor of 2 doubles: CV_in (column norms), CV_out (row norms)."""
    lib = load()
    _dev(W, "W", torch.float32)
    m, n = W.shape
    if out is None:
        out = torch.empty(2, dtype=torch.float64, device=W.device)
    need = lib.kronq_weight_cv_ws(m, n)
    if ws is None or ws.numel() < need:
        ws = _ws(need, W.device)
    _check(lib.kronq_weight_cv(_ptr(W), m, n, _ld(W), _ptr(out), _ptr(col_norms), _ptr(row_norms),
                               _ptr(ws), need, _stream(stream)), "kronq_weight_cv")
    return out


def kronq_signs(seed: int, n: int) -> torch.Tensor:
    """The library's documented sign draw: n floats of +-1 (host tensor)."""
    lib = load()
    out = torch.empty(max(n, 1), dtype=torch.float32)
    _check(lib.kronq_signs(ctypes.c_uint64(seed & (2 ** 64 - 1)), n, out.data_ptr()), "kronq_signs")
    return out[:n].clone()


def kronq_check_finite(A: torch.Tensor, flag: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Device int32 flag: 1 if A (fp32, 2-D row-major) holds a NaN or an infinity."""
    lib = load()
    _dev(A, "A", torch.float32)
    rows, cols = (A.shape if A.dim() == 2 else (1, A.numel()))
    if flag is None:
        flag = torch.empty(1, dtype=torch.int32, device=A.device)
    _check(lib.kronq_check_finite(_ptr(A), rows, cols, _ld(A) if A.dim() == 2 else cols, _ptr(flag),
                                  _stream(stream)), "kronq_check_finite")
    return flag


def kronq_gram_cross(A: torch.Tensor, B: torch.Tensor, C: torch.Tensor | None = None,
                     scale: float | None = None, sub: torch.Tensor | None = None, stream=None,
                     ws: torch.Tensor | None = None) -> torch.Tensor:
    """C = scale A^T B - sub (A, B: N x d bf16 with one layout; C, sub: d x d fp32).
    The drift term of the asymmetric objective: A = X_fp, B = X, sub = H_X."""
    lib = load()
    _dev(A, "A", torch.bfloat16)
    _dev(B, "B", torch.bfloat16)
    N, d = A.shape
    if tuple(B.shape) != (N, d) or _ld(A) != _ld(B):
        raise ValueError("A and B must have the same shape and leading dimension")
    if C is None:
        C = torch.empty((d, d), dtype=torch.float32, device=A.device)
    if sub is not None:
        _dev(sub, "sub", torch.float32)
    scale = 1.0 / N if scale is None else scale
    need = lib.kronq_gram_cross_ws(N, d)
    if ws is None or ws.numel() < need:
        ws = _ws(need, A.device)
    _check(lib.kronq_gram_cross(_ptr(A), _ptr(B), N, d, _ld(A), _ptr(C), _ld(C), scale, _ptr(sub),
                                _ld(sub) if sub is not None else d, _ptr(ws), need, _stream(stream)),
           "kronq_gram_cross")
    return C


def kronq_drift_cross(Xfp: torch.Tensor, X: torch.Tensor, C: torch.Tensor | None = None, stream=None,
                      ws: torch.Tensor | None = None) -> torch.Tensor:
    """C = (X_fp - X)^T X / N (X_fp, X: N x n bf16 with one layout; C n x n fp32)."""
    lib = load()
    _dev(Xfp, "Xfp", torch.bfloat16)
    _dev(X, "X", torch.bfloat16)
    N, n = X.shape
    if tuple(Xfp.shape) != (N, n) or _ld(Xfp) != _ld(X):
        raise ValueError("X_fp and X must have the same shape and leading dimension")
    if C is None:
        C = torch.empty((n, n), dtype=torch.float32, device=X.device)
    need = lib.kronq_drift_cross_ws(N, n)
    if ws is None or ws.numel() < need:
        ws = _ws(need, X.device)
    _check(lib.kronq_drift_cross(_ptr(Xfp), _ptr(X), N, n, _ld(X), _ptr(C), _ld(C), _ptr(ws), need,
                                 _stream(stream)), "kronq_drift_cross")
    return C


def kronq_gptaq_correction(C: torch.Tensor, R: torch.Tensor, perm: torch.Tensor | None, alpha: float,
                           P: torch.Tensor | None = None, stream=None,
                           ws: torch.Tensor | None = None) -> torch.Tensor:
    """P = alpha ((C_p R^T) (.) M) R, M strictly upper, C_p = C[perm][:, perm]."""
    lib = load()
    _dev(C, "C", torch.float32)
    _dev(R, "R", torch.float32)
    n = C.shape[0]
    if P is None:
        P = torch.empty((n, n), dtype=torch.float32, device=C.device)
    need = lib.kronq_gptaq_correction_ws(n)
    if ws is None or ws.numel() < need:
        ws = _ws(need, C.device)
    _check(lib.kronq_gptaq_correction(_ptr(C), n, _ld(C), _ptr(R), _ld(R), _ptr(perm), alpha, _ptr(P),
                                      _ld(P), _ptr(ws), need, _stream(stream)), "kronq_gptaq_correction")
    return P


def kronq_gptaq_quantize(W: torch.Tensor, R: torch.Tensor, perm: torch.Tensor | None, bits: int,
                         group: int, P: torch.Tensor, What: torch.Tensor | None = None,
                         want_pre: bool = False, want_row_loss: bool = False, stream=None,
                         ws: torch.Tensor | None = None, codes=None, scales=None, zeros=None):
    """The column loop with the asymmetric correction.  Returns the dict of
    kronq_gptq_quantize."""
    lib = load()
    _dev(W, "W", torch.float32)
    _dev(R, "R", torch.float32)
    _dev(P, "P", torch.float32)
    m, n = W.shape
    ng = 1 if group <= 0 else n // group
    dev = W.device
    codes = torch.empty((m, n), dtype=torch.uint8, device=dev) if codes is None else codes
    scales = torch.empty((m, ng), dtype=torch.float32, device=dev) if scales is None else scales
    zeros = torch.empty((m, ng), dtype=torch.float32, device=dev) if zeros is None else zeros
    What = torch.empty((m, n), dtype=torch.float32, device=dev) if What is None else What
    pre = torch.empty((m, n), dtype=torch.float32, device=dev) if want_pre else None
    row_loss = torch.empty(m, dtype=torch.float64, device=dev) if want_row_loss else None
    q = QCfg(bits, group)
    need = lib.kronq_gptaq_ws(m, n)
    if ws is None or ws.numel() < need:
        ws = _ws(need, dev)
    _check(lib.kronq_gptaq_quantize(_ptr(W), m, n, _ld(W), _ptr(R), _ld(R), _ptr(perm), ctypes.byref(q),
                                    _ptr(P), _ld(P), _ptr(codes), _ptr(scales), _ptr(zeros), _ptr(What),
                                    _ptr(pre), _ptr(row_loss), _ptr(ws), need, _stream(stream)),
           "kronq_gptaq_quantize")
    return dict(codes=codes, scales=scales, zeros=zeros, What=What, pre=pre, row_loss=row_loss)


# ------------------------------------------- 4-bit paged key/value cache

_KV_DTYPES = {torch.float32: KRONQ_F32, torch.bfloat16: KRONQ_BF16, torch.float16: KRONQ_F16}


def _same_device(device, *tensors):
    for t in tensors:
        if t.device != device:
            raise ValueError("all tensors must be on one device (%s and %s)" % (device, t.device))


class KVCache:
    """One layer's cache: codes uint8 (pages, heads, page, dim / 2) and grid
    words int32 (pages, heads, page), keys and values each (layouts in
    include/kronq.h).  Holds the tensors; a page's last three (two) dimensions
    are contiguous, the distance between pages is free."""

    def __init__(self, k_codes: torch.Tensor, v_codes: torch.Tensor, k_grid: torch.Tensor,
                 v_grid: torch.Tensor):
        if k_codes.dim() != 4:
            raise ValueError("k_codes must be (pages, heads, page, dim / 2)")
        pages, heads, page, half = k_codes.shape
        self.device = k_codes.device
        for t, nm, dt, shape in ((k_codes, "k_codes", torch.uint8, (pages, heads, page, half)),
                                 (v_codes, "v_codes", torch.uint8, (pages, heads, page, half)),
                                 (k_grid, "k_grid", torch.int32, (pages, heads, page)),
                                 (v_grid, "v_grid", torch.int32, (pages, heads, page))):
            _dev(t, nm, dt)
            if tuple(t.shape) != shape:
                raise ValueError("%s must have shape %s" % (nm, shape))
            # a dimension of one entry has no distance to speak of
            if any(n > 1 and t.stride(i) != math.prod(shape[i + 1:]) for i, n in enumerate(shape) if i):
                raise ValueError("%s: a page must be contiguous" % nm)
        _same_device(self.device, v_codes, k_grid, v_grid)
        self.k_codes, self.v_codes, self.k_grid, self.v_grid = k_codes, v_codes, k_grid, v_grid
        self.pages, self.heads, self.page, self.dim = pages, heads, page, 2 * half
        self._c = _Cache(k_codes.data_ptr(), v_codes.data_ptr(), k_grid.data_ptr(), v_grid.data_ptr(),
                         *(t.stride(0) if pages != 1 else math.prod(t.shape[1:])
                           for t in (k_codes, v_codes, k_grid, v_grid)),
                         pages, heads, page, 2 * half)

    @classmethod
    def empty(cls, pages: int, heads: int, page: int, dim: int, device="cuda:0") -> "KVCache":
        """A cache of `pages` pages with no content yet."""
        codes = [torch.zeros((pages, heads, page, dim // 2), dtype=torch.uint8, device=device) for _ in "kv"]
        grids = [torch.zeros((pages, heads, page), dtype=torch.int32, device=device) for _ in "kv"]
        return cls(*codes, *grids)


class KVBatch:
    """Which rows belong to which sequence, and where its positions are: table
    int32 (seqs, columns), ctx int32 (seqs), cu int32 (seqs + 1), on the device
    (include/kronq.h).  Holds the tensors; their content may change between
    calls (and between replays of a graph)."""

    def __init__(self, table: torch.Tensor, ctx: torch.Tensor, cu: torch.Tensor):
        self.device = table.device
        for t, nm, d in ((table, "table", 2), (ctx, "ctx", 1), (cu, "cu", 1)):
            # a dimension of one entry, or none, has no distance to speak of
            _dev(t.reshape(-1) if t.dim() == 2 and t.shape[1] < 2 else t, nm, torch.int32)
            if t.dim() != d or (d == 1 and not t.is_contiguous()):
                raise ValueError("%s must be a contiguous %d-D tensor" % (nm, d))
        _same_device(self.device, ctx, cu)
        seqs, columns = table.shape
        if ctx.shape[0] != seqs or cu.shape[0] != seqs + 1:
            raise ValueError("table, ctx and cu must be of seqs, seqs and seqs + 1 rows")
        self.table, self.ctx, self.cu, self.seqs = table, ctx, cu, seqs
        self._c = _Batch(table.data_ptr(), ctx.data_ptr(), cu.data_ptr(),
                         table.stride(0) if seqs > 1 else columns, seqs, columns)


class Rope:
    """Position rotation: cos and sin fp32 (positions, rotated dim / 2) on the
    device; pairs (i, i + rotated dim / 2), or (2 i, 2 i + 1) with `neighbours`."""

    def __init__(self, cos: torch.Tensor, sin: torch.Tensor, neighbours: bool = False):
        self.device = cos.device
        _dev(cos, "cos", torch.float32)
        _dev(sin, "sin", torch.float32)
        _same_device(self.device, sin)
        if cos.dim() != 2 or cos.shape != sin.shape or cos.stride() != sin.stride():
            raise ValueError("cos and sin must be 2-D with one shape and layout")
        self.cos, self.sin = cos, sin
        positions, half = cos.shape
        self._c = _Rope(cos.data_ptr(), sin.data_ptr(), cos.stride(0) if positions > 1 else half, positions,
                        2 * half, 1 if neighbours else 0)


def _heads3(t: torch.Tensor, name: str, rows: int, heads: int, dim: int, dtype, device) -> _Heads:
    if t.dtype is not dtype or t.device != device:
        raise ValueError("%s must be %s on %s" % (name, dtype, device))
    if t.shape != (rows, heads, dim):
        raise ValueError("%s must have shape (%d, %d, %d)" % (name, rows, heads, dim))
    sr, sh, sd = t.stride()
    if sd != 1:
        raise ValueError("%s must have unit stride in its last dimension" % name)
    # a dimension of one entry has no distance to speak of
    return _Heads(t.data_ptr(), sr if rows > 1 else heads * dim, sh if heads > 1 else dim)


def _new_heads3(shape, dtype, device):
    """A new tensor (rows, heads, dim) and its description."""
    t = torch.empty(shape, dtype=dtype, device=device)
    return t, _Heads(t.data_ptr(), shape[1] * shape[2], shape[2])


_AS_IT_IS = contextlib.nullcontext()


def _on_stream(device, stream):
    """(handle of the stream to run on, a context in which the device is current
    and torch allocates for that stream)."""
    if getattr(stream, "device", device) != device:    # default streams of all devices have one handle
        raise ValueError("stream must be one of %s" % device)
    # the current stream's handle without an object for it: calls for one token
    # cost as much as their parts in Python do
    cur = torch._C._cuda_getCurrentRawStream(device.index)
    handle = cur if stream is None else _stream(stream)
    if handle != cur:
        if not hasattr(stream, "cuda_stream"):
            stream = torch.cuda.ExternalStream(handle, device=device)
        return handle, torch.cuda.stream(stream)
    return handle, _AS_IT_IS if torch.cuda.current_device() == device.index else torch.cuda.device(device)


@functools.lru_cache(maxsize=1024)
def _kv_attention_ws(rows: int, seqs: int, q_heads: int, heads: int, dim: int) -> int:
    return load().kronq_kv_attention_ws(rows, seqs, q_heads, heads, dim)


def _kv_check(dtype, cache: KVCache, batch: KVBatch, rope: Rope | None):
    if dtype not in _KV_DTYPES:
        raise ValueError("dtype must be float32, bfloat16 or float16")
    if batch.device != cache.device or (rope is not None and rope.device != cache.device):
        _same_device(cache.device, batch, *(() if rope is None else (rope,)))


def kronq_kv_append(k: torch.Tensor, v: torch.Tensor, cache: KVCache, batch: KVBatch,
                    rope: Rope | None = None, stream=None) -> None:
    """k and v (rows, heads, dim) join the cache at the batch's positions, the
    keys rotated first when `rope` is given."""
    dtype = k.dtype
    _kv_check(dtype, cache, batch, rope)
    rows = k.shape[0]
    kh = _heads3(k, "k", rows, cache.heads, cache.dim, dtype, cache.device)
    vh = _heads3(v, "v", rows, cache.heads, cache.dim, dtype, cache.device)
    st, here = _on_stream(cache.device, stream)
    with here:
        _check(load().kronq_kv_append(kh, vh, _KV_DTYPES[dtype], rows, cache._c, batch._c,
                                      None if rope is None else rope._c, st), "kronq_kv_append")


def kronq_kv_read(cache: KVCache, batch: KVBatch, rows: int, dtype=torch.float32,
                  k: torch.Tensor | None = None, v: torch.Tensor | None = None, stream=None):
    """(k, v): the values held for the last cu[i + 1] - cu[i] positions of each
    sequence, (rows, heads, dim).  Rows of no sequence are left as they were
    (undefined when k or v is allocated here)."""
    _kv_check(dtype, cache, batch, None)
    shape = (rows, cache.heads, cache.dim)
    kh = None if k is None else _heads3(k, "k", *shape, dtype, cache.device)
    vh = None if v is None else _heads3(v, "v", *shape, dtype, cache.device)
    st, here = _on_stream(cache.device, stream)
    with here:
        if kh is None:
            k, kh = _new_heads3(shape, dtype, cache.device)
        if vh is None:
            v, vh = _new_heads3(shape, dtype, cache.device)
        _check(load().kronq_kv_read(kh, vh, _KV_DTYPES[dtype], rows, cache._c, batch._c, st), "kronq_kv_read")
    return k, v


def kronq_kv_attention(q: torch.Tensor, cache: KVCache, batch: KVBatch, scale: float | None = None,
                       window: int = 0, sinks: int = 0, rope: Rope | None = None,
                       out: torch.Tensor | None = None, want_lse: bool = False,
                       lse: torch.Tensor | None = None, stream=None, ws: torch.Tensor | None = None):
    """Causal attention of q (rows, q_heads, dim) over the cache: out in q's
    dtype, or (out, lse) when lse is asked for.  Rows of no sequence are left as
    they were (undefined when out is allocated here).  `ws`: device memory of at
    least the bytes that the call needs, not shared by calls that may run at the
    same time (one that is too small is replaced)."""
    dtype, device = q.dtype, cache.device
    _kv_check(dtype, cache, batch, rope)
    if q.dim() != 3:
        raise ValueError("q must be (rows, q_heads, dim)")
    rows, qheads, _ = q.shape
    shape = (rows, qheads, cache.dim)
    qh = _heads3(q, "q", *shape, dtype, device)
    oh = None if out is None else _heads3(out, "out", *shape, dtype, device)
    if lse is not None and (lse.dtype != torch.float32 or lse.shape != (rows, qheads) or
                            not lse.is_contiguous() or lse.device != device):
        raise ValueError("lse must be a contiguous float32 (rows, q_heads) tensor on %s" % device)
    need = _kv_attention_ws(rows, batch.seqs, qheads, cache.heads, cache.dim)
    if ws is not None and (ws.dtype != torch.uint8 or not ws.is_contiguous() or ws.device != device):
        raise ValueError("ws must be a contiguous uint8 tensor on %s" % device)
    st, here = _on_stream(device, stream)
    with here:
        if oh is None:
            out, oh = _new_heads3(shape, dtype, device)
        if lse is None and want_lse:
            lse = torch.empty((rows, qheads), dtype=torch.float32, device=device)
        if ws is None or ws.numel() < need:
            ws = _ws(need, device)
        _check(load().kronq_kv_attention(qh, _KV_DTYPES[dtype], rows, qheads, cache._c, batch._c,
                                         None if rope is None else rope._c,
                                         cache.dim ** -0.5 if scale is None else scale, window, sinks, oh,
                                         _ptr(lse), _ptr(ws), need, st), "kronq_kv_attention")
    return out if lse is None else (out, lse)


# ------------------------------------------- calibration pass

ROPE_SCALINGS = ("plain", "linear", "parts", "index")


def kronq_rope_tables(positions: int, dim: int, base: float = 10000.0, scaling: str = "plain",
                      factor: float = 1.0, original: float = 0.0, low: float = 1.0, high: float = 4.0,
                      magnitude: float = 1.0, neighbours: bool = False, first: int = 0, device=None,
                      stream=None) -> Rope:
    """The Rope of positions first .. first + positions - 1 for `dim` rotated
    values of a head: plain, or scaled for longer contexts (include/kronq.h has
    the formulas)."""
    if scaling not in ROPE_SCALINGS:
        raise ValueError("unknown scaling %r" % (scaling,))
    device = _cuda_device(device)
    c = _RopeScaling(base, factor, original, low, high, magnitude, ROPE_SCALINGS.index(scaling))
    st, here = _on_stream(device, stream)
    with here:
        if positions < 0 or dim < 2:
            raise ValueError("positions must be at least 0 and dim at least 2")
        cos, sin = torch.empty((2, positions, dim // 2), dtype=torch.float32, device=device)
        _check(load().kronq_rope_tables(cos.data_ptr(), sin.data_ptr(), dim // 2, first, positions, dim,
                                        ctypes.byref(c), st), "kronq_rope_tables")
    return Rope(cos, sin, neighbours)


def _cuda_device(device):
    device = torch.device("cuda" if device is None else device)
    if device.type != "cuda":
        raise ValueError("device must be a GPU")
    return device if device.index is not None else torch.device("cuda", torch.cuda.current_device())


def _ints(t: torch.Tensor, name: str, n: int, device):
    if t.dtype != torch.int32 or t.shape != (n,) or t.device != device or not t.is_contiguous():
        raise ValueError("%s must be a contiguous int32 tensor of %d entries on %s" % (name, n, device))


def _floats(t: torch.Tensor, name: str, shape, device):
    if t.dtype != torch.float32 or t.shape != shape or t.device != device or not t.is_contiguous():
        raise ValueError("%s must be a contiguous float32 tensor of shape %s on %s" % (name, tuple(shape), device))


def kronq_rotate(q: torch.Tensor, k: torch.Tensor | None, pos: torch.Tensor, rope: Rope, back: bool = False,
                 q_out: torch.Tensor | None = None, k_out: torch.Tensor | None = None, stream=None):
    """(q, k) turned by the angles of pos (int32, one a row): q (rows, q_heads,
    dim), k (rows, k_heads, dim) or None.  `back`: by the transpose, which is the
    gradient.  q_out may be q itself (k_out k); they are made where not given.
    Rows of pos < 0 are left as they were (undefined when made here)."""
    dtype, device = q.dtype, q.device
    if dtype not in _KV_DTYPES:
        raise ValueError("q must be float32, bfloat16 or float16")
    if q.dim() != 3 or not q.is_cuda:
        raise ValueError("q must be (rows, heads, dim) on a GPU")
    if k is None and k_out is not None:
        raise ValueError("k_out without k")
    rows, qh, dim = q.shape
    kh = 0
    qs, ks, ko = _heads3(q, "q", rows, qh, dim, dtype, device), None, None
    if k is not None:
        if k.dim() != 3:
            raise ValueError("k must be (rows, heads, dim)")
        kh = k.shape[1]
        ks = _heads3(k, "k", rows, kh, dim, dtype, device)
        if k_out is not None:
            ko = _heads3(k_out, "k_out", rows, kh, dim, dtype, device)
    qo = None if q_out is None else _heads3(q_out, "q_out", rows, qh, dim, dtype, device)
    _ints(pos, "pos", rows, device)
    _same_device(device, rope)
    st, here = _on_stream(device, stream)
    with here:
        if qo is None:
            q_out, qo = _new_heads3((rows, qh, dim), dtype, device)
        if k is not None and ko is None:
            k_out, ko = _new_heads3((rows, kh, dim), dtype, device)
        _check(load().kronq_rotate(qs, qh, ks, kh, _KV_DTYPES[dtype], rows, dim, pos.data_ptr(), rope._c,
                                   1 if back else 0, qo, ko, st), "kronq_rotate")
    return q_out, k_out


def _prompt_shapes(q: torch.Tensor, k: torch.Tensor, cu: torch.Tensor):
    """(rows, q_heads, heads, dim, seqs)"""
    if q.dtype not in _KV_DTYPES:
        raise ValueError("q must be float32, bfloat16 or float16")
    if q.dim() != 3 or k.dim() != 3 or not q.is_cuda:
        raise ValueError("q and k must be (rows, heads, dim) on a GPU")
    if cu.dim() != 1 or cu.shape[0] < 1:
        raise ValueError("cu must have seqs + 1 entries")
    _ints(cu, "cu", cu.shape[0], q.device)
    return *q.shape[:2], k.shape[1], q.shape[2], cu.shape[0] - 1


def kronq_prompt_attention(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, cu: torch.Tensor,
                           scale: float | None = None, window: int = 0, out: torch.Tensor | None = None,
                           want_lse: bool = False, lse: torch.Tensor | None = None, stream=None):
    """Causal attention over packed prompts: rows cu[i] .. cu[i + 1] - 1 (cu int32)
    of q (rows, q_heads, dim), k and v (rows, heads, dim) are sequence i's.  out in
    q's dtype, or (out, lse) when lse is asked for.  Rows of no sequence are left as
    they were (undefined when made here)."""
    rows, qheads, heads, dim, seqs = _prompt_shapes(q, k, cu)
    dtype, device = q.dtype, q.device
    qh = _heads3(q, "q", rows, qheads, dim, dtype, device)
    kh, vh = _heads3(k, "k", rows, heads, dim, dtype, device), _heads3(v, "v", rows, heads, dim, dtype, device)
    oh = None if out is None else _heads3(out, "out", rows, qheads, dim, dtype, device)
    if lse is not None:
        _floats(lse, "lse", (rows, qheads), device)
    st, here = _on_stream(device, stream)
    with here:
        if oh is None:
            out, oh = _new_heads3((rows, qheads, dim), dtype, device)
        if lse is None and want_lse:
            lse = torch.empty((rows, qheads), dtype=torch.float32, device=device)
        _check(load().kronq_prompt_attention(qh, kh, vh, _KV_DTYPES[dtype], rows, qheads, heads, dim, cu.data_ptr(),
                                             seqs, dim ** -0.5 if scale is None else scale, window, oh, _ptr(lse),
                                             st), "kronq_prompt_attention")
    return out if lse is None else (out, lse)


def kronq_prompt_attention_grad(dout: torch.Tensor, q: torch.Tensor, k: torch.Tensor, v: torch.Tensor,
                                out: torch.Tensor, lse: torch.Tensor, cu: torch.Tensor,
                                scale: float | None = None, window: int = 0, dq: torch.Tensor | None = None,
                                dk: torch.Tensor | None = None, dv: torch.Tensor | None = None, stream=None,
                                ws: torch.Tensor | None = None):
    """(dq, dk, dv) from dout, the gradient of out, and what kronq_prompt_attention
    was given and gave.  Rows of no sequence are left as they were (undefined when
    made here).  `ws`: device memory that calls that may run at the same time do not
    share."""
    rows, qheads, heads, dim, seqs = _prompt_shapes(q, k, cu)
    dtype, device = q.dtype, q.device
    wide, narrow = (rows, qheads, dim), (rows, heads, dim)
    h = [_heads3(t, nm, *shape, dtype, device)
         for t, nm, shape in ((dout, "dout", wide), (q, "q", wide), (k, "k", narrow), (v, "v", narrow), (out, "out", wide))]
    g = [None if t is None else _heads3(t, nm, *shape, dtype, device)
         for t, nm, shape in ((dq, "dq", wide), (dk, "dk", narrow), (dv, "dv", narrow))]
    _floats(lse, "lse", (rows, qheads), device)
    need = load().kronq_prompt_attention_grad_ws(rows, qheads)
    if ws is not None and (ws.dtype != torch.uint8 or not ws.is_contiguous() or ws.device != device):
        raise ValueError("ws must be a contiguous uint8 tensor on %s" % device)
    st, here = _on_stream(device, stream)
    with here:
        if dq is None:
            dq, g[0] = _new_heads3(wide, dtype, device)
        if dk is None:
            dk, g[1] = _new_heads3(narrow, dtype, device)
        if dv is None:
            dv, g[2] = _new_heads3(narrow, dtype, device)
        if need and (ws is None or ws.numel() < need):
            ws = _ws(need, device)
        _check(load().kronq_prompt_attention_grad(*h, lse.data_ptr(), _KV_DTYPES[dtype], rows, qheads, heads, dim,
                                                  cu.data_ptr(), seqs, dim ** -0.5 if scale is None else scale, window,
                                                  *g, _ptr(ws), need, st), "kronq_prompt_attention_grad")
    return dq, dk, dv


def _logits(t: torch.Tensor, name: str):
    """(rows, vocab, leading dimension)"""
    if t.dtype not in _KV_DTYPES:
        raise ValueError("%s must be float32, bfloat16 or float16" % name)
    if t.dim() != 2 or not t.is_cuda:
        raise ValueError("%s must be (rows, vocab) on a GPU" % name)
    rows, vocab = t.shape
    if vocab > 1 and t.stride(1) != 1:
        raise ValueError("%s must have unit stride in its last dimension" % name)
    return rows, vocab, t.stride(0) if rows > 1 else vocab


@functools.lru_cache(maxsize=1024)
def _token_logprobs_ws(rows: int, vocab: int, top: int) -> int:
    return load().kronq_token_logprobs_ws(rows, vocab, top)


def kronq_token_logprobs(logits: torch.Tensor, targets: torch.Tensor | None = None, top: int = 0,
                         want_entropy: bool = False, stream=None, ws: torch.Tensor | None = None) -> dict:
    """Of each row of logits (rows, vocab): lse, logp of its target (int32, below
    0: none), entropy when asked for, and with `top` the top_logp and top_ids of
    its largest (rows, top), equal ones by ascending index.  `ws`: device memory
    that calls that may run at the same time do not share."""
    rows, vocab, ld = _logits(logits, "logits")
    device = logits.device
    if targets is not None:
        _ints(targets, "targets", rows, device)
    need = _token_logprobs_ws(rows, vocab, top)
    if ws is not None and (ws.dtype != torch.uint8 or not ws.is_contiguous() or ws.device != device):
        raise ValueError("ws must be a contiguous uint8 tensor on %s" % device)
    st, here = _on_stream(device, stream)
    with here:
        new = lambda *shape: torch.empty(shape, dtype=torch.float32, device=device)  # noqa: E731
        got = dict(lse=new(rows))
        if targets is not None:
            got["logp"] = new(rows)
        if want_entropy:
            got["entropy"] = new(rows)
        if top > 0:
            got["top_logp"] = new(rows, top)
            got["top_ids"] = torch.empty((rows, top), dtype=torch.int32, device=device)
        if need and (ws is None or ws.numel() < need):
            ws = _ws(need, device)
        _check(load().kronq_token_logprobs(logits.data_ptr(), _KV_DTYPES[logits.dtype], rows, vocab, ld,
                                           _ptr(targets), _ptr(got.get("logp")), got["lse"].data_ptr(),
                                           _ptr(got.get("entropy")), top, _ptr(got.get("top_logp")),
                                           _ptr(got.get("top_ids")), _ptr(ws), need, st),
               "kronq_token_logprobs")
    return got


def kronq_token_logprobs_grad(logits: torch.Tensor, targets: torch.Tensor | None, lse: torch.Tensor,
                              d_logp: torch.Tensor | None = None, entropy: torch.Tensor | None = None,
                              d_entropy: torch.Tensor | None = None, top_ids: torch.Tensor | None = None,
                              d_top: torch.Tensor | None = None, out: torch.Tensor | None = None,
                              stream=None) -> torch.Tensor:
    """The gradient with respect to logits, in their type, of what
    kronq_token_logprobs gave: d_logp, d_entropy (rows) and d_top (rows, top) are
    the gradients of logp, entropy and top_logp, each None for none.  `out` may be
    logits itself."""
    rows, vocab, ld = _logits(logits, "logits")
    device = logits.device
    if targets is not None:
        _ints(targets, "targets", rows, device)
    for t, nm in ((lse, "lse"), (d_logp, "d_logp"), (entropy, "entropy"), (d_entropy, "d_entropy")):
        if t is not None:
            _floats(t, nm, (rows,), device)
    top = 0
    if d_top is not None:
        if top_ids is None or top_ids.dim() != 2:
            raise ValueError("d_top needs top_ids (rows, top)")
        top = top_ids.shape[1]
        _floats(d_top, "d_top", (rows, top), device)
        if top_ids.dtype != torch.int32 or top_ids.shape != (rows, top) or top_ids.device != device or \
                not top_ids.is_contiguous():
            raise ValueError("top_ids must be a contiguous int32 tensor of shape (%d, %d) on %s" % (rows, top, device))
    ld_out = vocab
    if out is not None:
        if out.dtype != logits.dtype or out.device != device or out.shape != logits.shape:
            raise ValueError("out must have the type, shape and device of logits")
        ld_out = _logits(out, "out")[2]
    st, here = _on_stream(device, stream)
    with here:
        if out is None:
            out = torch.empty((rows, vocab), dtype=logits.dtype, device=device)
        _check(load().kronq_token_logprobs_grad(logits.data_ptr(), _KV_DTYPES[logits.dtype], rows, vocab, ld,
                                                _ptr(targets), lse.data_ptr(), _ptr(entropy), _ptr(d_logp),
                                                _ptr(d_entropy), top, _ptr(top_ids) if top else None,
                                                _ptr(d_top) if top else None, out.data_ptr(), ld_out, st),
               "kronq_token_logprobs_grad")
    return out
