"""B200 (sm_100a) MLA decode over a paged latent KV cache.

A thin ctypes binding over ``libmla_b200.so`` (C ABI in ``include/mla.h``).  The
functions keep the C names and only marshal arguments: torch tensors become
device pointers and sizes, the current torch stream becomes the CUDA stream.
Every step of the computation runs in the library's CUDA kernels; there is no
fallback, and calling into a missing library raises.
"""

from __future__ import annotations

import ctypes
import os
from typing import Optional

PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(PKG, "libmla_b200.so")

D_C, D_R, D_N, D_V, PAGE = 512, 64, 128, 128, 64
MAX_SPLITS = 128
KV_BF16, KV_FP8_E4M3, KV_Q8_0, KV_Q4_0 = 0, 1, 2, 3
PROB_FP32, PROB_BF16 = 0, 1
Q8_BLOCKS = (D_C + D_R) // 32   # q8_0: scale blocks of a 576-value row

STATUS = {
    0: "MLA_OK", 1: "MLA_ERR_INVALID_VALUE", 2: "MLA_ERR_UNSUPPORTED", 3: "MLA_ERR_MISALIGNED",
    4: "MLA_ERR_WORKSPACE_TOO_SMALL", 5: "MLA_ERR_CUDA", 6: "MLA_ERR_DEVICE_TIMEOUT",
    7: "MLA_ERR_BAD_BLOCK_TABLE", 8: "MLA_ERR_BAD_SEQ_LEN", 9: "MLA_ERR_BAD_TOKEN",
}

# Every symbol include/mla.h declares.
EXPORTS = ("mla_absorb_q", "mla_decode_workspace_size", "mla_decode_num_splits",
           "mla_decode_paged", "mla_combine_splits", "mla_up_proj_v", "mla_get_status",
           "mla_status_string", "mla_decode_paged_noalloc", "mla_noalloc_init",
           "mla_get_status_noalloc", "mla_write_kv_workspace_size", "mla_write_kv",
           "mla_set_decode_kernel", "mla_set_device_wait_limit", "mla_fold_hadamard", "mla_prefill_workspace_size",
           "mla_prefill", "mla_decode_step_workspace_size", "mla_decode_step_launches", "mla_decode_step",
           "mla_append_workspace_size", "mla_append_kv", "mla_prefill_packed_workspace_size",
           "mla_prefill_packed", "mla_verify_workspace_size", "mla_verify_draft")

DECODE_AUTO, DECODE_WARP_MMA = 0, 1


class MlaError(RuntimeError):
    def __init__(self, fn, code):
        super().__init__(f"{fn} failed: {STATUS.get(code, code)}")
        self.code = code


class DecodeArgs(ctypes.Structure):
    """Mirror of ``mla_decode_args_t`` (field order and types must match)."""
    _fields_ = [
        ("q_lat", ctypes.c_void_p), ("q_pe", ctypes.c_void_p),
        ("kv_cache", ctypes.c_void_p), ("kv_scale", ctypes.c_void_p),
        ("block_table", ctypes.c_void_p), ("seq_lens", ctypes.c_void_p),
        ("o_lat", ctypes.c_void_p), ("lse", ctypes.c_void_p),
        ("workspace", ctypes.c_void_p), ("workspace_bytes", ctypes.c_size_t),
        ("B", ctypes.c_int32), ("s_q", ctypes.c_int32), ("H", ctypes.c_int32),
        ("d_c", ctypes.c_int32), ("d_r", ctypes.c_int32), ("page_size", ctypes.c_int32),
        ("num_pages", ctypes.c_int32), ("max_pages_per_seq", ctypes.c_int32),
        ("kv_dtype", ctypes.c_int32), ("causal", ctypes.c_int32),
        ("num_splits", ctypes.c_int32), ("max_seq_len", ctypes.c_int32),
        ("softmax_scale", ctypes.c_float),
    ]


class WriteKvArgs(ctypes.Structure):
    """Mirror of ``mla_write_kv_args_t`` (field order and types must match)."""
    _fields_ = [
        ("h", ctypes.c_void_p), ("w_dkv", ctypes.c_void_p),
        ("kv_cache", ctypes.c_void_p), ("kv_scale", ctypes.c_void_p),
        ("block_table", ctypes.c_void_p), ("seq_lens", ctypes.c_void_p),
        ("workspace", ctypes.c_void_p), ("workspace_bytes", ctypes.c_size_t),
        ("B", ctypes.c_int32), ("s_q", ctypes.c_int32), ("d_h", ctypes.c_int32),
        ("d_c", ctypes.c_int32), ("d_r", ctypes.c_int32), ("page_size", ctypes.c_int32),
        ("num_pages", ctypes.c_int32), ("max_pages_per_seq", ctypes.c_int32),
        ("kv_dtype", ctypes.c_int32), ("rope_base", ctypes.c_float),
    ]


class PrefillArgs(ctypes.Structure):
    """Mirror of ``mla_prefill_args_t`` (field order and types must match)."""
    _fields_ = [
        ("q_nope", ctypes.c_void_p), ("q_pe", ctypes.c_void_p),
        ("w_uk", ctypes.c_void_p), ("w_uv", ctypes.c_void_p),
        ("kv_cache", ctypes.c_void_p),
        ("block_table", ctypes.c_void_p), ("seq_lens", ctypes.c_void_p),
        ("out", ctypes.c_void_p), ("lse", ctypes.c_void_p),
        ("workspace", ctypes.c_void_p), ("workspace_bytes", ctypes.c_size_t),
        ("B", ctypes.c_int32), ("s_q", ctypes.c_int32), ("H", ctypes.c_int32),
        ("d_c", ctypes.c_int32), ("d_r", ctypes.c_int32), ("page_size", ctypes.c_int32),
        ("num_pages", ctypes.c_int32), ("max_pages_per_seq", ctypes.c_int32),
        ("kv_dtype", ctypes.c_int32), ("causal", ctypes.c_int32),
        ("max_seq_len", ctypes.c_int32), ("softmax_scale", ctypes.c_float),
    ]


class StepArgs(ctypes.Structure):
    """Mirror of ``mla_step_args_t`` (field order and types must match)."""
    _fields_ = [
        ("q_nope", ctypes.c_void_p), ("q_pe", ctypes.c_void_p),
        ("w_uk", ctypes.c_void_p), ("w_uv", ctypes.c_void_p),
        ("kv_cache", ctypes.c_void_p), ("kv_scale", ctypes.c_void_p),
        ("block_table", ctypes.c_void_p), ("seq_lens", ctypes.c_void_p),
        ("out", ctypes.c_void_p), ("lse", ctypes.c_void_p),
        ("workspace", ctypes.c_void_p), ("workspace_bytes", ctypes.c_size_t),
        ("B", ctypes.c_int32), ("s_q", ctypes.c_int32), ("H", ctypes.c_int32),
        ("d_c", ctypes.c_int32), ("d_r", ctypes.c_int32), ("page_size", ctypes.c_int32),
        ("num_pages", ctypes.c_int32), ("max_pages_per_seq", ctypes.c_int32),
        ("kv_dtype", ctypes.c_int32), ("causal", ctypes.c_int32), ("num_splits", ctypes.c_int32),
        ("max_seq_len", ctypes.c_int32), ("softmax_scale", ctypes.c_float), ("fuse", ctypes.c_int32),
    ]


class AppendArgs(ctypes.Structure):
    """Mirror of ``mla_append_args_t`` (field order and types must match)."""
    _fields_ = [
        ("c", ctypes.c_void_p), ("k_pe", ctypes.c_void_p), ("q_pe", ctypes.c_void_p),
        ("k_pe_out", ctypes.c_void_p), ("q_pe_out", ctypes.c_void_p),
        ("kv_cache", ctypes.c_void_p), ("kv_scale", ctypes.c_void_p),
        ("block_table", ctypes.c_void_p), ("cu_seqlens", ctypes.c_void_p), ("seq_lens", ctypes.c_void_p),
        ("workspace", ctypes.c_void_p), ("workspace_bytes", ctypes.c_size_t),
        ("c_tok", ctypes.c_int64), ("k_pe_tok", ctypes.c_int64),
        ("q_pe_tok", ctypes.c_int64), ("q_pe_head", ctypes.c_int64),
        ("k_pe_out_tok", ctypes.c_int64), ("q_pe_out_tok", ctypes.c_int64), ("q_pe_out_head", ctypes.c_int64),
        ("n_tok", ctypes.c_int32), ("B", ctypes.c_int32), ("H", ctypes.c_int32),
        ("d_c", ctypes.c_int32), ("d_r", ctypes.c_int32), ("page_size", ctypes.c_int32),
        ("num_pages", ctypes.c_int32), ("max_pages_per_seq", ctypes.c_int32),
        ("kv_dtype", ctypes.c_int32), ("rope_base", ctypes.c_float),
    ]


class PrefillPackedArgs(ctypes.Structure):
    """Mirror of ``mla_prefill_packed_args_t`` (field order and types must match)."""
    _fields_ = [
        ("q_nope", ctypes.c_void_p), ("q_pe", ctypes.c_void_p),
        ("k_nope", ctypes.c_void_p), ("k_pe", ctypes.c_void_p), ("v", ctypes.c_void_p),
        ("cu_seqlens", ctypes.c_void_p), ("out", ctypes.c_void_p), ("lse", ctypes.c_void_p),
        ("workspace", ctypes.c_void_p), ("workspace_bytes", ctypes.c_size_t),
        ("q_nope_tok", ctypes.c_int64), ("q_nope_head", ctypes.c_int64),
        ("q_pe_tok", ctypes.c_int64), ("q_pe_head", ctypes.c_int64),
        ("k_nope_tok", ctypes.c_int64), ("k_nope_head", ctypes.c_int64), ("k_pe_tok", ctypes.c_int64),
        ("v_tok", ctypes.c_int64), ("v_head", ctypes.c_int64),
        ("n_tok", ctypes.c_int32), ("B", ctypes.c_int32), ("H", ctypes.c_int32), ("H_kv", ctypes.c_int32),
        ("d_n", ctypes.c_int32), ("d_r", ctypes.c_int32), ("d_v", ctypes.c_int32),
        ("causal", ctypes.c_int32), ("softmax_scale", ctypes.c_float),
    ]


class VerifyArgs(ctypes.Structure):
    """Mirror of ``mla_verify_args_t`` (field order and types must match)."""
    _fields_ = [
        ("target_probs", ctypes.c_void_p), ("draft_probs", ctypes.c_void_p),
        ("draft_tokens", ctypes.c_void_p), ("num_draft", ctypes.c_void_p),
        ("u_accept", ctypes.c_void_p), ("u_sample", ctypes.c_void_p), ("seq_lens", ctypes.c_void_p),
        ("tokens", ctypes.c_void_p), ("num_accepted", ctypes.c_void_p), ("new_lens", ctypes.c_void_p),
        ("workspace", ctypes.c_void_p), ("workspace_bytes", ctypes.c_size_t),
        ("target_seq", ctypes.c_int64), ("target_row", ctypes.c_int64),
        ("draft_seq", ctypes.c_int64), ("draft_row", ctypes.c_int64),
        ("B", ctypes.c_int32), ("s_q", ctypes.c_int32), ("V", ctypes.c_int32), ("dtype", ctypes.c_int32),
    ]


_lib: Optional[ctypes.CDLL] = None


def load(path: str = LIB_PATH) -> ctypes.CDLL:
    """Load the CUDA library (built by ``head_latent_attention_06_b200.build``)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise RuntimeError(f"{path} is missing: run `python -m head_latent_attention_06_b200.build`")
    lib = ctypes.CDLL(path)
    vp, i32 = ctypes.c_void_p, ctypes.c_int32
    lib.mla_absorb_q.argtypes = [vp, vp, vp, i32, i32, i32, i32, vp]
    lib.mla_up_proj_v.argtypes = [vp, vp, vp, i32, i32, i32, i32, vp]
    pa = ctypes.POINTER(DecodeArgs)
    lib.mla_decode_workspace_size.argtypes = [pa, ctypes.POINTER(ctypes.c_size_t)]
    lib.mla_decode_num_splits.argtypes = [pa, ctypes.POINTER(ctypes.c_int32)]
    lib.mla_decode_paged.argtypes = [pa, vp]
    lib.mla_combine_splits.argtypes = [pa, vp]
    lib.mla_decode_paged_noalloc.argtypes = [pa, vp]
    lib.mla_noalloc_init.argtypes = []
    lib.mla_get_status_noalloc.argtypes = [vp]
    lib.mla_set_decode_kernel.argtypes = [i32]
    lib.mla_set_device_wait_limit.argtypes = [ctypes.c_uint64]
    pw = ctypes.POINTER(WriteKvArgs)
    lib.mla_write_kv_workspace_size.argtypes = [pw, ctypes.POINTER(ctypes.c_size_t)]
    lib.mla_write_kv.argtypes = [pw, vp]
    pp = ctypes.POINTER(PrefillArgs)
    lib.mla_prefill_workspace_size.argtypes = [pp, ctypes.POINTER(ctypes.c_size_t)]
    lib.mla_prefill.argtypes = [pp, vp]
    lib.mla_get_status.argtypes = [vp, vp]
    ps = ctypes.POINTER(StepArgs)
    lib.mla_decode_step_workspace_size.argtypes = [ps, ctypes.POINTER(ctypes.c_size_t)]
    lib.mla_decode_step_launches.argtypes = [ps, ctypes.POINTER(ctypes.c_int32)]
    lib.mla_decode_step.argtypes = [ps, vp]
    lib.mla_fold_hadamard.argtypes = [vp, i32, vp, vp, i32, vp]
    for name, kind in (("append", AppendArgs), ("prefill_packed", PrefillPackedArgs), ("verify", VerifyArgs)):
        getattr(lib, f"mla_{name}_workspace_size").argtypes = [ctypes.POINTER(kind), ctypes.POINTER(ctypes.c_size_t)]
    lib.mla_append_kv.argtypes = [ctypes.POINTER(AppendArgs), vp]
    lib.mla_prefill_packed.argtypes = [ctypes.POINTER(PrefillPackedArgs), vp]
    lib.mla_verify_draft.argtypes = [ctypes.POINTER(VerifyArgs), vp]
    lib.mla_status_string.argtypes = [ctypes.c_int]
    lib.mla_status_string.restype = ctypes.c_char_p
    for name in EXPORTS:
        if name != "mla_status_string":
            getattr(lib, name).restype = ctypes.c_int
    _lib = lib
    return lib


def _ptr(t) -> Optional[int]:
    return None if t is None else int(t.data_ptr())


_raw_stream = None


def _stream(stream) -> Optional[int]:
    """The CUDA stream handle: torch's current stream for None.  Its raw handle is asked
    for where this torch has the call (0.3 us; building the Stream object takes 3)."""
    if stream is None:
        global _raw_stream
        import torch
        if _raw_stream is None:
            _raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream",
                                  lambda index: torch.cuda.current_stream(index).cuda_stream)
        return int(_raw_stream(torch.cuda.current_device()))
    return int(stream) if isinstance(stream, int) else int(stream.cuda_stream)


def _check(fn, code):
    if code != 0:
        raise MlaError(fn, code)


def _want(specs):
    """Argument check of the tensor builders.  ``specs``: (tensor, name, dtype or
    tuple of dtypes, shape or None, optional).  Every tensor's dtype, shape and
    contiguity are checked first, then every tensor's device; the first problem
    raises ValueError naming the field."""
    for t, name, dtypes, shape, optional in specs:
        if t is None:
            if optional:
                continue
            raise ValueError(f"{name} is required")
        dtypes = dtypes if isinstance(dtypes, tuple) else (dtypes,)
        if t.dtype not in dtypes:
            raise ValueError(f"{name}: dtype {t.dtype}, expected {' or '.join(str(d) for d in dtypes)}")
        if shape is not None and tuple(t.shape) != tuple(shape):
            raise ValueError(f"{name}: shape {tuple(t.shape)}, expected {tuple(shape)}")
        if not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous")
    for t, name, _, _, _ in specs:
        if t is not None and not t.is_cuda:
            raise ValueError(f"{name} must be a CUDA tensor")


def _want_one_device(specs):
    """The last check of the packed and verification builders: every tensor on one
    CUDA device, which the entry points then make current.  Returns that device."""
    dev = None
    for t, name, *_ in specs:
        if t is None:
            continue
        if not t.is_cuda:
            raise ValueError(f"{name} must be a CUDA tensor")
        if dev is not None and t.device != dev:
            raise ValueError(f"{name} is on {t.device}, the others on {dev}")
        dev = t.device
    return dev


def _want_views(specs):
    """Like ``_want``, for tensors of which only the innermost dimension has to be
    contiguous (strided views); the device is left to ``_want_one_device``."""
    for t, name, dtypes, shape, optional in specs:
        if t is None:
            if optional:
                continue
            raise ValueError(f"{name} is required")
        dtypes = dtypes if isinstance(dtypes, tuple) else (dtypes,)
        if t.dtype not in dtypes:
            raise ValueError(f"{name}: dtype {t.dtype}, expected {' or '.join(str(d) for d in dtypes)}")
        if tuple(t.shape) != tuple(shape):
            raise ValueError(f"{name}: shape {tuple(t.shape)}, expected {tuple(shape)}")
        if t.shape[-1] > 1 and t.stride(-1) != 1:
            raise ValueError(f"{name}: its innermost dimension must be contiguous")


def _want_dense(specs):
    """``_want`` without the device check."""
    _want_views([(t, n, d, t.shape if t is not None and s is None else s, o) for t, n, d, s, o in specs])
    for t, name, *_ in specs:
        if t is not None and not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous")


def _call(fn, args, stream):
    """Calls entry point ``fn`` on ``stream`` (default: torch's current stream of the
    device that the arguments' tensors are on), with that device current."""
    import torch
    dev = getattr(args, "device", None)
    if dev is None or dev.index == torch.cuda.current_device():
        code = getattr(_lib or load(), fn)(ctypes.byref(args), _stream(stream))
    else:
        with torch.cuda.device(dev):
            code = getattr(_lib or load(), fn)(ctypes.byref(args), _stream(stream))
    if code != 0:
        raise MlaError(fn, code)


def _workspace_size(fn, args) -> int:
    n = ctypes.c_size_t(0)
    _check(fn, getattr(load(), fn)(ctypes.byref(args), ctypes.byref(n)))
    return int(n.value)


def _tokens(t, name, H, d):
    """Token count of a [..., H, d] tensor (any leading token dimensions)."""
    if t.dim() < 2 or tuple(t.shape[-2:]) != (H, d):
        raise ValueError(f"{name}: shape {tuple(t.shape)}, expected [..., {H}, {d}]")
    return t.numel() // (H * d)


# ------------------------------------------------------------------ entry points

def mla_absorb_q(q_nope, w_uk, q_lat, stream=None):
    """q_lat[t][h] = W_UK[h]^T q_nope[t][h]; q_nope [n_tok][H][128], w_uk [H][128][512],
    q_lat [n_tok][H][512], all bf16 on the device."""
    import torch
    H = w_uk.shape[0]
    n_tok = _tokens(q_nope, "q_nope", H, D_N)
    if _tokens(q_lat, "q_lat", H, D_C) != n_tok:
        raise ValueError("q_lat must hold as many tokens as q_nope")
    _want([(q_nope, "q_nope", torch.bfloat16, None, False), (w_uk, "w_uk", torch.bfloat16, (H, D_N, D_C), False),
           (q_lat, "q_lat", torch.bfloat16, None, False)])
    _check("mla_absorb_q", load().mla_absorb_q(_ptr(q_nope), _ptr(w_uk), _ptr(q_lat), n_tok, H,
                                               w_uk.shape[1], w_uk.shape[2], _stream(stream)))


def mla_up_proj_v(o_lat, w_uv, out, stream=None):
    """out[t][h] = W_UV[h] o_lat[t][h]; o_lat [n_tok][H][512], w_uv [H][128][512],
    out [n_tok][H][128], all bf16 on the device."""
    import torch
    H = w_uv.shape[0]
    n_tok = _tokens(o_lat, "o_lat", H, D_C)
    if _tokens(out, "out", H, D_V) != n_tok:
        raise ValueError("out must hold as many tokens as o_lat")
    _want([(o_lat, "o_lat", torch.bfloat16, None, False), (w_uv, "w_uv", torch.bfloat16, (H, D_V, D_C), False),
           (out, "out", torch.bfloat16, None, False)])
    _check("mla_up_proj_v", load().mla_up_proj_v(_ptr(o_lat), _ptr(w_uv), _ptr(out), n_tok, H,
                                                 w_uv.shape[1], w_uv.shape[2], _stream(stream)))


def mla_fold_hadamard(w_dkv=None, w_uk=None, w_uv=None, stream=None):
    """Folds the orthonormal 512-point Hadamard rotation into the weights, in place:
    w_dkv [576][d_h] (rows 0..511 -> H W_DKV), w_uk and w_uv [H][128][512] (each row
    -> row H); bf16 on the device, any of them may be None."""
    import torch
    H = (w_uk if w_uk is not None else w_uv).shape[0] if (w_uk is not None or w_uv is not None) else 0
    d_h = w_dkv.shape[1] if w_dkv is not None else 0
    _want([(w_dkv, "w_dkv", torch.bfloat16, (D_C + D_R, d_h), True),
           (w_uk, "w_uk", torch.bfloat16, (H, D_N, D_C), True),
           (w_uv, "w_uv", torch.bfloat16, (H, D_V, D_C), True)])
    _check("mla_fold_hadamard", load().mla_fold_hadamard(_ptr(w_dkv), d_h, _ptr(w_uk), _ptr(w_uv), H,
                                                         _stream(stream)))


def _cache_kind(kv_cache):
    """(kv_dtype code, scale dtype, scale shape tail, row width) of a cache tensor's
    dtype: bf16 values; float8_e4m3fn codes with fp32 row scales [pages][64]; int8
    q8_0 codes with fp16 block scales [pages][64][18]; uint8 q4_0 bytes (two codes
    a byte, 288 a row) with fp16 block scales [pages][64][18]."""
    import torch
    if kv_cache.dtype == torch.float8_e4m3fn:
        return KV_FP8_E4M3, torch.float32, (), D_C + D_R
    if kv_cache.dtype == torch.int8:
        return KV_Q8_0, torch.float16, (Q8_BLOCKS,), D_C + D_R
    if kv_cache.dtype == torch.uint8:
        return KV_Q4_0, torch.float16, (Q8_BLOCKS,), (D_C + D_R) // 2
    return KV_BF16, None, (), D_C + D_R


def make_decode_args(*, q_lat, q_pe, kv_cache, kv_scale, block_table, seq_lens, o_lat, lse,
                     workspace=None, causal=False, softmax_scale, num_splits=0,
                     max_seq_len=0) -> DecodeArgs:
    """Fill a ``DecodeArgs`` from device tensors.  Shapes: q_lat [B][s_q][H][512],
    q_pe [B][s_q][H][64], kv_cache [num_pages][64][576] (bf16, float8_e4m3fn or
    int8 for q8_0) or [num_pages][64][288] uint8 (q4_0), kv_scale [num_pages][64]
    fp32 (e4m3), [num_pages][64][18] fp16 (q8_0, q4_0) or None (bf16), block_table
    [B][max_pages] int32, seq_lens [B] int32, o_lat like q_lat, lse [B][s_q][H]
    fp32 or None."""
    import torch
    bf16, f32, i32 = torch.bfloat16, torch.float32, torch.int32
    if q_lat.dim() != 4 or kv_cache.dim() != 3 or block_table.dim() != 2:
        raise ValueError("q_lat must be [B][s_q][H][512], kv_cache [pages][64][576], block_table [B][pages]")
    B, s_q, H, _ = q_lat.shape
    P = kv_cache.shape[0]
    kind, sc_dtype, sc_tail, width = _cache_kind(kv_cache)
    _want([(q_lat, "q_lat", bf16, (B, s_q, H, D_C), False),
           (q_pe, "q_pe", bf16, (B, s_q, H, D_R), False),
           (kv_cache, "kv_cache", (bf16, torch.float8_e4m3fn, torch.int8, torch.uint8), (P, PAGE, width), False),
           (kv_scale, "kv_scale", sc_dtype or f32, (P, PAGE) + sc_tail, kind == KV_BF16),
           (block_table, "block_table", i32, (B, block_table.shape[1]), False),
           (seq_lens, "seq_lens", i32, (B,), False),
           (o_lat, "o_lat", bf16, (B, s_q, H, D_C), False),
           (lse, "lse", f32, (B, s_q, H), True),
           (workspace, "workspace", torch.uint8, None, True)])
    a = DecodeArgs()
    a.q_lat, a.q_pe = _ptr(q_lat), _ptr(q_pe)
    a.kv_cache, a.kv_scale = _ptr(kv_cache), _ptr(kv_scale)
    a.block_table, a.seq_lens = _ptr(block_table), _ptr(seq_lens)
    a.o_lat, a.lse = _ptr(o_lat), _ptr(lse)
    a.B, a.s_q, a.H = B, s_q, H
    a.d_c, a.d_r, a.page_size = D_C, D_R, PAGE
    a.num_pages = kv_cache.shape[0]
    a.max_pages_per_seq = block_table.shape[1]
    a.kv_dtype = kind
    a.causal = int(bool(causal))
    a.num_splits = int(num_splits)
    a.max_seq_len = int(max_seq_len)
    a.softmax_scale = float(softmax_scale)
    if workspace is not None:
        a.workspace, a.workspace_bytes = _ptr(workspace), workspace.numel() * workspace.element_size()
    return a


def mla_decode_workspace_size(args: DecodeArgs) -> int:
    n = ctypes.c_size_t(0)
    _check("mla_decode_workspace_size", load().mla_decode_workspace_size(ctypes.byref(args), ctypes.byref(n)))
    return int(n.value)


def mla_decode_num_splits(args: DecodeArgs) -> int:
    n = ctypes.c_int32(0)
    _check("mla_decode_num_splits", load().mla_decode_num_splits(ctypes.byref(args), ctypes.byref(n)))
    return int(n.value)


def mla_decode_paged(args: DecodeArgs, stream=None):
    _check("mla_decode_paged", load().mla_decode_paged(ctypes.byref(args), _stream(stream)))


def mla_combine_splits(args: DecodeArgs, stream=None):
    _check("mla_combine_splits", load().mla_combine_splits(ctypes.byref(args), _stream(stream)))


def mla_decode_paged_noalloc(args: DecodeArgs, stream=None):
    """Decode plus split merge with the library's built-in scratch (args.workspace is
    ignored); for callers that cannot allocate device memory."""
    _check("mla_decode_paged_noalloc", load().mla_decode_paged_noalloc(ctypes.byref(args), _stream(stream)))


def mla_noalloc_init():
    """Set-up of the built-in scratch on the current device (address lookup, status
    word zeroed); call at start-up, before any stream capture."""
    _check("mla_noalloc_init", load().mla_noalloc_init())


def mla_get_status_noalloc(stream=None) -> int:
    """Waits for the stream and returns (and clears) the built-in scratch's device
    status word."""
    return int(load().mla_get_status_noalloc(_stream(stream)))


def mla_set_decode_kernel(kernel: int):
    """Process-wide decode kernel choice: DECODE_AUTO or DECODE_WARP_MMA."""
    _check("mla_set_decode_kernel", load().mla_set_decode_kernel(int(kernel)))


def mla_set_device_wait_limit(ns: int):
    """Process-wide limit of the decode kernels' bounded waits (0: the 2 s default)."""
    _check("mla_set_device_wait_limit", load().mla_set_device_wait_limit(int(ns)))


def make_write_kv_args(*, h, w_dkv, kv_cache, kv_scale, block_table, seq_lens, workspace=None,
                       rope_base=10000.0) -> WriteKvArgs:
    """Fill a ``WriteKvArgs`` from device tensors.  Shapes: h [B][s_q][d_h] bf16,
    w_dkv [576][d_h] bf16 (W_DKV rows, then W_KR rows), kv_cache [num_pages][64][576]
    (bf16, float8_e4m3fn or int8 for q8_0) or [num_pages][64][288] uint8 (q4_0),
    kv_scale [num_pages][64] fp32 (e4m3), [num_pages][64][18] fp16 (q8_0, q4_0) or
    None (bf16), block_table [B][max_pages] int32, seq_lens [B] int32."""
    import torch
    bf16, f32, i32 = torch.bfloat16, torch.float32, torch.int32
    if h.dim() != 3 or kv_cache.dim() != 3 or block_table.dim() != 2:
        raise ValueError("h must be [B][s_q][d_h], kv_cache [pages][64][576], block_table [B][pages]")
    B, s_q, d_h = h.shape
    P = kv_cache.shape[0]
    kind, sc_dtype, sc_tail, width = _cache_kind(kv_cache)
    _want([(h, "h", bf16, (B, s_q, d_h), False),
           (w_dkv, "w_dkv", bf16, (D_C + D_R, d_h), False),
           (kv_cache, "kv_cache", (bf16, torch.float8_e4m3fn, torch.int8, torch.uint8), (P, PAGE, width), False),
           (kv_scale, "kv_scale", sc_dtype or f32, (P, PAGE) + sc_tail, kind == KV_BF16),
           (block_table, "block_table", i32, (B, block_table.shape[1]), False),
           (seq_lens, "seq_lens", i32, (B,), False),
           (workspace, "workspace", torch.uint8, None, True)])
    a = WriteKvArgs()
    a.h, a.w_dkv = _ptr(h), _ptr(w_dkv)
    a.kv_cache, a.kv_scale = _ptr(kv_cache), _ptr(kv_scale)
    a.block_table, a.seq_lens = _ptr(block_table), _ptr(seq_lens)
    a.B, a.s_q, a.d_h = B, s_q, d_h
    a.d_c, a.d_r, a.page_size = D_C, D_R, PAGE
    a.num_pages = kv_cache.shape[0]
    a.max_pages_per_seq = block_table.shape[1]
    a.kv_dtype = kind
    a.rope_base = float(rope_base)
    if workspace is not None:
        a.workspace, a.workspace_bytes = _ptr(workspace), workspace.numel() * workspace.element_size()
    return a


def mla_write_kv_workspace_size(args: WriteKvArgs) -> int:
    n = ctypes.c_size_t(0)
    _check("mla_write_kv_workspace_size", load().mla_write_kv_workspace_size(ctypes.byref(args), ctypes.byref(n)))
    return int(n.value)


def mla_write_kv(args: WriteKvArgs, stream=None):
    """Appends the new tokens' latent and RoPE key rows to the paged cache."""
    _check("mla_write_kv", load().mla_write_kv(ctypes.byref(args), _stream(stream)))


def make_step_args(*, q_nope, q_pe, w_uk, w_uv, kv_cache, kv_scale, block_table, seq_lens, out, lse,
                   workspace=None, causal=False, softmax_scale, num_splits=0, max_seq_len=0,
                   fuse=0) -> StepArgs:
    """Fill a ``StepArgs`` (the whole decode step, ``mla_decode_step``) from device
    tensors.  Shapes: q_nope [B][s_q][H][128], q_pe [B][s_q][H][64], w_uk and w_uv
    [H][128][512] bf16; the cache, scales, block table and lengths as for
    ``make_decode_args``; out [B][s_q][H][128] bf16, lse [B][s_q][H] fp32 or None;
    fuse: 0 automatic, 1 one launch wherever possible, -1 never."""
    import torch
    bf16, f32, i32 = torch.bfloat16, torch.float32, torch.int32
    if q_nope.dim() != 4 or kv_cache.dim() != 3 or block_table.dim() != 2:
        raise ValueError("q_nope must be [B][s_q][H][128], kv_cache [pages][64][row], block_table [B][pages]")
    B, s_q, H, _ = q_nope.shape
    P = kv_cache.shape[0]
    kind, sc_dtype, sc_tail, width = _cache_kind(kv_cache)
    _want([(q_nope, "q_nope", bf16, (B, s_q, H, D_N), False),
           (q_pe, "q_pe", bf16, (B, s_q, H, D_R), False),
           (w_uk, "w_uk", bf16, (H, D_N, D_C), False),
           (w_uv, "w_uv", bf16, (H, D_V, D_C), False),
           (kv_cache, "kv_cache", (bf16, torch.float8_e4m3fn, torch.int8, torch.uint8), (P, PAGE, width), False),
           (kv_scale, "kv_scale", sc_dtype or f32, (P, PAGE) + sc_tail, kind == KV_BF16),
           (block_table, "block_table", i32, (B, block_table.shape[1]), False),
           (seq_lens, "seq_lens", i32, (B,), False),
           (out, "out", bf16, (B, s_q, H, D_V), False),
           (lse, "lse", f32, (B, s_q, H), True),
           (workspace, "workspace", torch.uint8, None, True)])
    a = StepArgs()
    a.q_nope, a.q_pe, a.w_uk, a.w_uv = _ptr(q_nope), _ptr(q_pe), _ptr(w_uk), _ptr(w_uv)
    a.kv_cache, a.kv_scale = _ptr(kv_cache), _ptr(kv_scale)
    a.block_table, a.seq_lens = _ptr(block_table), _ptr(seq_lens)
    a.out, a.lse = _ptr(out), _ptr(lse)
    a.B, a.s_q, a.H = B, s_q, H
    a.d_c, a.d_r, a.page_size = D_C, D_R, PAGE
    a.num_pages = P
    a.max_pages_per_seq = block_table.shape[1]
    a.kv_dtype = kind
    a.causal = int(bool(causal))
    a.num_splits = int(num_splits)
    a.max_seq_len = int(max_seq_len)
    a.softmax_scale = float(softmax_scale)
    a.fuse = int(fuse)
    if workspace is not None:
        a.workspace, a.workspace_bytes = _ptr(workspace), workspace.numel() * workspace.element_size()
    return a


def mla_decode_step_workspace_size(args: StepArgs) -> int:
    n = ctypes.c_size_t(0)
    _check("mla_decode_step_workspace_size",
           load().mla_decode_step_workspace_size(ctypes.byref(args), ctypes.byref(n)))
    return int(n.value)


def mla_decode_step_launches(args: StepArgs) -> int:
    """Kernel launches one mla_decode_step call makes (1: fused)."""
    n = ctypes.c_int32(0)
    _check("mla_decode_step_launches", load().mla_decode_step_launches(ctypes.byref(args), ctypes.byref(n)))
    return int(n.value)


def mla_decode_step(args: StepArgs, stream=None):
    """The whole decode step (absorption, decode, split merge, up-projection)."""
    _check("mla_decode_step", load().mla_decode_step(ctypes.byref(args), _stream(stream)))


def make_prefill_args(*, q_nope, q_pe, w_uk, w_uv, kv_cache, block_table, seq_lens, out, lse,
                      max_seq_len, workspace=None, causal=True, softmax_scale) -> PrefillArgs:
    """Fill a ``PrefillArgs`` from device tensors.  Shapes: q_nope [B][s_q][H][128],
    q_pe [B][s_q][H][64], w_uk [H][128][512], w_uv [H][128][512], kv_cache
    [num_pages][64][576] bf16, block_table [B][max_pages] int32, seq_lens [B] int32,
    out [B][s_q][H][128] bf16, lse [B][s_q][H] fp32 or None; max_seq_len bounds
    seq_lens and sizes the workspace."""
    import torch
    bf16, f32, i32 = torch.bfloat16, torch.float32, torch.int32
    if q_nope.dim() != 4 or kv_cache.dim() != 3 or block_table.dim() != 2:
        raise ValueError("q_nope must be [B][s_q][H][128], kv_cache [pages][64][576], block_table [B][pages]")
    B, s_q, H, _ = q_nope.shape
    P = kv_cache.shape[0]
    _want([(q_nope, "q_nope", bf16, (B, s_q, H, D_N), False),
           (q_pe, "q_pe", bf16, (B, s_q, H, D_R), False),
           (w_uk, "w_uk", bf16, (H, D_N, D_C), False),
           (w_uv, "w_uv", bf16, (H, D_V, D_C), False),
           (kv_cache, "kv_cache", bf16, (P, PAGE, D_C + D_R), False),
           (block_table, "block_table", i32, (B, block_table.shape[1]), False),
           (seq_lens, "seq_lens", i32, (B,), False),
           (out, "out", bf16, (B, s_q, H, D_V), False),
           (lse, "lse", f32, (B, s_q, H), True),
           (workspace, "workspace", torch.uint8, None, True)])
    a = PrefillArgs()
    a.q_nope, a.q_pe, a.w_uk, a.w_uv = _ptr(q_nope), _ptr(q_pe), _ptr(w_uk), _ptr(w_uv)
    a.kv_cache = _ptr(kv_cache)
    a.block_table, a.seq_lens = _ptr(block_table), _ptr(seq_lens)
    a.out, a.lse = _ptr(out), _ptr(lse)
    a.B, a.s_q, a.H = B, s_q, H
    a.d_c, a.d_r, a.page_size = D_C, D_R, PAGE
    a.num_pages = P
    a.max_pages_per_seq = block_table.shape[1]
    a.kv_dtype = KV_BF16
    a.causal = int(bool(causal))
    a.max_seq_len = int(max_seq_len)
    a.softmax_scale = float(softmax_scale)
    if workspace is not None:
        a.workspace, a.workspace_bytes = _ptr(workspace), workspace.numel() * workspace.element_size()
    return a


def mla_prefill_workspace_size(args: PrefillArgs) -> int:
    n = ctypes.c_size_t(0)
    _check("mla_prefill_workspace_size", load().mla_prefill_workspace_size(ctypes.byref(args), ctypes.byref(n)))
    return int(n.value)


def mla_prefill(args: PrefillArgs, stream=None):
    """Explicit-form attention of the s_q new tokens of every sequence (per-head
    keys and values formed in the workspace, then a FlashAttention forward)."""
    _check("mla_prefill", load().mla_prefill(ctypes.byref(args), _stream(stream)))


def make_append_args(*, c, k_pe, q_pe=None, k_pe_out=None, q_pe_out=None, kv_cache, kv_scale, block_table,
                     cu_seqlens, seq_lens, workspace=None, rope_base=10000.0) -> AppendArgs:
    """Fill an ``AppendArgs`` (packed tokens into the paged cache, rotation on the
    way) from device tensors.  Shapes: c [n_tok][512], k_pe and k_pe_out [n_tok][64],
    q_pe and q_pe_out [n_tok][H][64], all bf16 and strided views at will (the outputs
    may be the inputs); the cache, scales and block table as for
    ``make_write_kv_args``; cu_seqlens [B + 1] and seq_lens [B] int32."""
    import torch
    bf16, f32, i32 = torch.bfloat16, torch.float32, torch.int32
    if c.dim() != 2 or kv_cache.dim() != 3 or block_table.dim() != 2 or (q_pe is not None and q_pe.dim() != 3):
        raise ValueError("c must be [n_tok][512], q_pe [n_tok][H][64], kv_cache [pages][64][row], block_table [B][pages]")
    if q_pe is None and q_pe_out is not None:
        raise ValueError("q_pe_out without q_pe")
    n, B, P = c.shape[0], block_table.shape[0], kv_cache.shape[0]
    H = 0 if q_pe is None else q_pe.shape[1]
    kind, sc_dtype, sc_tail, width = _cache_kind(kv_cache)
    views = [(c, "c", bf16, (n, D_C), False), (k_pe, "k_pe", bf16, (n, D_R), False),
             (q_pe, "q_pe", bf16, (n, H, D_R), True), (k_pe_out, "k_pe_out", bf16, (n, D_R), True),
             (q_pe_out, "q_pe_out", bf16, (n, H, D_R), q_pe is None)]
    dense = [(kv_cache, "kv_cache", (bf16, torch.float8_e4m3fn, torch.int8, torch.uint8), (P, PAGE, width), False),
             (kv_scale, "kv_scale", sc_dtype or f32, (P, PAGE) + sc_tail, kind == KV_BF16),
             (block_table, "block_table", i32, (B, block_table.shape[1]), False),
             (cu_seqlens, "cu_seqlens", i32, (B + 1,), False), (seq_lens, "seq_lens", i32, (B,), False),
             (workspace, "workspace", torch.uint8, None, True)]
    _want_views(views)
    _want_dense(dense)
    a = AppendArgs()
    a.device = _want_one_device(views + dense)
    a.c, a.k_pe, a.q_pe, a.k_pe_out, a.q_pe_out = (_ptr(t) for t in (c, k_pe, q_pe, k_pe_out, q_pe_out))
    a.c_tok, a.k_pe_tok = c.stride(0), k_pe.stride(0)
    if k_pe_out is not None:
        a.k_pe_out_tok = k_pe_out.stride(0)
    if q_pe is not None:
        a.q_pe_tok, a.q_pe_head = q_pe.stride(0), q_pe.stride(1)
        a.q_pe_out_tok, a.q_pe_out_head = q_pe_out.stride(0), q_pe_out.stride(1)
    a.kv_cache, a.kv_scale, a.block_table = _ptr(kv_cache), _ptr(kv_scale), _ptr(block_table)
    a.cu_seqlens, a.seq_lens = _ptr(cu_seqlens), _ptr(seq_lens)
    a.n_tok, a.B, a.H = n, B, H
    a.d_c, a.d_r, a.page_size = D_C, D_R, PAGE
    a.num_pages, a.max_pages_per_seq = P, block_table.shape[1]
    a.kv_dtype = kind
    a.rope_base = float(rope_base)
    if workspace is not None:
        a.workspace, a.workspace_bytes = _ptr(workspace), workspace.numel()
    return a


def mla_append_workspace_size(args: AppendArgs) -> int:
    return _workspace_size("mla_append_workspace_size", args)


def mla_append_kv(args: AppendArgs, stream=None):
    """Appends packed tokens' latents and rotated RoPE keys to the paged cache and
    rotates their queries' RoPE parts."""
    _call("mla_append_kv", args, stream)


def make_prefill_packed_args(*, q_nope, q_pe, k_nope, k_pe, v, cu_seqlens, out, lse, workspace=None,
                             causal=True, softmax_scale) -> PrefillPackedArgs:
    """Fill a ``PrefillPackedArgs`` (attention over packed prompts) from device
    tensors.  Shapes: q_nope [n_tok][H][128], q_pe [n_tok][H][64] or None, k_nope and
    v [n_tok][H_kv][128], k_pe [n_tok][64] or None with q_pe, all bf16 and strided
    views at will; cu_seqlens [B + 1] int32; out [n_tok][H][128] bf16 and lse
    [n_tok][H] fp32 or None, dense."""
    import torch
    bf16, f32, i32 = torch.bfloat16, torch.float32, torch.int32
    if q_nope.dim() != 3 or k_nope.dim() != 3 or cu_seqlens.dim() != 1 or cu_seqlens.shape[0] < 1:
        raise ValueError("q_nope must be [n_tok][H][128], k_nope [n_tok][H_kv][128], cu_seqlens [B + 1]")
    n, H, _ = q_nope.shape
    H_kv = k_nope.shape[1]
    if (q_pe is None) != (k_pe is None):
        raise ValueError("q_pe and k_pe come together")
    views = [(q_nope, "q_nope", bf16, (n, H, D_N), False), (q_pe, "q_pe", bf16, (n, H, D_R), True),
             (k_nope, "k_nope", bf16, (n, H_kv, D_N), False), (k_pe, "k_pe", bf16, (n, D_R), True),
             (v, "v", bf16, (n, H_kv, D_V), False)]
    dense = [(cu_seqlens, "cu_seqlens", i32, None, False), (out, "out", bf16, (n, H, D_V), False),
             (lse, "lse", f32, (n, H), True), (workspace, "workspace", torch.uint8, None, True)]
    _want_views(views)
    _want_dense(dense)
    a = PrefillPackedArgs()
    a.device = _want_one_device(views + dense)
    a.q_nope, a.q_pe, a.k_nope, a.k_pe, a.v = (_ptr(t) for t in (q_nope, q_pe, k_nope, k_pe, v))
    a.cu_seqlens, a.out, a.lse = _ptr(cu_seqlens), _ptr(out), _ptr(lse)
    a.q_nope_tok, a.q_nope_head = q_nope.stride(0), q_nope.stride(1)
    a.k_nope_tok, a.k_nope_head = k_nope.stride(0), k_nope.stride(1)
    a.v_tok, a.v_head = v.stride(0), v.stride(1)
    if q_pe is not None:
        a.q_pe_tok, a.q_pe_head, a.k_pe_tok = q_pe.stride(0), q_pe.stride(1), k_pe.stride(0)
    a.n_tok, a.B, a.H, a.H_kv = n, cu_seqlens.shape[0] - 1, H, H_kv
    a.d_n, a.d_r, a.d_v = D_N, 0 if q_pe is None else D_R, D_V
    a.causal = int(bool(causal))
    a.softmax_scale = float(softmax_scale)
    if workspace is not None:
        a.workspace, a.workspace_bytes = _ptr(workspace), workspace.numel()
    return a


def mla_prefill_packed_workspace_size(args: PrefillPackedArgs) -> int:
    return _workspace_size("mla_prefill_packed_workspace_size", args)


def mla_prefill_packed(args: PrefillPackedArgs, stream=None):
    """Attention over packed prompts in the explicit form."""
    _call("mla_prefill_packed", args, stream)


def make_verify_args(*, target_probs, draft_probs, draft_tokens, u_accept, u_sample, tokens, num_accepted,
                     num_draft=None, seq_lens=None, new_lens=None, workspace=None) -> VerifyArgs:
    """Fill a ``VerifyArgs`` (verification of drafted tokens) from device tensors.
    Shapes: target_probs [B][s_q][V] and draft_probs [B][s_q - 1][V] (or None: certain
    drafts), both fp32 or both bf16, strided rows at will; draft_tokens int32 and
    u_accept fp32 [B][s_q - 1]; num_draft [B] int32 or None; u_sample [B] fp32;
    tokens [B][s_q], num_accepted, seq_lens and new_lens [B] int32."""
    import torch
    f32, i32 = torch.float32, torch.int32
    if target_probs.dim() != 3:
        raise ValueError("target_probs must be [B][s_q][V]")
    B, s_q, V = target_probs.shape
    if s_q < 1:
        raise ValueError("target_probs must have at least one row per sequence")
    views = [(target_probs, "target_probs", (f32, torch.bfloat16), (B, s_q, V), False),
             (draft_probs, "draft_probs", target_probs.dtype, (B, s_q - 1, V), True)]
    dense = [(draft_tokens, "draft_tokens", i32, (B, s_q - 1), False), (num_draft, "num_draft", i32, (B,), True),
             (u_accept, "u_accept", f32, (B, s_q - 1), False), (u_sample, "u_sample", f32, (B,), False),
             (seq_lens, "seq_lens", i32, (B,), new_lens is None), (tokens, "tokens", i32, (B, s_q), False),
             (num_accepted, "num_accepted", i32, (B,), False), (new_lens, "new_lens", i32, (B,), True),
             (workspace, "workspace", torch.uint8, None, True)]
    _want_views(views)
    _want_dense(dense)
    a = VerifyArgs()
    a.device = _want_one_device(views + dense)
    a.target_probs, a.draft_probs, a.draft_tokens = _ptr(target_probs), _ptr(draft_probs), _ptr(draft_tokens)
    a.num_draft, a.u_accept, a.u_sample = _ptr(num_draft), _ptr(u_accept), _ptr(u_sample)
    a.seq_lens, a.tokens, a.num_accepted, a.new_lens = _ptr(seq_lens), _ptr(tokens), _ptr(num_accepted), _ptr(new_lens)
    a.target_seq, a.target_row = target_probs.stride(0), target_probs.stride(1)
    if draft_probs is not None:
        a.draft_seq, a.draft_row = draft_probs.stride(0), draft_probs.stride(1)
    a.B, a.s_q, a.V = B, s_q, V
    a.dtype = PROB_FP32 if target_probs.dtype == f32 else PROB_BF16
    if workspace is not None:
        a.workspace, a.workspace_bytes = _ptr(workspace), workspace.numel()
    return a


def mla_verify_workspace_size(args: VerifyArgs) -> int:
    return _workspace_size("mla_verify_workspace_size", args)


def mla_verify_draft(args: VerifyArgs, stream=None):
    """Accepts drafted tokens against the target's probabilities, draws the token
    after them and shortens the cached lengths by the rejected ones."""
    _call("mla_verify_draft", args, stream)


def mla_get_status(workspace, stream=None) -> int:
    """Waits for the stream and returns (and clears) the device status word."""
    import torch
    dev = getattr(workspace, "device", None)
    if dev is None or dev.type != "cuda" or dev.index == torch.cuda.current_device():
        return int(load().mla_get_status(_ptr(workspace), _stream(stream)))
    with torch.cuda.device(dev):
        return int(load().mla_get_status(_ptr(workspace), _stream(stream)))


def mla_status_string(code: int) -> str:
    return load().mla_status_string(int(code)).decode()


def alloc_workspace(args, device="cuda"):
    """A zeroed workspace tensor sized for ``args`` (any of the ``*Args``); also
    stored into ``args``."""
    import torch
    if isinstance(args, (AppendArgs, PrefillPackedArgs, VerifyArgs)):
        n = {AppendArgs: mla_append_workspace_size, PrefillPackedArgs: mla_prefill_packed_workspace_size,
             VerifyArgs: mla_verify_workspace_size}[type(args)](args)
        if device == "cuda" and getattr(args, "device", None) is not None:
            device = args.device
    elif isinstance(args, WriteKvArgs):
        n = mla_write_kv_workspace_size(args)
    elif isinstance(args, StepArgs):
        n = mla_decode_step_workspace_size(args)
    elif isinstance(args, PrefillArgs):
        n = mla_prefill_workspace_size(args)
    else:
        n = mla_decode_workspace_size(args)
    ws = torch.zeros(n, dtype=torch.uint8, device=device)
    args.workspace, args.workspace_bytes = _ptr(ws), n
    return ws
