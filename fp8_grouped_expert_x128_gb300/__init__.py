"""Python binding of libmoe_fp8.so, the GB300 (sm_103a) routed-expert FP8 MoE FFN.

Argument marshalling only: every step runs in the library's CUDA kernels;
PyTorch supplies device memory and the current stream.  Each function has the
name of the C entry point it calls (see include/moe_fp8.h for the definitions,
layouts and error rules).  A non-zero status raises ``MoeError``.

The library is built in-tree by ``fp8_grouped_expert_x128_gb300/_build.py``
(``__graft_entry__.build()`` does it).  Importing this package without the
built library raises ImportError: there is no fallback path.
"""
from __future__ import annotations

import ctypes
import os
import struct

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libmoe_fp8.so")

if not os.path.exists(LIB_PATH):
    raise ImportError(
        f"{LIB_PATH} is missing: build it with `python fp8_grouped_expert_x128_gb300/_build.py` "
        "(the CUDA library is the only implementation; there is no CPU fallback)")

_lib = ctypes.CDLL(LIB_PATH)

# ---------------------------------------------------------------- constants
MOE_OK = 0
MOE_ERR_INVALID_ARG = -1
MOE_ERR_UNSUPPORTED = -2
MOE_ERR_CUDA = -3
MOE_ERR_OVERFLOW = -4
MOE_ERR_TIMEOUT = -5
MOE_ERR_BAD_INDEX = -6
MOE_DEV_OVERFLOW, MOE_DEV_TIMEOUT, MOE_DEV_BAD_INDEX = 0x1, 0x2, 0x4
MOE_LAYOUT_MASKED, MOE_LAYOUT_CONTIG = 0, 1
MOE_GEMM_DEFAULT = 0
MOE_GEMM_FORCE_TOKENS_M = 0x1
MOE_GEMM_FORCE_WEIGHTS_M = 0x2
MOE_FFN_FUSE_SWIGLU = 0x4
MOE_GEMM_CTA_PAIR = 0x8
MOE_FFN_UE8M0 = 0x10
MOE_GEMM_EARLY_WEIGHTS = 0x20
MOE_GEMM_DEBUG_STALL = 0x100
MOE_QUANT_UE8M0 = 0x1
MOE_COMBINE_ACCUMULATE = 0x1
MOE_DTYPE_BF16, MOE_DTYPE_F16 = 0, 1
MOE_KV_INTERLEAVED = 0x1
MOE_KV_FULL = 0x1

EXPORTED = [
    "moe_status_string", "moe_version", "moe_read_device_status", "moe_quant_fp8",
    "moe_quant_weight_fp8", "moe_contig_rows_bound", "moe_permute", "moe_gemm_fp8_contig",
    "moe_gemm_fp8_masked", "moe_gemm_fp8_masked_variant", "moe_swiglu_quant", "moe_combine", "moe_ffn_workspace_size", "moe_ffn",
    "moe_ffn_noalloc", "moe_ffn_noalloc_capacity", "moe_ffn_kernel_count", "moe_quant_fp8_ue8m0",
    "moe_ue8m0_scale", "moe_quant_weight_fp8_ue8m0", "moe_ue8m0_act_words", "moe_ue8m0_weight_words",
    "moe_pack_ue8m0_act", "moe_pack_ue8m0_weight", "moe_gemm_fp8_contig_ue8m0", "moe_gemm_fp8_masked_ue8m0",
    "moe_kv_append", "moe_kv_attention", "moe_kv_attention_workspace_size",
]

_P = ctypes.c_void_p
_I64 = ctypes.c_int64
_I32 = ctypes.c_int32


class moe_ffn_desc(ctypes.Structure):
    _fields_ = [
        ("T", _I64), ("H", _I32), ("I", _I32), ("k", _I32), ("expert_begin", _I32), ("E", _I32),
        ("layout", _I32), ("max_m", _I32), ("expected_m", _I32), ("gemm_flags", _I32),
        ("x", _P), ("topk_ids", _P), ("topk_w", _P), ("w13", _P), ("w13_s", _P), ("w2", _P),
        ("w2_s", _P), ("out", _P), ("err", _P), ("stage_events", _P), ("w13_sf", _P), ("w2_sf", _P),
    ]


class moe_kv_cache(ctypes.Structure):
    _fields_ = [
        ("k", _P), ("v", _P), ("k_scale", _P), ("v_scale", _P), ("page_table", _P), ("cu_new", _P), ("kv_len", _P),
        ("k_page_ld", _I64), ("k_head_ld", _I64), ("k_slot_ld", _I64), ("v_page_ld", _I64), ("v_head_ld", _I64),
        ("v_slot_ld", _I64), ("table_ld", _I64), ("pages", _I64), ("batch", _I32), ("max_pages", _I32),
        ("page_size", _I32), ("kv_heads", _I32), ("dim", _I32), ("dtype", _I32),
    ]


class moe_kv_append_desc(ctypes.Structure):
    _fields_ = [
        ("cache", moe_kv_cache), ("T", _I64), ("k", _P), ("v", _P), ("q", _P), ("q_out", _P), ("cos_sin", _P), ("err", _P),
        ("k_token_ld", _I64), ("k_head_ld", _I64), ("v_token_ld", _I64), ("v_head_ld", _I64), ("q_token_ld", _I64),
        ("q_head_ld", _I64), ("qo_token_ld", _I64), ("qo_head_ld", _I64), ("q_heads", _I32), ("rot_dim", _I32),
        ("max_pos", _I32), ("flags", _I32),
    ]


class moe_kv_attention_desc(ctypes.Structure):
    _fields_ = [
        ("cache", moe_kv_cache), ("T", _I64), ("q", _P), ("out", _P), ("lse", _P), ("err", _P),
        ("q_token_ld", _I64), ("q_head_ld", _I64), ("o_token_ld", _I64), ("o_head_ld", _I64),
        ("sm_scale", ctypes.c_float), ("softcap", ctypes.c_float), ("q_heads", _I32), ("max_q", _I32), ("window", _I32),
        ("flags", _I32),
    ]


def _sig(name, res, args):
    f = getattr(_lib, name)
    f.restype = res
    f.argtypes = args
    return f


_sig("moe_status_string", ctypes.c_char_p, [ctypes.c_int])
_sig("moe_version", ctypes.c_int, [])
_sig("moe_read_device_status", ctypes.c_int,
     [_P, _P, ctypes.POINTER(ctypes.c_int), ctypes.POINTER(_I32)])
_sig("moe_quant_fp8", ctypes.c_int, [_P, _I64, _I64, _I64, _P, _I64, _P, _I64, _I32, _P, _P])
_sig("moe_quant_fp8_ue8m0", ctypes.c_int, [_P, _I64, _I64, _I64, _P, _I64, _P, _P, _I64, _P, _P])
_sig("moe_ue8m0_scale", ctypes.c_float, [ctypes.c_float, ctypes.POINTER(ctypes.c_uint8)])
_sig("moe_quant_weight_fp8", ctypes.c_int, [_P, _I64, _I64, _I64, _P, _P, _P])
_sig("moe_quant_weight_fp8_ue8m0", ctypes.c_int, [_P, _I64, _I64, _I64, _P, _P, _P, _P])
_sig("moe_contig_rows_bound", _I64, [_I64, _I32])
_sig("moe_permute", ctypes.c_int,
     [_P, _P, _I64, _P, _I64, _I32, _I32, _I32, _I32, _I32, _I32, _P, _P, _I64, _P, _P, _P, _P,
      _P, _I64, _P, _P])
_sig("moe_gemm_fp8_contig", ctypes.c_int,
     [_P, _I64, _P, _I64, _P, _P, _P, _P, _I64, _I32, _I32, _I32, _P, _I64, _I32, _P, _P])
_sig("moe_gemm_fp8_masked", ctypes.c_int,
     [_P, _P, _P, _P, _P, _I32, _I32, _I32, _I32, _I32, _P, _I32, _P, _P])
_sig("moe_gemm_fp8_masked_variant", ctypes.c_int, [_I32, _I32, _I32])
_sig("moe_swiglu_quant", ctypes.c_int, [_P, _I64, _I32, _P, _I32, _P, _P, _P, _I64, _I32, _P, _P])
_sig("moe_combine", ctypes.c_int, [_P, _I64, _I64, _P, _P, _I64, _I32, _I32, _P, _I64, _I32, _P, _I64, _P, _P])
_sig("moe_ue8m0_act_words", _I64, [_I64, _I64, _I64])
_sig("moe_ue8m0_weight_words", _I64, [_I64, _I64, _I64])
_sig("moe_pack_ue8m0_act", ctypes.c_int, [_P, _I64, _I64, _I64, _I64, _P, _P])
_sig("moe_pack_ue8m0_weight", ctypes.c_int, [_P, _I64, _I64, _I64, _P, _P])
_sig("moe_gemm_fp8_contig_ue8m0", ctypes.c_int,
     [_P, _I64, _P, _I64, _P, _P, _P, _P, _I64, _I32, _I32, _I32, _P, _I64, _I32, _P, _P])
_sig("moe_gemm_fp8_masked_ue8m0", ctypes.c_int,
     [_P, _P, _P, _P, _P, _I32, _I32, _I32, _I32, _I32, _P, _I32, _P, _P])
_sig("moe_ffn_workspace_size", ctypes.c_size_t, [ctypes.POINTER(moe_ffn_desc)])
_sig("moe_ffn_kernel_count", ctypes.c_int, [ctypes.POINTER(moe_ffn_desc)])
_sig("moe_ffn", ctypes.c_int, [ctypes.POINTER(moe_ffn_desc), _P, ctypes.c_size_t, _P])
_sig("moe_ffn_noalloc", ctypes.c_int, [ctypes.POINTER(moe_ffn_desc), _P])
_sig("moe_ffn_noalloc_capacity", ctypes.c_size_t, [])
_sig("moe_kv_append", ctypes.c_int, [_P, _P])
_sig("moe_kv_attention_workspace_size", ctypes.c_size_t, [ctypes.POINTER(moe_kv_attention_desc)])
_sig("moe_kv_attention", ctypes.c_int, [_P, _P, ctypes.c_size_t, _P])


class MoeError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {moe_status_string(status)} ({status})")


def moe_status_string(status: int) -> str:
    return _lib.moe_status_string(status).decode()


def moe_version() -> int:
    return _lib.moe_version()


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream=None):
    s = torch.cuda.current_stream() if stream is None else stream
    return ctypes.c_void_p(s.cuda_stream)


def _stream_of(device: int, stream=None) -> int:
    """The handle of `stream`, or of the current stream of GPU `device`."""
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(device)
    if stream.device_index != device:
        raise ValueError(f"stream: on GPU {stream.device_index}, the cache on GPU {device}")
    return stream.cuda_stream


def _check(rc: int, where: str):
    if rc != MOE_OK:
        raise MoeError(rc, where)


def _dev(t, dtype=None, name="tensor"):
    if t is None:
        return
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if dtype is not None and t.dtype not in (dtype if isinstance(dtype, tuple) else (dtype,)):
        raise ValueError(f"{name}: expected {dtype}, got {t.dtype}")


_U8 = (torch.uint8, torch.float8_e4m3fn)


def _u8(t):
    return t.view(torch.uint8) if t is not None and t.dtype == torch.float8_e4m3fn else t


def new_error_word(device=None) -> torch.Tensor:
    """A zeroed device int32 word for the library's device-side error bits."""
    return torch.zeros(1, dtype=torch.int32, device=device or "cuda")


def moe_read_device_status(err: torch.Tensor, stream=None) -> tuple[int, int]:
    """Synchronise, read and clear the device error word -> (status, raw bits)."""
    st = ctypes.c_int(0)
    bits = _I32(0)
    _check(_lib.moe_read_device_status(_ptr(err), _stream(stream), ctypes.byref(st),
                                       ctypes.byref(bits)), "moe_read_device_status")
    return st.value, bits.value


def moe_contig_rows_bound(assignments: int, E: int) -> int:
    return int(_lib.moe_contig_rows_bound(assignments, E))


def moe_quant_fp8(x, q, s, s_ld=None, flags=0, err=None, stream=None):
    """a1: x bf16 [M, K] -> q uint8 [M, K], s fp32 [K/128, s_ld] (s[kb, m]);
    flags = MOE_QUANT_UE8M0 for power-of-two scales."""
    _dev(x, torch.bfloat16, "x"); _dev(q, _U8, "q"); _dev(s, torch.float32, "s")
    M, K = x.shape
    s_ld = s.shape[-1] if s_ld is None else s_ld
    _check(_lib.moe_quant_fp8(_ptr(x), M, K, x.stride(0), _ptr(_u8(q)), q.stride(0), _ptr(s), s_ld,
                              flags, _ptr(err), _stream(stream)), "moe_quant_fp8")
    return q, s


def moe_quant_fp8_ue8m0(x, q, s, e8=None, s_ld=None, err=None, stream=None):
    """a1 with power-of-two block scales: s fp32 [K/128, s_ld] holds 2^e, e8 uint8
    (optional, same shape) holds e + 127."""
    _dev(x, torch.bfloat16, "x"); _dev(q, _U8, "q"); _dev(s, torch.float32, "s"); _dev(e8, _U8, "e8")
    M, K = x.shape
    s_ld = s.shape[-1] if s_ld is None else s_ld
    _check(_lib.moe_quant_fp8_ue8m0(_ptr(x), M, K, x.stride(0), _ptr(_u8(q)), q.stride(0), _ptr(s),
                                    _ptr(e8), s_ld, _ptr(err), _stream(stream)), "moe_quant_fp8_ue8m0")
    return q, s


def moe_ue8m0_scale(amax: float) -> tuple[float, int]:
    """The UE8M0 block-scale rule for one block maximum (host): (2^e, e + 127)."""
    b = ctypes.c_uint8(0)
    s = float(_lib.moe_ue8m0_scale(ctypes.c_float(amax), ctypes.byref(b)))
    return s, int(b.value)


def moe_quant_weight_fp8(w, q, s, stream=None):
    """a3: w bf16 [E, N, K] -> q uint8 [E, N, K], s fp32 [E, N/128, K/128]."""
    _dev(w, torch.bfloat16, "w"); _dev(q, _U8, "q"); _dev(s, torch.float32, "s")
    E, N, K = w.shape
    assert w.is_contiguous() and q.is_contiguous() and s.is_contiguous()
    _check(_lib.moe_quant_weight_fp8(_ptr(w), E, N, K, _ptr(_u8(q)), _ptr(s), _stream(stream)),
           "moe_quant_weight_fp8")
    return q, s


def moe_quant_weight_fp8_ue8m0(w, q, s, e8=None, stream=None):
    """a3 with power-of-two tile scales: s fp32 [E, N/128, K/128] holds 2^e, e8
    uint8 (optional, same shape) holds e + 127."""
    _dev(w, torch.bfloat16, "w"); _dev(q, _U8, "q"); _dev(s, torch.float32, "s"); _dev(e8, _U8, "e8")
    E, N, K = w.shape
    assert w.is_contiguous() and q.is_contiguous() and s.is_contiguous()
    _check(_lib.moe_quant_weight_fp8_ue8m0(_ptr(w), E, N, K, _ptr(_u8(q)), _ptr(s), _ptr(e8), _stream(stream)),
           "moe_quant_weight_fp8_ue8m0")
    return q, s


def moe_permute(q, s, topk_ids, expert_begin, E, layout, max_m, q_out, s_out, counts, offsets,
                m_indices, row_src, dst_row, rows_capacity=0, s_ld=None, s_out_ld=None, err=None,
                stream=None):
    """a2: token-order q/s -> grouped layout.  See moe_fp8.h for the layouts."""
    T, H = q.shape
    k = topk_ids.shape[1]
    s_ld = s.shape[-1] if s_ld is None else s_ld
    if s_out_ld is None:
        s_out_ld = s_out.shape[-1] if layout == MOE_LAYOUT_CONTIG else max_m
    _check(_lib.moe_permute(_ptr(_u8(q)), _ptr(s), s_ld, _ptr(topk_ids), T, H, k, expert_begin, E,
                            layout, max_m, _ptr(_u8(q_out)), _ptr(s_out), s_out_ld, _ptr(counts),
                            _ptr(offsets), _ptr(m_indices), _ptr(row_src), _ptr(dst_row),
                            rows_capacity, _ptr(err), _stream(stream)), "moe_permute")


def moe_gemm_fp8_contig(A, sA, B, sB, offsets, m_indices, D, sA_ld=None, flags=0, err=None,
                        stream=None):
    """a4/a6, contiguous layout: A [M_cap, K], sA [K/128, sA_ld], B [E, N, K], D [M_cap, N]."""
    E, N, K = B.shape
    M_cap = A.shape[0]
    sA_ld = sA.shape[-1] if sA_ld is None else sA_ld
    _check(_lib.moe_gemm_fp8_contig(_ptr(_u8(A)), A.stride(0), _ptr(sA), sA_ld, _ptr(_u8(B)),
                                    _ptr(sB), _ptr(offsets), _ptr(m_indices), M_cap, E, N, K,
                                    _ptr(D), D.stride(0), flags, _ptr(err), _stream(stream)),
           "moe_gemm_fp8_contig")
    return D


def moe_gemm_fp8_masked(A, sA, B, sB, counts, D, expected_m=0, flags=0, err=None, stream=None):
    """a4/a6, masked layout: A [E, max_m, K], sA [E, K/128, max_m], D [E, max_m, N]."""
    E, max_m, K = A.shape
    N = B.shape[1]
    _check(_lib.moe_gemm_fp8_masked(_ptr(_u8(A)), _ptr(sA), _ptr(_u8(B)), _ptr(sB), _ptr(counts),
                                    E, max_m, N, K, expected_m, _ptr(D), flags, _ptr(err),
                                    _stream(stream)), "moe_gemm_fp8_masked")
    return D


def moe_gemm_fp8_masked_variant(max_m: int, expected_m: int = 0, flags: int = 0) -> int:
    """0 = tokens-as-M kernel; 64/128/256 = weights-as-M token-tile width."""
    return int(_lib.moe_gemm_fp8_masked_variant(max_m, expected_m, flags))


def moe_ue8m0_act_words(groups: int, G: int, K: int) -> int:
    return int(_lib.moe_ue8m0_act_words(groups, G, K))


def moe_ue8m0_weight_words(E: int, N: int, K: int) -> int:
    return int(_lib.moe_ue8m0_weight_words(E, N, K))


def moe_pack_ue8m0_act(s, groups, G, rows, K, sfA, stream=None):
    """Power-of-two fp32 scales in the grouped layout (groups of G rows) -> packed
    UE8M0 words sfA (int32 tensor of moe_ue8m0_act_words(groups, G, K) words)."""
    _dev(s, torch.float32, "s"); _dev(sfA, torch.int32, "sfA")
    _check(_lib.moe_pack_ue8m0_act(_ptr(s), groups, G, rows, K, _ptr(sfA), _stream(stream)), "moe_pack_ue8m0_act")
    return sfA


def moe_pack_ue8m0_weight(s, sfB, K, stream=None):
    """Power-of-two fp32 weight scales [E, N/128, K/128] -> packed records sfB."""
    _dev(s, torch.float32, "s"); _dev(sfB, torch.int32, "sfB")
    E, NB, _ = s.shape
    _check(_lib.moe_pack_ue8m0_weight(_ptr(s), E, NB * 128, K, _ptr(sfB), _stream(stream)), "moe_pack_ue8m0_weight")
    return sfB


def moe_gemm_fp8_contig_ue8m0(A, sfA, sfA_ld, B, sfB, offsets, m_indices, D, flags=0, err=None, stream=None):
    """a4/a6 with packed UE8M0 scales, contiguous layout."""
    E, N, K = B.shape
    _check(_lib.moe_gemm_fp8_contig_ue8m0(_ptr(_u8(A)), A.stride(0), _ptr(sfA), sfA_ld, _ptr(_u8(B)), _ptr(sfB),
                                          _ptr(offsets), _ptr(m_indices), A.shape[0], E, N, K, _ptr(D),
                                          D.stride(0), flags, _ptr(err), _stream(stream)), "moe_gemm_fp8_contig_ue8m0")
    return D


def moe_gemm_fp8_masked_ue8m0(A, sfA, B, sfB, counts, D, expected_m=0, flags=0, err=None, stream=None):
    """a4/a6 with packed UE8M0 scales, masked layout: A [E, max_m, K], D [E, max_m, N]."""
    E, max_m, K = A.shape
    N = B.shape[1]
    _check(_lib.moe_gemm_fp8_masked_ue8m0(_ptr(_u8(A)), _ptr(sfA), _ptr(_u8(B)), _ptr(sfB), _ptr(counts), E, max_m,
                                          N, K, expected_m, _ptr(D), flags, _ptr(err), _stream(stream)),
           "moe_gemm_fp8_masked_ue8m0")
    return D


def moe_swiglu_quant(Y1, q, s, counts=None, max_m=0, m_indices=None, s_ld=0, flags=0, err=None,
                     stream=None):
    """a5: Y1 bf16 [rows, 2I] -> q uint8 [rows, I] + scales (groups of max_m rows when
    ``counts`` is given, else one group of ``s_ld`` rows selected by ``m_indices``);
    flags = MOE_QUANT_UE8M0 for power-of-two scales."""
    two_i = Y1.shape[-1]
    rows = Y1.numel() // two_i
    _check(_lib.moe_swiglu_quant(_ptr(Y1), rows, two_i // 2, _ptr(counts), max_m, _ptr(m_indices),
                                 _ptr(_u8(q)), _ptr(s), s_ld, flags, _ptr(err), _stream(stream)),
           "moe_swiglu_quant")


def moe_combine(Y2, dst_row, topk_w, out, shared=None, flags=0, err=None, stream=None):
    """a7: out[t] = bf16((out[t] if ACCUMULATE) + sum_j w[t,j] * Y2[dst_row[t*k+j]] + shared[t]);
    Y2 viewed as [rows, H]; shared (optional) bf16 [T, H]."""
    H = Y2.shape[-1]
    rows = Y2.numel() // H
    T, k = topk_w.shape
    _dev(shared, torch.bfloat16, "shared")
    _check(_lib.moe_combine(_ptr(Y2), H, rows, _ptr(dst_row), _ptr(topk_w), T, k, H, _ptr(shared),
                            shared.stride(0) if shared is not None else 0, flags, _ptr(out),
                            out.stride(0), _ptr(err), _stream(stream)), "moe_combine")
    return out


def make_ffn_desc(x, topk_ids, topk_w, w13, w13_s, w2, w2_s, out, expert_begin, E, layout,
                  max_m=0, expected_m=0, gemm_flags=0, err=None, stage_events=None, w13_sf=None, w2_sf=None):
    T, H = x.shape
    I = w2.shape[2]
    d = moe_ffn_desc(T=T, H=H, I=I, k=topk_ids.shape[1], expert_begin=expert_begin, E=E,
                     layout=layout, max_m=max_m, expected_m=expected_m, gemm_flags=gemm_flags,
                     x=x.data_ptr(), topk_ids=topk_ids.data_ptr(), topk_w=topk_w.data_ptr(),
                     w13=_u8(w13).data_ptr(), w13_s=w13_s.data_ptr() if w13_s is not None else None,
                     w2=_u8(w2).data_ptr(),
                     w2_s=w2_s.data_ptr() if w2_s is not None else None, out=out.data_ptr(),
                     err=err.data_ptr() if err is not None else None, stage_events=None,
                     w13_sf=w13_sf.data_ptr() if w13_sf is not None else None,
                     w2_sf=w2_sf.data_ptr() if w2_sf is not None else None)
    if stage_events is not None:
        if len(stage_events) != 7:
            raise ValueError("stage_events needs 7 events")
        for ev in stage_events:
            if not ev.cuda_event:          # torch creates the CUDA event on first record
                ev.record()
        arr = (ctypes.c_void_p * len(stage_events))(*[ev.cuda_event for ev in stage_events])
        d._events_keepalive = arr
        d.stage_events = ctypes.cast(arr, ctypes.c_void_p)
    return d


def moe_ffn_kernel_count(desc: moe_ffn_desc) -> int:
    """Kernels one moe_ffn call with `desc` launches (host-only)."""
    n = int(_lib.moe_ffn_kernel_count(ctypes.byref(desc)))
    _check(n if n < 0 else MOE_OK, "moe_ffn_kernel_count")
    return n


def moe_ffn_workspace_size(desc: moe_ffn_desc) -> int:
    return int(_lib.moe_ffn_workspace_size(ctypes.byref(desc)))


def moe_ffn(desc: moe_ffn_desc, workspace: torch.Tensor, stream=None):
    """a8: the whole FFN on one stream; ``workspace`` is a uint8 device tensor of at
    least moe_ffn_workspace_size(desc) bytes, 256-byte aligned."""
    _check(_lib.moe_ffn(ctypes.byref(desc), _ptr(workspace), workspace.numel(), _stream(stream)),
           "moe_ffn")


def moe_ffn_noalloc(desc: moe_ffn_desc, stream=None):
    """a8 without a workspace argument: the intermediates live in the library's
    fixed device scratch (moe_ffn_noalloc_capacity() bytes, shared by all calls;
    calls that overlap on the GPU race).  For callers that cannot allocate."""
    _check(_lib.moe_ffn_noalloc(ctypes.byref(desc), _stream(stream)), "moe_ffn_noalloc")


def moe_ffn_noalloc_capacity() -> int:
    return int(_lib.moe_ffn_noalloc_capacity())


def alloc_workspace(desc: moe_ffn_desc, device=None) -> torch.Tensor:
    n = moe_ffn_workspace_size(desc)
    if n == 0:
        raise MoeError(MOE_ERR_INVALID_ARG, "moe_ffn_workspace_size")
    return torch.empty(n, dtype=torch.uint8, device=device or "cuda")


# ---------------------------------------------------------------- paged 8-bit key/value cache
_KV_TYPES = {torch.bfloat16: MOE_DTYPE_BF16, torch.float16: MOE_DTYPE_F16}


# Descriptors as the C structures lay them out; packing one is what a call costs on
# the host beside the launch, so the checks below are written to pass quickly and
# leave the telling of what is wrong to functions that run only then.
_KV_CACHE_FIELDS = "7Q8q6i"
_kv_append_pack = struct.Struct("@" + _KV_CACHE_FIELDS + "q6Q8q4i").pack
_kv_attention_pack = struct.Struct("@" + _KV_CACHE_FIELDS + "q4Q4q2f4i").pack


def _kv_rows(t, name, T, heads, dim, dtype, device):
    """Strides (token, head) of a [T, heads, dim] tensor of the step's rows."""
    st, sh, sd = t.stride()
    if t.shape != (T, heads, dim) or t.dtype is not dtype or t.get_device() != device or (sd != 1 and t.numel()):
        raise ValueError(f"{name}: expected {dtype} [{T}, {heads}, {dim}] on the cache's GPU with the elements of a row next to "
                         f"each other, got {t.dtype} {list(t.shape)}, strides {list(t.stride())}")
    return st, sh


def _kv_rows2(a, a_name, b, b_name, T, heads, dim, dtype, device):
    """_kv_rows of two tensors of one shape: (token, head) strides of each."""
    shape = (T, heads, dim)
    at, ah, ad = a.stride()
    bt, bh, bd = b.stride()
    if not (a.shape == shape == b.shape and a.dtype is dtype is b.dtype and ad == 1 == bd
            and a.get_device() == device == b.get_device()):
        return (*_kv_rows(a, a_name, T, heads, dim, dtype, device), *_kv_rows(b, b_name, T, heads, dim, dtype, device))
    return at, ah, bt, bh


def _kv_cache_refused(k_cache, v_cache, k_scale, v_scale, page_table, cu_new, kv_len, dtype):
    pages, heads, page, dim = k_cache.shape
    device = k_cache.get_device()
    if device < 0:
        return ValueError("k_cache must be a CUDA tensor")
    if v_cache.shape != k_cache.shape or k_cache.dtype not in _U8 or v_cache.dtype not in _U8:
        return ValueError("k_cache and v_cache: expected uint8 or float8_e4m3fn [pages, kv_heads, page_size, dim]")
    if k_cache.stride(3) != 1 or v_cache.stride(3) != 1:
        return ValueError("k_cache, v_cache: the elements of a row must be next to each other")
    for t, name in ((k_scale, "k_scale"), (v_scale, "v_scale")):
        if t.shape != (pages, heads) or t.dtype != torch.float32 or not t.is_contiguous():
            return ValueError(f"{name}: expected contiguous float32 [{pages}, {heads}]")
    batch = page_table.shape[0]
    if page_table.dim() != 2 or page_table.dtype != torch.int32 or page_table.stride(1) != 1:
        return ValueError("page_table: expected int32 [batch, max_pages], rows contiguous")
    if (cu_new.shape != (batch + 1,) or kv_len.shape != (batch,) or cu_new.dtype != torch.int32
            or kv_len.dtype != torch.int32 or not cu_new.is_contiguous() or not kv_len.is_contiguous()):
        return ValueError(f"cu_new, kv_len: expected contiguous int32 [{batch + 1}] and [{batch}]")
    if dtype not in _KV_TYPES:
        return ValueError(f"token tensors: expected bfloat16 or float16, got {dtype}")
    for t, name in ((v_cache, "v_cache"), (k_scale, "k_scale"), (v_scale, "v_scale"), (page_table, "page_table"),
                    (cu_new, "cu_new"), (kv_len, "kv_len")):
        if t.get_device() != device:
            return ValueError(f"{name}: not on the GPU that holds k_cache")
    if torch.cuda.current_device() != device:        # the library launches on the current one
        return ValueError(f"k_cache: on GPU {device}, but GPU {torch.cuda.current_device()} is current (torch.cuda.set_device)")
    return ValueError("paged cache: tensors not as moe_fp8.h has them")


def _kv_cache(k_cache, v_cache, k_scale, v_scale, page_table, cu_new, kv_len, dtype):
    """The cache part of a descriptor, as a tuple in the order of its fields."""
    shape = k_cache.shape
    pages, heads, page, dim = shape
    kp, kh, ks, kd = k_cache.stride()
    vp, vh, vs, vd = v_cache.stride()
    batch, max_pages = page_table.shape
    table_ld, table_one = page_table.stride()
    device = k_cache.get_device()
    i32, f32 = torch.int32, torch.float32
    if not (v_cache.shape == shape and kd == 1 == vd and table_one == 1 and device >= 0
            and k_cache.dtype in _U8 and v_cache.dtype in _U8 and dtype in _KV_TYPES
            and k_scale.shape == (pages, heads) == v_scale.shape and k_scale.is_contiguous() and v_scale.is_contiguous()
            and cu_new.shape == (batch + 1,) and kv_len.shape == (batch,) and cu_new.is_contiguous() and kv_len.is_contiguous()
            and k_scale.dtype is f32 and v_scale.dtype is f32
            and page_table.dtype is i32 and cu_new.dtype is i32 and kv_len.dtype is i32
            and v_cache.get_device() == device and k_scale.get_device() == device and v_scale.get_device() == device
            and page_table.get_device() == device and cu_new.get_device() == device and kv_len.get_device() == device
            and torch.cuda.current_device() == device):
        raise _kv_cache_refused(k_cache, v_cache, k_scale, v_scale, page_table, cu_new, kv_len, dtype)
    return (k_cache.data_ptr(), v_cache.data_ptr(), k_scale.data_ptr(), v_scale.data_ptr(), page_table.data_ptr(),
            cu_new.data_ptr(), kv_len.data_ptr(), kp, kh, ks, vp, vh, vs, table_ld, pages, batch, max_pages,
            page, heads, dim, _KV_TYPES[dtype])


def _kv_err(err, device):
    if err is None:
        return 0
    if err.dtype != torch.int32 or err.get_device() != device:
        raise ValueError("err: expected an int32 word on the cache's GPU (new_error_word)")
    return err.data_ptr()


def moe_kv_append(k, v, k_cache, v_cache, k_scale, v_scale, page_table, cu_new, kv_len, cos_sin=None, flags=0, q=None,
                  q_out=None, err=None, stream=None):
    """Append the step's keys and values k, v [T, kv_heads, dim] (bf16 or f16, any
    token and head strides) to the paged E4M3 cache k_cache, v_cache [pages,
    kv_heads, page_size, dim] (any strides but the last) with scales k_scale,
    v_scale fp32 [pages, kv_heads]; see moe_fp8.h for the rule.  Sequence b's new
    tokens are rows cu_new[b] .. cu_new[b + 1] - 1, the last of its kv_len[b].
    cos_sin fp32 [max_pos, rot_dim] rotates the keys, and q [T, q_heads, dim] into
    q_out (which may be q); flags = MOE_KV_INTERLEAVED for adjacent pairs."""
    dtype = k.dtype
    c = _kv_cache(k_cache, v_cache, k_scale, v_scale, page_table, cu_new, kv_len, dtype)
    device, heads, dim, T = k_cache.get_device(), c[18], c[19], k.shape[0]
    kt, kh, vt, vh = _kv_rows2(k, "k", v, "v", T, heads, dim, dtype, device)
    qt = qh = ot = oh = q_heads = max_pos = rot = q_ptr = o_ptr = cs_ptr = 0
    if q is not None:
        if q_out is None:
            raise ValueError("q_out: queries need a tensor to be written to")
        q_heads = q.shape[1]
        qt, qh, ot, oh = _kv_rows2(q, "q", q_out, "q_out", T, q_heads, dim, dtype, device)
        q_ptr, o_ptr = q.data_ptr(), q_out.data_ptr()
    elif q_out is not None:
        raise ValueError("q_out without q")
    if cos_sin is not None:
        if (cos_sin.dtype is not torch.float32 or cos_sin.dim() != 2 or not cos_sin.is_contiguous()
                or cos_sin.get_device() != device):
            raise ValueError("cos_sin: expected contiguous float32 [max_pos, rot_dim] on the cache's GPU")
        max_pos, rot = cos_sin.shape
        cs_ptr = cos_sin.data_ptr()
    d = _kv_append_pack(*c, T, k.data_ptr(), v.data_ptr(), q_ptr, o_ptr, cs_ptr, _kv_err(err, device), kt, kh, vt, vh, qt, qh,
                        ot, oh, q_heads, rot, max_pos, flags)
    rc = _lib.moe_kv_append(d, _stream_of(device, stream))
    if rc != MOE_OK:
        raise MoeError(rc, "moe_kv_append")


def _kv_attention_fields(q, k_cache, v_cache, k_scale, v_scale, page_table, cu_new, kv_len, out, sm_scale, max_q, window, softcap,
                         flags, lse, err):
    dtype = q.dtype
    c = _kv_cache(k_cache, v_cache, k_scale, v_scale, page_table, cu_new, kv_len, dtype)
    device, dim = k_cache.get_device(), c[19]
    T, heads, _ = q.shape
    qt, qh, ot, oh = _kv_rows2(q, "q", out, "out", T, heads, dim, dtype, device)
    lse_ptr = 0
    if lse is not None:
        if lse.shape != (T, heads) or lse.dtype != torch.float32 or not lse.is_contiguous() or lse.get_device() != device:
            raise ValueError(f"lse: expected contiguous float32 [{T}, {heads}] on the cache's GPU")
        lse_ptr = lse.data_ptr()
    return c, (T, q.data_ptr(), out.data_ptr(), lse_ptr, _kv_err(err, device), qt, qh, ot, oh, sm_scale, softcap, heads, max_q,
               window, flags)


def make_kv_attention_desc(q, k_cache, v_cache, k_scale, v_scale, page_table, cu_new, kv_len, out, sm_scale, max_q=0, window=0,
                           softcap=0.0, flags=0, lse=None, err=None):
    """Descriptor of a moe_kv_attention call, for moe_kv_attention_workspace_size and alloc_kv_workspace."""
    c, rest = _kv_attention_fields(q, k_cache, v_cache, k_scale, v_scale, page_table, cu_new, kv_len, out, sm_scale, max_q, window,
                                   softcap, flags, lse, err)
    return moe_kv_attention_desc(c, *rest)


def moe_kv_attention_workspace_size(desc: moe_kv_attention_desc) -> int:
    return int(_lib.moe_kv_attention_workspace_size(ctypes.byref(desc)))


def moe_kv_attention(q, k_cache, v_cache, k_scale, v_scale, page_table, cu_new, kv_len, out, workspace, sm_scale, max_q=0,
                     window=0, softcap=0.0, flags=0, lse=None, err=None, stream=None):
    """Attention of the step's queries q [T, q_heads, dim] over the paged cache
    (arguments as in moe_kv_append) into out; see moe_fp8.h for the definition.
    max_q: the largest number of new tokens of a sequence (0 = not known).
    workspace: a uint8 device tensor of at least moe_kv_attention_workspace_size
    bytes, zeroed once before its first use.  lse: optional fp32 [T, q_heads]."""
    c, rest = _kv_attention_fields(q, k_cache, v_cache, k_scale, v_scale, page_table, cu_new, kv_len, out, sm_scale, max_q, window,
                                   softcap, flags, lse, err)
    device = q.get_device()
    if workspace.get_device() != device or not workspace.is_contiguous():
        raise ValueError("workspace: expected a contiguous tensor on the cache's GPU")
    rc = _lib.moe_kv_attention(_kv_attention_pack(*c, *rest), workspace.data_ptr(), workspace.nbytes, _stream_of(device, stream))
    if rc != MOE_OK:
        raise MoeError(rc, "moe_kv_attention")
    return out


def alloc_kv_workspace(desc: moe_kv_attention_desc, device=None) -> torch.Tensor:
    n = moe_kv_attention_workspace_size(desc)
    if n == 0:
        raise MoeError(MOE_ERR_INVALID_ARG, "moe_kv_attention_workspace_size")
    return torch.zeros(n, dtype=torch.uint8, device=device or "cuda")
