"""Batch-invariant verify pass for GB300 (sm_103a): Python binding of the W8A8
linear and LM head, the verify-pass executor, the block-scaled variant, the
split-KV verify attention, the decoder-step operators (norm, rotation with the
4-bit paged cache, attention over it, logit rules), and the e4m3 linears with the
mixture of experts made of them.

A thin ctypes layer over ``libbi.so`` (C ABI declared in ``include/bi.h``).
Each function has the name of the C entry point it calls and only marshals
arguments: tensor pointers, shapes and the current CUDA stream.  All
arithmetic runs in the library's CUDA kernels; there is no other code path.
If ``libbi.so`` is missing or fails to load, importing this package raises.

PyTorch supplies device memory and streams.  bf16 tensors may be passed as
``torch.bfloat16`` or as their ``int16``/``uint16`` bit patterns.
"""
from __future__ import annotations

import ctypes
import os

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libbi.so")

if not os.path.exists(LIB_PATH):
    raise ImportError("libbi.so is not built: run invariant_quantized_linear_gb300/build.py "
                      "(or __graft_entry__.build()) first")

lib = ctypes.CDLL(LIB_PATH)

_vp, _i64, _ci, _cu, _sz = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_uint, ctypes.c_size_t
lib.bi_status_string.argtypes = [_ci]
lib.bi_status_string.restype = ctypes.c_char_p
lib.bi_quantize_act.argtypes = [_vp, _i64, _ci, _ci, _vp, _vp, _cu, _vp]
lib.bi_quantize_act.restype = _ci
lib.bi_residual_quantize.argtypes = [_vp, _vp, _i64, _ci, _ci, _vp, _vp, _cu, _vp]
lib.bi_residual_quantize.restype = _ci
lib.bi_relu_mul_quantize.argtypes = [_vp, _i64, _ci, _ci, _vp, _vp, _vp, _cu, _vp]
lib.bi_relu_mul_quantize.restype = _ci
lib.bi_quantize_weight.argtypes = [_vp, _i64, _ci, _ci, _vp, _vp, _vp]
lib.bi_quantize_weight.restype = _ci
lib.bi_requant_pow2.argtypes = [_vp, _vp, _ci, _ci, _vp, _vp, _vp]
lib.bi_requant_pow2.restype = _ci
lib.bi_linear_workspace_size.argtypes = [_ci, _ci, _ci]
lib.bi_linear_workspace_size.restype = _sz
lib.bi_lmhead_workspace_size.argtypes = [_ci, _ci, _ci]
lib.bi_lmhead_workspace_size.restype = _sz
lib.bi_linear_w8a8.argtypes = [_vp, _vp, _ci, _ci, _vp, _vp, _ci, _vp, _vp, _sz, _cu, _vp]
lib.bi_linear_w8a8.restype = _ci
lib.bi_lmhead_argmax.argtypes = [_vp, _vp, _ci, _ci, _vp, _vp, _ci, _vp, _vp, _vp, _sz, _cu, _vp]
lib.bi_lmhead_argmax.restype = _ci
lib.bi_greedy_verify.argtypes = [_vp, _vp, _ci, _vp, _vp]
lib.bi_greedy_verify.restype = _ci
lib.bi_selftest_wait_timeout.argtypes = [_vp, _sz, _vp]
lib.bi_selftest_wait_timeout.restype = _ci
lib.bi_selftest_quotient.argtypes = [_vp, _vp]
lib.bi_selftest_quotient.restype = _ci
lib.bi_workspace_status.argtypes = [_vp, _sz, _vp]
lib.bi_workspace_status.restype = _ci
lib.bi_linear_w8a8_noalloc.argtypes = [_vp, _vp, _ci, _ci, _vp, _vp, _ci, _vp, _cu, _vp]
lib.bi_linear_w8a8_noalloc.restype = _ci
lib.bi_linear_w8a8_noalloc_status.argtypes = [_vp]
lib.bi_linear_w8a8_noalloc_status.restype = _ci
lib.bi_quantize_weight_q6.argtypes = [_vp, _i64, _ci, _ci, _vp, _vp, _vp, _vp, _vp]
lib.bi_quantize_weight_q6.restype = _ci
lib.bi_quantize_act_blocks.argtypes = [_vp, _i64, _ci, _ci, _vp, _vp, _vp]
lib.bi_quantize_act_blocks.restype = _ci
lib.bi_linear_q6.argtypes = [_vp, _vp, _ci, _ci, _vp, _vp, _vp, _vp, _ci, _vp, _cu, _vp]
lib.bi_linear_q6.restype = _ci
lib.bi_attention_workspace_size.argtypes = [_ci, _ci, _ci, _ci]
lib.bi_attention_workspace_size.restype = _sz
lib.bi_attention_verify.argtypes = [_vp, _vp, _vp, _ci, _ci, _ci, _ci, _ci, _ci, ctypes.c_float, _vp, _vp, _sz,
                                    _vp]
lib.bi_attention_verify.restype = _ci


class bi_kv4_cache(ctypes.Structure):
    """A paged 4-bit key/value cache (struct bi_kv4_cache of include/bi.h)."""
    _fields_ = [("pool", _vp), ("page_stride", _i64), ("num_pages", _ci), ("page_size", _ci), ("Hkv", _ci), ("D", _ci)]


class bi_kv4_batch(ctypes.Structure):
    """Sequences with new tokens (struct bi_kv4_batch of include/bi.h)."""
    _fields_ = [("cu_q", _vp), ("kv_len", _vp), ("pages", _vp), ("ld_pages", _i64), ("B", _ci), ("T", _ci),
                ("max_q", _ci), ("max_kv", _ci)]


class bi_logits_rules(ctypes.Structure):
    """Rules applied to logits (struct bi_logits_rules of include/bi.h)."""
    _fields_ = [("ids", _vp), ("begin", _vp), ("mid", _vp), ("end", _vp), ("repetition", _vp), ("presence", _vp),
                ("frequency", _vp), ("bias_ids", _vp), ("bias", _vp), ("n_bias", _ci), ("mask", _vp), ("ld_mask", _i64)]
    # rows that there are rules for, and elements of a row that the mask reaches, as far as logits_rules knows
    rows = reach = 1 << 62


def _holding(s, *tensors):
    """A structure of addresses that keeps the tensors behind them alive as long as it lives."""
    s.tensors = tensors
    return s


_cache_p, _batch_p = ctypes.POINTER(bi_kv4_cache), ctypes.POINTER(bi_kv4_batch)
lib.bi_rmsnorm_quantize.argtypes = [_vp, _i64, _vp, _i64, _vp, ctypes.c_float, _ci, _ci, _vp, _i64, _vp, _vp, _cu, _vp]
lib.bi_rmsnorm_quantize.restype = _ci
lib.bi_kv4_block_bytes.argtypes = [_ci, _ci]
lib.bi_kv4_block_bytes.restype = _sz
lib.bi_rope_table.argtypes = [_vp, _ci, ctypes.c_float, _ci, _vp, _vp]
lib.bi_rope_table.restype = _ci
lib.bi_rope_append_kv4.argtypes = [_vp, _i64, _ci, _vp, _i64, _vp, _i64, _vp, _vp, ctypes.c_float, _vp, _ci, _ci, _ci,
                                   _vp, _cache_p, _batch_p, _cu, _vp]
lib.bi_rope_append_kv4.restype = _ci
lib.bi_kv4_gather.argtypes = [_cache_p, _batch_p, _vp, _vp, _vp]
lib.bi_kv4_gather.restype = _ci
lib.bi_attention_kv4_workspace_size.argtypes = [_ci, _cache_p, _batch_p]
lib.bi_attention_kv4_workspace_size.restype = _sz
lib.bi_attention_kv4.argtypes = [_vp, _i64, _ci, _cache_p, _batch_p, ctypes.c_float, _vp, _vp, _sz, _cu, _vp]
lib.bi_attention_kv4.restype = _ci
lib.bi_logits_workspace_size.argtypes = [_ci]
lib.bi_logits_workspace_size.restype = _sz
lib.bi_logits_process.argtypes = [_vp, _i64, _ci, _ci, ctypes.POINTER(bi_logits_rules), _vp, _i64, _vp, _vp, _sz, _cu,
                                  _vp]
lib.bi_logits_process.restype = _ci
lib.bi_quantize_act_f8.argtypes = [_vp, _i64, _ci, _ci, _vp, _vp, _cu, _vp]
lib.bi_quantize_act_f8.restype = _ci
lib.bi_gated_quantize_f8.argtypes = [_vp, _i64, _ci, _ci, _ci, _vp, _vp, _cu, _vp]
lib.bi_gated_quantize_f8.restype = _ci
lib.bi_quantize_weight_f8.argtypes = [_vp, _i64, _ci, _ci, _vp, _vp, _vp]
lib.bi_quantize_weight_f8.restype = _ci
lib.bi_f8_workspace_size.argtypes = []
lib.bi_f8_workspace_size.restype = _sz
lib.bi_linear_f8.argtypes = [_vp, _vp, _ci, _ci, _vp, _vp, _ci, _vp, _vp, _sz, _cu, _vp]
lib.bi_linear_f8.restype = _ci
lib.bi_linear_f8_grouped.argtypes = [_vp, _vp, _ci, _ci, _vp, _ci, _vp, _ci, _vp, _vp, _ci, _vp, _vp, _sz, _cu, _vp]
lib.bi_linear_f8_grouped.restype = _ci
lib.bi_moe_route_workspace_size.argtypes = [_ci, _ci]
lib.bi_moe_route_workspace_size.restype = _sz
lib.bi_moe_route.argtypes = [_vp, _i64, _ci, _ci, _ci, _ci, _ci, _ci, ctypes.c_float, _vp, _vp, _vp, _vp, _vp, _vp, _sz, _cu,
                             _vp]
lib.bi_moe_route.restype = _ci
lib.bi_moe_combine.argtypes = [_vp, _ci, _vp, _vp, _ci, _ci, _ci, _vp, _vp, _cu, _vp]
lib.bi_moe_combine.restype = _ci
lib.bi_probe_read.argtypes = [_vp, _sz, _vp, _vp]
lib.bi_probe_read.restype = _ci
lib.bi_probe_copy.argtypes = [_vp, _vp, _sz, _vp]
lib.bi_probe_copy.restype = _ci

lib.bi_program_bytes.argtypes = [_ci]
lib.bi_program_bytes.restype = _sz
lib.bi_program_workspace_size.argtypes = []
lib.bi_program_workspace_size.restype = _sz


class bi_op(ctypes.Structure):
    """One op of a verify-pass program (struct bi_op of include/bi.h)."""
    _fields_ = [("kind", _ci), ("M", _ci), ("N", _ci), ("K", _ci),
                ("x", _vp), ("ldx", _i64), ("q", _vp), ("s_a", _vp),
                ("w_q", _vp), ("s_w", _vp), ("y", _vp), ("argmax", _vp),
                ("draft", _vp), ("accept", _vp)]


lib.bi_program_build.argtypes = [ctypes.POINTER(bi_op), _ci, _vp, _sz]
lib.bi_program_build.restype = _ci
lib.bi_program_run.argtypes = [_vp, _ci, _vp, _sz, _vp]
lib.bi_program_run.restype = _ci

BI_OP_QUANTIZE_ACT = 1
BI_OP_LINEAR = 2
BI_OP_LMHEAD = 3
BI_OP_RESIDUAL_QUANT = 4
BI_OP_RELU_MUL_QUANT = 5

BI_OK = 0
BI_ERR_INVALID_ARG = 1
BI_ERR_ALIGNMENT = 2
BI_ERR_INT32_BOUND = 3
BI_ERR_WORKSPACE = 4
BI_ERR_UNSUPPORTED = 5
BI_ERR_TIMEOUT = 6
BI_ERR_CUDA = 7
BI_FLAG_PDL = 1
BI_ROPE_HALF = 0
BI_ROPE_INTERLEAVED = 1
BI_GATE_RELU = 0
BI_GATE_SILU = 1
BI_TYPE_F32 = 0
BI_TYPE_BF16 = 1
BI_ROUTE_SOFTMAX = 0
BI_ROUTE_SIGMOID = 1


class BiError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        super().__init__("%s: %s" % (what, lib.bi_status_string(status).decode()))


def _check(status: int, what: str) -> None:
    if status != BI_OK:
        raise BiError(status, what)


def _stream(stream) -> int:
    if stream is None:
        # the raw handle of torch's current stream, without building a Stream object (3 us less a call)
        return torch._C._cuda_getCurrentRawStream(torch._C._cuda_getDevice())
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _ptr(t) -> int | None:
    return None if t is None else t.data_ptr()


def bi_status_string(status: int) -> str:
    return lib.bi_status_string(status).decode()


def bi_quantize_act(x: torch.Tensor, q: torch.Tensor, s_a: torch.Tensor, K: int | None = None,
                    flags: int = 0, stream=None) -> None:
    """x: bf16 [M, ldx] (row stride ldx = x.stride(0)); q: int8 [M, K]; s_a: fp32 [M]."""
    M = x.shape[0]
    K = x.shape[1] if K is None else K
    _check(lib.bi_quantize_act(_ptr(x), x.stride(0), M, K, _ptr(q), _ptr(s_a), flags, _stream(stream)),
           "bi_quantize_act")


def bi_residual_quantize(h: torch.Tensor, y: torch.Tensor, q: torch.Tensor, s_a: torch.Tensor,
                         flags: int = 0, stream=None) -> None:
    """h: bf16 [M, K] contiguous, updated in place; y: bf16 [M, >= K] (row stride
    y.stride(0)), first K columns added; q: int8 [M, K]; s_a: fp32 [M]."""
    M, K = h.shape
    assert h.stride(0) == K
    _check(lib.bi_residual_quantize(_ptr(h), _ptr(y), y.stride(0), M, K, _ptr(q), _ptr(s_a), flags,
                                    _stream(stream)), "bi_residual_quantize")


def bi_relu_mul_quantize(gu: torch.Tensor, K: int, q: torch.Tensor, s_a: torch.Tensor,
                         m_out: torch.Tensor | None = None, flags: int = 0, stream=None) -> None:
    """gu: bf16 [M, >= 2K] packed gate|up (row stride gu.stride(0)); q: int8 [M, K];
    s_a: fp32 [M]; m_out: bf16 [M, K] or None."""
    M = gu.shape[0]
    _check(lib.bi_relu_mul_quantize(_ptr(gu), gu.stride(0), M, K, _ptr(q), _ptr(s_a), _ptr(m_out), flags,
                                    _stream(stream)), "bi_relu_mul_quantize")


def bi_quantize_weight(w: torch.Tensor, w_q: torch.Tensor, s_w: torch.Tensor, stream=None) -> None:
    N, K = w.shape
    _check(lib.bi_quantize_weight(_ptr(w), w.stride(0), N, K, _ptr(w_q), _ptr(s_w), _stream(stream)),
           "bi_quantize_weight")


def bi_requant_pow2(w_q: torch.Tensor, s_w: torch.Tensor, w_q_out: torch.Tensor, s_w_out: torch.Tensor,
                    stream=None) -> None:
    N, K = w_q.shape
    _check(lib.bi_requant_pow2(_ptr(w_q), _ptr(s_w), N, K, _ptr(w_q_out), _ptr(s_w_out), _stream(stream)),
           "bi_requant_pow2")


def bi_linear_workspace_size(M: int, N: int, K: int) -> int:
    return int(lib.bi_linear_workspace_size(M, N, K))


def bi_lmhead_workspace_size(M: int, N: int, K: int) -> int:
    return int(lib.bi_lmhead_workspace_size(M, N, K))


def bi_linear_w8a8(q: torch.Tensor, s_a: torch.Tensor, w_q: torch.Tensor, s_w: torch.Tensor,
                   y: torch.Tensor, ws: torch.Tensor, flags: int = 0, stream=None) -> None:
    M, K = q.shape
    N = w_q.shape[0]
    _check(lib.bi_linear_w8a8(_ptr(q), _ptr(s_a), M, K, _ptr(w_q), _ptr(s_w), N, _ptr(y), _ptr(ws),
                              ws.numel() * ws.element_size(), flags, _stream(stream)), "bi_linear_w8a8")


def bi_lmhead_argmax(q: torch.Tensor, s_a: torch.Tensor, w_q: torch.Tensor, s_w: torch.Tensor,
                     logits: torch.Tensor | None, argmax: torch.Tensor, ws: torch.Tensor,
                     flags: int = 0, stream=None) -> None:
    M, K = q.shape
    N = w_q.shape[0]
    _check(lib.bi_lmhead_argmax(_ptr(q), _ptr(s_a), M, K, _ptr(w_q), _ptr(s_w), N, _ptr(logits),
                                _ptr(argmax), _ptr(ws), ws.numel() * ws.element_size(), flags,
                                _stream(stream)), "bi_lmhead_argmax")


def bi_quantize_weight_q6(w: torch.Tensor, ql: torch.Tensor, qh: torch.Tensor, sc: torch.Tensor, d: torch.Tensor,
                          stream=None) -> None:
    """w fp32 [N, K] -> block-scaled ql uint8 [N, K/2], qh uint8 [N, K/4], sc int8 [N, K/16], d fp32 [N, K/256]."""
    N, K = w.shape
    _check(lib.bi_quantize_weight_q6(_ptr(w), w.stride(0), N, K, _ptr(ql), _ptr(qh), _ptr(sc), _ptr(d),
                                     _stream(stream)), "bi_quantize_weight_q6")


def bi_quantize_act_blocks(x: torch.Tensor, q: torch.Tensor, d_a: torch.Tensor, stream=None) -> None:
    """x bf16 bits [M, K] (int16/uint16/bfloat16) -> q int8 [M, K], d_a fp32 [M, K/32]."""
    M, K = x.shape
    _check(lib.bi_quantize_act_blocks(_ptr(x), x.stride(0), M, K, _ptr(q), _ptr(d_a), _stream(stream)),
           "bi_quantize_act_blocks")


def bi_linear_q6(q: torch.Tensor, d_a: torch.Tensor, ql: torch.Tensor, qh: torch.Tensor, sc: torch.Tensor,
                 d: torch.Tensor, y: torch.Tensor, flags: int = 0, stream=None) -> None:
    """y fp32 [M, N] = the block-scaled linear (1 <= M <= 16)."""
    M, K = q.shape
    N = ql.shape[0]
    _check(lib.bi_linear_q6(_ptr(q), _ptr(d_a), M, K, _ptr(ql), _ptr(qh), _ptr(sc), _ptr(d), N, _ptr(y), flags,
                            _stream(stream)), "bi_linear_q6")


def bi_attention_workspace_size(M: int, Hq: int, D: int, T0: int) -> int:
    return int(lib.bi_attention_workspace_size(M, Hq, D, T0))


def bi_attention_verify(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, T0: int, scale: float, o: torch.Tensor,
                        ws: torch.Tensor | None = None, stream=None) -> None:
    """Split-KV verify attention: q bf16 [M, Hq, D], k/v bf16 [S, Hkv, D]
    (contiguous), o bf16 [M, Hq, D] out; query m sees positions 0 .. T0 + m.
    ws: device buffer of at least bi_attention_workspace_size(M, Hq, D, T0)
    bytes, or None when that is 0."""
    M, Hq, D = q.shape
    S, Hkv = k.shape[0], k.shape[1]
    nbytes = 0 if ws is None else ws.numel() * ws.element_size()
    _check(lib.bi_attention_verify(_ptr(q), _ptr(k), _ptr(v), M, Hq, Hkv, D, T0, S, scale, _ptr(o), _ptr(ws),
                                   nbytes, _stream(stream)), "bi_attention_verify")


def _rows(t: torch.Tensor, M: int, K: int, size: int) -> int:
    """The row stride of elements of `size` bytes [>= M, >= K]; of a single row, whose stride may be anything, K."""
    assert t.dim() == 2
    m, k = t.shape
    ld, s = t.stride()
    assert m >= M and k >= K and (s == 1 or k == 1) and t.element_size() == size
    return ld if M > 1 else K


def _vector(t: torch.Tensor, n: int, size: int) -> int:
    """The address of at least n elements of `size` bytes side by side."""
    assert t.is_contiguous() and t.numel() >= n and t.element_size() == size
    return t.data_ptr()


def bi_rmsnorm_quantize(h: torch.Tensor, y: torch.Tensor | None, w: torch.Tensor, eps: float,
                        h_out: torch.Tensor | None, q: torch.Tensor, s_a: torch.Tensor, flags: int = 0,
                        stream=None) -> None:
    """h, y: bf16 [M, >= K] (row strides h.stride(0), y.stride(0)); w: bf16 [K]; h_out: bf16 [M, >= K], given with y
    (it may be h); q: int8 [M, K]; s_a: fp32 [M]."""
    M, K = q.shape
    assert q.element_size() == 1 and q.is_contiguous()
    ldh = _rows(h, M, K, 2)
    ldy = K if y is None else _rows(y, M, K, 2)
    ldo = K if h_out is None else _rows(h_out, M, K, 2)
    _check(lib.bi_rmsnorm_quantize(h.data_ptr(), ldh, _ptr(y), ldy, _vector(w, K, 2), eps, M, K, _ptr(h_out), ldo,
                                   q.data_ptr(), _vector(s_a, M, 4), flags, _stream(stream)), "bi_rmsnorm_quantize")


def bi_kv4_block_bytes(page_size: int, D: int) -> int:
    return int(lib.bi_kv4_block_bytes(page_size, D))


def kv4_cache(pool: torch.Tensor, page_size: int, D: int) -> bi_kv4_cache:
    """A cache over `pool`, uint8 [num_pages, Hkv, bi_kv4_block_bytes(page_size, D)] with any page stride (for
    instance one layer of a pool of all layers).  The cache holds the tensor."""
    n, Hkv, block = pool.shape
    assert pool.dtype == torch.uint8 and block == bi_kv4_block_bytes(page_size, D)
    assert pool.stride(2) == 1 and pool.stride(1) == block
    return _holding(bi_kv4_cache(pool.data_ptr(), pool.stride(0) if n > 1 else Hkv * block, n, page_size, Hkv, D), pool)


def new_kv4_pool(num_pages: int, Hkv: int, page_size: int, D: int, device="cuda") -> torch.Tensor:
    """Device memory for a cache of num_pages pages."""
    return torch.zeros((num_pages, Hkv, bi_kv4_block_bytes(page_size, D)), dtype=torch.uint8, device=device)


def kv4_batch(cu_q: torch.Tensor, kv_len: torch.Tensor, pages: torch.Tensor, T: int, max_q: int,
              max_kv: int) -> bi_kv4_batch:
    """cu_q int32 [B + 1], kv_len int32 [B], pages int32 [B, n]; T, max_q, max_kv: bounds
    known to the host.  The batch holds the tensors."""
    B = kv_len.shape[0]
    assert cu_q.dtype == kv_len.dtype == pages.dtype == torch.int32
    assert cu_q.shape[0] == B + 1 and cu_q.is_contiguous() and kv_len.is_contiguous()
    assert pages.shape[0] == B and pages.is_contiguous()
    return _holding(bi_kv4_batch(cu_q.data_ptr(), kv_len.data_ptr(), pages.data_ptr(), pages.shape[1], B, T, max_q, max_kv),
                    cu_q, kv_len, pages)


def _heads(t: torch.Tensor, T: int, H: int, D: int) -> int:
    """The row stride of 16-bit elements [>= T, H, D], the heads of a row side by side; of a single row, whose stride may
    be anything, its length."""
    n, h, d = t.shape
    ld, sh, sd = t.stride()
    assert n >= T and h == H and d == D and sd == 1 and (sh == D or h == 1) and t.element_size() == 2
    return ld if n > 1 else H * D


def bi_rope_table(inv_freq: torch.Tensor, rope: torch.Tensor, amp: float = 1.0, stream=None) -> None:
    """inv_freq: fp64 [n]; rope: fp32 [positions, n, 2] out."""
    assert inv_freq.dtype == torch.float64 and rope.dtype == torch.float32 and rope.is_contiguous()
    assert rope.shape[1:] == (inv_freq.shape[0], 2)
    n = inv_freq.shape[0]
    _check(lib.bi_rope_table(_vector(inv_freq, n, 8), n, amp, rope.shape[0], _ptr(rope), _stream(stream)), "bi_rope_table")


def bi_rope_append_kv4(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, rope: torch.Tensor, rot: int, layout: int,
                       q_out: torch.Tensor, cache: bi_kv4_cache, batch: bi_kv4_batch, q_norm: torch.Tensor | None = None,
                       k_norm: torch.Tensor | None = None, eps: float = 0.0, flags: int = 0, stream=None) -> None:
    """q: bf16 [T, Hq, D], k, v: bf16 [T, Hkv, D] (row strides stride(0); parts of one packed tensor will do);
    rope: fp32 [positions, rot / 2, 2] (any width with rot 0); q_norm, k_norm: bf16 [D] or None; q_out: bf16 [T, Hq, D]."""
    T, D, Hq, Hkv = batch.T, cache.D, q.shape[1], cache.Hkv
    ldq, ldk, ldv = _heads(q, T, Hq, D), _heads(k, T, Hkv, D), _heads(v, T, Hkv, D)
    table = rope.shape
    assert _heads(q_out, T, Hq, D) == Hq * D and rope.is_contiguous() and rope.dtype == torch.float32
    assert rot == 0 or table == (table[0], rot // 2, 2)
    qn = None if q_norm is None else _vector(q_norm, D, 2)
    kn = None if k_norm is None else _vector(k_norm, D, 2)
    _check(lib.bi_rope_append_kv4(q.data_ptr(), ldq, Hq, k.data_ptr(), ldk, v.data_ptr(), ldv, qn, kn, eps,
                                  rope.data_ptr(), table[0], rot, layout, q_out.data_ptr(), cache, batch, flags,
                                  _stream(stream)), "bi_rope_append_kv4")


def bi_kv4_gather(cache: bi_kv4_cache, batch: bi_kv4_batch, k_out: torch.Tensor, v_out: torch.Tensor,
                  stream=None) -> None:
    """k_out, v_out: bf16 [T, Hkv, D], the cached values of the batch's token rows."""
    T, Hkv, D = batch.T, cache.Hkv, cache.D
    assert _heads(k_out, T, Hkv, D) == _heads(v_out, T, Hkv, D) == Hkv * D
    _check(lib.bi_kv4_gather(cache, batch, k_out.data_ptr(), v_out.data_ptr(), _stream(stream)), "bi_kv4_gather")


def bi_attention_kv4_workspace_size(Hq: int, cache: bi_kv4_cache, batch: bi_kv4_batch) -> int:
    return int(lib.bi_attention_kv4_workspace_size(Hq, cache, batch))


def new_attention_kv4_workspace(Hq: int, cache: bi_kv4_cache, batch: bi_kv4_batch, device="cuda") -> torch.Tensor:
    """A zero-filled workspace for bi_attention_kv4 calls up to this size."""
    return torch.zeros(bi_attention_kv4_workspace_size(Hq, cache, batch), dtype=torch.uint8, device=device)


def bi_attention_kv4(q: torch.Tensor, cache: bi_kv4_cache, batch: bi_kv4_batch, scale: float, o: torch.Tensor,
                     ws: torch.Tensor, flags: int = 0, stream=None) -> None:
    """q: bf16 [T, Hq, D] (row stride q.stride(0)); o: bf16 [T, Hq, D] out; ws: from new_attention_kv4_workspace."""
    T, Hq, D = batch.T, q.shape[1], cache.D
    ldq = _heads(q, T, Hq, D)
    assert _heads(o, T, Hq, D) == Hq * D
    _check(lib.bi_attention_kv4(q.data_ptr(), ldq, Hq, cache, batch, scale, o.data_ptr(), ws.data_ptr(), ws.nbytes,
                                flags, _stream(stream)), "bi_attention_kv4")


def logits_rules(ids: torch.Tensor | None = None, begin: torch.Tensor | None = None, mid: torch.Tensor | None = None,
                 end: torch.Tensor | None = None, repetition: torch.Tensor | None = None,
                 presence: torch.Tensor | None = None, frequency: torch.Tensor | None = None,
                 bias_ids: torch.Tensor | None = None, bias: torch.Tensor | None = None,
                 mask: torch.Tensor | None = None) -> bi_logits_rules:
    """ids int32; begin, mid, end int32 [M]; repetition, presence, frequency fp32 [M]; bias_ids int32 [M, n] and bias
    fp32 [M, n]; mask int32 words [M, >= ceil(V / 32)].  The rules hold the tensors."""
    for t in (ids, begin, mid, end, bias_ids, mask):
        assert t is None or t.dtype == torch.int32
    for t in (repetition, presence, frequency, bias):
        assert t is None or t.dtype == torch.float32
    for t in (ids, begin, mid, end, repetition, presence, frequency, bias_ids, bias):
        assert t is None or t.is_contiguous()
    assert mask is None or mask.stride(1) == 1 or mask.shape[1] == 1
    assert bias_ids is None or bias is None or bias.shape == bias_ids.shape
    n = 0 if bias_ids is None else bias_ids.shape[1]
    r = bi_logits_rules(_ptr(ids), _ptr(begin), _ptr(mid), _ptr(end), _ptr(repetition), _ptr(presence),
                        _ptr(frequency), _ptr(bias_ids), _ptr(bias), n, _ptr(mask),
                        0 if mask is None else mask.stride(0) if mask.shape[0] > 1 else mask.shape[1])
    r.rows = min((t.shape[0] for t in (begin, mid, end, repetition, presence, frequency, bias_ids, bias, mask) if t is not None),
                 default=r.rows)
    if mask is not None:
        r.reach = 32 * mask.shape[1]
    return _holding(r, ids, begin, mid, end, repetition, presence, frequency, bias_ids, bias, mask)


def bi_logits_workspace_size(M: int) -> int:
    return int(lib.bi_logits_workspace_size(M))


def new_logits_workspace(M: int, device="cuda") -> torch.Tensor:
    """A zero-filled workspace for bi_logits_process on up to M rows."""
    return torch.zeros(bi_logits_workspace_size(M), dtype=torch.uint8, device=device)


def bi_logits_process(logits: torch.Tensor, rules: bi_logits_rules, out: torch.Tensor | None,
                      argmax: torch.Tensor | None, ws: torch.Tensor, flags: int = 0, stream=None) -> None:
    """logits: bf16 [M, V] (row stride logits.stride(0)); rules: for at least M rows; out: fp32 [M, V] or None; argmax:
    int32 [M] or None."""
    M, V = logits.shape
    ldl, ldo = _rows(logits, M, V, 2), V
    if out is not None:
        assert out.dtype == torch.float32
        ldo = _rows(out, M, V, 4)
    assert argmax is None or argmax.dtype == torch.int32
    assert rules.rows >= M and rules.reach >= V
    _check(lib.bi_logits_process(logits.data_ptr(), ldl, M, V, rules, _ptr(out), ldo,
                                 None if argmax is None else _vector(argmax, M, 4), ws.data_ptr(), ws.nbytes, flags,
                                 _stream(stream)), "bi_logits_process")


_BF16, _F32, _I32 = torch.bfloat16, torch.float32, torch.int32
_E4M3 = (torch.float8_e4m3fn, torch.uint8)       # codes as such, or as bytes


def _codes(t: torch.Tensor) -> int:
    """The address of e4m3 codes side by side."""
    assert t.dtype in _E4M3 and t.is_contiguous()
    return t.data_ptr()


def _flat(t: torch.Tensor, dtype: torch.dtype) -> int:
    """The address of elements side by side."""
    assert t.dtype is dtype and t.is_contiguous()
    return t.data_ptr()


def _dense(t: torch.Tensor, shape: tuple, dtype: torch.dtype) -> int:
    """The same of this shape."""
    assert t.dtype is dtype and t.shape == shape and t.is_contiguous()
    return t.data_ptr()


def _matrix(t: torch.Tensor, M: int, K: int, dtype: torch.dtype) -> int:
    """The row stride of elements [>= M, >= K]; of a single row, whose stride may be anything, K."""
    (m, k), (ld, s) = t.shape, t.stride()
    assert t.dtype is dtype and m >= M and k >= K and (s == 1 or k == 1)
    return ld if M > 1 else K


def _blocks(n: int) -> int:
    """Blocks of 128 elements, the last one may be short."""
    return (n + 127) // 128


def _here(d: int, name: str) -> None:
    """Refuses a call unless d, where its tensors are (-1: host memory), is the current GPU.  The library takes addresses and
    cannot see whose memory they are; its kernels would fault on them."""
    if d < 0 or d != torch._C._cuda_getDevice():
        raise BiError(BI_ERR_INVALID_ARG, name + ", a tensor that is not on the current GPU")


def _stream_at(d: int, stream) -> int:
    """The handle of a stream; None: torch's current one of GPU d."""
    return torch._C._cuda_getCurrentRawStream(d) if stream is None else _stream(stream)


def bi_quantize_act_f8(x: torch.Tensor, q: torch.Tensor, s_a: torch.Tensor, flags: int = 0, stream=None) -> None:
    """x: bf16 [M, >= K] (row stride x.stride(0)); q: e4m3 [M, K] (float8_e4m3fn or bytes); s_a: fp32 [M, ceil(K / 128)]."""
    M, K = q.shape
    ld, at_q, at_s = _matrix(x, M, K, _BF16), _codes(q), _dense(s_a, (M, (K + 127) // 128), _F32)
    d = x.get_device()
    _here(d if d == q.get_device() == s_a.get_device() else -1, "bi_quantize_act_f8")
    _check(lib.bi_quantize_act_f8(x.data_ptr(), ld, M, K, at_q, at_s, flags, _stream_at(d, stream)), "bi_quantize_act_f8")


def bi_gated_quantize_f8(gu: torch.Tensor, gate: int, q: torch.Tensor, s_a: torch.Tensor, flags: int = 0, stream=None) -> None:
    """gu: bf16 [M, >= 2K] packed gate|up (row stride gu.stride(0)); gate: BI_GATE_RELU or BI_GATE_SILU; q: e4m3 [M, K];
    s_a: fp32 [M, ceil(K / 128)]."""
    M, K = q.shape
    ld, at_q, at_s = _matrix(gu, M, 2 * K, _BF16), _codes(q), _dense(s_a, (M, (K + 127) // 128), _F32)
    d = gu.get_device()
    _here(d if d == q.get_device() == s_a.get_device() else -1, "bi_gated_quantize_f8")
    _check(lib.bi_gated_quantize_f8(gu.data_ptr(), ld, M, K, gate, at_q, at_s, flags, _stream_at(d, stream)),
           "bi_gated_quantize_f8")


def bi_quantize_weight_f8(w: torch.Tensor, w_q: torch.Tensor, s_w: torch.Tensor, stream=None) -> None:
    """w: fp32 [N, K] (row stride w.stride(0)); w_q: e4m3 [N, K]; s_w: fp32 [ceil(N / 128), ceil(K / 128)]."""
    N, K = w_q.shape
    ld, at_q, at_s = _matrix(w, N, K, _F32), _codes(w_q), _dense(s_w, (_blocks(N), _blocks(K)), _F32)
    d = w.get_device()
    _here(d if d == w_q.get_device() == s_w.get_device() else -1, "bi_quantize_weight_f8")
    _check(lib.bi_quantize_weight_f8(w.data_ptr(), ld, N, K, at_q, at_s, _stream_at(d, stream)), "bi_quantize_weight_f8")


def bi_f8_workspace_size() -> int:
    return int(lib.bi_f8_workspace_size())


def new_f8_workspace(device="cuda") -> torch.Tensor:
    """A zero-filled workspace for bi_linear_f8 and bi_linear_f8_grouped calls of any size."""
    return torch.zeros(bi_f8_workspace_size(), dtype=torch.uint8, device=device)


def bi_linear_f8(q: torch.Tensor, s_a: torch.Tensor, w: torch.Tensor, s_w: torch.Tensor, y: torch.Tensor, ws: torch.Tensor,
                 flags: int = 0, stream=None) -> None:
    """q: e4m3 [M, K], s_a: fp32 [M, ceil(K / 128)]; w: e4m3 [N, K], s_w: fp32 [ceil(N / 128), ceil(K / 128)]; y: bf16 [M, N];
    ws: from new_f8_workspace."""
    (M, K), (N, k) = q.shape, w.shape
    assert k == K
    kb = _blocks(K)
    at_q, at_sa, at_w = _codes(q), _dense(s_a, (M, kb), _F32), _codes(w)
    at_sw, at_y = _dense(s_w, (_blocks(N), kb), _F32), _dense(y, (M, N), _BF16)
    d = q.get_device()
    _here(d if d == s_a.get_device() == w.get_device() == s_w.get_device() == y.get_device() == ws.get_device() else -1,
          "bi_linear_f8")
    _check(lib.bi_linear_f8(at_q, at_sa, M, K, at_w, at_sw, N, at_y, ws.data_ptr(), ws.nbytes, flags, _stream_at(d, stream)),
           "bi_linear_f8")


def bi_linear_f8_grouped(q: torch.Tensor, s_a: torch.Tensor, src: torch.Tensor | None, offsets: torch.Tensor, w: torch.Tensor,
                         s_w: torch.Tensor, y: torch.Tensor, ws: torch.Tensor, flags: int = 0, stream=None) -> None:
    """y: bf16 [R, N], expert e's rows offsets[e] .. offsets[e + 1] - 1 (int32 [E + 1]) = rows src[r] (int32 [R], None: r) of
    q: e4m3 [n, K], s_a: fp32 [n, ceil(K / 128)] by w: e4m3 [E, N, K], s_w: fp32 [E, ceil(N / 128), ceil(K / 128)]."""
    (n, K), (R, N), (E, _, k) = q.shape, y.shape, w.shape
    assert w.shape[1] == N and k == K
    kb = _blocks(K)
    at_src = None if src is None else _dense(src, (R,), _I32)
    at_q, at_sa, at_off, at_w = _codes(q), _dense(s_a, (n, kb), _F32), _dense(offsets, (E + 1,), _I32), _codes(w)
    at_sw, at_y = _dense(s_w, (E, _blocks(N), kb), _F32), _flat(y, _BF16)
    d = q.get_device()
    _here(d if d == s_a.get_device() == offsets.get_device() == w.get_device() == s_w.get_device() == y.get_device() ==
          ws.get_device() and (src is None or d == src.get_device()) else -1, "bi_linear_f8_grouped")
    _check(lib.bi_linear_f8_grouped(at_q, at_sa, n, K, at_src, R, at_off, E, at_w, at_sw, N, at_y, ws.data_ptr(), ws.nbytes,
                                    flags, _stream_at(d, stream)), "bi_linear_f8_grouped")


def bi_moe_route_workspace_size(M: int, E: int) -> int:
    return int(lib.bi_moe_route_workspace_size(M, E))


def new_moe_route_workspace(M: int, E: int, device="cuda") -> torch.Tensor:
    """A workspace for bi_moe_route calls of M tokens and E experts."""
    return torch.empty(bi_moe_route_workspace_size(M, E), dtype=torch.uint8, device=device)


def bi_moe_route(logits: torch.Tensor, score: int, renorm: bool, scale: float, ids: torch.Tensor, weights: torch.Tensor,
                 offsets: torch.Tensor, src: torch.Tensor, pos: torch.Tensor, ws: torch.Tensor, flags: int = 0,
                 stream=None) -> None:
    """logits: fp32 or bf16 [M, E] (row stride logits.stride(0)); score: BI_ROUTE_SOFTMAX or BI_ROUTE_SIGMOID; ids: int32
    [M, k]; weights: fp32 [M, k]; offsets: int32 [E + 1]; src: int32 [M k]; pos: int32 [M, k]."""
    (M, E), k = logits.shape, ids.shape[1]
    half = logits.dtype is _BF16
    ld = _matrix(logits, M, E, _BF16 if half else _F32)
    at_ids, at_w, at_off = _dense(ids, (M, k), _I32), _dense(weights, (M, k), _F32), _dense(offsets, (E + 1,), _I32)
    at_src, at_pos = _dense(src, (M * k,), _I32), _dense(pos, (M, k), _I32)
    d = logits.get_device()
    _here(d if d == ids.get_device() == weights.get_device() == offsets.get_device() == src.get_device() ==
          pos.get_device() == ws.get_device() else -1, "bi_moe_route")
    _check(lib.bi_moe_route(logits.data_ptr(), ld, BI_TYPE_BF16 if half else BI_TYPE_F32, M, E, k, score, renorm, scale,
                            at_ids, at_w, at_off, at_src, at_pos, ws.data_ptr(), ws.nbytes, flags, _stream_at(d, stream)),
           "bi_moe_route")


def bi_moe_combine(rows: torch.Tensor, pos: torch.Tensor, weights: torch.Tensor, base: torch.Tensor | None, y: torch.Tensor,
                   flags: int = 0, stream=None) -> None:
    """rows: bf16 [R, N]; pos: int32 [M, k]; weights: fp32 [M, k]; base: bf16 [M, N] or None; y: bf16 [M, N], it may be
    base."""
    (M, k), (R, N) = pos.shape, rows.shape
    at_rows, at_pos, at_w = _flat(rows, _BF16), _flat(pos, _I32), _dense(weights, (M, k), _F32)
    at_base, at_y = None if base is None else _dense(base, (M, N), _BF16), _dense(y, (M, N), _BF16)
    d = rows.get_device()
    _here(d if d == pos.get_device() == weights.get_device() == y.get_device() and
          (base is None or d == base.get_device()) else -1, "bi_moe_combine")
    _check(lib.bi_moe_combine(at_rows, R, at_pos, at_w, M, k, N, at_base, at_y, flags, _stream_at(d, stream)), "bi_moe_combine")


def bi_probe_read(buf: torch.Tensor, out: torch.Tensor, stream=None) -> None:
    """Read all of `buf` once (bandwidth probe); out: int64 device tensor, receives the xor of its 64-bit words."""
    _check(lib.bi_probe_read(_ptr(buf), buf.numel() * buf.element_size(), _ptr(out), _stream(stream)),
           "bi_probe_read")


def bi_probe_copy(src: torch.Tensor, dst: torch.Tensor, stream=None) -> None:
    """dst = src (bandwidth probe), same byte size, not overlapping."""
    _check(lib.bi_probe_copy(_ptr(src), _ptr(dst), src.numel() * src.element_size(), _stream(stream)),
           "bi_probe_copy")


def bi_linear_w8a8_noalloc(q: torch.Tensor, s_a: torch.Tensor, w_q: torch.Tensor, s_w: torch.Tensor,
                           y: torch.Tensor, flags: int = 0, stream=None) -> None:
    """bi_linear_w8a8 without a workspace argument, for callers that cannot
    allocate device memory: the library keeps the kernel's scratch in a fixed
    array of its own (M <= 16; calls on one stream only, never overlapping)."""
    M, K = q.shape
    N = w_q.shape[0]
    _check(lib.bi_linear_w8a8_noalloc(_ptr(q), _ptr(s_a), M, K, _ptr(w_q), _ptr(s_w), N, _ptr(y), flags,
                                      _stream(stream)), "bi_linear_w8a8_noalloc")


def bi_linear_w8a8_noalloc_status(stream=None) -> int:
    """Status of the no-alloc entry point's scratch after `stream`: BI_OK, or
    BI_ERR_TIMEOUT (once; the scratch is then restored)."""
    return int(lib.bi_linear_w8a8_noalloc_status(_stream(stream)))


def bi_program_bytes(n_ops: int) -> int:
    return int(lib.bi_program_bytes(n_ops))


def bi_program_workspace_size() -> int:
    return int(lib.bi_program_workspace_size())


def bi_program_build(ops, program: torch.Tensor) -> None:
    """ops: a sequence of bi_op; program: device uint8 tensor of at least
    bi_program_bytes(len(ops)) bytes, 128-byte aligned."""
    arr = (bi_op * len(ops))(*ops)
    _check(lib.bi_program_build(arr, len(ops), _ptr(program), program.numel() * program.element_size()),
           "bi_program_build")


def bi_program_run(program: torch.Tensor, max_tokens: int, ws: torch.Tensor, stream=None) -> None:
    _check(lib.bi_program_run(_ptr(program), max_tokens, _ptr(ws), ws.numel() * ws.element_size(),
                              _stream(stream)), "bi_program_run")


def op_quantize_act(x: torch.Tensor, q: torch.Tensor, s_a: torch.Tensor, K: int | None = None) -> bi_op:
    M = x.shape[0]
    K = x.shape[1] if K is None else K
    return bi_op(BI_OP_QUANTIZE_ACT, M, 0, K, _ptr(x), x.stride(0), _ptr(q), _ptr(s_a), None, None, None, None)


def op_residual_quant(h: torch.Tensor, y: torch.Tensor, q: torch.Tensor, s_a: torch.Tensor) -> bi_op:
    """h (in/out, contiguous [M, K]) <- rescale(bf16(h + y[:, :K])); q, s_a <- quant(h)."""
    M, K = h.shape
    assert h.stride(0) == K
    return bi_op(BI_OP_RESIDUAL_QUANT, M, 0, K, _ptr(y), y.stride(0), _ptr(q), _ptr(s_a), None, None, _ptr(h), None)


def op_relu_mul_quant(gu: torch.Tensor, K: int, q: torch.Tensor, s_a: torch.Tensor,
                      m_out: torch.Tensor | None = None) -> bi_op:
    """q, s_a <- quant(bf16(relu(gu[:, :K]) * gu[:, K:2K])); m_out receives the product if given."""
    M = gu.shape[0]
    return bi_op(BI_OP_RELU_MUL_QUANT, M, 0, K, _ptr(gu), gu.stride(0), _ptr(q), _ptr(s_a), None, None,
                 _ptr(m_out), None)


def op_linear(q: torch.Tensor, s_a: torch.Tensor, w_q: torch.Tensor, s_w: torch.Tensor, y: torch.Tensor) -> bi_op:
    M, K = q.shape
    return bi_op(BI_OP_LINEAR, M, w_q.shape[0], K, None, 0, _ptr(q), _ptr(s_a), _ptr(w_q), _ptr(s_w), _ptr(y), None)


def op_lmhead(q: torch.Tensor, s_a: torch.Tensor, w_q: torch.Tensor, s_w: torch.Tensor,
              logits: torch.Tensor | None, argmax: torch.Tensor, draft: torch.Tensor | None = None,
              accept: torch.Tensor | None = None) -> bi_op:
    """LM head; with `accept` (int32 [2]) also greedy verification against `draft` (int32 [M - 1])."""
    M, K = q.shape
    return bi_op(BI_OP_LMHEAD, M, w_q.shape[0], K, None, 0, _ptr(q), _ptr(s_a), _ptr(w_q), _ptr(s_w),
                 _ptr(logits), _ptr(argmax), _ptr(draft), _ptr(accept))


def new_program(n_ops: int, device="cuda") -> torch.Tensor:
    """Device memory for a program of n_ops ops (128-byte aligned)."""
    n = bi_program_bytes(n_ops)
    buf = torch.empty(n + 128, dtype=torch.uint8, device=device)
    off = (-buf.data_ptr()) % 128
    return buf[off:off + n]


def bi_greedy_verify(argmax: torch.Tensor, draft: torch.Tensor | None, out: torch.Tensor, stream=None) -> None:
    """argmax int32 [M], draft int32 [M - 1] (or None when M == 1), out int32 [2]:
    accepted draft count and next token."""
    _check(lib.bi_greedy_verify(_ptr(argmax), _ptr(draft), argmax.shape[0], _ptr(out), _stream(stream)),
           "bi_greedy_verify")


def bi_selftest_wait_timeout(ws: torch.Tensor, stream=None) -> None:
    """Launch a bounded wait that nothing satisfies (about 2 s); the workspace
    status then reads BI_ERR_TIMEOUT."""
    _check(lib.bi_selftest_wait_timeout(_ptr(ws), ws.numel() * ws.element_size(), _stream(stream)),
           "bi_selftest_wait_timeout")


def bi_selftest_quotient(out: torch.Tensor, stream=None) -> None:
    """out int64 [3] on the device: pairs checked, mismatches, one mismatching
    (amax bits << 16 | v bits) of the executor's quotient against IEEE division."""
    assert out.dtype == torch.int64 and out.numel() >= 3 and out.is_cuda
    _check(lib.bi_selftest_quotient(_ptr(out), _stream(stream)), "bi_selftest_quotient")


def bi_workspace_status(ws: torch.Tensor, stream=None) -> int:
    """BI_OK or BI_ERR_TIMEOUT (returned, not raised); clears the status word."""
    return int(lib.bi_workspace_status(_ptr(ws), ws.numel() * ws.element_size(), _stream(stream)))


def new_workspace(M: int, N: int, K: int, device="cuda") -> torch.Tensor:
    """A zero-filled workspace large enough for bi_linear_w8a8 and bi_lmhead_argmax."""
    n = max(bi_linear_workspace_size(M, N, K), bi_lmhead_workspace_size(M, N, K))
    return torch.zeros(n, dtype=torch.uint8, device=device)
