"""Python binding of libmoe, the MI355X (gfx950) quantized mixture-of-experts layer.

This module only marshals arguments to the C ABI declared in ``include/moe.h``
(same entry-point names); every step of the layer runs in the library's HIP
kernels.  PyTorch supplies device memory and streams.  There is no fallback:
if ``libmoe.so`` is missing or fails to load, importing the binding raises.
"""
from __future__ import annotations

import ctypes
import os

import numpy as np

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libmoe.so")

MOE_OK = 0
MOE_ERR_INVALID_ARG = -1
MOE_ERR_UNSUPPORTED = -2
MOE_ERR_WORKSPACE = -3
MOE_ERR_BUDGET = -4
MOE_ERR_HIP = -5
MOE_ERR_HOST_ALLOC = -6

MOE_FMT_NVFP4 = 1
MOE_FMT_Q6K = 2
MOE_FMT_Q8_0 = 3
MOE_FMT_IQ3G = 4
MOE_FMT_IQ1G = 5
MOE_FMT_BF16 = 6  # key/value cache only
MOE_FMT_MXFP4 = 7  # dense projections and their rows
MOE_FMT_MXFP8 = 8  # rows only
MOE_DTYPE_F32 = 0
MOE_DTYPE_BF16 = 1

MOE_NOALLOC_WORKSPACE_BYTES = 32 << 20

MOE_ROPE_PLAIN = 0
MOE_ROPE_LINEAR = 1
MOE_ROPE_BASE = 2
MOE_ROPE_PARTS = 3

MOE_FFN_AUTO = 0
MOE_FFN_GEMV = 1
MOE_FFN_GEMM = 2


class MoeError(RuntimeError):
    def __init__(self, status: int, msg: str):
        super().__init__(f"status {status}: {msg}")
        self.status = status


class ExpertRef(ctypes.Structure):
    _fields_ = [("blob", ctypes.c_void_p), ("ts_gate", ctypes.c_float),
                ("ts_up", ctypes.c_float), ("ts_down", ctypes.c_float),
                ("reserved", ctypes.c_uint32)]


class LayerDesc(ctypes.Structure):
    _fields_ = [("E", ctypes.c_int32), ("k", ctypes.c_int32), ("H", ctypes.c_int32),
                ("I", ctypes.c_int32), ("fmt_gate_up", ctypes.c_int32),
                ("fmt_down", ctypes.c_int32), ("renormalize", ctypes.c_int32),
                ("ffn_mode", ctypes.c_int32), ("experts", ctypes.c_void_p),
                ("w_router", ctypes.c_void_p), ("router_bias", ctypes.c_void_p)]


class Buckets(ctypes.Structure):
    _fields_ = [("counts", ctypes.c_void_p), ("offsets", ctypes.c_void_p),
                ("sorted_asg", ctypes.c_void_p), ("asg_pos", ctypes.c_void_p),
                ("active", ctypes.c_void_p), ("n_active", ctypes.c_void_p),
                ("T_max", ctypes.c_int64), ("E", ctypes.c_int32), ("k", ctypes.c_int32)]


class TierDesc(ctypes.Structure):
    _fields_ = [("L", ctypes.c_int32), ("E", ctypes.c_int32),
                ("resident_per_layer", ctypes.c_int32), ("staging_slots", ctypes.c_int32),
                ("expert_bytes", ctypes.c_size_t), ("host_blobs", ctypes.c_void_p),
                ("scales", ctypes.c_void_p), ("hbm_pool", ctypes.c_void_p),
                ("hbm_pool_bytes", ctypes.c_size_t), ("copy_stream", ctypes.c_void_p)]


class TierStats(ctypes.Structure):
    _fields_ = [(n, ctypes.c_uint64) for n in
                ("hits", "misses", "h2d_bytes", "promotions", "prepares", "rebalances")]


class KvCacheDesc(ctypes.Structure):
    """moe_kv_cache: a layer's paged key/value cache."""
    _fields_ = [("fmt", ctypes.c_int32), ("n_kv", ctypes.c_int32), ("D", ctypes.c_int32),
                ("page_tokens", ctypes.c_int32), ("n_pages", ctypes.c_int32),
                ("k_scale", ctypes.c_float), ("v_scale", ctypes.c_float),
                ("pool", ctypes.c_void_p)]


class SeqBatch(ctypes.Structure):
    """moe_seq_batch: a step's sequences (device pointers)."""
    _fields_ = [("n_seq", ctypes.c_int32), ("max_pages", ctypes.c_int32),
                ("row_start", ctypes.c_void_p), ("kv_len", ctypes.c_void_p),
                ("page_table", ctypes.c_void_p)]


class QkvDesc(ctypes.Structure):
    """moe_qkv_desc: norms and rotation of a step's queries and keys."""
    _fields_ = [("n_q", ctypes.c_int32), ("eps", ctypes.c_float), ("q_norm", ctypes.c_void_p),
                ("k_norm", ctypes.c_void_p), ("rot_dim", ctypes.c_int32),
                ("interleaved", ctypes.c_int32), ("inv_freq", ctypes.c_void_p),
                ("rope_scale", ctypes.c_float)]


class MxMatrix(ctypes.Structure):
    """moe_mx_matrix: a dense projection's packed weights (device pointers)."""
    _fields_ = [("N", ctypes.c_int32), ("K", ctypes.c_int32), ("packed", ctypes.c_void_p),
                ("bias", ctypes.c_void_p)]


assert ctypes.sizeof(MxMatrix) == 24
assert ctypes.sizeof(KvCacheDesc) == 40
assert ctypes.sizeof(SeqBatch) == 32
assert ctypes.sizeof(QkvDesc) == 48
assert ctypes.sizeof(ExpertRef) == 24
assert ctypes.sizeof(TierDesc) == 64
assert ctypes.sizeof(LayerDesc) == 56
assert ctypes.sizeof(Buckets) == 64

# name -> (restype, argtypes); mirrors include/moe.h
_vp, _i32, _i64, _sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t
_LP = ctypes.POINTER(LayerDesc)
_BP = ctypes.POINTER(Buckets)
_CP = ctypes.POINTER(KvCacheDesc)
_SP = ctypes.POINTER(SeqBatch)
_MP = ctypes.POINTER(MxMatrix)
_f32, _f64 = ctypes.c_float, ctypes.c_double
SIGNATURES = {
    "moe_abi_version": (ctypes.c_int, []),
    "moe_last_error": (ctypes.c_char_p, []),
    "moe_expert_blob_bytes": (_sz, [_i32, _i32, _i32, _i32]),
    "moe_pack_experts": (ctypes.c_int, [_i32, _i32, _i32, _i32, _i32, _vp, _vp, _vp, _vp, _vp,
                                        _vp, _vp, _sz, _vp]),
    "moe_buckets_bytes": (_sz, [_i32, _i64, _i32]),
    "moe_buckets_carve": (ctypes.c_int, [_vp, _sz, _i32, _i64, _i32, _BP]),
    "moe_workspace_bytes": (_sz, [_LP, _i64]),
    "moe_route": (ctypes.c_int, [_LP, _vp, _i64, _vp, _vp, _vp, _vp]),
    "moe_bucket": (ctypes.c_int, [_LP, _vp, _i64, _BP, _vp, _sz, _vp]),
    "moe_expert_ffn": (ctypes.c_int, [_LP, _vp, _i64, _BP, _vp, _i32, _vp, _sz, _vp]),
    "moe_expert_ffn_noalloc": (ctypes.c_int, [_LP, _vp, _i64, _BP, _vp, _i32, _vp]),
    "moe_combine": (ctypes.c_int, [_LP, _vp, _i32, _BP, _vp, _i64, _vp, _vp, _vp]),
    "moe_expert_hist": (ctypes.c_int, [_LP, _BP, _vp, _i32, _i32, _vp]),
    "moe_route_ffn": (ctypes.c_int, [_LP, _vp, _i64, _vp, _vp, _vp, _BP, _vp, _i32, _i32, _vp,
                                      _i32, _vp, _sz, _vp]),
    "moe_layer_forward": (ctypes.c_int, [_LP, _vp, _i64, _vp, _vp, _vp, _vp, _vp, _BP, _vp, _i32,
                                          _i32, _vp, _i32, _vp, _sz, _vp]),
    "moe_route_bucket": (ctypes.c_int, [_LP, _vp, _i64, _vp, _vp, _vp, _BP, _vp, _sz, _vp, _i32,
                                         _i32, _vp]),
    "moe_kv_page_bytes": (_sz, [_i32, _i32, _i32, _i32]),
    "moe_rope_freqs": (ctypes.c_int, [_i32, _i32, _f64, _f64, _f64, _f64, _f64, _vp, _vp]),
    "moe_kv_append": (ctypes.c_int, [_CP, ctypes.POINTER(QkvDesc), _SP, _vp, _i64, _i64, _vp, _vp,
                                     _i64, _vp, _i64, _vp]),
    "moe_kv_read": (ctypes.c_int, [_CP, _SP, _vp, _vp, _i64, _vp, _i64, _vp, _i64, _vp]),
    "moe_attn_workspace_bytes": (_sz, [_CP, _i32, _i32, _i64, _i64]),
    "moe_attn_decode": (ctypes.c_int, [_CP, _SP, _i32, _vp, _i64, _i64, _i64, _f32, _vp, _i64, _vp,
                                       _sz, _vp]),
    "moe_attn_chunk_workspace_bytes": (_sz, [_CP, _i32, _i32, _i64, _i64]),
    "moe_attn_chunk": (ctypes.c_int, [_CP, _SP, _i32, _vp, _i64, _i64, _i64, _f32, _vp, _i64, _vp,
                                      _sz, _vp]),
    "moe_attn_prompt": (ctypes.c_int, [_i32, _i32, _i32, _i32, _vp, _vp, _i64, _i64, _vp, _i64, _vp,
                                       _i64, _vp, _i64, _f32, _vp, _i64, _vp]),
    "moe_add_norm": (ctypes.c_int, [_i32, _i64, _vp, _i64, _vp, _i64, _vp, _f32, _vp, _i64, _vp, _i64,
                                    _i32, _vp, _vp, _vp]),
    "moe_mx_quant": (ctypes.c_int, [_i32, _i32, _i64, _vp, _i64, _vp, _vp, _vp]),
    "moe_mx_matrix_bytes": (_sz, [_i32, _i32]),
    "moe_mx_pack": (ctypes.c_int, [_i32, _i32, _vp, _vp, _vp, _vp]),
    "moe_mx_linear": (ctypes.c_int, [_MP, _i32, _vp, _vp, _i64, _vp, _i64, _i32, _vp]),
    "moe_mx_workspace_bytes": (_sz, [_i32, _i32, _i64]),
    "moe_mx_linear_rows": (ctypes.c_int, [_MP, _i32, _vp, _i64, _i64, _vp, _i64, _i32, _vp, _sz, _vp]),
    "moe_tier_create": (ctypes.c_int, [ctypes.POINTER(TierDesc), ctypes.POINTER(ctypes.c_void_p)]),
    "moe_tier_prepare": (ctypes.c_int, [_vp, _i32, _BP, _vp, _vp]),
    "moe_tier_prepare_async": (ctypes.c_int, [_vp, _i32, _BP, _vp, _vp]),
    "moe_tier_rebalance": (ctypes.c_int, [_vp, _i32, _vp, _vp]),
    "moe_tier_stats_get": (ctypes.c_int, [_vp, ctypes.POINTER(TierStats), _i32, _vp]),
    "moe_tier_destroy": (None, [_vp]),
}

_lib = None


def lib():
    """The loaded libmoe.so (raises if it is not built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise ImportError(f"libmoe.so not built at {LIB_PATH}; run __graft_entry__.build()")
        L = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in SIGNATURES.items():
            f = getattr(L, name)
            f.restype = res
            f.argtypes = args
        _lib = L
    return _lib


def last_error() -> str:
    return lib().moe_last_error().decode()


def _check(status: int):
    if status != MOE_OK:
        raise MoeError(status, last_error())


def _ptr(t) -> int | None:
    """Device (or host) address of a tensor / int / None."""
    if t is None:
        return None
    if isinstance(t, int):
        return t
    return t.data_ptr()


def _stream(stream) -> int | None:
    if stream is None:
        import torch
        if torch.cuda.is_initialized() and hasattr(torch._C, "_cuda_getCurrentRawStream"):
            # the current stream's handle without its Python object (0.3 us, not 2.9)
            return torch._C._cuda_getCurrentRawStream(torch._C._cuda_getDevice())
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _stream_object(stream, device):
    """torch's object for a stream that may be given as a raw handle, or None: the current one."""
    import torch
    if stream is None:
        return torch.cuda.current_stream(device)
    if not isinstance(stream, int):
        return stream
    # (torch takes a handle of 0 for no handle, and makes a stream)
    return torch.cuda.ExternalStream(stream, device) if stream else torch.cuda.default_stream(device)


# ---------------------------------------------------------------- raw ABI

def moe_abi_version() -> int:
    return lib().moe_abi_version()


def moe_expert_blob_bytes(H, I, fmt_gate_up, fmt_down) -> int:
    return lib().moe_expert_blob_bytes(H, I, fmt_gate_up, fmt_down)


def moe_pack_experts(E, H, I, fmt_gate_up, fmt_down, gate_q, gate_s, up_q, up_s, down_q, down_s,
                     blobs, blob_stride, stream=None):
    _check(lib().moe_pack_experts(E, H, I, fmt_gate_up, fmt_down, _ptr(gate_q), _ptr(gate_s),
                                  _ptr(up_q), _ptr(up_s), _ptr(down_q), _ptr(down_s), _ptr(blobs),
                                  blob_stride, _stream(stream)))


def moe_buckets_bytes(E, T_max, k) -> int:
    return lib().moe_buckets_bytes(E, T_max, k)


def moe_buckets_carve(buf, nbytes, E, T_max, k) -> Buckets:
    b = Buckets()
    _check(lib().moe_buckets_carve(_ptr(buf), nbytes, E, T_max, k, ctypes.byref(b)))
    return b


def moe_workspace_bytes(desc: LayerDesc, T_max) -> int:
    return lib().moe_workspace_bytes(ctypes.byref(desc), T_max)


def moe_route(desc, x, T, logits, topk_idx, topk_w, stream=None):
    _check(lib().moe_route(ctypes.byref(desc), _ptr(x), T, _ptr(logits), _ptr(topk_idx),
                           _ptr(topk_w), _stream(stream)))


def moe_bucket(desc, topk_idx, T, buckets, ws, ws_bytes, stream=None):
    _check(lib().moe_bucket(ctypes.byref(desc), _ptr(topk_idx), T, ctypes.byref(buckets),
                            _ptr(ws), ws_bytes, _stream(stream)))


def moe_expert_ffn(desc, x, T, buckets, y, y_dtype, ws, ws_bytes, stream=None):
    _check(lib().moe_expert_ffn(ctypes.byref(desc), _ptr(x), T, ctypes.byref(buckets), _ptr(y),
                                y_dtype, _ptr(ws), ws_bytes, _stream(stream)))


def moe_expert_ffn_noalloc(desc, x, T, buckets, y, y_dtype, stream=None):
    _check(lib().moe_expert_ffn_noalloc(ctypes.byref(desc), _ptr(x), T, ctypes.byref(buckets),
                                        _ptr(y), y_dtype, _stream(stream)))


def moe_combine(desc, y, y_dtype, buckets, topk_w, T, residual, out, stream=None):
    _check(lib().moe_combine(ctypes.byref(desc), _ptr(y), y_dtype, ctypes.byref(buckets),
                             _ptr(topk_w), T, _ptr(residual), _ptr(out), _stream(stream)))


def moe_expert_hist(desc, buckets, hist, decay_shift, unit_shift, stream=None):
    _check(lib().moe_expert_hist(ctypes.byref(desc), ctypes.byref(buckets), _ptr(hist),
                                 decay_shift, unit_shift, _stream(stream)))


def moe_route_bucket(desc, x, T, logits, topk_idx, topk_w, buckets, ws, ws_bytes, hist=None,
                     decay_shift=0, unit_shift=0, stream=None):
    _check(lib().moe_route_bucket(ctypes.byref(desc), _ptr(x), T, _ptr(logits), _ptr(topk_idx),
                                  _ptr(topk_w), ctypes.byref(buckets), _ptr(ws), ws_bytes,
                                  _ptr(hist), decay_shift, unit_shift, _stream(stream)))


def moe_route_ffn(desc, x, T, logits, topk_idx, topk_w, buckets, hist, decay_shift, unit_shift,
                  y, y_dtype, ws, ws_bytes, stream=None):
    _check(lib().moe_route_ffn(ctypes.byref(desc), _ptr(x), T, _ptr(logits), _ptr(topk_idx),
                               _ptr(topk_w), ctypes.byref(buckets), _ptr(hist), decay_shift,
                               unit_shift, _ptr(y), y_dtype, _ptr(ws), ws_bytes, _stream(stream)))


def moe_layer_forward(desc, x, T, residual, out, logits, topk_idx, topk_w, buckets, hist,
                      decay_shift, unit_shift, y, y_dtype, ws, ws_bytes, stream=None):
    _check(lib().moe_layer_forward(ctypes.byref(desc), _ptr(x), T, _ptr(residual), _ptr(out),
                                   _ptr(logits), _ptr(topk_idx), _ptr(topk_w),
                                   ctypes.byref(buckets), _ptr(hist), decay_shift, unit_shift,
                                   _ptr(y), y_dtype, _ptr(ws), ws_bytes, _stream(stream)))


def moe_kv_page_bytes(fmt, n_kv, D, page_tokens) -> int:
    return lib().moe_kv_page_bytes(fmt, n_kv, D, page_tokens)


def moe_rope_freqs(kind, rot_dim, base, factor=1.0, orig_len=0.0, turns_lo=1.0, turns_hi=32.0):
    """(frequencies float64 [rot_dim/2], rope_scale) of rotary positions."""
    f, scale = np.zeros(max(rot_dim // 2, 1), np.float64), ctypes.c_float()
    _check(lib().moe_rope_freqs(kind, rot_dim, base, factor, orig_len, turns_lo, turns_hi,
                                f.ctypes.data, ctypes.addressof(scale)))
    return f, scale.value


def moe_kv_append(cache, qkv_desc, seqs, qkv, qkv_stride, T, pos, q_out, q_stride, k_out=None,
                  k_stride=0, stream=None):
    _check(lib().moe_kv_append(ctypes.byref(cache), ctypes.byref(qkv_desc), ctypes.byref(seqs),
                               _ptr(qkv), qkv_stride, T, _ptr(pos), _ptr(q_out), q_stride,
                               _ptr(k_out), k_stride, _stream(stream)))


def moe_kv_read(cache, seqs, first, out_start, R, k_out, k_stride, v_out, v_stride, stream=None):
    _check(lib().moe_kv_read(ctypes.byref(cache), ctypes.byref(seqs), _ptr(first), _ptr(out_start),
                             R, _ptr(k_out), k_stride, _ptr(v_out), v_stride, _stream(stream)))


def moe_attn_workspace_bytes(cache, n_q, n_seq, T, max_len=0) -> int:
    return lib().moe_attn_workspace_bytes(ctypes.byref(cache), n_q, n_seq, T, max_len)


def moe_attn_decode(cache, seqs, n_q, q, q_stride, T, max_len, scale, out, out_stride, ws, ws_bytes,
                    stream=None):
    _check(lib().moe_attn_decode(ctypes.byref(cache), ctypes.byref(seqs), n_q, _ptr(q), q_stride, T,
                                 max_len, scale, _ptr(out), out_stride, _ptr(ws), ws_bytes,
                                 _stream(stream)))


def moe_attn_chunk_workspace_bytes(cache, n_q, n_seq, T, max_len=0) -> int:
    return lib().moe_attn_chunk_workspace_bytes(ctypes.byref(cache), n_q, n_seq, T, max_len)


def moe_attn_chunk(cache, seqs, n_q, q, q_stride, T, max_len, scale, out, out_stride, ws, ws_bytes,
                   stream=None):
    _check(lib().moe_attn_chunk(ctypes.byref(cache), ctypes.byref(seqs), n_q, _ptr(q), q_stride, T,
                                max_len, scale, _ptr(out), out_stride, _ptr(ws), ws_bytes,
                                _stream(stream)))


def moe_attn_prompt(n_q, n_kv, D, n_seq, q_start, kv_start, T, Tk, q, q_stride, k, k_stride, v,
                    v_stride, scale, out, out_stride, stream=None):
    _check(lib().moe_attn_prompt(n_q, n_kv, D, n_seq, _ptr(q_start), _ptr(kv_start), T, Tk, _ptr(q),
                                 q_stride, _ptr(k), k_stride, _ptr(v), v_stride, scale, _ptr(out),
                                 out_stride, _stream(stream)))


def moe_add_norm(H, T, x, x_stride, residual, residual_stride, weight, eps, sum, sum_stride, out,
                 out_stride, fmt=0, codes=None, scales=None, stream=None):
    _check(lib().moe_add_norm(H, T, _ptr(x), x_stride, _ptr(residual), residual_stride, _ptr(weight), eps,
                              _ptr(sum), sum_stride, _ptr(out), out_stride, fmt, _ptr(codes),
                              _ptr(scales), _stream(stream)))


def moe_mx_quant(fmt, K, T, x, x_stride, codes, scales, stream=None):
    _check(lib().moe_mx_quant(fmt, K, T, _ptr(x), x_stride, _ptr(codes), _ptr(scales), _stream(stream)))


def moe_mx_matrix_bytes(N, K) -> int:
    return lib().moe_mx_matrix_bytes(N, K)


def moe_mx_pack(N, K, codes, scales, packed, stream=None):
    _check(lib().moe_mx_pack(N, K, _ptr(codes), _ptr(scales), _ptr(packed), _stream(stream)))


def moe_mx_linear(w, fmt, codes, scales, T, y, y_stride, y_dtype, stream=None):
    _check(lib().moe_mx_linear(ctypes.byref(w), fmt, _ptr(codes), _ptr(scales), T, _ptr(y), y_stride,
                               y_dtype, _stream(stream)))


def moe_mx_workspace_bytes(fmt, K, T) -> int:
    return lib().moe_mx_workspace_bytes(fmt, K, T)


def moe_mx_linear_rows(w, fmt, x, x_stride, T, y, y_stride, y_dtype, ws, ws_bytes, stream=None):
    _check(lib().moe_mx_linear_rows(ctypes.byref(w), fmt, _ptr(x), x_stride, T, _ptr(y), y_stride, y_dtype,
                                    _ptr(ws), ws_bytes, _stream(stream)))


def moe_tier_create(desc: TierDesc) -> int:
    h = ctypes.c_void_p()
    _check(lib().moe_tier_create(ctypes.byref(desc), ctypes.byref(h)))
    return h.value


def moe_tier_prepare(tier, layer, buckets, table_dev, stream=None):
    _check(lib().moe_tier_prepare(tier, layer, ctypes.byref(buckets), _ptr(table_dev),
                                  _stream(stream)))


def moe_tier_prepare_async(tier, layer, buckets, table_dev, stream=None):
    _check(lib().moe_tier_prepare_async(tier, layer, ctypes.byref(buckets), _ptr(table_dev),
                                        _stream(stream)))


def moe_tier_rebalance(tier, layer, hist, stream=None):
    _check(lib().moe_tier_rebalance(tier, layer, _ptr(hist), _stream(stream)))


def moe_tier_stats_get(tier, layer=0, R=0):
    st = TierStats()
    res = np.zeros(max(R, 1), np.int32)
    _check(lib().moe_tier_stats_get(tier, ctypes.byref(st), layer,
                                    res.ctypes.data if R else None))
    return {n: getattr(st, n) for n, _ in TierStats._fields_}, res[:R]


def moe_tier_destroy(tier):
    lib().moe_tier_destroy(tier)


# ---------------------------------------------------------------- device plumbing

class DeviceLayer:
    """One layer's weights resident in HBM: router weights/bias, packed expert
    blobs (packed on the GPU by moe_pack_experts) and the expert table.
    ffn_mode: MOE_FFN_AUTO, _GEMV or _GEMM, carried in the layer descriptor
    (desc.ffn_mode may be changed between calls)."""

    def __init__(self, w, device="cuda", stream=None, ffn_mode=MOE_FFN_AUTO):
        import torch
        self.E, self.k, self.H, self.I = w.E, w.k, w.H, w.I
        self.fmt_down = w.fmt_down
        dev = torch.device(device)
        t = lambda a: torch.from_numpy(np.ascontiguousarray(a)).to(dev)  # noqa: E731
        self.w_router = t(w.w_router)
        self.bias = None if w.bias is None else t(w.bias)
        self.blob_bytes = moe_expert_blob_bytes(self.H, self.I, MOE_FMT_NVFP4, self.fmt_down)
        if self.blob_bytes == 0:
            raise MoeError(MOE_ERR_UNSUPPORTED, last_error())
        self.blobs = torch.empty(self.E * self.blob_bytes, dtype=torch.uint8, device=dev)
        canon = [t(a) if a is not None else None
                 for a in (w.gate_q, w.gate_s, w.up_q, w.up_s, w.down_q, w.down_s)]
        moe_pack_experts(self.E, self.H, self.I, MOE_FMT_NVFP4, self.fmt_down, *canon,
                         self.blobs, self.blob_bytes, stream)
        refs = np.zeros(self.E, dtype=[("blob", "<u8"), ("tg", "<f4"), ("tu", "<f4"),
                                       ("td", "<f4"), ("r", "<u4")])
        base = self.blobs.data_ptr()
        refs["blob"] = base + np.arange(self.E, dtype=np.uint64) * self.blob_bytes
        refs["tg"] = w.gate_ts
        refs["tu"] = w.up_ts
        refs["td"] = w.down_ts if w.down_ts is not None else 1.0
        self.refs = t(refs.view(np.uint8))
        _stream_object(stream, dev).synchronize()
        del canon
        self.desc = LayerDesc(self.E, self.k, self.H, self.I, MOE_FMT_NVFP4, self.fmt_down,
                              w.renormalize, ffn_mode, self.refs.data_ptr(), self.w_router.data_ptr(),
                              None if self.bias is None else self.bias.data_ptr())


class StepBuffers:
    """Per-step device buffers for up to T_max tokens of a layer."""

    def __init__(self, layer: DeviceLayer, T_max: int, y_dtype=MOE_DTYPE_F32, device="cuda"):
        import torch
        dev = torch.device(device)
        E, k, H = layer.E, layer.k, layer.H
        self.T_max = T_max
        self.y_dtype = y_dtype
        self.logits = torch.empty((T_max, E), dtype=torch.float32, device=dev)
        self.idx = torch.empty((T_max, k), dtype=torch.int32, device=dev)
        self.w = torch.empty((T_max, k), dtype=torch.float32, device=dev)
        nb = moe_buckets_bytes(E, T_max, k)
        self.bucket_buf = torch.zeros(nb, dtype=torch.uint8, device=dev)
        self.buckets = moe_buckets_carve(self.bucket_buf, nb, E, T_max, k)
        self.ws_bytes = moe_workspace_bytes(layer.desc, T_max)
        self.ws = torch.empty(self.ws_bytes, dtype=torch.uint8, device=dev)
        ydt = torch.float32 if y_dtype == MOE_DTYPE_F32 else torch.bfloat16
        self.y = torch.empty((max(T_max * k, 1), H), dtype=ydt, device=dev)
        self.out = torch.empty((T_max, H), dtype=torch.int16, device=dev)
        self.hist = torch.zeros(E, dtype=torch.int32, device=dev)

    def counts_view(self, E: int):
        """The per-expert assignment counts of the last step as an int32
        device tensor view [E] (no copy)."""
        import torch
        off = self.buckets.counts - self.bucket_buf.data_ptr()
        return self.bucket_buf[off:off + 4 * E].view(torch.int32)

    def bucket_view(self, E: int, T: int, k: int) -> dict:
        """Host copies of the bucket outputs of the last step (synchronizes)."""
        b = self.bucket_buf.cpu().numpy()
        base = self.bucket_buf.data_ptr()

        def arr(ptr, n, dt):
            off = ptr - base
            return b[off: off + n * 4].view(dt).copy()
        bk = self.buckets
        A = T * k
        n_active = int(arr(bk.n_active, 1, np.int32)[0])
        return dict(counts=arr(bk.counts, E, np.uint32), offsets=arr(bk.offsets, E + 1, np.int32),
                    sorted_asg=arr(bk.sorted_asg, A, np.int32),
                    asg_pos=arr(bk.asg_pos, A, np.int32),
                    active=arr(bk.active, E, np.int32)[:n_active], n_active=n_active)


def layer_forward(layer: DeviceLayer, buf: StepBuffers, x, T: int, residual=None,
                  hist_shifts=(5, 10), stream=None, fused_gating=True, keep_y=True):
    """One pass of the layer: route, bucket, expert FFN, combine, histogram.
    fused_gating: one moe_route_ffn call (routing, gating, buckets, histogram
    and the expert FFN) in place of moe_route + moe_bucket + moe_expert_ffn +
    moe_expert_hist.  keep_y=False (with fused_gating): one moe_layer_forward
    call, which for decode batches fuses the down projection with the
    combine and leaves buf.y unwritten."""
    d = layer.desc
    if fused_gating and not keep_y:
        h = None if hist_shifts is None else buf.hist
        ds, us = (0, 0) if hist_shifts is None else hist_shifts
        moe_layer_forward(d, x, T, residual, buf.out, buf.logits, buf.idx, buf.w, buf.buckets, h,
                          ds, us, buf.y, buf.y_dtype, buf.ws, buf.ws_bytes, stream)
        return buf.out
    if fused_gating:
        h = None if hist_shifts is None else buf.hist
        ds, us = (0, 0) if hist_shifts is None else hist_shifts
        moe_route_ffn(d, x, T, buf.logits, buf.idx, buf.w, buf.buckets, h, ds, us, buf.y,
                      buf.y_dtype, buf.ws, buf.ws_bytes, stream)
    else:
        moe_route(d, x, T, buf.logits, buf.idx, buf.w, stream)
        moe_bucket(d, buf.idx, T, buf.buckets, buf.ws, buf.ws_bytes, stream)
        moe_expert_ffn(d, x, T, buf.buckets, buf.y, buf.y_dtype, buf.ws, buf.ws_bytes, stream)
    moe_combine(d, buf.y, buf.y_dtype, buf.buckets, buf.w, T, residual, buf.out, stream)
    if hist_shifts is not None and not fused_gating:
        moe_expert_hist(d, buf.buckets, buf.hist, hist_shifts[0], hist_shifts[1], stream)
    return buf.out


class KvCache:
    """A layer's paged key/value cache in HBM (n_pages pages of page_tokens
    tokens; fmt MOE_FMT_NVFP4, _Q8_0 or _BF16), with the norm weights and rotary
    frequencies of its layer: q_norm, k_norm float32 [D] or None, rope a pair
    (frequencies, scale) as moe_rope_freqs returns it, or None."""

    def __init__(self, fmt, n_q, n_kv, D, page_tokens, n_pages, q_norm=None, k_norm=None, rope=None,
                 interleaved=0, eps=1e-6, k_scale=1.0, v_scale=1.0, device="cuda"):
        import torch
        dev = torch.device(device)
        self.n_q, self.n_kv, self.D = n_q, n_kv, D
        self.page_bytes = moe_kv_page_bytes(fmt, n_kv, D, page_tokens)
        if self.page_bytes == 0:
            raise MoeError(MOE_ERR_UNSUPPORTED, last_error())
        self.pool = torch.empty(n_pages * self.page_bytes, dtype=torch.uint8, device=dev)
        t = lambda a, dt: None if a is None else torch.as_tensor(a, dtype=dt, device=dev).contiguous()  # noqa: E731
        self.q_norm, self.k_norm = t(q_norm, torch.float32), t(k_norm, torch.float32)
        for name, w in (("q_norm", self.q_norm), ("k_norm", self.k_norm)):
            if w is not None and w.numel() != D:
                raise MoeError(MOE_ERR_INVALID_ARG, f"KvCache: {name} has {w.numel()} weights, not D={D}")
        freqs, scale = (None, 1.0) if rope is None else rope
        self.inv_freq = t(freqs, torch.float64)
        rot = 0 if freqs is None else 2 * len(freqs)
        self.desc = KvCacheDesc(fmt, n_kv, D, page_tokens, n_pages, k_scale, v_scale,
                                self.pool.data_ptr())
        self.qkv_desc = QkvDesc(n_q, eps, _ptr(self.q_norm), _ptr(self.k_norm), rot, interleaved,
                                _ptr(self.inv_freq), scale)


class AttnBuffers:
    """Per-step device buffers for up to T_max rows of n_seq sequences with page
    tables of max_pages pages; the host fills row_start, kv_len and page_table
    (int32 device tensors) before a step.  chunk: with the workspace of
    attention_forward's chunk steps."""

    def __init__(self, cache: KvCache, n_seq: int, T_max: int, max_pages: int, device="cuda", chunk=False):
        import torch
        dev = torch.device(device)
        self.T_max = T_max
        self.heads = (cache.n_q, cache.n_kv, cache.D)
        i32 = lambda *shape: torch.zeros(shape, dtype=torch.int32, device=dev)  # noqa: E731
        bf16 = lambda heads: torch.empty((T_max, heads * cache.D), dtype=torch.bfloat16, device=dev)  # noqa: E731
        self.row_start, self.kv_len, self.page_table = i32(n_seq + 1), i32(n_seq), i32(n_seq, max_pages)
        self.seqs = SeqBatch(n_seq, max_pages, self.row_start.data_ptr(), self.kv_len.data_ptr(),
                             self.page_table.data_ptr())
        self.max_len = max_pages * cache.desc.page_tokens
        self.q, self.k, self.out = bf16(cache.n_q), bf16(cache.n_kv), bf16(cache.n_q)
        self.ws_bytes = moe_attn_workspace_bytes(cache.desc, cache.n_q, n_seq, T_max, self.max_len)
        self.chunk_bytes = moe_attn_chunk_workspace_bytes(cache.desc, cache.n_q, n_seq, T_max, self.max_len) if chunk else None
        self.ws = torch.empty(max(self.ws_bytes, self.chunk_bytes or 0, 1), dtype=torch.uint8, device=dev)
        self.spans = _spans(self.q, self.k, self.out, self.ws)


def _check_rows(t, numel, device, name, call="attention_forward", other="the cache"):
    """t: contiguous bf16 values (or their bits) on the device of `other`, numel
    of them or more.  (An address cannot be checked.)"""
    import torch
    if isinstance(t, int):
        return
    if t.dtype not in (torch.bfloat16, torch.int16, torch.uint16) or not t.is_contiguous():
        raise MoeError(MOE_ERR_INVALID_ARG, f"{call}: {name} must be bf16 and contiguous")
    if t.numel() < numel:
        raise MoeError(MOE_ERR_INVALID_ARG, f"{call}: {name} has {t.numel()} elements of {numel}")
    if t.device != device:
        raise MoeError(MOE_ERR_INVALID_ARG, f"{call}: {name} is on {t.device}, {other} on {device}")


def _spans(*tensors):
    """The addresses that contiguous tensors lie at: (first, past the last) of each."""
    return [(t.data_ptr(), t.data_ptr() + t.numel() * t.element_size()) for t in tensors]


def _launches_on(device, stream):
    """Whether a call's kernels run on this device: the stream's, or the current
    one if no stream is given.  (A raw handle does not tell.)"""
    import torch
    if device.type != "cuda":
        return False
    if stream is None:
        return device.index == torch.cuda.current_device()
    return getattr(stream, "device", device) == device


def attention_forward(cache: KvCache, buf: AttnBuffers, qkv, T: int, scale: float, prompt=None,
                      max_len=0, stream=None, chunk=False):
    """One layer's attention over the step's rows qkv (bf16 [T][n_q + 2 n_kv][D],
    the projections' output): norms, rotation and cache write, then attention
    over the cache.  prompt: None for decode and verification steps; for
    prompts kv_start (int32 device [n_seq + 1], the running sum of kv_len), the
    total Tk and buffers k, v (bf16 [Tk][n_kv][D]) as a tuple: the keys and
    values, those cached earlier included, are read back into k, v first, so
    that every chunk of a prompt attends to what the cache holds.  chunk, in
    place of prompt: the same straight over the cache, without k and v
    (buffers made with chunk=True; decode rows of other slots may be among the
    step's).  The answers are the same but for rounding.  Time (32 query and 4
    key/value heads of 128, NVFP4): with neither, a few rows a sequence, up to
    some 128 behind 8192 tokens, are the fastest (8 slots of one row behind 16000
    22 us, chunk 51, prompt 301); chunk is for more rows behind a long cache (512
    behind 8192: 99 us, else 118, prompt 133), alone or among decode rows; prompt
    for thousands of rows (4096 behind 12288: 775 us, chunk 897; 2048 behind none:
    53 us, else 67, chunk 86)."""
    c, D = cache.desc, cache.D
    qw, kw = cache.n_q * D, cache.n_kv * D
    if chunk and prompt is not None:
        raise MoeError(MOE_ERR_INVALID_ARG, "attention_forward: chunk steps take no prompt buffers")
    if chunk and buf.chunk_bytes is None:
        raise MoeError(MOE_ERR_INVALID_ARG, "attention_forward: buffers made without chunk=True")
    if T > buf.T_max:
        raise MoeError(MOE_ERR_INVALID_ARG, f"attention_forward: T={T} > T_max={buf.T_max}")
    if prompt is not None and min(prompt[2].numel(), prompt[3].numel()) < prompt[1] * kw:
        raise MoeError(MOE_ERR_INVALID_ARG, f"attention_forward: k, v are smaller than Tk={prompt[1]} rows")
    if buf.heads != (cache.n_q, cache.n_kv, D):
        raise MoeError(MOE_ERR_INVALID_ARG, f"attention_forward: buffers for heads {buf.heads}, "
                       f"the cache has {(cache.n_q, cache.n_kv, D)}")
    dev = cache.pool.device
    _check_rows(qkv, T * (qw + 2 * kw), dev, "qkv")
    if prompt is not None:
        import torch
        start = prompt[0]
        if start.dtype != torch.int32 or start.numel() <= buf.seqs.n_seq or not start.is_contiguous() or start.device != dev:
            raise MoeError(MOE_ERR_INVALID_ARG, f"attention_forward: kv_start must be int32 [{buf.seqs.n_seq + 1}] on {dev}")
        _check_rows(prompt[2], prompt[1] * kw, dev, "k")
        _check_rows(prompt[3], prompt[1] * kw, dev, "v")
    if buf.q.device != dev:
        raise MoeError(MOE_ERR_INVALID_ARG, f"attention_forward: buffers on {buf.q.device}, the cache on {dev}")
    if T > 0 and not _launches_on(dev, stream):
        raise MoeError(MOE_ERR_INVALID_ARG, f"attention_forward: the cache is on {dev}, not the current GPU or the stream's")
    moe_kv_append(c, cache.qkv_desc, buf.seqs, qkv, qw + 2 * kw, T, None, buf.q, qw, buf.k, kw, stream)
    if chunk:
        moe_attn_chunk(c, buf.seqs, cache.n_q, buf.q, qw, T, max_len, scale, buf.out, qw, buf.ws,
                       buf.chunk_bytes, stream)
    elif prompt is None:
        moe_attn_decode(c, buf.seqs, cache.n_q, buf.q, qw, T, max_len, scale, buf.out, qw, buf.ws,
                        buf.ws_bytes, stream)
    else:
        kv_start, Tk, k, v = prompt
        moe_kv_read(c, buf.seqs, None, kv_start, Tk, k, kw, v, kw, stream)
        moe_attn_prompt(cache.n_q, cache.n_kv, D, buf.seqs.n_seq, buf.row_start, kv_start, T, Tk,
                        buf.q, qw, k, kw, v, kw, scale, buf.out, qw, stream)
    return buf.out


class MxLinear:
    """A dense projection's weights in 4-bit microscaled form, packed for
    moe_mx_linear: from bf16 weight [N][K] on the GPU (quantised there), or from
    codes uint8 [N][K/2] with scales uint8 [N][K/32].  bias: float32 [N] or None."""

    def __init__(self, weight, scales=None, bias=None, stream=None):
        import torch
        bad = lambda msg: MoeError(MOE_ERR_INVALID_ARG, f"MxLinear: {msg}")  # noqa: E731
        if weight.dim() != 2 or not weight.is_contiguous():
            raise bad("weight must be [N][K] and contiguous")
        if weight.dtype != (torch.bfloat16 if scales is None else torch.uint8):
            raise bad("weight must be bf16 without scales and uint8 codes with them")
        dev = weight.device
        N, K = weight.shape[0], weight.shape[1] * (1 if scales is None else 2)
        nb = moe_mx_matrix_bytes(N, K)
        if nb == 0:
            raise MoeError(MOE_ERR_UNSUPPORTED, last_error())
        if scales is not None and (scales.dtype != torch.uint8 or tuple(scales.shape) != (N, K // 32) or
                                   not scales.is_contiguous() or scales.device != dev):
            raise bad(f"scales must be uint8 [{N}][{K // 32}] on {dev}")
        if bias is not None and (bias.dtype != torch.float32 or tuple(bias.shape) != (N,) or
                                 not bias.is_contiguous() or bias.device != dev):
            raise bad(f"bias must be float32 [{N}] on {dev}")
        if not _launches_on(dev, stream):
            raise bad(f"weight is on {dev}, not the current GPU or the stream's")
        self.N, self.K, self.device = N, K, dev
        self.packed = torch.empty(nb, dtype=torch.uint8, device=dev)
        codes, quantise = weight, scales is None
        if quantise:
            codes = torch.empty((N, K // 2), dtype=torch.uint8, device=dev)
            scales = torch.empty((N, K // 32), dtype=torch.uint8, device=dev)
        # The current stream may still be writing weight, and using the memory that its allocator
        # has just handed out again.
        stream = _stream_object(stream, dev)
        stream.wait_stream(torch.cuda.current_stream(dev))
        if quantise:
            moe_mx_quant(MOE_FMT_MXFP4, K, N, weight, K, codes, scales, stream)
        moe_mx_pack(N, K, codes, scales, self.packed, stream)
        stream.synchronize()
        self.bias = bias
        self.mat = MxMatrix(N, K, self.packed.data_ptr(), None if bias is None else bias.data_ptr())


class BlockWeights:
    """What stands around a layer's attention and experts: the norms before them
    (float32 [H]), the projections qkv (MxLinear H -> (n_q + 2 n_kv) D) and out
    (n_q D -> H), and the form fmt that rows take before a projection
    (MOE_FMT_MXFP8 or MOE_FMT_MXFP4)."""

    def __init__(self, attn_norm, qkv: MxLinear, out: MxLinear, ffn_norm, eps=1e-6, fmt=MOE_FMT_MXFP8):
        import torch
        bad = lambda msg: MoeError(MOE_ERR_INVALID_ARG, f"BlockWeights: {msg}")  # noqa: E731
        H, dev = qkv.K, qkv.device
        if fmt not in (MOE_FMT_MXFP4, MOE_FMT_MXFP8):
            raise bad(f"fmt {fmt} is no form of rows")
        if out.N != H or out.device != dev:
            raise bad(f"out gives {out.N} values on {out.device}, qkv takes {H} on {dev}")
        for name, w in (("attn_norm", attn_norm), ("ffn_norm", ffn_norm)):
            if w.dtype != torch.float32 or tuple(w.shape) != (H,) or not w.is_contiguous() or w.device != dev:
                raise bad(f"{name} must be float32 [{H}] on {dev}")
        self.H, self.device, self.eps, self.fmt = H, dev, eps, fmt
        self.attn_norm, self.ffn_norm, self.qkv, self.out = attn_norm, ffn_norm, qkv, out


class BlockBuffers:
    """Per-step device buffers of block_forward for up to T_max rows."""

    def __init__(self, w: BlockWeights, T_max: int):
        import torch
        u8 = lambda *shape: torch.empty(shape, dtype=torch.uint8, device=w.device)  # noqa: E731
        bf16 = lambda n: torch.empty((T_max, n), dtype=torch.bfloat16, device=w.device)  # noqa: E731
        self.T_max, self.shape = T_max, (w.H, w.qkv.N, w.out.K, w.fmt)
        self.codes = u8(T_max, w.H if w.fmt == MOE_FMT_MXFP8 else w.H // 2)
        self.scales = u8(T_max, w.H // 32)
        self.qkv, self.proj, self.sum, self.z = bf16(w.qkv.N), bf16(w.H), bf16(w.H), bf16(w.H)
        self.ws_bytes = moe_mx_workspace_bytes(w.fmt, w.out.K, T_max)
        self.ws = u8(max(self.ws_bytes, 1))
        self.spans = _spans(self.qkv, self.proj, self.ws)


def block_forward(w: BlockWeights, layer: DeviceLayer, cache: KvCache, buf: BlockBuffers, attn: AttnBuffers,
                  step: StepBuffers, x, T: int, scale: float, prompt=None, max_len=0, stream=None, chunk=False,
                  **layer_options):
    """One layer from residual to residual over the step's rows x (bf16 [T][H]):
      a = attention_forward(qkv(norm(x))), h = x + out(a), h + layer_forward(norm(h)),
    the norms' rows going to the projection as codes.  x is read twice: it may
    be step.out (a layer's rows from the one before), but not lie in a buffer that
    the step writes in between (buf.qkv, proj and ws, attn's, prompt's k and v).
    attn, prompt, max_len and chunk as for attention_forward, step and
    layer_options as for layer_forward.
    Returns step.out (bf16 bits [T_max][H]; the first T rows are the step's)."""
    call = "block_forward"
    bad = lambda msg: MoeError(MOE_ERR_INVALID_ARG, f"{call}: {msg}")  # noqa: E731
    H, width, kwidth = w.H, w.qkv.N, w.out.K
    if layer.H != H:
        raise bad(f"the experts' rows have {layer.H} values, the norms' {H}")
    if width != (cache.n_q + 2 * cache.n_kv) * cache.D or kwidth != cache.n_q * cache.D:
        raise bad(f"projections to {width} and from {kwidth} do not fit the cache's heads")
    if buf.shape != (H, width, kwidth, w.fmt):
        raise bad("buffers of other weights")
    if (step.out.shape[1], step.logits.shape[1], step.idx.shape[1]) != (H, layer.E, layer.k):
        raise bad("step's buffers of another layer")
    if T < 0 or T > min(buf.T_max, attn.T_max, step.T_max):
        raise bad(f"T={T} for buffers of {buf.T_max}, {attn.T_max} and {step.T_max} rows")
    dev = cache.pool.device
    for name, d in (("weights", w.device), ("buffers", buf.z.device), ("experts", layer.blobs.device),
                    ("step's buffers", step.out.device)):
        if d != dev:
            raise bad(f"the {name} are on {d}, the cache on {dev}")
    _check_rows(x, T * H, dev, "x", call)
    lo = _ptr(x)
    hi = lo + 2 * T * H
    for a, b in buf.spans + attn.spans + ([] if prompt is None else _spans(*prompt[2:])):
        if a < hi and lo < b:
            raise bad("x lies in a buffer that the step writes before it reads x again")
    if T > 0 and not _launches_on(dev, stream):
        raise bad(f"the cache is on {dev}, not the current GPU or the stream's")
    moe_add_norm(H, T, x, H, None, 0, w.attn_norm, w.eps, None, 0, None, 0, w.fmt, buf.codes, buf.scales, stream)
    moe_mx_linear(w.qkv.mat, w.fmt, buf.codes, buf.scales, T, buf.qkv, width, MOE_DTYPE_BF16, stream)
    a = attention_forward(cache, attn, buf.qkv, T, scale, prompt, max_len, stream, chunk)
    moe_mx_linear_rows(w.out.mat, w.fmt, a, kwidth, T, buf.proj, H, MOE_DTYPE_BF16, buf.ws, buf.ws_bytes, stream)
    moe_add_norm(H, T, buf.proj, H, x, H, w.ffn_norm, w.eps, buf.sum, H, buf.z, H, 0, None, None, stream)
    return layer_forward(layer, step, buf.z, T, buf.sum, stream=stream, **layer_options)
