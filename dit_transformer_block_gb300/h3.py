"""ctypes binding of libh3block.so (argument marshalling only).

Every function takes torch tensors that already live on the current CUDA
device, passes their data pointers and sizes to the C entry point of the same
name (h3_<name>) and raises H3Error when the call returns a non-OK status.
All compute happens in the library's kernels; there is no fallback: if the
library is missing, the first call raises.
"""
from __future__ import annotations

import ctypes
import os
import re

import torch

PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(PKG, "libh3block.so")
HEADER = os.path.join(os.path.dirname(PKG), "include", "h3block.h")

H3_OK = 0
STATUS = {0: "H3_OK", 1: "H3_ERR_INVALID_ARG", 2: "H3_ERR_UNSUPPORTED", 3: "H3_ERR_MISALIGNED",
          4: "H3_ERR_WORKSPACE", 5: "H3_ERR_CUDA", 6: "H3_ERR_TIMEOUT"}


class H3Error(RuntimeError):
    def __init__(self, fn: str, status: int, msg: str):
        super().__init__(f"h3_{fn}: {STATUS.get(status, status)}: {msg}")
        self.status = status
        self.msg = msg


class BlockConfig(ctypes.Structure):
    _fields_ = [("S", ctypes.c_int), ("L", ctypes.c_int), ("D", ctypes.c_int), ("H", ctypes.c_int),
                ("Dh", ctypes.c_int), ("F", ctypes.c_int), ("axis_dims", ctypes.c_int * 3),
                ("theta", ctypes.c_float), ("eps_ln", ctypes.c_float), ("eps_qk", ctypes.c_float),
                ("rope_pairing", ctypes.c_int)]


class BlockWeightsFp8(ctypes.Structure):
    _fields_ = [("w_qkv", ctypes.c_void_p), ("s_qkv", ctypes.c_void_p),
                ("w_o", ctypes.c_void_p), ("s_o", ctypes.c_void_p),
                ("w_gu", ctypes.c_void_p), ("s_gu", ctypes.c_void_p),
                ("w_down", ctypes.c_void_p), ("s_down", ctypes.c_void_p),
                ("q_gain", ctypes.c_void_p), ("k_gain", ctypes.c_void_p)]


class BlockWeights(ctypes.Structure):
    _fields_ = [("w_qkv", ctypes.c_void_p), ("w_o", ctypes.c_void_p), ("w_gu", ctypes.c_void_p),
                ("w_down", ctypes.c_void_p), ("q_gain", ctypes.c_void_p),
                ("k_gain", ctypes.c_void_p)]


class KvCache(ctypes.Structure):
    device = None  # of the tensors, where kv_cache made it

    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("num_pages", ctypes.c_int),
                ("page_size", ctypes.c_int), ("Hkv", ctypes.c_int), ("Dh", ctypes.c_int)]


class KvBatch(ctypes.Structure):
    device = None

    _fields_ = [("T", ctypes.c_int), ("B", ctypes.c_int), ("max_pages", ctypes.c_int),
                ("cu_q", ctypes.c_void_p), ("kv_len", ctypes.c_void_p),
                ("page_table", ctypes.c_void_p)]


_P, _I, _F, _U64, _SZ = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_uint64, ctypes.c_size_t
_I64 = ctypes.c_int64
_SIGS = {
    "h3_version": (_I, []),
    "h3_last_error": (ctypes.c_char_p, []),
    "h3_status_string": (ctypes.c_char_p, [_I]),
    "h3_check_device_error": (_I, [_P]),
    "h3_set_wait_timeout_ns": (None, [_U64]),
    "h3_mod_norm_residual": (_I, [_P, _P, _P, _P, _P, _P, _I, _I, _I, _F, _P]),
    "h3_qk_norm_rope": (_I, [_P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _F, _F, _P]),
    "h3_attention_varlen": (_I, [_P, _P, _P, _P, _I, _I, _I, _I, _F, _P]),
    "h3_swiglu": (_I, [_P, _P, _I, _I, _I, _P]),
    "h3_sage_scratch_bytes": (_SZ, [_I, _I]),
    "h3_sage_quantize": (_I, [_P, _P, _P, _I, _I, _I, _I, _P, _P, _P, _P, _P, _P, _P, _P, _SZ,
                              _P]),
    "h3_attention_fp8": (_I, [_P, _P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _F, _P]),
    "h3_attention_fp8_skip": (_I, [_P, _P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _F, _F, _P, _P]),
    "h3_attention_varlen_skip": (_I, [_P, _P, _P, _P, _I, _I, _I, _I, _F, _F, _P, _P]),
    "h3_linear": (_I, [_P, _P, _P, _I, _I, _I, _I, _P]),
    "h3_linear_swiglu": (_I, [_P, _P, _P, _I, _I, _I, _I, _P]),
    "h3_rope_table": (_I, [_P, _P, _I, _I, _F, _P, _P]),
    "h3_linear_qk_norm_rope": (_I, [_P, _P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _F, _P]),
    "h3_qk_norm_rope_layout": (_I, [_P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _F, _F, _I, _P]),
    "h3_linear_residual": (_I, [_P, _P, _P, _P, _I, _I, _I, _I, _P]),
    "h3_block_workspace_bytes": (_SZ, [ctypes.POINTER(BlockConfig)]),
    "h3_block_forward": (_I, [ctypes.POINTER(BlockConfig), ctypes.POINTER(BlockWeights), _P, _P,
                              _P, _P, _SZ, _P]),
    "h3_block_forward_events": (_I, [ctypes.POINTER(BlockConfig), ctypes.POINTER(BlockWeights),
                                     _P, _P, _P, _P, _SZ, _P, ctypes.POINTER(_P), _I]),
    "h3_block_forward_noalloc": (_I, [ctypes.POINTER(BlockConfig), ctypes.POINTER(BlockWeights),
                                      _P, _P, _P, _P]),
    "h3_debug_wait_timeout": (_I, [_U64, _P]),
    "h3_mod_norm_residual_seg": (_I, [_P, _P, _P, _P, _P, _P, _I, ctypes.c_int64, _P, _I, _I, _I,
                                      _F, _P]),
    "h3_frames_to_u8": (_I, [_P, _P, _I, _I, _I, _I, _I, _P]),
    "h3_quantize_fp8_rows": (_I, [_P, _P, _P, _I, _I, _P]),
    "h3_linear_fp8": (_I, [_P, _P, _P, _P, _P, _I, _I, _I, _I, _P]),
    "h3_linear_swiglu_fp8": (_I, [_P, _P, _P, _P, _P, _I, _I, _I, _I, _P]),
    "h3_block_workspace_bytes_fp8": (_SZ, [ctypes.POINTER(BlockConfig)]),
    "h3_block_forward_fp8": (_I, [ctypes.POINTER(BlockConfig), ctypes.POINTER(BlockWeightsFp8),
                                  _P, _P, _P, _I, _P, _SZ, _P]),
    "h3_kv_append_paged": (_I, [_P, _I64, _P, _I64, _P, _I64, _P, _I, _P, _P, _P, _P, _I, _F, _F,
                                _P, _P, _P]),
    "h3_attention_paged_workspace_bytes": (_SZ, [_I, _I, _I]),
    "h3_attention_paged": (_I, [_P, _I64, _P, _I64, _I, _F, _I, _P, _P, _P, _SZ, _P]),
    "h3_attention_paged_prefix": (_I, [_P, _I64, _P, _I64, _I, _F, _I, _P, _P, _P, _I, _P, _SZ,
                                       _P]),
    "h3_sandwich_norm": (_I, [_P, _P, _P, _P, _I, _P, _P, _F, _P, _P, _P, _P, _I, _I64, _I, _I, _I,
                              _I, _F, _P]),
    "h3_fp4_scale_bytes": (_SZ, [_I, _I, _I]),
    "h3_quantize_fp4_rows": (_I, [_P, _I64, _P, _P, _P, _I, _I, _I, _P]),
    "h3_linear_fp4": (_I, [_P, _P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _P]),
    "h3_linear_swiglu_fp4": (_I, [_P, _P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _P]),
    "h3_block_scores_workspace_bytes": (_SZ, [_I, _I, _I, _I, _I]),
    "h3_block_scores": (_I, [_P, _I64, _P, _I64, _P, _I, _I, _I, _I, _I, _I, _F, _P, _SZ, _P]),
    "h3_block_select": (_I, [_P, _P, _P, _I, _I, _I, _I, _I, _P]),
    "h3_attention_blocks": (_I, [_P, _I64, _P, _I64, _P, _I64, _P, _I64, _P, _P, _I, _I, _I, _I,
                                 _I, _I, _I, _F, _P]),
    "h3_stack_forward": (_I, [ctypes.POINTER(BlockConfig), ctypes.POINTER(BlockWeights), _I, _P,
                              _P, _I, _P, _P, _P, _SZ, _P]),
}

_lib = None


def lib() -> ctypes.CDLL:
    """Load libh3block.so (built by dit_transformer_block_gb300.build)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is not built; run `python -m "
                               "dit_transformer_block_gb300.build`")
        L = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in _SIGS.items():
            f = getattr(L, name)
            f.restype = res
            f.argtypes = args
        _lib = L
    return _lib


def header_functions() -> list[str]:
    """Names of the functions include/h3block.h declares."""
    text = open(HEADER).read()
    return sorted(set(re.findall(r"^\s*(?:const\s+)?[A-Za-z_0-9]+\*?\s+\*?(h3_[a-z0-9_]+)\s*\(",
                                 text, flags=re.M)))


def last_error() -> str:
    return lib().h3_last_error().decode()


def _check(fn: str, status: int):
    if status != H3_OK:
        raise H3Error(fn, status, last_error())


def _p(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _s(stream):
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def _need(t, dtype, name):
    if t is None:
        return
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def version() -> int:
    return lib().h3_version()


def set_wait_timeout_ns(ns: int):
    lib().h3_set_wait_timeout_ns(int(ns))


def check_device_error(stream=None):
    _check("check_device_error", lib().h3_check_device_error(_s(stream)))


def debug_wait_timeout(ns: int, stream=None):
    _check("debug_wait_timeout", lib().h3_debug_wait_timeout(int(ns), _s(stream)))


def mod_norm_residual(resid, delta=None, gate=None, shift=None, scale=None, normed=None, L=None,
                      eps=1e-6, stream=None):
    """resid [S,D] f32 in/out; optional delta [S,D] bf16 + gate [D]; optional normed [S,D] bf16."""
    _need(resid, torch.float32, "resid")
    _need(delta, torch.bfloat16, "delta")
    _need(normed, torch.bfloat16, "normed")
    S, D = resid.shape
    L = S if L is None else L
    _check("mod_norm_residual", lib().h3_mod_norm_residual(
        _p(resid), _p(delta), _p(gate), _p(shift), _p(scale), _p(normed), S, L, D, eps, _s(stream)))


def mod_norm_residual_seg(resid, table, seg, delta=None, gate_idx=None, shift_idx=None,
                          scale_idx=None, normed=None, L=None, eps=1e-6, stream=None):
    """mod_norm_residual with token-group modulation: table [G, 6, D] f32,
    seg [S] int32; row i uses table[seg[i], idx] for the gate/shift/scale
    indices given (0..5), e.g. gate_idx=2, shift_idx=3, scale_idx=4."""
    _need(resid, torch.float32, "resid")
    _need(table, torch.float32, "table")
    _need(seg, torch.int32, "seg")
    S, D = resid.shape
    G = table.shape[0]
    L = S if L is None else L
    row = lambda i: None if i is None else ctypes.c_void_p(table[0, i].data_ptr())
    _check("mod_norm_residual_seg", lib().h3_mod_norm_residual_seg(
        _p(resid), _p(delta), row(gate_idx), row(shift_idx), row(scale_idx), _p(seg), G, 6 * D,
        _p(normed), S, L, D, eps, _s(stream)))


def qk_norm_rope(q, k, q_gain, k_gain, pos, axis_dims, L=None, theta=1e4, eps=1e-6, stream=None,
                 pairing=0):
    """In-place per-head RMSNorm + RoPE of q, k [S,H,Dh] bf16 (pairing 0:
    interleaved pairs, 1: split-half pairs per section)."""
    _need(q, torch.bfloat16, "q")
    _need(k, torch.bfloat16, "k")
    _need(pos, torch.int32, "pos")
    S, H, Dh = q.shape
    L = S if L is None else L
    ax = ctypes.cast((ctypes.c_int * 3)(*axis_dims), ctypes.c_void_p)
    if pairing == 0:
        _check("qk_norm_rope", lib().h3_qk_norm_rope(
            _p(q), _p(k), _p(q_gain), _p(k_gain), _p(pos), ax, S, L, H, Dh, theta, eps,
            _s(stream)))
    else:
        _check("qk_norm_rope_layout", lib().h3_qk_norm_rope_layout(
            _p(q), _p(k), _p(q_gain), _p(k_gain), _p(pos), ax, S, L, H, Dh, theta, eps, pairing,
            _s(stream)))


def attention_varlen(q, k, v, o, L=None, scale=None, stream=None):
    """o[:L] = softmax(q k^T * scale) v over keys < L; all [S,H,Dh] bf16."""
    for n, t in (("q", q), ("k", k), ("v", v), ("o", o)):
        _need(t, torch.bfloat16, n)
    S, H, Dh = q.shape
    L = S if L is None else L
    scale = Dh ** -0.5 if scale is None else scale
    _check("attention_varlen", lib().h3_attention_varlen(
        _p(q), _p(k), _p(v), _p(o), S, L, H, Dh, scale, _s(stream)))


def attention_varlen_skip(q, k, v, o, L=None, scale=None, skip_eps=0.0, kept=None, stream=None):
    """attention_varlen with Skip-Softmax tile skipping (skip_eps = 0: dense).
    kept (optional): int32 [ceil(L/128), H], receives the key tiles kept per
    (query tile, head)."""
    for n, t in (("q", q), ("k", k), ("v", v), ("o", o)):
        _need(t, torch.bfloat16, n)
    S, H, Dh = q.shape
    L = S if L is None else L
    scale = Dh ** -0.5 if scale is None else scale
    if kept is not None:
        _need(kept, torch.int32, "kept")
        if tuple(kept.shape) != ((L + 127) // 128, H):
            raise ValueError(f"kept must be [{(L + 127) // 128}, {H}]")
    _check("attention_varlen_skip", lib().h3_attention_varlen_skip(
        _p(q), _p(k), _p(v), _p(o), S, L, H, Dh, scale, skip_eps, _p(kept), _s(stream)))


def sage_quantize(q, k, v, L=None, stream=None) -> dict:
    """FP8 operands for attention_fp8 (allocated here, from torch): codes qc,
    kc, vc (uint8 [S, H, Dh]), scales sq, sk ([ceil(L/128), H]), sv and
    k_mean ([H, Dh])."""
    S, H, Dh = q.shape
    L = S if L is None else L
    dev = q.device
    nt = max(1, (L + 127) // 128)
    out = dict(qc=torch.zeros(S, H, Dh, dtype=torch.uint8, device=dev),
               kc=torch.zeros(S, H, Dh, dtype=torch.uint8, device=dev),
               vc=torch.zeros(S, H, Dh, dtype=torch.uint8, device=dev),
               sq=torch.zeros(nt, H, device=dev), sk=torch.zeros(nt, H, device=dev),
               sv=torch.zeros(H, Dh, device=dev), k_mean=torch.zeros(H, Dh, device=dev))
    nbytes = lib().h3_sage_scratch_bytes(L, H)
    scratch = torch.empty(max(nbytes, 16), dtype=torch.uint8, device=dev)
    _check("sage_quantize", lib().h3_sage_quantize(
        _p(q), _p(k), _p(v), S, L, H, Dh, _p(out["qc"]), _p(out["kc"]), _p(out["vc"]),
        _p(out["sq"]), _p(out["sk"]), _p(out["sv"]), _p(out["k_mean"]), _p(scratch), nbytes,
        _s(stream)))
    return out


def attention_fp8(ops: dict, o, L=None, scale=None, stream=None):
    """FP8 attention on sage_quantize's operands into o [S, H, Dh] bf16."""
    S, H, Dh = o.shape
    L = S if L is None else L
    scale = Dh ** -0.5 if scale is None else scale
    _check("attention_fp8", lib().h3_attention_fp8(
        _p(ops["qc"]), _p(ops["kc"]), _p(ops["vc"]), _p(ops["sq"]), _p(ops["sk"]),
        _p(ops["sv"]), _p(o), S, L, H, Dh, scale, _s(stream)))


def attention_fp8_skip(ops: dict, o, L=None, scale=None, skip_eps=0.0, kept=None, stream=None):
    """attention_fp8 with Skip-Softmax tile skipping on the FP8 logits
    (skip_eps = 0: attention_fp8 bit for bit). kept (optional): int32
    [ceil(L/128), H], receives the key tiles kept per (query tile, head)."""
    S, H, Dh = o.shape
    L = S if L is None else L
    scale = Dh ** -0.5 if scale is None else scale
    if kept is not None:
        _need(kept, torch.int32, "kept")
        if tuple(kept.shape) != ((L + 127) // 128, H):
            raise ValueError(f"kept must be [{(L + 127) // 128}, {H}]")
    _check("attention_fp8_skip", lib().h3_attention_fp8_skip(
        _p(ops["qc"]), _p(ops["kc"]), _p(ops["vc"]), _p(ops["sq"]), _p(ops["sk"]),
        _p(ops["sv"]), _p(o), S, L, H, Dh, scale, skip_eps, _p(kept), _s(stream)))


# The paged calls run once per layer and token: their checks are kept to a few
# attribute reads, and the device and stream are asked for by number.
_INT3 = ctypes.c_int * 3
_AXES = {}  # axis_dims as the library takes them


def _device() -> int:
    return torch._C._cuda_getDevice() if torch.cuda.is_initialized() else -1


def _on(t, name, dev):
    if t.get_device() != dev or dev < 0:
        raise ValueError(f"{name} must be on the current CUDA device, is on {t.device}")


def _raw_stream(stream, dev):
    return torch._C._cuda_getCurrentRawStream(dev) if stream is None else stream.cuda_stream


def _made_on(cache, batch, dev):
    if cache.device != dev and cache.device is not None:
        raise ValueError(f"the cache must be on the current CUDA device, is on device {cache.device}")
    if batch.device != dev and batch.device is not None:
        raise ValueError(f"the batch must be on the current CUDA device, is on device {batch.device}")


def _heads(t, name, T, dev):
    """Row stride and heads of a [T, heads, 128] bf16 tensor whose rows may be
    strided (columns of a merged projection's output)."""
    if t.dtype is not torch.bfloat16:
        raise TypeError(f"{name} must be {torch.bfloat16}, got {t.dtype}")
    shape = t.shape
    if len(shape) != 3 or shape[2] != 128 or shape[0] != T:
        raise ValueError(f"{name} must be [{T}, heads, 128], got {list(shape)}")
    ld, head, one = t.stride()
    heads = shape[1]
    if one != 1 or (head != 128 and heads > 1):
        raise ValueError(f"the heads of a row of {name} must be contiguous")
    if t.get_device() != dev or dev < 0:
        _on(t, name, dev)
    return (ld if T > 1 else heads * 128), heads


def _flat(t, name, dtype, dev):
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    _on(t, name, dev)


def _gain(g, dev):
    _flat(g, "a gain", torch.float32, dev)
    if g.numel() != 128:
        raise ValueError(f"a gain must have 128 values, has {g.numel()}")
    return g.data_ptr()


def kv_cache(k, v) -> KvCache:
    """A paged key/value cache on k, v [num_pages, Hkv, page_size, 128] bf16,
    for kv_append_paged and attention_paged; it holds on to both tensors."""
    dev = _device()
    for n, t in (("k", k), ("v", v)):
        _flat(t, n, torch.bfloat16, dev)
    if k.dim() != 4 or k.shape != v.shape:
        raise ValueError(f"k and v must both be [num_pages, Hkv, page_size, 128], got "
                         f"{list(k.shape)} and {list(v.shape)}")
    c = KvCache(k.data_ptr(), v.data_ptr(), k.shape[0], k.shape[2], k.shape[1], k.shape[3])
    c.tensors, c.device = (k, v), dev
    return c


def kv_batch(cu_q, kv_len, page_table, T: int) -> KvBatch:
    """The rows of a call (T of them, sequence b's being [cu_q[b], cu_q[b+1]))
    and their sequences: cu_q [B+1], kv_len [B] (with the call's rows in it),
    page_table [B, max_pages], int32 on the device. It holds on to the tensors,
    whose values are read when a call runs; one batch serves every layer. The
    attention's kernel is chosen by max_pages * page_size: a table no wider than the
    sequences can get is faster where they are short."""
    dev = _device()
    for n, t in (("cu_q", cu_q), ("kv_len", kv_len), ("page_table", page_table)):
        _flat(t, n, torch.int32, dev)
    B = kv_len.shape[0]
    if cu_q.shape != (B + 1,) or kv_len.dim() != 1 or page_table.dim() != 2 \
            or page_table.shape[0] != B:
        raise ValueError(f"cu_q [B+1], kv_len [B], page_table [B, max_pages] wanted, got "
                         f"{list(cu_q.shape)}, {list(kv_len.shape)}, {list(page_table.shape)}")
    b = KvBatch(T, B, page_table.shape[1], cu_q.data_ptr(), kv_len.data_ptr(),
                page_table.data_ptr())
    b.tensors, b.device = (cu_q, kv_len, page_table), dev
    return b


def kv_append_paged(q, k, v, q_out, cache: KvCache, batch: KvBatch, pos, axis_dims, q_gain=None,
                    k_gain=None, theta=1e4, eps=1e-6, pairing=0, stream=None):
    """q_out <- RoPE(RMSNorm(q)); the rows' places in the cache get
    RoPE(RMSNorm(k)) and v. q [T,H,128], k, v [T,Hkv,128] bf16 (rows may be
    strided), q_out [T,H,128] contiguous (q and q_out None: cache only), pos
    [T,3] int32, gains [128] f32 (None: no norm)."""
    dev, T = _device(), batch.T
    _made_on(cache, batch, dev)
    H, pq, ldq, po = 0, None, 0, None
    if q is not None:
        ldq, H = _heads(q, "q", T, dev)
        if q_out is None or q_out.shape != q.shape:
            raise ValueError("q_out must have q's shape")
        _flat(q_out, "q_out", torch.bfloat16, dev)
        pq, po = q.data_ptr(), q_out.data_ptr()
    elif q_out is not None:
        raise ValueError("q_out without q")
    ldk, hk = _heads(k, "k", T, dev)
    ldv, hv = _heads(v, "v", T, dev)
    if hk != cache.Hkv or hv != cache.Hkv:
        raise ValueError(f"k and v have {hk} and {hv} heads, the cache {cache.Hkv}")
    if pos.shape != (T, 3):
        raise ValueError(f"pos must be [{T}, 3], got {list(pos.shape)}")
    _flat(pos, "pos", torch.int32, dev)
    pg = [None, None]
    if q_gain is not None:
        pg[0] = _gain(q_gain, dev)
    if k_gain is not None:
        pg[1] = _gain(k_gain, dev)
    axis = tuple(axis_dims)
    ax = _AXES.get(axis)
    if ax is None:
        ax = _AXES[axis] = _INT3(*axis)
    _check("kv_append_paged", lib().h3_kv_append_paged(
        pq, ldq, k.data_ptr(), ldk, v.data_ptr(), ldv, po, H, pg[0], pg[1], pos.data_ptr(),
        ctypes.addressof(ax), pairing, theta, eps, ctypes.addressof(cache),
        ctypes.addressof(batch), _raw_stream(stream, dev)))


def attention_paged_workspace_bytes(T: int, H: int, prefix_len: int = 0) -> int:
    n = lib().h3_attention_paged_workspace_bytes(T, H, prefix_len)
    if n == 0:
        raise H3Error("attention_paged_workspace_bytes", 1, last_error())
    return n


def attention_paged(q, o, cache: KvCache, batch: KvBatch, workspace, scale=None, causal=False,
                    stream=None):
    """o = softmax(q k^T * scale) v over the keys of every row's own sequence
    (causal: those up to the row itself); q, o [T,H,128] bf16, rows may be
    strided; workspace: device tensor of attention_paged_workspace_bytes."""
    attention_paged_prefix(q, o, cache, batch, None, 0, workspace, scale, causal, stream)


def attention_paged_prefix(q, o, cache: KvCache, batch: KvBatch, prefix_pages, prefix_len: int,
                           workspace, scale=None, causal=False, stream=None):
    """attention_paged with prefix_len keys in prefix_pages (int32) before the
    own keys of every sequence, read once for the whole batch (by few rows behind
    a short prefix once for each)."""
    dev, T = _device(), batch.T
    _made_on(cache, batch, dev)
    ldq, H = _heads(q, "q", T, dev)
    ldo, Ho = _heads(o, "o", T, dev)
    if Ho != H:
        raise ValueError(f"q has {H} heads, o {Ho}")
    pages = None
    if prefix_pages is not None:
        _flat(prefix_pages, "prefix_pages", torch.int32, dev)
        if prefix_pages.numel() * cache.page_size < prefix_len:
            raise ValueError(f"prefix_pages holds {prefix_pages.numel()} pages of "
                             f"{cache.page_size} keys, prefix_len is {prefix_len}")
        pages = prefix_pages.data_ptr()
    _flat(workspace, "workspace", workspace.dtype, dev)
    _check("attention_paged_prefix", lib().h3_attention_paged_prefix(
        q.data_ptr(), ldq, o.data_ptr(), ldo, H, 128 ** -0.5 if scale is None else scale,
        int(causal), ctypes.addressof(cache), ctypes.addressof(batch), pages, prefix_len,
        workspace.data_ptr(), workspace.nbytes, _raw_stream(stream, dev)))


def swiglu(gate_up, out, L=None, stream=None):
    _need(gate_up, torch.bfloat16, "gate_up")
    _need(out, torch.bfloat16, "out")
    S, F = out.shape
    L = S if L is None else L
    _check("swiglu", lib().h3_swiglu(_p(gate_up), _p(out), S, L, F, _s(stream)))


def linear(x, w, y, L=None, stream=None):
    """y[:L] = x[:L] @ w^T; x [S,K], w [N,K], y [S,N] bf16."""
    for n, t in (("x", x), ("w", w), ("y", y)):
        _need(t, torch.bfloat16, n)
    S, K = x.shape
    N = w.shape[0]
    L = S if L is None else L
    _check("linear", lib().h3_linear(_p(x), _p(w), _p(y), S, L, N, K, _s(stream)))


def linear_swiglu(x, w_gu, out, L=None, stream=None):
    """out[:L] = SiLU(x w_g^T) * (x w_u^T); w_gu [2F,K] rows [gate | up]."""
    for n, t in (("x", x), ("w_gu", w_gu), ("out", out)):
        _need(t, torch.bfloat16, n)
    S, K = x.shape
    F = out.shape[1]
    L = S if L is None else L
    _check("linear_swiglu", lib().h3_linear_swiglu(_p(x), _p(w_gu), _p(out), S, L, F, K,
                                                    _s(stream)))


def rope_table(pos, axis_dims, table, L=None, theta=1e4, stream=None):
    """table[:L] = (cos, sin) of every RoPE angle; pos [S,3] int32, table [S,64,2] f32."""
    _need(pos, torch.int32, "pos")
    _need(table, torch.float32, "table")
    S = pos.shape[0]
    L = S if L is None else L
    ax = (ctypes.c_int * 3)(*axis_dims)
    _check("rope_table", lib().h3_rope_table(_p(pos), ctypes.cast(ax, ctypes.c_void_p), S, L,
                                              theta, _p(table), _s(stream)))


def linear_qk_norm_rope(x, w_qkv, qkv, q_gain, k_gain, table, axis_dims, L=None, eps=1e-6,
                        pairing=0, stream=None):
    """qkv[:L] = x @ w_qkv^T with per-head Q/K RMSNorm + RoPE (table from
    rope_table, sections axis_dims, pairing as qk_norm_rope) in the epilogue;
    x [S,K], w_qkv [3D,K], qkv [S,3D] bf16."""
    for n, t in (("x", x), ("w_qkv", w_qkv), ("qkv", qkv)):
        _need(t, torch.bfloat16, n)
    S, K = x.shape
    H = w_qkv.shape[0] // 3 // 128
    L = S if L is None else L
    ax = ctypes.cast((ctypes.c_int * 3)(*axis_dims), ctypes.c_void_p)
    _check("linear_qk_norm_rope", lib().h3_linear_qk_norm_rope(
        _p(x), _p(w_qkv), _p(qkv), _p(q_gain), _p(k_gain), _p(table), ax, pairing, S, L, H, K,
        eps, _s(stream)))


def linear_residual(x, w, resid, gate, L=None, stream=None):
    """resid[:L] += gate * bf16(x @ w^T) in FP32; x [S,K], w [N,K] bf16, resid [S,N] f32."""
    _need(x, torch.bfloat16, "x")
    _need(w, torch.bfloat16, "w")
    _need(resid, torch.float32, "resid")
    S, K = x.shape
    N = w.shape[0]
    L = S if L is None else L
    _check("linear_residual", lib().h3_linear_residual(_p(x), _p(w), _p(resid), _p(gate), S, L,
                                                        N, K, _s(stream)))


def block_config(S, L, D, H, Dh, F, axis_dims, theta=1e4, eps_ln=1e-6, eps_qk=1e-6,
                 rope_pairing=0) -> BlockConfig:
    return BlockConfig(S, L, D, H, Dh, F, (ctypes.c_int * 3)(*axis_dims), theta, eps_ln, eps_qk,
                       rope_pairing)


NOALLOC_SCRATCH_BYTES = 32 * 1024 * 1024


def block_forward_noalloc(cfg: BlockConfig, weights, resid, mod, pos, stream=None):
    """h3_block_forward_noalloc: the block forward with the library's own
    fixed scratch array instead of a caller workspace, for callers that cannot
    allocate device memory (blocks up to NOALLOC_SCRATCH_BYTES of workspace)."""
    w = weights if isinstance(weights, BlockWeights) else block_weights(weights)
    _check("block_forward_noalloc", lib().h3_block_forward_noalloc(
        ctypes.byref(cfg), ctypes.byref(w), _p(resid), _p(mod), _p(pos), _s(stream)))


def stack_forward(cfg: BlockConfig, weights_list, resid, mods, pos, workspace, seg=None,
                  stream=None):
    """Blocks applied in order: weights_list[b] (dict or BlockWeights) with
    mods [num_blocks, G, 6, D] f32 (or [num_blocks, 6, D] when seg is None);
    seg [S] int32 picks each row's group."""
    n = len(weights_list)
    arr = (BlockWeights * n)(*(w if isinstance(w, BlockWeights) else block_weights(w)
                               for w in weights_list))
    G = 1 if mods.dim() == 3 else mods.shape[1]
    _need(mods, torch.float32, "mods")
    _check("stack_forward", lib().h3_stack_forward(
        ctypes.byref(cfg), arr, n, _p(resid), _p(mods), G, _p(seg), _p(pos), _p(workspace),
        workspace.numel() * workspace.element_size(), _s(stream)))


def frames_to_u8(frames, out, stream=None):
    """frames [B, C, T, H, W] f32 -> out [B, T, H, W, C] uint8."""
    _need(frames, torch.float32, "frames")
    _need(out, torch.uint8, "out")
    B, C, T, H, W = frames.shape
    _check("frames_to_u8", lib().h3_frames_to_u8(_p(frames), _p(out), B, C, T, H, W,
                                                  _s(stream)))


def quantize_fp8_rows(x, q, scale, stream=None):
    """x [R, K] bf16 -> q [R, K] uint8 (E4M3 codes), scale [R] f32."""
    _need(x, torch.bfloat16, "x")
    _need(q, torch.uint8, "q")
    _need(scale, torch.float32, "scale")
    R, K = x.shape
    _check("quantize_fp8_rows", lib().h3_quantize_fp8_rows(_p(x), _p(q), _p(scale), R, K,
                                                            _s(stream)))


def linear_fp8(qx, sx, qw, sw, y, L=None, stream=None):
    S, K = qx.shape
    N = qw.shape[0]
    L = S if L is None else L
    _check("linear_fp8", lib().h3_linear_fp8(_p(qx), _p(sx), _p(qw), _p(sw), _p(y), S, L, N, K,
                                              _s(stream)))


def linear_swiglu_fp8(qx, sx, qw_gu, sw_gu, out, L=None, stream=None):
    S, K = qx.shape
    F = out.shape[1]
    L = S if L is None else L
    _check("linear_swiglu_fp8", lib().h3_linear_swiglu_fp8(
        _p(qx), _p(sx), _p(qw_gu), _p(sw_gu), _p(out), S, L, F, K, _s(stream)))


def quantize_block_weights_fp8(weights: dict, stream=None) -> dict:
    """Load-time FP8 quantisation of a block's four projection weights:
    returns a dict with codes (uint8) and per-row scales for each, plus the
    Q/K gains, ready for block_forward_fp8."""
    out = {"q_gain": weights["q_gain"], "k_gain": weights["k_gain"]}
    for k in ("w_qkv", "w_o", "w_gu", "w_down"):
        w = weights[k]
        q = torch.empty(w.shape, dtype=torch.uint8, device=w.device)
        sc = torch.empty(w.shape[0], dtype=torch.float32, device=w.device)
        quantize_fp8_rows(w, q, sc, stream)
        out[k] = q
        out["s_" + k[2:]] = sc
    return out


def block_weights_fp8(w: dict) -> BlockWeightsFp8:
    return BlockWeightsFp8(*(w[k].data_ptr() for k in (
        "w_qkv", "s_qkv", "w_o", "s_o", "w_gu", "s_gu", "w_down", "s_down", "q_gain", "k_gain")))


def block_workspace_bytes_fp8(cfg: BlockConfig) -> int:
    n = lib().h3_block_workspace_bytes_fp8(ctypes.byref(cfg))
    if n == 0:
        raise H3Error("block_workspace_bytes_fp8", 1, last_error())
    return n


def block_forward_fp8(cfg: BlockConfig, weights_fp8, resid, mod, pos, workspace, stream=None,
                      fp8_attention=False):
    w = weights_fp8 if isinstance(weights_fp8, BlockWeightsFp8) else block_weights_fp8(weights_fp8)
    _check("block_forward_fp8", lib().h3_block_forward_fp8(
        ctypes.byref(cfg), ctypes.byref(w), _p(resid), _p(mod), _p(pos), int(fp8_attention),
        _p(workspace), workspace.numel() * workspace.element_size(), _s(stream)))


def block_workspace_bytes(cfg: BlockConfig) -> int:
    n = lib().h3_block_workspace_bytes(ctypes.byref(cfg))
    if n == 0:
        raise H3Error("block_workspace_bytes", 1, last_error())
    return n


BLOCK_STAGES = 7
STAGE_NAMES = ("mod_norm", "qkv_proj_qk_norm_rope", "attention", "out_proj",
               "residual_mod_norm", "gate_up_swiglu", "down_proj_residual")
# kernels one block launches: one per stage
BLOCK_LAUNCHES = BLOCK_STAGES


def block_weights(weights: dict) -> BlockWeights:
    return BlockWeights(*(weights[k].data_ptr() for k in
                          ("w_qkv", "w_o", "w_gu", "w_down", "q_gain", "k_gain")))


def block_forward(cfg: BlockConfig, weights, resid, mod, pos, workspace, stream=None,
                  events=None):
    """One block forward, in place on resid [S,D] f32. weights: dict with
    w_qkv, w_o, w_gu, w_down (bf16) and q_gain, k_gain (f32), or a prepared
    BlockWeights; workspace: uint8 device tensor. events: optional list of
    BLOCK_STAGES + 1 recorded-once torch.cuda.Event, marked before each stage."""
    w = weights if isinstance(weights, BlockWeights) else block_weights(weights)
    nbytes = workspace.numel() * workspace.element_size()
    if events is None:
        _check("block_forward", lib().h3_block_forward(
            ctypes.byref(cfg), ctypes.byref(w), _p(resid), _p(mod), _p(pos), _p(workspace),
            nbytes, _s(stream)))
        return
    arr = (_P * len(events))(*(e.cuda_event for e in events))
    _check("block_forward_events", lib().h3_block_forward_events(
        ctypes.byref(cfg), ctypes.byref(w), _p(resid), _p(mod), _p(pos), _p(workspace), nbytes,
        _s(stream), arr, len(events)))


# Norms around a branch, 4-bit rows and block-sparse attention: like the paged calls they run
# several times per layer, so a tensor that is as it should be costs a few attribute reads.
_F32, _BF16, _I32 = torch.float32, torch.bfloat16, torch.int32


def _here(t, name) -> int:
    """The device of the first tensor of a call, which has to be the current one."""
    dev = t.get_device()
    if dev < 0 or dev != torch._C._cuda_getDevice():
        raise ValueError(f"{name} must be on the current CUDA device, is on {t.device}")
    return dev


def _tensor(t, name, dtype, shape, dev):
    """Pointer of a contiguous tensor of this type and shape, or NULL for None."""
    if t is None:
        return None
    if t.dtype is not dtype or t.get_device() != dev or t.shape != shape or not t.is_contiguous():
        if t.shape != shape:
            raise ValueError(f"{name} must be {list(shape)}, got {list(t.shape)}")
        _flat(t, name, dtype, dev)
    return t.data_ptr()


def _table(t, name, shape, stride, dev):
    """Pointer of the first row of a [groups, D] f32 table, or NULL for None."""
    if t is None:
        return None
    if t.dtype is not _F32:
        raise TypeError(f"{name} must be {_F32}, got {t.dtype}")
    if t.shape != shape or t.stride(1) != 1 or (shape[0] > 1 and t.stride(0) != stride):
        raise ValueError(f"{name} must be {list(shape)} with neighbouring values and rows as far "
                         f"apart as the other tables', got {list(t.shape)} of strides {t.stride()}")
    _on(t, name, dev)
    return t.data_ptr()


def sandwich_norm(resid, delta=None, normed=None, resid_out=None, post_norm=True, post_gain=None,
                  gate=None, resid_scale=1.0, pre_gain=None, shift=None, scale=None, seg=None,
                  rms=False, L=None, eps=1e-6, stream=None):
    """r = resid_scale * resid + gate * n(delta) * post_gain (post_norm False: delta as it
    is), stored to resid_out (default: resid itself where there is a delta or a
    resid_scale); normed <- bf16(n(r) * pre_gain * (1 + scale) + shift); n: LayerNorm
    without affine, or with rms the division by the root mean square. resid, resid_out
    [S,D] f32, delta, normed [S,D] bf16; vectors [D] f32, left out where None. With seg [S]
    int32, gate, shift and scale are [G,D] tables (rows equally far apart, as columns of a
    [G,6,D] one are) and row i takes row seg[i] of them."""
    shape = resid.shape
    S, D = shape
    dev = _here(resid, "resid")
    pr = _tensor(resid, "resid", _F32, shape, dev)
    pd = _tensor(delta, "delta", _BF16, shape, dev)
    pn = _tensor(normed, "normed", _BF16, shape, dev)
    if delta is None:
        post_norm = False
    if resid_out is None:
        po = pr if delta is not None or resid_scale != 1.0 else None
    else:
        po = _tensor(resid_out, "resid_out", _F32, shape, dev)
    vec = (D,)
    if seg is None:
        pseg, groups, stride = None, 1, 0
        pg = _tensor(gate, "gate", _F32, vec, dev)
        ph = _tensor(shift, "shift", _F32, vec, dev)
        pc = _tensor(scale, "scale", _F32, vec, dev)
    else:
        pseg = _tensor(seg, "seg", _I32, (S,), dev)
        first = gate if gate is not None else shift if shift is not None else scale
        groups = 1 if first is None else first.shape[0]
        stride = D if groups == 1 else first.stride(0)
        pg = _table(gate, "gate", (groups, D), stride, dev)
        ph = _table(shift, "shift", (groups, D), stride, dev)
        pc = _table(scale, "scale", (groups, D), stride, dev)
    status = (_lib or lib()).h3_sandwich_norm(
        pr, pd, po, pn, post_norm, _tensor(post_gain, "post_gain", _F32, vec, dev), pg, resid_scale,
        _tensor(pre_gain, "pre_gain", _F32, vec, dev), ph, pc, pseg, groups, stride, rms, S,
        S if L is None else L, D, eps, _raw_stream(stream, dev))
    if status:
        _check("sandwich_norm", status)


FP4_FORMATS = {"mx": 0, "nv": 1}


def _fp4_format(format) -> int:
    if format not in FP4_FORMATS:
        raise ValueError(f"format must be one of {sorted(FP4_FORMATS)}, got {format!r}")
    return FP4_FORMATS[format]


class Fp4Rows:
    """A matrix [R, K] of 4-bit rows: codes [R, K/2] uint8, scales (bytes, in the library's
    tiles), row_scale [R] f32 ("nv") or None ("mx"). fp4_rows makes room for one."""
    __slots__ = ("codes", "scales", "row_scale", "format", "R", "K", "shape", "device", "pointers",
                 "number")

    def __init__(self, codes, scales, row_scale, format):
        number = _fp4_format(format)
        dev = codes.get_device()
        _flat(codes, "codes", torch.uint8, dev)
        _flat(scales, "scales", torch.uint8, dev)
        if codes.dim() != 2:
            raise ValueError(f"codes must be [R, K/2], got {list(codes.shape)}")
        self.R, self.K = codes.shape[0], codes.shape[1] * 2
        need = fp4_scale_bytes(self.R, self.K, format)
        if scales.numel() < need:
            raise ValueError(f"scales have {scales.numel()} bytes, {need} are needed")
        if (row_scale is not None) != (format == "nv"):
            raise ValueError('row_scale belongs to format "nv", and only to it')
        if row_scale is not None:
            _flat(row_scale, "row_scale", torch.float32, dev)
            if row_scale.shape != (self.R,):
                raise ValueError(f"row_scale must be [{self.R}], got {list(row_scale.shape)}")
        self.codes, self.scales, self.row_scale = codes, scales, row_scale
        self.format, self.number, self.device = format, number, dev
        self.shape = (self.R, self.K)
        self.pointers = (codes.data_ptr(), scales.data_ptr(),
                         None if row_scale is None else row_scale.data_ptr())


def fp4_scale_bytes(R: int, K: int, format: str = "nv") -> int:
    n = lib().h3_fp4_scale_bytes(R, K, _fp4_format(format))
    if n == 0:
        raise H3Error("fp4_scale_bytes", 1, last_error())
    return n


def fp4_rows(R: int, K: int, format: str = "nv", device=None) -> Fp4Rows:
    """Room for [R, K] 4-bit rows on a device (default: the current one): "nv" (16 values
    share an E4M3 scale, a row an FP32 one) or "mx" (32 share a power of two). The scales are
    zeros, so that a program which fills in packed weights itself need not clear the places
    past a row's last block, which a product reads where K is no multiple of 64."""
    device = torch.device("cuda") if device is None else device
    n = fp4_scale_bytes(R, K, format)
    return Fp4Rows(torch.empty(R, K // 2, dtype=torch.uint8, device=device),
                   torch.zeros(n, dtype=torch.uint8, device=device),
                   torch.empty(R, dtype=torch.float32, device=device) if format == "nv" else None,
                   format)


def _same_device(q: Fp4Rows, name, dev):
    if q.device != dev:
        raise ValueError(f"{name} must be on the current CUDA device, is on device {q.device}")


def quantize_fp4_rows(x, out: Fp4Rows, L=None, stream=None):
    """x [R, K] bf16 (rows may be strided) -> out, its first L rows."""
    dev = _here(x, "x")
    if x.dtype is not _BF16:
        raise TypeError(f"x must be {_BF16}, got {x.dtype}")
    if x.shape != out.shape:
        raise ValueError(f"x must be {list(out.shape)}, got {list(x.shape)}")
    ld, one = x.stride()
    if one != 1:
        raise ValueError("the values of a row of x must be neighbours")
    if out.device != dev:
        _same_device(out, "out", dev)
    R = out.R
    if L is None:
        L = R
    elif not 0 <= L <= R:
        raise ValueError(f"L={L} exceeds the {R} rows")
    codes, scales, row_scale = out.pointers
    status = (_lib or lib()).h3_quantize_fp4_rows(
        x.data_ptr(), ld if R > 1 else out.K, codes, scales, row_scale, L, out.K, out.number,
        _raw_stream(stream, dev))
    if status:
        _check("quantize_fp4_rows", status)


def _fp4_product(name, call, x, w, y, N, L, stream):
    dev = _here(y, "the output")
    if x.number != w.number or x.K != w.K:
        raise ValueError(f"x is {x.format!r} rows of {x.K}, the weights {w.format!r} of {w.K}")
    py = _tensor(y, "the output", _BF16, (x.R, N), dev)
    if x.device != dev or w.device != dev:
        _same_device(x, "x", dev)
        _same_device(w, "the weights", dev)
    status = call(*x.pointers, *w.pointers, py, x.R, x.R if L is None else L, N, x.K, x.number,
                  _raw_stream(stream, dev))
    if status:
        _check(name, status)


def linear_fp4(x: Fp4Rows, w: Fp4Rows, y, L=None, stream=None):
    """y[:L] = x w^T of 4-bit rows x [S, K], w [N, K]; y [S, N] bf16."""
    _fp4_product("linear_fp4", (_lib or lib()).h3_linear_fp4, x, w, y, w.R, L, stream)


def linear_swiglu_fp4(x: Fp4Rows, w_gu: Fp4Rows, out, L=None, stream=None):
    """out[:L] = SiLU(x Wg^T) * (x Wu^T) of 4-bit rows x [S, K], w_gu [2F, K] (rows
    [gate | up]); out [S, F] bf16."""
    if w_gu.R % 2:
        raise ValueError(f"the weights have {w_gu.R} rows, an odd number")
    _fp4_product("linear_swiglu_fp4", (_lib or lib()).h3_linear_swiglu_fp4, x, w_gu, out,
                 w_gu.R // 2, L, stream)


QUERY_BLOCK = 256


def block_scores_workspace_bytes(Lq: int, Lk: int, H: int, Hkv: int, k_block: int = 64) -> int:
    n = lib().h3_block_scores_workspace_bytes(Lq, Lk, H, Hkv, k_block)
    if n == 0:
        raise H3Error("block_scores_workspace_bytes", 1, last_error())
    return n


def _block_shape(Lq, Lk, H, k_block):
    if k_block not in (64, 128):
        raise ValueError(f"k_block must be 64 or 128, got {k_block}")
    return H, -(-Lq // QUERY_BLOCK), -(-Lk // k_block)


def block_scores(q, k, scores, workspace, k_block=64, scale=None, stream=None):
    """scores [H, nq, nk] f32 of every (block of QUERY_BLOCK query rows, block of k_block
    keys): scale times the product of their mean rows. q [Lq,H,128], k [Lk,Hkv,128] bf16
    (rows may be strided), workspace of block_scores_workspace_bytes."""
    dev = _here(scores, "scores")
    Lq, Lk = q.shape[0], k.shape[0]
    ldq, H = _heads(q, "q", Lq, dev)
    ldk, Hkv = _heads(k, "k", Lk, dev)
    ps = _tensor(scores, "scores", _F32, _block_shape(Lq, Lk, H, k_block), dev)
    _flat(workspace, "workspace", workspace.dtype, dev)
    status = (_lib or lib()).h3_block_scores(
        q.data_ptr(), ldq, k.data_ptr(), ldk, ps, Lq, Lk, H, Hkv, 128, k_block,
        128 ** -0.5 if scale is None else scale, workspace.data_ptr(), workspace.nbytes,
        _raw_stream(stream, dev))
    if status:
        _check("block_scores", status)


def block_select(scores, ids, counts, keep_first=0, keep_last=0, stream=None):
    """The best-scored blocks of every row of scores [..., nk] f32: ids [..., max_blocks]
    int32 in ascending order (then -1), counts [...] int32. The first keep_first and the
    last keep_last blocks are always among them; -inf and NaN never are otherwise."""
    shape, listed, rows = scores.shape, ids.shape, counts.shape
    nk, most = shape[-1], listed[-1]
    if listed[:-1] != rows or shape[:-1] != rows:
        raise ValueError(f"scores [..., nk], ids [..., max_blocks] and counts [...] wanted, got "
                         f"{list(shape)}, {list(listed)} and {list(rows)}")
    dev = _here(scores, "scores")
    status = (_lib or lib()).h3_block_select(
        _tensor(scores, "scores", _F32, shape, dev), _tensor(ids, "ids", _I32, listed, dev),
        _tensor(counts, "counts", _I32, rows, dev), counts.numel(), nk, most, keep_first, keep_last,
        _raw_stream(stream, dev))
    if status:
        _check("block_select", status)


def attention_blocks(q, k, v, o, ids, counts, k_block=64, scale=None, stream=None):
    """Attention of every block of QUERY_BLOCK query rows over its listed key blocks: ids
    [H, nq, max_blocks], counts [H, nq] int32 (block_select's), q, o [Lq,H,128], k, v
    [Lk,Hkv,128] bf16 (rows may be strided)."""
    dev = _here(counts, "counts")
    Lq, Lk = q.shape[0], k.shape[0]
    ldq, H = _heads(q, "q", Lq, dev)
    ldk, Hkv = _heads(k, "k", Lk, dev)
    ldv, hv = _heads(v, "v", Lk, dev)
    ldo, ho = _heads(o, "o", Lq, dev)
    if hv != Hkv or ho != H:
        raise ValueError(f"q and o have {H} and {ho} heads, k and v {Hkv} and {hv}")
    shape = _block_shape(Lq, Lk, H, k_block)[:2]
    if ids.dim() != 3:
        raise ValueError(f"ids must be {list(shape)} x max_blocks, got {list(ids.shape)}")
    most = ids.shape[2]
    status = (_lib or lib()).h3_attention_blocks(
        q.data_ptr(), ldq, k.data_ptr(), ldk, v.data_ptr(), ldv, o.data_ptr(), ldo,
        _tensor(ids, "ids", _I32, (*shape, most), dev), _tensor(counts, "counts", _I32, shape, dev),
        most, Lq, Lk, H, Hkv, 128, k_block, 128 ** -0.5 if scale is None else scale,
        _raw_stream(stream, dev))
    if status:
        _check("attention_blocks", status)
