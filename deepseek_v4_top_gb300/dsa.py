"""Python binding of libdsa.so: the C ABI of include/dsa.h under the same names.

Argument marshalling only.  Every step of the attention runs in the CUDA
kernels of libdsa.so; PyTorch provides device memory and the current stream.
There is no fallback: if the library is missing or the GPU is unsupported,
the calls raise.
"""

from __future__ import annotations

import ctypes
import os
import threading

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libdsa.so")

DSA_OK = 0
DSA_ERR_INVALID_ARG = 1
DSA_ERR_UNSUPPORTED = 2
DSA_ERR_CUDA = 3
DSA_ERR_DEVICE_CHECK = 4

DSA_F32 = 0
DSA_BF16 = 1

DSA_DEVERR_IDX_RANGE = 0x1
DSA_DEVERR_NSEL_RANGE = 0x2
DSA_DEVERR_TIMEOUT = 0x4
DSA_DEVERR_LAYOUT = 0x8
DSA_DEVERR_NVALID_RANGE = 0x10
DSA_DEVERR_PAGE_RANGE = 0x20
DSA_DEVERR_POS_RANGE = 0x40
DSA_DEVERR_SEQ_RANGE = 0x80

DSA_ROPE_PAIRS = 0
DSA_ROPE_HALVES = 1

# Every function declared in include/dsa.h.
EXPORTS = ("dsa_sparse_attn_decode", "dsa_sparse_attn_decode_rows", "dsa_sparse_attn_prefill",
           "dsa_sparse_attn", "dsa_sparse_attn_decode_whole_rows", "dsa_oproj", "dsa_sparse_attn_prefill_oproj",
           "dsa_sparse_attn_decode_noalloc",
           "dsa_qk_norm_rope", "dsa_paged_append", "dsa_paged_attn", "dsa_paged_sparse_attn",
           "dsa_paged_workspace_bytes",
           "dsa_topk_select", "dsa_head_shard", "dsa_shard_heads", "dsa_unshard_heads",
           "dsa_selftest_wait_limit", "dsa_get_device_error", "dsa_status_string", "dsa_shutdown")
DSA_NOALLOC_MAX_UNITS = 64

_lib = None
_lock = threading.Lock()


class HeadShardPlan(ctypes.Structure):
    """dsa_head_shard_plan of include/dsa.h."""
    _fields_ = [("heads_per_rank", ctypes.c_int), ("padded_heads", ctypes.c_int),
                ("first_head", ctypes.c_int), ("real_heads", ctypes.c_int)]


class DsaError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__("%s returned %s" % (where, status_string(status)))


def load():
    """Load libdsa.so (it must have been built; see __graft_entry__.build)."""
    global _lib
    with _lock:
        if _lib is None:
            if not os.path.exists(LIB_PATH):
                raise RuntimeError("libdsa.so is not built: run __graft_entry__.build() first")
            lib = ctypes.CDLL(LIB_PATH)
            P, I, F = ctypes.c_void_p, ctypes.c_int, ctypes.c_float
            sig = [P, P, P, P, P, F, P, I, I, I, I, I, P]
            for name in ("dsa_sparse_attn_decode", "dsa_sparse_attn_prefill",
                         "dsa_sparse_attn_decode_noalloc"):
                fn = getattr(lib, name)
                fn.argtypes = sig
                fn.restype = I
            lib.dsa_sparse_attn_decode_rows.argtypes = [P, P, P, P, P, F, P, I, I, I, I, I, I, P]
            lib.dsa_sparse_attn_decode_rows.restype = I
            lib.dsa_sparse_attn.argtypes = [P, P, P, P, P, F, P, I, I, I, I, I, I, I, P]
            lib.dsa_sparse_attn.restype = I
            lib.dsa_sparse_attn_decode_whole_rows.argtypes = [P, P, P, P, P, F, P, I, I, I, I, I, I, I, P]
            lib.dsa_sparse_attn_decode_whole_rows.restype = I
            lib.dsa_oproj.argtypes = [P, P, P, I, I, I, P]
            lib.dsa_oproj.restype = I
            lib.dsa_sparse_attn_prefill_oproj.argtypes = [P, P, P, P, P, F, P, P, P, I, I, I, I, I, P]
            lib.dsa_sparse_attn_prefill_oproj.restype = I
            lib.dsa_topk_select.argtypes = [P, I, P, I, I, P, I, P, P]
            lib.dsa_topk_select.restype = I
            lib.dsa_qk_norm_rope.argtypes = [P, P, P, P, F, P, I, I, I, P, P, P, I, I, I, I, P]
            lib.dsa_qk_norm_rope.restype = I
            lib.dsa_paged_append.argtypes = [P, P, F, P, I, I, I, P, P, P, P, P, I, I, I, I, I, I, I, P]
            lib.dsa_paged_append.restype = I
            Z = ctypes.c_size_t
            lib.dsa_paged_attn.argtypes = [P, P, P, P, P, P, F, P, P, Z, I, I, I, I, I, I, I, P]
            lib.dsa_paged_attn.restype = I
            lib.dsa_paged_sparse_attn.argtypes = [P, P, P, P, P, P, P, P, F, P, P, Z, I, I, I, I, I, I, I, I, P]
            lib.dsa_paged_sparse_attn.restype = I
            lib.dsa_paged_workspace_bytes.argtypes = [I, I]
            lib.dsa_paged_workspace_bytes.restype = Z
            lib.dsa_head_shard.argtypes = [I, I, I, ctypes.POINTER(HeadShardPlan)]
            lib.dsa_head_shard.restype = I
            lib.dsa_shard_heads.argtypes = [P, P, P, P, I, I, I, I, I, P]
            lib.dsa_shard_heads.restype = I
            lib.dsa_unshard_heads.argtypes = [P, P, I, I, I, I, P]
            lib.dsa_unshard_heads.restype = I
            lib.dsa_selftest_wait_limit.argtypes = [P]
            lib.dsa_selftest_wait_limit.restype = I
            lib.dsa_get_device_error.argtypes = [P, ctypes.POINTER(ctypes.c_uint32)]
            lib.dsa_get_device_error.restype = I
            lib.dsa_status_string.argtypes = [I]
            lib.dsa_status_string.restype = ctypes.c_char_p
            lib.dsa_shutdown.argtypes = []
            lib.dsa_shutdown.restype = I
            _lib = lib
    return _lib


def status_string(status: int) -> str:
    return load().dsa_status_string(int(status)).decode()


# ------------------------------------------------------------- raw pointers
def call_raw(name: str, q: int, kv: int, idx: int, n_sel: int, sink: int, scale: float, out: int,
             R: int, H: int, N: int, k_max: int, dtype: int, stream: int = 0) -> int:
    """Call an entry point with integer device addresses; returns the status."""
    fn = getattr(load(), name)
    return int(fn(q, kv, idx, n_sel, sink, ctypes.c_float(scale), out, R, H, N, k_max, dtype,
                  stream))


# ------------------------------------------------------------ torch tensors
def _same_device(*pairs):
    """Every tensor must be on the current CUDA device: the library launches
    there, and another device's addresses are not valid in its kernels."""
    import torch
    cur = torch.cuda.current_device()
    for name, t in pairs:
        if t.device.index != cur:
            raise ValueError("%s is on cuda:%s, but the calls run on the current device cuda:%d "
                             "(torch.cuda.set_device)" % (name, t.device.index, cur))


def _dtype_code(t):
    import torch
    if t.dtype == torch.float32:
        return DSA_F32
    if t.dtype == torch.bfloat16:
        return DSA_BF16
    raise TypeError("q and kv_cache must be float32 or bfloat16, got %s" % t.dtype)


def _check(q, kv, idx, n_sel, sink, out, decode, rows_per_slot=1, out_dtype=None):
    import torch
    for name, t in (("q", q), ("kv_cache", kv), ("idx", idx), ("n_sel", n_sel), ("sink", sink),
                    ("out", out)):
        if not isinstance(t, torch.Tensor):
            raise TypeError("%s must be a torch.Tensor" % name)
        if not t.is_cuda:
            raise ValueError("%s must be a CUDA tensor" % name)
        if not t.is_contiguous():
            raise ValueError("%s must be contiguous" % name)
    _same_device(("q", q), ("kv_cache", kv), ("idx", idx), ("n_sel", n_sel), ("sink", sink), ("out", out))
    if kv.dtype != q.dtype:
        raise TypeError("q and kv_cache must have the same dtype")
    if idx.dtype != torch.int32 or n_sel.dtype != torch.int32:
        raise TypeError("idx and n_sel must be int32")
    if sink.dtype != torch.float32:
        raise TypeError("sink must be float32")
    if out.dtype != (torch.float32 if out_dtype is None else out_dtype):
        raise TypeError("out must be %s" % ("float32" if out_dtype is None else out_dtype))
    if q.dim() != 3 or q.shape[2] != 512:
        raise ValueError("q must be [rows, heads, 512]")
    R, H = q.shape[0], q.shape[1]
    if decode:
        if kv.dim() != 3 or kv.shape[0] * rows_per_slot != R or kv.shape[2] != 512:
            raise ValueError("decode kv_cache must be [slots, N, 512] with slots * rows_per_slot = rows")
        N = kv.shape[1]
    else:
        if kv.dim() != 2 or kv.shape[1] != 512:
            raise ValueError("prefill kv_cache must be [N, 512]")
        N = kv.shape[0]
    if idx.dim() != 2 or idx.shape[0] != R:
        raise ValueError("idx must be [rows, k_max]")
    if tuple(n_sel.shape) != (R,) or tuple(sink.shape) != (H,) or tuple(out.shape) != (R, H, 512):
        raise ValueError("n_sel [rows], sink [heads] and out [rows, heads, 512] expected")
    return R, H, N, idx.shape[1]


def _stream_handle(stream):
    import torch
    if stream is None:
        stream = torch.cuda.current_stream()
    if hasattr(stream, "device") and getattr(stream.device, "index", None) is not None:
        if stream.device.index != torch.cuda.current_device():
            raise ValueError("the stream belongs to cuda:%d, but the calls run on the current device cuda:%d"
                             % (stream.device.index, torch.cuda.current_device()))
    return int(stream.cuda_stream) if hasattr(stream, "cuda_stream") else int(stream)


def _run(name, decode, q, kv_cache, idx, n_sel, sink, scale, out, stream):
    R, H, N, k_max = _check(q, kv_cache, idx, n_sel, sink, out, decode)
    st = call_raw(name, q.data_ptr(), kv_cache.data_ptr(), idx.data_ptr(), n_sel.data_ptr(),
                  sink.data_ptr(), float(scale), out.data_ptr(), R, H, N, k_max,
                  _dtype_code(q), _stream_handle(stream))
    if st != DSA_OK:
        raise DsaError(st, name)
    return out


def dsa_sparse_attn_decode(q, kv_cache, idx, n_sel, sink, scale, out, stream=None):
    """Decode attention: q [B,H,512], kv_cache [B,N,512], out [B,H,512] fp32."""
    return _run("dsa_sparse_attn_decode", True, q, kv_cache, idx, n_sel, sink, scale, out, stream)


def dsa_sparse_attn_decode_rows(q, kv_cache, idx, n_sel, sink, scale, out, rows_per_slot, stream=None):
    """Decode with T = rows_per_slot query rows a slot: q [B*T,H,512], kv_cache [B,N,512],
    idx [B*T,k_max], n_sel [B*T], out [B*T,H,512] fp32; row r reads slot r // T."""
    T = int(rows_per_slot)
    if T < 1:
        raise ValueError("rows_per_slot must be >= 1")
    if kv_cache.dim() != 3 or q.dim() != 3 or q.shape[0] != kv_cache.shape[0] * T:
        raise ValueError("q must be [slots * rows_per_slot, heads, 512] for kv_cache [slots, N, 512]")
    R, H, N, k_max = _check(q, kv_cache, idx, n_sel, sink, out, decode=True, rows_per_slot=T)
    st = load().dsa_sparse_attn_decode_rows(q.data_ptr(), kv_cache.data_ptr(), idx.data_ptr(),
                                            n_sel.data_ptr(), sink.data_ptr(), ctypes.c_float(float(scale)),
                                            out.data_ptr(), R // T, T, H, N, k_max, _dtype_code(q),
                                            _stream_handle(stream))
    if st != DSA_OK:
        raise DsaError(st, "dsa_sparse_attn_decode_rows")
    return out


def dsa_sparse_attn_prefill(q, kv_cache, idx, n_sel, sink, scale, out, stream=None):
    """Prefill attention: q [R,H,512], kv_cache [N,512], out [R,H,512] fp32."""
    return _run("dsa_sparse_attn_prefill", False, q, kv_cache, idx, n_sel, sink, scale, out, stream)


def dsa_sparse_attn(q, kv_cache, idx, n_sel, sink, scale, out, rows_per_slot=0, stream=None):
    """Attention with the output type taken from `out` (float32 or bfloat16):
    rows_per_slot 0 is prefill (kv_cache [N,512]), T >= 1 decode with T rows a
    slot (kv_cache [R/T,N,512]).  A bf16 out holds the float32 result rounded
    to nearest even."""
    import torch
    T = int(rows_per_slot)
    if T < 0:
        raise ValueError("rows_per_slot must be >= 0")
    if not isinstance(out, torch.Tensor) or out.dtype not in (torch.float32, torch.bfloat16):
        raise TypeError("out must be a float32 or bfloat16 tensor")
    R, H, N, k_max = _check(q, kv_cache, idx, n_sel, sink, out, decode=T > 0, rows_per_slot=max(T, 1),
                            out_dtype=out.dtype)
    st = load().dsa_sparse_attn(q.data_ptr(), kv_cache.data_ptr(), idx.data_ptr(), n_sel.data_ptr(),
                                sink.data_ptr(), ctypes.c_float(float(scale)), out.data_ptr(), R, T, H, N,
                                k_max, _dtype_code(q), _dtype_code(out), _stream_handle(stream))
    if st != DSA_OK:
        raise DsaError(st, "dsa_sparse_attn")
    return out


def dsa_sparse_attn_decode_whole_rows(q, kv_cache, idx, n_sel, sink, scale, out, rows_per_slot=1, stream=None):
    """Decode without the key split (each row whole in one CTA, no partials):
    q [B*T,H,512], kv_cache [B,N,512], idx [B*T,k_max], n_sel [B*T], out
    [B*T,H,512] float32 or bfloat16; row r reads slot r // T (T =
    rows_per_slot).  For batches of about as many rows as SMs or more."""
    import torch
    T = int(rows_per_slot)
    if T < 1:
        raise ValueError("rows_per_slot must be >= 1")
    if not isinstance(out, torch.Tensor) or out.dtype not in (torch.float32, torch.bfloat16):
        raise TypeError("out must be a float32 or bfloat16 tensor")
    if kv_cache.dim() != 3 or q.dim() != 3 or q.shape[0] != kv_cache.shape[0] * T:
        raise ValueError("q must be [slots * rows_per_slot, heads, 512] for kv_cache [slots, N, 512]")
    R, H, N, k_max = _check(q, kv_cache, idx, n_sel, sink, out, decode=True, rows_per_slot=T, out_dtype=out.dtype)
    st = load().dsa_sparse_attn_decode_whole_rows(q.data_ptr(), kv_cache.data_ptr(), idx.data_ptr(),
                                                  n_sel.data_ptr(), sink.data_ptr(), ctypes.c_float(float(scale)),
                                                  out.data_ptr(), R, T, H, N, k_max, _dtype_code(q),
                                                  _dtype_code(out), _stream_handle(stream))
    if st != DSA_OK:
        raise DsaError(st, "dsa_sparse_attn_decode_whole_rows")
    return out


def _check_oproj(attn, w_o, out):
    import torch
    for name, t in (("attn", attn), ("w_o", w_o), ("out", out)):
        if not isinstance(t, torch.Tensor) or not t.is_cuda or not t.is_contiguous():
            raise ValueError("%s must be a contiguous CUDA tensor" % name)
    _same_device(("attn", attn), ("w_o", w_o), ("out", out))
    if attn.dtype != torch.bfloat16 or w_o.dtype != torch.bfloat16 or out.dtype != torch.float32:
        raise TypeError("attn and w_o must be bfloat16, out float32")
    if w_o.dim() != 2 or out.dim() != 2:
        raise ValueError("w_o [K, d_out] and out [rows, d_out] expected")
    R, K, d_out = attn.shape[0], w_o.shape[0], w_o.shape[1]
    if attn.numel() != R * K or tuple(out.shape) != (R, d_out):
        raise ValueError("attn [rows, K] (or [rows, H, 512] with H*512 = K) and out [rows, d_out] expected")
    return R, K, d_out


def dsa_oproj(attn, w_o, out, stream=None):
    """Output projection: out [R,d_out] fp32 = attn [R,K] bf16 . w_o [K,d_out] bf16."""
    R, K, d_out = _check_oproj(attn, w_o, out)
    st = load().dsa_oproj(attn.data_ptr(), w_o.data_ptr(), out.data_ptr(), R, K, d_out, _stream_handle(stream))
    if st != DSA_OK:
        raise DsaError(st, "dsa_oproj")
    return out


def dsa_sparse_attn_prefill_oproj(q, kv_cache, idx, n_sel, sink, scale, w_o, attn, out, stream=None):
    """Prefill attention (bf16 q/kv) into attn [R,H,512] bf16, then
    out [R,d_out] fp32 = attn . w_o [H*512,d_out] bf16."""
    R, H, N, k_max = _check(q, kv_cache, idx, n_sel, sink, attn, decode=False, out_dtype=attn.dtype)
    R2, K, d_out = _check_oproj(attn, w_o, out)
    if K != H * 512 or R2 != R:
        raise ValueError("w_o must be [heads * 512, d_out]")
    st = load().dsa_sparse_attn_prefill_oproj(q.data_ptr(), kv_cache.data_ptr(), idx.data_ptr(), n_sel.data_ptr(),
                                              sink.data_ptr(), ctypes.c_float(float(scale)), w_o.data_ptr(),
                                              attn.data_ptr(), out.data_ptr(), R, H, N, k_max, d_out,
                                              _stream_handle(stream))
    if st != DSA_OK:
        raise DsaError(st, "dsa_sparse_attn_prefill_oproj")
    return out


def dsa_sparse_attn_decode_noalloc(q, kv_cache, idx, n_sel, sink, scale, out, stream=None):
    """Decode attention that allocates no device memory (fixed static scratch;
    see include/dsa.h for its size limit and its sharing rules)."""
    return _run("dsa_sparse_attn_decode_noalloc", True, q, kv_cache, idx, n_sel, sink, scale, out,
                stream)


def dsa_topk_select(scores, n_valid, k, idx, n_sel, stream=None):
    """Top-k selection of each row of scores [R, ld] (float32) among positions
    [0, n_valid[r]) into idx [R, k_max] and n_sel [R] (int32)."""
    import torch
    for name, t in (("scores", scores), ("n_valid", n_valid), ("idx", idx), ("n_sel", n_sel)):
        if not isinstance(t, torch.Tensor) or not t.is_cuda or not t.is_contiguous():
            raise ValueError("%s must be a contiguous CUDA tensor" % name)
    _same_device(("scores", scores), ("n_valid", n_valid), ("idx", idx), ("n_sel", n_sel))
    if scores.dtype != torch.float32 or scores.dim() != 2:
        raise TypeError("scores must be a float32 [rows, ld] tensor")
    if n_valid.dtype != torch.int32 or idx.dtype != torch.int32 or n_sel.dtype != torch.int32:
        raise TypeError("n_valid, idx and n_sel must be int32")
    R, ld = scores.shape
    if tuple(n_valid.shape) != (R,) or tuple(n_sel.shape) != (R,) or idx.dim() != 2 or idx.shape[0] != R:
        raise ValueError("n_valid [rows], idx [rows, k_max] and n_sel [rows] expected")
    st = load().dsa_topk_select(scores.data_ptr(), ld, n_valid.data_ptr(), R, int(k), idx.data_ptr(),
                                idx.shape[1], n_sel.data_ptr(), _stream_handle(stream))
    if st != DSA_OK:
        raise DsaError(st, "dsa_topk_select")
    return idx, n_sel


# ------------------------------------------------------ paged 8-bit cache
# These calls are made once a layer and step with up to a dozen tensors each, so their checks are kept cheap:
# the current device and stream are asked for once a call, and what is right takes one pass.
_types = None


def _row_types():
    """((float32,), (bfloat16,), (int32,), (float32, bfloat16), (uint8, float8_e4m3fn), (uint8,)) of torch."""
    global _types
    if _types is None:
        import torch
        _types = ((torch.float32,), (torch.bfloat16,), (torch.int32,), (torch.float32, torch.bfloat16),
                  (torch.uint8, torch.float8_e4m3fn), (torch.uint8,))
    return _types


def _device(name, t):
    """The current CUDA device's index, for a call whose first tensor is t."""
    import torch
    if not isinstance(t, torch.Tensor):
        raise TypeError("%s must be a torch.Tensor" % name)
    if not t.is_cuda:
        raise ValueError("%s must be a contiguous CUDA tensor" % name)
    return torch.cuda.current_device()


def _shape(name, t, what, n):
    """t.shape, of n extents (`what` says which)."""
    try:
        got = t.shape
    except AttributeError:
        raise TypeError("%s must be a torch.Tensor" % name) from None
    if len(got) != n:
        raise ValueError("%s must be %s, got %s" % (name, what, list(got)))
    return got


def _tensor(name, t, dtypes, shape, dev):
    """Checks one argument: a contiguous CUDA tensor on device `dev`, of one of `dtypes` and of `shape`.
    Returns its address."""
    try:
        if t.shape == shape and t.dtype in dtypes and t.get_device() == dev and t.is_contiguous():
            return t.data_ptr()
    except AttributeError:
        raise TypeError("%s must be a torch.Tensor" % name) from None
    if not t.is_cuda or not t.is_contiguous():
        raise ValueError("%s must be a contiguous CUDA tensor" % name)
    if t.dtype not in dtypes:
        raise TypeError("%s must be %s, got %s" % (name, " or ".join(str(d) for d in dtypes), t.dtype))
    _same_device((name, t))
    raise ValueError("%s must be %s, got %s" % (name, list(shape), list(t.shape)))


def _stream_of(stream, dev):
    """The handle of `stream`, or of torch's current one."""
    if stream is None:
        import torch
        return torch._C._cuda_getCurrentRawStream(dev)
    return _stream_handle(stream)


def rope_table(n_positions, rope_dim, base=10000.0, device="cuda"):
    """float32 [n_positions, rope_dim / 2, 2] of cos, sin of position * base^(-2 i / rope_dim), for
    dsa_qk_norm_rope and dsa_paged_append.  The angles are computed in 64 bits: float32 angles of far
    positions would be off by more than the table's own rounding."""
    import torch
    f = float(base) ** (-torch.arange(0, rope_dim, 2, dtype=torch.float64, device=device) / rope_dim)
    a = torch.arange(n_positions, dtype=torch.float64, device=device)[:, None] * f[None, :]
    return torch.stack((a.cos(), a.sin()), dim=-1).float().contiguous()


def _rope_args(rope, f32, dev):
    """(address, n_positions, rope_dim) of a rotation table, or of none."""
    if rope is None:
        return 0, 0, 0
    n, half, _ = _shape("rope", rope, "[positions, rope_dim / 2, 2]", 3)
    return _tensor("rope", rope, f32, (n, half, 2), dev), n, 2 * half


def dsa_qk_norm_rope(q, positions, q_out, k=None, k_out=None, q_weight=None, k_weight=None, eps=1e-6, rope=None,
                     rope_style=DSA_ROPE_PAIRS, stream=None):
    """RMS norm of every 512-wide row of q [R,H,512] (and k [R,Hk,512]) and rotation of its last
    2 * rope.shape[1] columns by positions [R] (int32), into q_out (and k_out); float32 or bfloat16.
    rope is a float32 [n_positions, rope_dim / 2, 2] table of cos, sin (rope_table), or None for no
    rotation (positions may then be None); eps < 0 leaves the norm out; weights are float32 [512] or
    None (ones).  q_out may be q, k_out may be k."""
    f32, _, i32, rows, _, _ = _row_types()
    dev = _device("q", q)
    R, H, _ = _shape("q", q, "[rows, heads, 512]", 3)
    aq = _tensor("q", q, rows, (R, H, 512), dev)
    same = (q.dtype,)
    ao = _tensor("q_out", q_out, same, (R, H, 512), dev)
    if (k is None) != (k_out is None):
        raise ValueError("k and k_out go together")
    Hk = ak = ako = 0
    if k is not None:
        _, Hk, _ = _shape("k", k, "[rows, heads, 512]", 3)
        ak = _tensor("k", k, same, (R, Hk, 512), dev)
        ako = _tensor("k_out", k_out, same, (R, Hk, 512), dev)
    at, n_pos, rope_dim = _rope_args(rope, f32, dev)
    if rope is not None and positions is None:
        raise ValueError("a rotation needs positions")
    ap = _tensor("positions", positions, i32, (R,), dev) if positions is not None else 0
    wq = _tensor("q_weight", q_weight, f32, (512,), dev) if q_weight is not None else 0
    wk = _tensor("k_weight", k_weight, f32, (512,), dev) if k_weight is not None else 0
    st = (_lib or load()).dsa_qk_norm_rope(aq, ak, wq, wk, eps, at, n_pos, rope_dim, rope_style, ap, ao, ako, R, H, Hk,
                                           DSA_F32 if same == f32 else DSA_BF16, _stream_of(stream, dev))
    if st != DSA_OK:
        raise DsaError(st, "dsa_qk_norm_rope")
    return q_out if k is None else (q_out, k_out)


def _cache_args(cache, cache_scale, page_table, B, dev):
    """(addresses of cache, cache_scale, page_table, then n_pages, page_size, scale_block, max_pages)."""
    f32, _, i32, _, codes, _ = _row_types()
    n_pages, page_size, _ = _shape("cache", cache, "[pages, page_size, 512]", 3)
    ac = _tensor("cache", cache, codes, (n_pages, page_size, 512), dev)
    _, blocks = _shape("cache_scale", cache_scale, "[pages, page_size / scale_block]", 2)
    asc = _tensor("cache_scale", cache_scale, f32, (n_pages, blocks), dev)
    if blocks < 1 or page_size % blocks != 0:
        raise ValueError("cache_scale must be [pages, page_size / scale_block]")
    _, max_pages = _shape("page_table", page_table, "[sequences, max_pages]", 2)
    ap = _tensor("page_table", page_table, i32, (B, max_pages), dev)
    return ac, asc, ap, n_pages, page_size, page_size // blocks, max_pages


def dsa_paged_append(kv, row_offsets, seq_start, page_table, cache, cache_scale, norm_weight=None, eps=None,
                     rope=None, rope_style=DSA_ROPE_PAIRS, stream=None):
    """Append latent rows kv [R,512] (float32 or bfloat16) to a paged 8-bit cache: rows
    [row_offsets[b], row_offsets[b+1]) are tokens seq_start[b], ... of sequence b (int32 [B+1], [B]),
    normed (eps >= 0; by default 1e-6 with a norm_weight, no norm without one) and rotated (rope) as by
    dsa_qk_norm_rope, stored as e4m3 in cache
    [pages, page_size, 512] (uint8 or float8_e4m3fn) with a power-of-two scale for each block of
    scale_block tokens in cache_scale [pages, page_size / scale_block].  Returns (cache, cache_scale)."""
    f32, _, i32, rows, _, _ = _row_types()
    dev = _device("kv", kv)
    R, _ = _shape("kv", kv, "[rows, 512]", 2)
    ak = _tensor("kv", kv, rows, (R, 512), dev)
    B, = _shape("seq_start", seq_start, "[sequences]", 1)
    a_s = _tensor("seq_start", seq_start, i32, (B,), dev)
    ao = _tensor("row_offsets", row_offsets, i32, (B + 1,), dev)
    ac, asc, ap, n_pages, page_size, block, max_pages = _cache_args(cache, cache_scale, page_table, B, dev)
    at, n_pos, rope_dim = _rope_args(rope, f32, dev)
    w = _tensor("norm_weight", norm_weight, f32, (512,), dev) if norm_weight is not None else 0
    if eps is None:
        eps = 1e-6 if w else -1.0
    st = (_lib or load()).dsa_paged_append(ak, w, eps, at, n_pos, rope_dim, rope_style, ac, asc, ap, a_s, ao, R, B,
                                           n_pages, page_size, block, max_pages,
                                           DSA_F32 if kv.dtype in f32 else DSA_BF16, _stream_of(stream, dev))
    if st != DSA_OK:
        raise DsaError(st, "dsa_paged_append")
    return cache, cache_scale


def dsa_paged_workspace_bytes(rows: int, max_keys: int) -> int:
    """Bytes of workspace of a paged attention call over `rows` rows of at most max_keys keys."""
    return int(load().dsa_paged_workspace_bytes(int(rows), int(max_keys)))


def _paged_args(q, cache, cache_scale, page_table, seq_len, sink, out, rows_per_seq, idx, workspace, stream):
    """(addresses of q, cache, cache_scale, page_table, seq_len), (of idx), (of sink, out, workspace and its
    bytes), the sizes, the stream's handle and the workspace itself."""
    T = int(rows_per_seq)
    if T < 1:
        raise ValueError("rows_per_seq must be >= 1")
    f32, bf16, i32, _, _, u8 = _row_types()
    dev = _device("q", q)
    B, = _shape("seq_len", seq_len, "[sequences]", 1)
    a_l = _tensor("seq_len", seq_len, i32, (B,), dev)
    R = B * T
    _, H, _ = _shape("q", q, "[sequences * rows_per_seq, heads, 512]", 3)
    aq = _tensor("q", q, bf16, (R, H, 512), dev)
    ao = _tensor("out", out, bf16, (R, H, 512), dev)
    asi = _tensor("sink", sink, f32, (H,), dev) if sink is not None else 0
    ac, asc, ap, n_pages, page_size, block, max_pages = _cache_args(cache, cache_scale, page_table, B, dev)
    ai, max_keys = 0, max_pages * page_size
    if idx is not None:
        _, max_keys = _shape("idx", idx, "[rows, k_max]", 2)
        ai = _tensor("idx", idx, i32, (R, max_keys), dev)
    handle = _stream_of(stream, dev)
    if workspace is None:
        import torch
        nw = (_lib or load()).dsa_paged_workspace_bytes(R, max_keys)
        # from torch's allocator for this call alone, on the stream that the call runs on: the memory is
        # reused in that stream's order
        if stream is None or handle == torch.cuda.current_stream().cuda_stream:
            workspace = torch.empty(nw, dtype=torch.uint8, device=q.device)
        else:
            with torch.cuda.stream(torch.cuda.ExternalStream(handle) if handle else torch.cuda.default_stream()):
                workspace = torch.empty(nw, dtype=torch.uint8, device=q.device)
        aw = workspace.data_ptr()
    else:
        nw, = _shape("workspace", workspace, "[bytes]", 1)
        aw = _tensor("workspace", workspace, u8, (nw,), dev)
    return (aq, ac, asc, ap, a_l), ai, (ao, aw, nw), asi, (B, T, H, n_pages, page_size, block, max_pages), handle, workspace


def dsa_paged_attn(q, cache, cache_scale, page_table, seq_len, sink, scale, out, rows_per_seq=1, workspace=None,
                   stream=None):
    """Attention of the rows_per_seq = T newest tokens of each sequence over its whole paged context:
    q [B*T,H,512] bfloat16, cache [pages,page_size,512] e4m3, cache_scale [pages,page_size/scale_block],
    page_table [B,max_pages] int32, seq_len [B] int32 (the T rows' tokens included; row t sees all but
    the T-1-t newest), sink [H] float32 or None, out [B*T,H,512] bfloat16.  workspace: uint8 of
    dsa_paged_workspace_bytes(B*T, max_pages*page_size) bytes, or None to allocate it for the call."""
    ins, _, outs, asi, dims, handle, workspace = _paged_args(q, cache, cache_scale, page_table, seq_len, sink, out,
                                                             rows_per_seq, None, workspace, stream)
    st = (_lib or load()).dsa_paged_attn(*ins, asi, scale, *outs, *dims, handle)
    if st != DSA_OK:
        raise DsaError(st, "dsa_paged_attn")
    return out


def dsa_paged_sparse_attn(q, cache, cache_scale, page_table, seq_len, idx, n_sel, sink, scale, out, rows_per_seq=1,
                          workspace=None, stream=None):
    """dsa_paged_attn over a selection: row r attends to positions idx[r, :n_sel[r]] of its sequence
    (idx [B*T,k_max], n_sel [B*T] int32).  Prefill is one sequence with rows_per_seq rows.  workspace:
    dsa_paged_workspace_bytes(B*T, k_max) bytes, or None."""
    if idx is None:
        raise TypeError("idx must be a torch.Tensor")
    ins, ai, outs, asi, dims, handle, workspace = _paged_args(q, cache, cache_scale, page_table, seq_len, sink, out,
                                                              rows_per_seq, idx, workspace, stream)
    R, k_max = idx.shape
    an = _tensor("n_sel", n_sel, _row_types()[2], (R,), q.get_device())
    st = (_lib or load()).dsa_paged_sparse_attn(*ins, ai, an, asi, scale, *outs, *dims, k_max, handle)
    if st != DSA_OK:
        raise DsaError(st, "dsa_paged_sparse_attn")
    return out


# ------------------------------------------------- head-sharded parallelism
def dsa_head_shard(H: int, world: int, rank: int) -> HeadShardPlan:
    """Which heads rank `rank` of `world` owns (host only; see include/dsa.h)."""
    plan = HeadShardPlan()
    st = load().dsa_head_shard(int(H), int(world), int(rank), ctypes.byref(plan))
    if st != DSA_OK:
        raise DsaError(st, "dsa_head_shard")
    return plan


def dsa_shard_heads(q, sink, q_local, sink_local, world: int, rank: int, stream=None):
    """q_local [R,hpr,512], sink_local [hpr] = rank's heads of q [R,H,512],
    sink [H] (zero for padding heads)."""
    import torch
    for name, t in (("q", q), ("sink", sink), ("q_local", q_local), ("sink_local", sink_local)):
        if not isinstance(t, torch.Tensor) or not t.is_cuda or not t.is_contiguous():
            raise ValueError("%s must be a contiguous CUDA tensor" % name)
    _same_device(("q", q), ("sink", sink), ("q_local", q_local), ("sink_local", sink_local))
    if q.dim() != 3 or q.shape[2] != 512 or q_local.dtype != q.dtype:
        raise ValueError("q [rows, heads, 512] and q_local of the same dtype expected")
    R, H = q.shape[0], q.shape[1]
    plan = dsa_head_shard(H, world, rank)
    if tuple(q_local.shape) != (R, plan.heads_per_rank, 512) or tuple(sink.shape) != (H,) \
            or tuple(sink_local.shape) != (plan.heads_per_rank,):
        raise ValueError("q_local [rows, heads_per_rank, 512], sink [heads], sink_local [heads_per_rank] expected")
    if sink.dtype != torch.float32 or sink_local.dtype != torch.float32:
        raise TypeError("sinks must be float32")
    st = load().dsa_shard_heads(q.data_ptr(), sink.data_ptr(), q_local.data_ptr(), sink_local.data_ptr(),
                                R, H, int(world), int(rank), _dtype_code(q), _stream_handle(stream))
    if st != DSA_OK:
        raise DsaError(st, "dsa_shard_heads")
    return q_local, sink_local


def dsa_unshard_heads(gathered, out, world: int, stream=None):
    """out [R,H,512] from gathered [world,R,hpr,512] (padding heads dropped)."""
    import torch
    for name, t in (("gathered", gathered), ("out", out)):
        if not isinstance(t, torch.Tensor) or not t.is_cuda or not t.is_contiguous():
            raise ValueError("%s must be a contiguous CUDA tensor" % name)
    _same_device(("gathered", gathered), ("out", out))
    if out.dim() != 3 or out.shape[2] != 512 or gathered.dtype != out.dtype:
        raise ValueError("out [rows, heads, 512] and gathered of the same dtype expected")
    R, H = out.shape[0], out.shape[1]
    plan = dsa_head_shard(H, world, 0)
    if tuple(gathered.shape) != (world, R, plan.heads_per_rank, 512):
        raise ValueError("gathered must be [world, rows, heads_per_rank, 512]")
    st = load().dsa_unshard_heads(gathered.data_ptr(), out.data_ptr(), R, H, int(world), _dtype_code(out),
                                  _stream_handle(stream))
    if st != DSA_OK:
        raise DsaError(st, "dsa_unshard_heads")
    return out


def tp_sparse_attn(q_local, kv_cache, idx, n_sel, sink_local, scale, out_local, gathered, out, group=None,
                   rows_per_slot=0, stream=None):
    """One rank's step of head-sharded attention, all on one stream (torch's
    current one unless `stream` is given): the attention call over the rank's
    heads into out_local [R,hpr,512], an all-gather of every rank's out_local
    into gathered [world,R,hpr,512] (torch.distributed on `group`; NCCL on
    GPUs), then the gathered outputs laid out as out [R,H,512].  With one
    rank, out_local itself is the gathered array."""
    import torch
    import torch.distributed as dist
    world = dist.get_world_size(group) if dist.is_available() and dist.is_initialized() else 1
    with torch.cuda.stream(stream if stream is not None else torch.cuda.current_stream()):
        dsa_sparse_attn(q_local, kv_cache, idx, n_sel, sink_local, scale, out_local,
                        rows_per_slot=rows_per_slot)
        if world > 1:
            dist.all_gather_into_tensor(gathered.view(-1), out_local.view(-1), group=group)
            src = gathered
        else:
            src = out_local.view((1,) + tuple(out_local.shape))
        return dsa_unshard_heads(src, out, world)


def tp_oproj_weights(w_o, H: int, world: int, rank: int):
    """The rank's rows of the output projection w_o [H*512, d_out] (bf16) for
    tp_sparse_attn_oproj: its heads' 512-row blocks, then zero blocks for its
    padding heads, whose attention outputs (q = 0, sink = 0) must not reach
    the projection.  One-time weight preparation: a view of w_o when the rank
    has no padding heads, else a padded copy."""
    import torch
    if not isinstance(w_o, torch.Tensor) or w_o.dim() != 2 or w_o.shape[0] != H * 512:
        raise ValueError("w_o must be a [heads * 512, d_out] tensor")
    plan = dsa_head_shard(H, world, rank)
    lo, n = plan.first_head * 512, plan.real_heads * 512
    if plan.real_heads == plan.heads_per_rank:
        return w_o[lo:lo + n]
    local = torch.zeros((plan.heads_per_rank * 512, w_o.shape[1]), dtype=w_o.dtype, device=w_o.device)
    local[:n].copy_(w_o[lo:lo + n])
    return local


def tp_sparse_attn_oproj(q_local, kv_cache, idx, n_sel, sink_local, scale, w_o_local, attn_local, out,
                         group=None, rows_per_slot=0, stream=None, scatter_out=None):
    """One rank's step of head-sharded attention followed by the output
    projection, row-parallel, all on one stream (torch's current one unless
    `stream` is given): the attention over the rank's heads into attn_local
    [R,hpr,512] (bf16), the rank's share of the projection out [R,d_out] fp32
    = attn_local . w_o_local (w_o_local from tp_oproj_weights), then a sum
    of every rank's share over `group` (torch.distributed all-reduce; NCCL on
    GPUs), so that every rank holds the whole projection.  Against
    tp_sparse_attn followed by the projection, the ranks exchange the
    projected rows (R x d_out fp32) instead of the attention outputs
    (R x H x 512 bf16).  The shares are summed in the collective's order, so
    the result differs from the one-GPU projection by fp32 rounding.

    With `scatter_out` ([R / world, d_out] float32, R a multiple of the world
    size) the sum is reduce-scattered instead: rank w receives rows
    [w R / world, (w + 1) R / world) of the projection in scatter_out, and
    `out` keeps the rank's own unsummed share.  Returns the tensor that holds
    the summed rows."""
    import torch
    import torch.distributed as dist
    world = dist.get_world_size(group) if dist.is_available() and dist.is_initialized() else 1
    if attn_local.dtype != torch.bfloat16:
        raise TypeError("attn_local must be bfloat16 (the projection's A operand)")
    R = attn_local.shape[0]
    if scatter_out is not None:
        if (not isinstance(scatter_out, torch.Tensor) or scatter_out.dtype != torch.float32
                or not scatter_out.is_contiguous() or R % world != 0
                or tuple(scatter_out.shape) != (R // world, out.shape[-1])):
            raise ValueError("scatter_out must be a contiguous float32 [rows / world, d_out] tensor, "
                             "rows a multiple of the world size")
        _same_device(("out", out), ("scatter_out", scatter_out))
    with torch.cuda.stream(stream if stream is not None else torch.cuda.current_stream()):
        dsa_sparse_attn(q_local, kv_cache, idx, n_sel, sink_local, scale, attn_local,
                        rows_per_slot=rows_per_slot)
        dsa_oproj(attn_local.view(R, -1), w_o_local, out)
        if scatter_out is not None:
            if world > 1:
                dist.reduce_scatter_tensor(scatter_out, out, op=dist.ReduceOp.SUM, group=group)
            else:
                scatter_out.copy_(out)
            return scatter_out
        if world > 1:
            dist.all_reduce(out, op=dist.ReduceOp.SUM, group=group)
        return out


def dsa_selftest_wait_limit(stream=None) -> None:
    """Queue the bounded-wait self-test (sets DSA_DEVERR_TIMEOUT after ~2 s)."""
    st = load().dsa_selftest_wait_limit(_stream_handle(stream))
    if st != DSA_OK:
        raise DsaError(st, "dsa_selftest_wait_limit")


def dsa_get_device_error(stream=None) -> int:
    """Synchronise the stream, return and clear the device error word."""
    code = ctypes.c_uint32(0)
    st = load().dsa_get_device_error(_stream_handle(stream), ctypes.byref(code))
    if st != DSA_OK:
        raise DsaError(st, "dsa_get_device_error")
    return int(code.value)


def dsa_shutdown() -> None:
    st = load().dsa_shutdown()
    if st != DSA_OK:
        raise DsaError(st, "dsa_shutdown")
