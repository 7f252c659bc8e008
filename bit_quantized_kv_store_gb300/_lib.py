"""ctypes binding of libkvq (include/kvq.h).

Argument marshalling only: every step of the path runs in the CUDA kernels of
libkvq.so.  Tensors are torch tensors on a CUDA device; their ``data_ptr()`` and
the current torch stream are passed straight to the C entry points.  If the
library has not been built, loading raises: there is no fallback.
"""
from __future__ import annotations

import ctypes
import os

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
# KVQ_SANITIZE=1: the host-sanitizer build (argument validation checked on the CPU)
LIB_PATH = os.path.join(_PKG, "_build_san" if os.environ.get("KVQ_SANITIZE") == "1" else "_build", "libkvq.so")

OK, ERR_INVALID_ARG, ERR_UNSUPPORTED, ERR_CUDA, ERR_WORKSPACE_TOO_SMALL = 0, -1, -2, -3, -4
DEV_BAD_SLOT, DEV_BAD_PAGE, DEV_BAD_LENGTH, DEV_BAD_INDEX, DEV_TIMEOUT = 1, 2, 4, 8, 16
DT_F32, DT_BF16 = 0, 1
# Q4_0: the 4-bit rows without the rotation; TQ4: randomized-Hadamard rows with the Lloyd-Max codebook
FMT_Q4_HAD32, FMT_BF16, FMT_FP8_ROW, FMT_Q4_0, FMT_TQ4 = 0, 1, 2, 3, 4

_P = ctypes.c_void_p
_I32 = ctypes.c_int32
_I64 = ctypes.c_int64
_SZ = ctypes.c_size_t
_F = ctypes.c_float


class CacheDesc(ctypes.Structure):
    _fields_ = [("format", _I32), ("num_kv_heads", _I32), ("head_dim", _I32), ("rope_dim", _I32),
                ("page_size", _I32), ("num_pages", _I32), ("k", _P), ("k_scale", _P), ("v", _P), ("v_scale", _P),
                ("signs", _P)]


class RowsDesc(ctypes.Structure):
    _fields_ = [("data", _P), ("dtype", _I32), ("heads", _I32), ("tok_stride", _I64), ("head_stride", _I64)]


class NormDesc(ctypes.Structure):
    _fields_ = [("weight", _P), ("dtype", _I32), ("eps", _F), ("offset", _F)]


class RopeDesc(ctypes.Structure):
    _fields_ = [("rot_dim", _I32), ("interleaved", _I32), ("num_axes", _I32), ("reserved", _I32), ("table", _P)]


_ROWS, _NORM, _ROPE, _CACHE = (ctypes.POINTER(c) for c in (RowsDesc, NormDesc, RopeDesc, CacheDesc))

# name -> (restype, argtypes); mirrors include/kvq.h
SIGNATURES = {
    "kvq_version": (_I32, []),
    "kvq_status_string": (ctypes.c_char_p, [_I32]),
    "kvq_last_cuda_error": (_I32, []),
    "kvq_plane_bytes": (_SZ, [ctypes.POINTER(CacheDesc), _I32]),
    "kvq_store": (_I32, [ctypes.POINTER(CacheDesc), _P, _P, _I32, _I64, _P, _P, _P]),
    "kvq_rotate_query": (_I32, [_P, _I32, _P, _I64, _I32, _P]),
    "kvq_tq4_rotate": (_I32, [ctypes.POINTER(CacheDesc), _P, _I32, _P, _I64, _I32, _P]),
    "kvq_store_rotate": (_I32, [ctypes.POINTER(CacheDesc), _P, _P, _I32, _I64, _P, _P, _P, _I32, _P, _I64, _P]),
    "kvq_decode_workspace_size": (_SZ, [ctypes.POINTER(CacheDesc), _I32, _I32, _I32, _I32]),
    "kvq_decode_attn": (_I32, [ctypes.POINTER(CacheDesc), _P, _I32, _I32, _P, _P, _I32, _I32, _P, _I32, _F, _P,
                               _SZ, _P]),
    "kvq_decode_window": (_I32, [ctypes.POINTER(CacheDesc), _P, _I32, _I32, _P, _P, _I32, _I32, _F, _P, _SZ, _P]),
    "kvq_decode_merged": (_I32, [ctypes.POINTER(CacheDesc), _P, _I32, _I32, _P, _P, _I32, _I32, _F, _P, _SZ, _P,
                                 _P]),
    "kvq_decode_attn_unrotated": (_I32, [ctypes.POINTER(CacheDesc), _P, _I32, _I32, _I32, _P, _P, _I32, _I32, _P,
                                         _I32, _F, _P, _SZ, _P]),
    "kvq_decode_step": (_I32, [ctypes.POINTER(CacheDesc), _P, _P, _I32, _P, _I32, _I32, _I32, _P, _P, _I32, _I32, _F,
                               _P, _SZ, _P]),
    "kvq_merge": (_I32, [ctypes.POINTER(CacheDesc), _P, _SZ, _I32, _I32, _P, _I32, _I32, _I32, _P, _P]),
    "kvq_prefill_attn": (_I32, [ctypes.POINTER(CacheDesc), _P, _I32, _I32, _I32, _I32, _P, _I32, _F, _P, _P, _P]),
    "kvq_read_status": (_I32, [_P, _P, _P]),
    "kvq_prefill_fp8_workspace_size": (_SZ, [ctypes.POINTER(CacheDesc), _I32, _I32]),
    "kvq_selftest_wait_timeout": (_I32, [_P, _P]),
    "kvq_prefill_attn_fp8": (_I32, [ctypes.POINTER(CacheDesc), _P, _I32, _I32, _I32, _P, _I32, _F, _P, _SZ, _P, _P]),
    "kvq_noalloc_scratch_bytes": (_SZ, []),
    "kvq_decode_noalloc": (_I32, [ctypes.POINTER(CacheDesc), _P, _I32, _I32, _P, _P, _I32, _I32, _P, _I32, _F, _I32,
                                  _P, _P, _P]),
    "kvq_rope_table": (_I32, [_P, _P, _I32, _P]),
    "kvq_norm_rope": (_I32, [_ROWS, _ROWS, _I64, _I32, _NORM, _ROPE, _P, _I64, _P, _P]),
    "kvq_norm_rope_store": (_I32, [_CACHE, _ROWS, _ROWS, _ROWS, _I64, _NORM, _NORM, _ROPE, _P, _I64, _P, _ROWS, _I32,
                                   _P, _P]),
    "kvq_load": (_I32, [_CACHE, _P, _I64, _I32, _ROWS, _ROWS, _P, _P]),
    "kvq_load_seqs": (_I32, [_CACHE, _P, _I32, _I32, _P, _P, _I64, _I32, _ROWS, _ROWS, _P, _P]),
    "kvq_merge_diff": (_I32, [_CACHE, _P, _SZ, _I32, _I32, _P, _I32, _I32, _I32, _P, _I64, _NORM, _F, _P, _I32, _P]),
    "kvq_diff_heads": (_I32, [_P, _I64, _I32, _I32, _P, _I64, _NORM, _F, _P, _I32, _P]),
}

_lib = None


def lib():
    """Load libkvq.so (raises if it is missing: the CUDA path has no substitute)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"libkvq.so is not built ({LIB_PATH}); run bit_quantized_kv_store_gb300.build.build()")
        L = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in SIGNATURES.items():
            f = getattr(L, name)
            f.restype = res
            f.argtypes = args
        _lib = L
    return _lib


class KvqError(RuntimeError):
    def __init__(self, status, where):
        msg = lib().kvq_status_string(status).decode()
        if status == ERR_CUDA:
            msg += f" (cudaError {lib().kvq_last_cuda_error()})"
        super().__init__(f"{where}: {msg} [{status}]")
        self.status = status


def _check(status, where):
    if status != OK:
        raise KvqError(status, where)


def _ptr(t):
    """Device address of a tensor for the C ABI (None -> NULL).  The kernels read
    plain row-major device memory, so a host tensor (whose address the GPU would
    fault on) or a strided view (read with the wrong layout) is refused here."""
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError(f"kvq: expected a CUDA tensor, got one on {t.device}")
    if not t.is_contiguous():
        raise ValueError("kvq: expected a contiguous tensor (call .contiguous())")
    return t.data_ptr()


# The current stream's handle without building a torch Stream object (the
# accessor torch's own compiler uses; the public route is the fallback).
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream(stream=None):
    """The CUDA stream handle to launch on: `stream`'s, else the current
    device's current torch stream."""
    if stream is not None:
        return stream.cuda_stream
    if _raw_stream is not None:
        return _raw_stream(torch.cuda.current_device())
    return torch.cuda.current_stream().cuda_stream


def _dtype_code(t):
    if t.dtype == torch.float32:
        return DT_F32
    if t.dtype == torch.bfloat16:
        return DT_BF16
    raise TypeError(f"unsupported activation dtype {t.dtype}")


class Cache:
    """A paged KV cache: the planes are caller-owned torch tensors on one device.

    Q4:   k, v codes [num_pages, Hk, page_size, D/2] uint8; k_scale, v_scale
          [num_pages, Hk, page_size, D/32] float16.
    BF16: k, v [num_pages, Hk, page_size, D] bfloat16.
    FP8:  k (latent codes) [num_pages, page_size, D] uint8, v (rope codes)
          [num_pages, page_size, R] uint8, k_scale / v_scale [num_pages, page_size] f32.
    TQ4:  k, v codes [num_pages, Hk, page_size, D/2] uint8; k_scale, v_scale
          [num_pages, Hk, page_size] float16; `signs` the rotation's sign mask,
          int32 [D/32] (bit i set: element i negated), given by the caller.
    """

    def __init__(self, fmt, num_kv_heads, head_dim, page_size, num_pages, device="cuda", rope_dim=0, signs=None):
        if torch.device(device).type != "cuda":
            raise ValueError(f"kvq: the cache planes live in device memory, not on {device}")
        self.fmt, self.Hk, self.D, self.page_size, self.num_pages = fmt, num_kv_heads, head_dim, page_size, num_pages
        self.rope = rope_dim
        self.signs = None
        rows = (num_pages, num_kv_heads, page_size)
        if fmt == FMT_TQ4:
            if signs is None or signs.numel() != head_dim // 32:
                raise ValueError("TQ4 needs a sign mask of head_dim / 32 words")
            self.signs = signs.to(device=device, dtype=torch.int32).contiguous()
            self.k = torch.zeros(rows + (head_dim // 2,), dtype=torch.uint8, device=device)
            self.v = torch.zeros_like(self.k)
            self.k_scale = torch.zeros(rows, dtype=torch.float16, device=device)
            self.v_scale = torch.zeros_like(self.k_scale)
        elif fmt in (FMT_Q4_HAD32, FMT_Q4_0):
            self.k = torch.zeros(rows + (head_dim // 2,), dtype=torch.uint8, device=device)
            self.v = torch.zeros_like(self.k)
            self.k_scale = torch.zeros(rows + (head_dim // 32,), dtype=torch.float16, device=device)
            self.v_scale = torch.zeros_like(self.k_scale)
        elif fmt == FMT_BF16:
            self.k = torch.zeros(rows + (head_dim,), dtype=torch.bfloat16, device=device)
            self.v = torch.zeros_like(self.k)
            self.k_scale = self.v_scale = None
        elif fmt == FMT_FP8_ROW:
            assert num_kv_heads == 1
            self.k = torch.zeros(rows + (head_dim,), dtype=torch.uint8, device=device)
            self.v = torch.zeros(rows + (rope_dim,), dtype=torch.uint8, device=device)
            self.k_scale = torch.zeros(rows, dtype=torch.float32, device=device)
            self.v_scale = torch.zeros(rows, dtype=torch.float32, device=device)
        else:
            raise ValueError(fmt)
        self.refresh()

    def refresh(self):
        for t in (self.k, self.v, self.k_scale, self.v_scale, self.signs):
            if t is not None and not (t.is_cuda and t.is_contiguous()):
                raise ValueError("kvq: cache planes must be contiguous CUDA tensors")
        self.desc = CacheDesc(self.fmt, self.Hk, self.D, self.rope, self.page_size, self.num_pages,
                              self.k.data_ptr(), 0 if self.k_scale is None else self.k_scale.data_ptr(),
                              self.v.data_ptr(), 0 if self.v_scale is None else self.v_scale.data_ptr(),
                              0 if self.signs is None else self.signs.data_ptr())

    @property
    def ref(self):
        return ctypes.byref(self.desc)

    def nbytes(self):
        return sum(t.numel() * t.element_size() for t in (self.k, self.v, self.k_scale, self.v_scale) if t is not None)


def store(cache: Cache, k, v, slot_mapping, status=None, stream=None):
    n_tok = k.shape[0]
    _check(lib().kvq_store(cache.ref, _ptr(k), _ptr(v), _dtype_code(k), n_tok, _ptr(slot_mapping), _ptr(status),
                           _stream(stream)), "kvq_store")


def rotate_query(x, out=None, stream=None):
    D = x.shape[-1]
    rows = x.numel() // D
    if out is None:
        out = torch.empty(x.shape, dtype=torch.float32, device=x.device)
    _check(lib().kvq_rotate_query(_ptr(x), _dtype_code(x), _ptr(out), rows, D, _stream(stream)), "kvq_rotate_query")
    return out


def tq4_rotate(cache: Cache, x, inverse=False, out=None, stream=None):
    """The TQ4 cache's signed row transform (queries in; inverse: outputs back)."""
    rows = x.numel() // cache.D
    if out is None:
        out = torch.empty(x.shape, dtype=torch.float32, device=x.device)
    _check(lib().kvq_tq4_rotate(cache.ref, _ptr(x), _dtype_code(x), _ptr(out), rows, int(inverse), _stream(stream)),
           "kvq_tq4_rotate")
    return out


def store_rotate(cache: Cache, k, v, slot_mapping, q, out=None, status=None, stream=None):
    """store(cache, k, v, slot_mapping) and rotate_query(q, out) in one launch
    (4-bit format, a few tokens); returns the rotated queries."""
    if out is None:
        out = torch.empty(q.shape, dtype=torch.float32, device=q.device)
    rows = q.numel() // q.shape[-1]
    _check(lib().kvq_store_rotate(cache.ref, _ptr(k), _ptr(v), _dtype_code(k), k.shape[0], _ptr(slot_mapping),
                                  _ptr(status), _ptr(q), _dtype_code(q), _ptr(out), rows, _stream(stream)),
           "kvq_store_rotate")
    return out


def workspace_size(cache: Cache, num_seqs, num_q_heads, max_seq_len, n_sel=0):
    return lib().kvq_decode_workspace_size(cache.ref, num_seqs, num_q_heads, max_seq_len, n_sel)


def alloc_workspace(cache: Cache, num_seqs, num_q_heads, max_seq_len, n_sel=0, device="cuda"):
    n = workspace_size(cache, num_seqs, num_q_heads, max_seq_len, n_sel)
    return torch.zeros(n, dtype=torch.uint8, device=device)


def decode_attn(cache: Cache, q, seq_lens, block_tables, max_seq_len, sm_scale, workspace, sel=None, stream=None):
    B, Hq = q.shape[0], q.shape[1]
    n_sel = 0 if sel is None else sel.shape[1]
    _check(lib().kvq_decode_attn(cache.ref, _ptr(q), B, Hq, _ptr(seq_lens), _ptr(block_tables),
                                 block_tables.shape[1], max_seq_len, _ptr(sel), n_sel, float(sm_scale),
                                 _ptr(workspace), workspace.numel(), _stream(stream)), "kvq_decode_attn")


def decode_step(cache: Cache, k_new, v_new, q, seq_lens, block_tables, max_seq_len, sm_scale, workspace,
                stream=None):
    """Store each sequence's new K/V rows at position seq_lens[b] - 1, rotate the
    (unrotated) queries and write the split-T partials, in one launch (4-bit
    formats); merge with merge()."""
    B, Hq = q.shape[0], q.shape[1]
    _check(lib().kvq_decode_step(cache.ref, _ptr(k_new), _ptr(v_new), _dtype_code(k_new), _ptr(q), _dtype_code(q), B,
                                 Hq, _ptr(seq_lens), _ptr(block_tables), block_tables.shape[1], max_seq_len,
                                 float(sm_scale), _ptr(workspace), workspace.numel(), _stream(stream)),
           "kvq_decode_step")


def decode_merged(cache: Cache, q_rot, seq_lens, block_tables, max_seq_len, sm_scale, workspace, out=None,
                  stream=None):
    """Decode partials and their merge in one launch (4-bit formats); q_rot as for
    decode_attn.  Returns out [B, Hq, 256]."""
    B, Hq = q_rot.shape[0], q_rot.shape[1]
    if out is None:
        out = torch.empty((B, Hq, cache.D), dtype=torch.float32, device=q_rot.device)
    _check(lib().kvq_decode_merged(cache.ref, _ptr(q_rot), B, Hq, _ptr(seq_lens), _ptr(block_tables),
                                   block_tables.shape[1], max_seq_len, float(sm_scale), _ptr(workspace),
                                   workspace.numel(), _ptr(out), _stream(stream)), "kvq_decode_merged")
    return out


def decode_window(cache: Cache, q_rot, row_lens, block_table, max_seq_len, sm_scale, workspace, stream=None):
    """Partials for a window of rows of one sequence sharing its block table
    (row i attends keys 0 .. row_lens[i] - 1); merge with merge(num_seqs=rows)."""
    R, Hq = q_rot.shape[0], q_rot.shape[1]
    bt = block_table.reshape(-1)
    _check(lib().kvq_decode_window(cache.ref, _ptr(q_rot), R, Hq, _ptr(row_lens), _ptr(bt), bt.numel(), max_seq_len,
                                   float(sm_scale), _ptr(workspace), workspace.numel(), _stream(stream)),
           "kvq_decode_window")


def decode_window_causal(cache: Cache, q, prefix_len, block_table, sm_scale, workspace, out=None, stream=None):
    """One speculative-decoding verify step: the R rows of q sit at positions
    prefix_len .. prefix_len + R - 1 (their keys already stored) and row i attends
    keys 0 .. prefix_len + i.  Rotates the queries (Hadamard format), decodes the
    window, merges; returns the outputs [R, Hq, D]."""
    R, Hq = q.shape[0], q.shape[1]
    row_lens = torch.arange(prefix_len + 1, prefix_len + R + 1, dtype=torch.int32, device=q.device)
    qq = rotate_query(q, stream=stream) if cache.fmt == FMT_Q4_HAD32 else q.float()
    decode_window(cache, qq, row_lens, block_table, prefix_len + R, sm_scale, workspace, stream=stream)
    if out is None:
        out = torch.empty((R, Hq, cache.D), dtype=torch.float32, device=q.device)
    return merge(cache, workspace, R, Hq, row_lens, prefix_len + R, out, stream=stream)


def decode_attn_unrotated(cache: Cache, q, seq_lens, block_tables, max_seq_len, sm_scale, workspace, sel=None,
                          stream=None):
    """Decode partials from an unrotated query (4-bit format): the rotation runs in the decode kernel."""
    B, Hq = q.shape[0], q.shape[1]
    n_sel = 0 if sel is None else sel.shape[1]
    _check(lib().kvq_decode_attn_unrotated(cache.ref, _ptr(q), _dtype_code(q), B, Hq, _ptr(seq_lens), _ptr(block_tables),
                                           block_tables.shape[1], max_seq_len, _ptr(sel), n_sel, float(sm_scale),
                                           _ptr(workspace), workspace.numel(), _stream(stream)),
           "kvq_decode_attn_unrotated")


def merge(cache: Cache, workspace, num_seqs, num_q_heads, seq_lens, max_seq_len, out, n_sel=0, rotate_back=None,
          stream=None):
    if rotate_back is None:
        rotate_back = cache.fmt in (FMT_Q4_HAD32, FMT_TQ4)
    _check(lib().kvq_merge(cache.ref, _ptr(workspace), workspace.numel(), num_seqs, num_q_heads, _ptr(seq_lens),
                           max_seq_len, n_sel, int(rotate_back), _ptr(out), _stream(stream)), "kvq_merge")
    return out


def decode(cache: Cache, q, seq_lens, block_tables, max_seq_len, sm_scale, workspace, out=None, sel=None,
           stream=None):
    """Rotate the query (4-bit formats), decode partials, merge: one decode step."""
    B, Hq = q.shape[0], q.shape[1]
    qq = q
    if cache.fmt == FMT_Q4_HAD32:
        qq = rotate_query(q, stream=stream)
    elif cache.fmt == FMT_TQ4:
        qq = tq4_rotate(cache, q, stream=stream)
    elif q.dtype != torch.float32:
        qq = q.float()
    decode_attn(cache, qq, seq_lens, block_tables, max_seq_len, sm_scale, workspace, sel=sel, stream=stream)
    if out is None:
        out = torch.empty((B, Hq, cache.D), dtype=torch.float32, device=q.device)
    return merge(cache, workspace, B, Hq, seq_lens, max_seq_len, out, n_sel=0 if sel is None else sel.shape[1],
                 stream=stream)


def prefill_attn(cache: Cache, q, q_start, block_table, sm_scale, out=None, status=None, stream=None):
    n_q, Hq = q.shape[0], q.shape[1]
    if out is None:
        out = torch.empty((n_q, Hq, cache.D), dtype=torch.float32, device=q.device)
    bt = block_table.reshape(-1)
    _check(lib().kvq_prefill_attn(cache.ref, _ptr(q), _dtype_code(q), n_q, Hq, int(q_start), _ptr(bt), bt.numel(),
                                  float(sm_scale), _ptr(out), _ptr(status), _stream(stream)), "kvq_prefill_attn")
    return out


def decode_noalloc(cache: Cache, q_rot, seq_lens, block_tables, max_seq_len, sm_scale, out, sel=None,
                   rotate_back=None, status=None, stream=None):
    """Decode partials + merge without a caller workspace (the library's fixed
    device scratch array is used instead; see kvq_decode_noalloc in kvq.h)."""
    B, Hq = q_rot.shape[0], q_rot.shape[1]
    n_sel = 0 if sel is None else sel.shape[1]
    if rotate_back is None:
        rotate_back = cache.fmt in (FMT_Q4_HAD32, FMT_TQ4)
    _check(lib().kvq_decode_noalloc(cache.ref, _ptr(q_rot), B, Hq, _ptr(seq_lens), _ptr(block_tables),
                                    block_tables.shape[1], max_seq_len, _ptr(sel), n_sel, float(sm_scale),
                                    int(rotate_back), _ptr(out), _ptr(status), _stream(stream)), "kvq_decode_noalloc")
    return out


def prefill_attn_fp8(cache: Cache, q, q_start, block_table, sm_scale, workspace=None, out=None, stream=None):
    """Causal prefill of q [n_q, Hq, 576] (positions q_start ..) over the fp8
    latent cache; returns out [n_q, Hq, 512] (the workspace's first word is the
    status)."""
    n_q, Hq = q.shape[0], q.shape[1]
    if workspace is None:
        workspace = torch.zeros(lib().kvq_prefill_fp8_workspace_size(cache.ref, n_q, Hq), dtype=torch.uint8,
                                device=q.device)
    if out is None:
        out = torch.empty((n_q, Hq, cache.D), dtype=torch.float32, device=q.device)
    bt = block_table.reshape(-1)
    _check(lib().kvq_prefill_attn_fp8(cache.ref, _ptr(q), n_q, Hq, int(q_start), _ptr(bt), bt.numel(),
                                      float(sm_scale), _ptr(workspace), workspace.numel(), _ptr(out),
                                      _stream(stream)), "kvq_prefill_attn_fp8")
    return out


_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)
_DTYPES = {torch.float32: DT_F32, torch.bfloat16: DT_BF16}


def _device(t):
    """The current device, on which a call's first tensor has to be."""
    dev = t.get_device()
    if dev < 0 or dev != _current_device():
        _refuse_device(t, "a tensor", _current_device() if dev >= 0 else 0)
    return dev


def _refuse_device(t, what, dev):
    if not t.is_cuda:
        raise ValueError(f"kvq: expected a CUDA tensor, got one on {t.device}")
    raise ValueError(f"kvq: {what} is on {t.device}, the current device is cuda:{dev}")


def _at(t, what, dev, dtype=None):
    """Address of a tensor the calls below hand to the library: on the call's
    device (the kernels are launched there), of the type the call reads."""
    if t.get_device() != dev:
        _refuse_device(t, what, dev)
    if dtype is not None and t.dtype is not dtype:
        raise TypeError(f"kvq: {what} must be {dtype}, got {t.dtype}")
    return t.data_ptr()


def _ints(t, what, dev, shape):
    """Address of contiguous int32 metadata of a given shape."""
    at = _at(t, what, dev, torch.int32)
    if t.shape != shape or not t.is_contiguous():
        raise ValueError(f"kvq: {what} must be contiguous {shape}, got {tuple(t.shape)}")
    return at


def _status_at(t, dev):
    return None if t is None else _at(t, "status", dev, torch.int32)


def _code(t, what):
    code = _DTYPES.get(t.dtype)
    if code is None:
        raise TypeError(f"kvq: {what} must be fp32 or bf16, got {t.dtype}")
    return code


def _rows(t, what, dev, tokens, heads, width):
    """kvq_rows of a tensor [tokens, heads, width] whose last dimension is contiguous."""
    if t.shape != (tokens, heads, width):
        raise ValueError(f"kvq: {what} must be [{tokens}, {heads}, {width}], got {tuple(t.shape)}")
    ts, hs, es = t.stride()
    if es != 1:
        raise ValueError(f"kvq: the last dimension of {what} must be contiguous")
    return RowsDesc(_at(t, what, dev), _code(t, what), heads, ts, hs)


def _three(t, what):
    if t.dim() != 3:
        raise ValueError(f"kvq: {what} must be [tokens, heads, width], got {tuple(t.shape)}")
    return t.shape


def _new(shape, dtype, like, stream):
    """An output tensor that belongs to the stream it is written on."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=like.device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=like.device)


def _new_rows(n, heads, width, dtype, like, stream):
    """A new contiguous tensor [n, heads, width] and its kvq_rows."""
    code = _DTYPES.get(dtype)
    if code is None:
        raise TypeError(f"kvq: an output must be fp32 or bf16, got {dtype}")
    t = _new((n, heads, width), dtype, like, stream)
    return t, RowsDesc(t.data_ptr(), code, heads, heads * width, width)


def _launch_stream(stream, dev):
    if stream is not None:
        return stream.cuda_stream
    return _raw_stream(dev) if _raw_stream is not None else torch.cuda.current_stream().cuda_stream


class Norm:
    """Root-mean-square norm of a head's row: x / sqrt(mean(x^2) + eps) * (weight +
    offset).  weight: [width] fp32 or bf16 on the device (kept, not copied)."""

    def __init__(self, weight, eps=1e-6, offset=0.0):
        self.weight, self.eps, self.offset, self.width = weight, eps, offset, weight.numel()
        self.desc = NormDesc(_ptr(weight), _dtype_code(weight), eps, offset)
        self.ref = ctypes.byref(self.desc)


class Rope:
    """Rotary positions of the first 2 * len(inv_freq) elements of a row: pair i is
    turned by position * inv_freq[i] radians.  inv_freq: floats (theta ** (-2 i /
    rot_dim), or a model's scaled ones).  axes: the position axis of every pair
    (default 0: one axis).  interleaved: pairs (2i, 2i + 1) instead of
    (i, i + rot_dim / 2)."""

    def __init__(self, inv_freq, axes=None, interleaved=False, device="cuda"):
        n = len(inv_freq)
        if axes is not None and len(axes) != n:
            raise ValueError("kvq: one axis for every pair")
        words = (ctypes.c_uint64 * max(n, 1))()
        _check(lib().kvq_rope_table((ctypes.c_double * max(n, 1))(*inv_freq),
                                    None if axes is None else (_I32 * max(n, 1))(*axes), n, words), "kvq_rope_table")
        self.num_axes = 1 if axes is None else max(axes) + 1
        self.rot_dim, self.interleaved = 2 * n, bool(interleaved)
        signed = [w - (1 << 64) if w >= 1 << 63 else w for w in words]
        self.table = torch.tensor(signed, dtype=torch.int64).to(device)
        self.desc = RopeDesc(2 * n, int(self.interleaved), self.num_axes, 0, _ptr(self.table))
        self.ref = ctypes.byref(self.desc)


def _norm_ref(norm, what, dev, width):
    if norm is None:
        return None
    if norm.width != width:
        raise ValueError(f"kvq: {what} is for rows of {norm.width}, not {width}")
    if norm.weight.get_device() != dev:
        _refuse_device(norm.weight, what, dev)
    return norm.ref


def _rope_args(rope, positions, dev, n):
    """(kvq_rope, positions, axis stride) of a call over n tokens; positions int32
    [n] (one axis) or [axes, n]."""
    if rope is None:
        return None, None, 0
    if positions is None:
        raise ValueError("kvq: rotary positions need positions")
    at = _at(positions, "positions", dev, torch.int32)
    if rope.table.get_device() != dev:
        _refuse_device(rope.table, "the rope's table", dev)
    axes, shape = rope.num_axes, positions.shape
    if shape != (axes, n) and (axes != 1 or shape != (n,)):
        raise ValueError(f"kvq: positions must be [{axes}, {n}], got {tuple(shape)}")
    st = positions.stride()
    if n > 1 and st[-1] != 1:
        raise ValueError("kvq: positions of an axis must be contiguous")
    return rope.ref, at, (st[0] if axes > 1 else n)


def norm_rope(x, positions=None, rope=None, norm=None, out=None, dtype=None, status=None, stream=None):
    """Norm and rotary positions of rows x [tokens, heads, width] (any strides with a
    contiguous last dimension) in one pass; returns out (default: a new tensor of
    `dtype`, x's own if None).  out may be x."""
    n, heads, width = _three(x, "x")
    dev = _device(x)
    rx = _rows(x, "x", dev, n, heads, width)
    if out is None:
        out, ry = _new_rows(n, heads, width, dtype or x.dtype, x, stream)
    else:
        ry = _rows(out, "out", dev, n, heads, width)
    ref, pos, ps = _rope_args(rope, positions, dev, n)
    _check(lib().kvq_norm_rope(rx, ry, n, width, _norm_ref(norm, "norm", dev, width), ref, pos, ps,
                               _status_at(status, dev), _launch_stream(stream, dev)), "kvq_norm_rope")
    return out


def norm_rope_store(cache: Cache, q, k, v, slot_mapping, positions=None, rope=None, q_norm=None, k_norm=None,
                    q_out=None, rotate=True, status=None, stream=None):
    """One launch from a layer's projections to the cache: the queries q [tokens, Hq,
    D] normed, position-rotated and (rotate) turned into the cache's space, the
    keys normed, position-rotated and stored, the values stored.  Returns q_out
    (default: a new fp32 tensor) for decode_attn, or with rotate=False for the
    calls that take unrotated queries.  q None: keys and values only."""
    n = k.shape[0]
    D, Hk, dev = cache.D, cache.Hk, _device(k)
    rk, rv = _rows(k, "k", dev, n, Hk, D), _rows(v, "v", dev, n, Hk, D)
    rq = ro = None
    if q is not None:
        Hq = _three(q, "q")[1]
        rq = _rows(q, "q", dev, n, Hq, D)
        if q_out is None:
            q_out, ro = _new_rows(n, Hq, D, torch.float32, q, stream)
        else:
            ro = _rows(q_out, "q_out", dev, n, Hq, D)
    elif q_out is not None:
        raise ValueError("kvq: q_out without q")
    ref, pos, ps = _rope_args(rope, positions, dev, n)
    _check(lib().kvq_norm_rope_store(cache.ref, rq, rk, rv, n, _norm_ref(q_norm, "q_norm", dev, D),
                                     _norm_ref(k_norm, "k_norm", dev, D), ref, pos, ps,
                                     _ints(slot_mapping, "slot_mapping", dev, (n,)), ro, int(rotate),
                                     _status_at(status, dev), _launch_stream(stream, dev)), "kvq_norm_rope_store")
    return q_out


def _load_outputs(cache, n, k, v, dtype, like, dev, stream):
    """The outputs of a load and their kvq_rows: new ones where both are None."""
    fp8 = cache.fmt == FMT_FP8_ROW
    Hk, width = cache.Hk, cache.D + cache.rope if fp8 else cache.D
    if k is None and v is None:
        k, rk = _new_rows(n, Hk, width, dtype, like, stream)
        v, rv = (None, None) if fp8 else _new_rows(n, Hk, width, dtype, like, stream)
        return k, v, rk, rv
    return (k, v, None if k is None else _rows(k, "k", dev, n, Hk, width),
            None if v is None else _rows(v, "v", dev, n, Hk, width))


def _rotates(cache, rotate_back):
    return int(cache.fmt in (FMT_Q4_HAD32, FMT_TQ4) if rotate_back is None else rotate_back)


def load(cache: Cache, slots, k=None, v=None, dtype=torch.bfloat16, rotate_back=None, status=None, stream=None):
    """The rows at slots (int32 [n]) as the values they stand for: (k, v), each [n,
    Hk, D] (fp8: k [n, 1, 576], v None).  Given k and / or v are written instead of
    new ones (one alone: only that plane); a negative slot leaves its rows as they were."""
    n, dev = slots.shape[0], _device(slots)
    k, v, rk, rv = _load_outputs(cache, n, k, v, dtype, slots, dev, stream)
    _check(lib().kvq_load(cache.ref, _ints(slots, "slots", dev, (n,)), n, _rotates(cache, rotate_back), rk, rv,
                          _status_at(status, dev), _launch_stream(stream, dev)), "kvq_load")
    return k, v


def load_seqs(cache: Cache, block_tables, cu_lens, n_tok, starts=None, k=None, v=None, dtype=torch.bfloat16,
              rotate_back=None, status=None, stream=None):
    """Runs of positions of several sequences, packed: output rows cu_lens[b] ..
    cu_lens[b + 1] - 1 are positions starts[b] (default 0) onwards of the sequence
    whose pages block_tables[b] lists.  n_tok: rows of the outputs; those past
    cu_lens[-1] are left as they were.  Outputs as for load()."""
    B, pages, dev = cu_lens.shape[0] - 1, block_tables.shape[-1], _device(cu_lens)
    k, v, rk, rv = _load_outputs(cache, n_tok, k, v, dtype, cu_lens, dev, stream)
    _check(lib().kvq_load_seqs(cache.ref, _ints(block_tables, "block_tables", dev, (B, pages)), pages, B,
                               None if starts is None else _ints(starts, "starts", dev, (B,)),
                               _ints(cu_lens, "cu_lens", dev, (B + 1,)), n_tok, _rotates(cache, rotate_back), rk, rv,
                               _status_at(status, dev), _launch_stream(stream, dev)), "kvq_load_seqs")
    return k, v


def _lambda(lam, dev, rows, heads):
    """Address and row stride of lambda: fp32 [heads] (one set) or [rows, heads]."""
    at, shape = _at(lam, "lam", dev, torch.float32), lam.shape
    if (shape != (rows, heads) and shape != (heads,)) or (heads > 1 and lam.stride(-1) != 1):
        raise ValueError(f"kvq: lam must be [{heads}] or [{rows}, {heads}] with contiguous rows, got {tuple(shape)}")
    return at, (lam.stride(0) if len(shape) == 2 else 0)


def _diff_out(out, rows, heads, width, dtype, like, dev, stream):
    if out is None:
        return _new((rows, heads, width), dtype, like, stream)
    if out.shape != (rows, heads, width) or not out.is_contiguous():
        raise ValueError(f"kvq: out must be contiguous [{rows}, {heads}, {width}], got {tuple(out.shape)}")
    _at(out, "out", dev)
    return out


def merge_diff(cache: Cache, workspace, num_seqs, num_q_heads, seq_lens, max_seq_len, lam, norm=None, out_scale=1.0,
               out=None, dtype=torch.float32, n_sel=0, rotate_back=None, stream=None):
    """merge() for differential attention: output head h is query head 2h's merged
    output minus lam[.., h] times head 2h + 1's, rotated back, normed (norm) and
    scaled.  lam: fp32 [num_q_heads / 2] or [num_seqs, num_q_heads / 2].  Returns
    out [num_seqs, num_q_heads / 2, D]."""
    dev, heads = _device(seq_lens), num_q_heads // 2
    out = _diff_out(out, num_seqs, heads, cache.D, dtype, seq_lens, dev, stream)
    lp, ls = _lambda(lam, dev, num_seqs, heads)
    _check(lib().kvq_merge_diff(cache.ref, _ptr(workspace), workspace.numel(), num_seqs, num_q_heads,
                                _ints(seq_lens, "seq_lens", dev, (num_seqs,)), max_seq_len, n_sel,
                                _rotates(cache, rotate_back), lp, ls, _norm_ref(norm, "norm", dev, cache.D),
                                out_scale, out.data_ptr(), _code(out, "out"), _launch_stream(stream, dev)),
           "kvq_merge_diff")
    return out


def diff_heads(x, lam, norm=None, out_scale=1.0, out=None, dtype=torch.float32, stream=None):
    """The same difference of heads already merged: x fp32 [rows, Hq, width]
    (prefill_attn's output) to [rows, Hq / 2, width]."""
    rows, Hq, width = _three(x, "x")
    dev = _device(x)
    _at(x, "x", dev, torch.float32)
    out = _diff_out(out, rows, Hq // 2, width, dtype, x, dev, stream)
    lp, ls = _lambda(lam, dev, rows, Hq // 2)
    _check(lib().kvq_diff_heads(_ptr(x), rows, Hq, width, lp, ls, _norm_ref(norm, "norm", dev, width), out_scale,
                                out.data_ptr(), _code(out, "out"), _launch_stream(stream, dev)), "kvq_diff_heads")
    return out


def decode_diff(cache: Cache, q, seq_lens, block_tables, max_seq_len, sm_scale, workspace, lam, norm=None,
                out_scale=1.0, out=None, dtype=torch.float32, sel=None, stream=None):
    """One differential decode step: decode() of the Hq query heads with merge_diff();
    returns [B, Hq / 2, D]."""
    B, Hq, D = _three(q, "q")
    if cache.fmt in (FMT_Q4_HAD32, FMT_Q4_0):
        decode_attn_unrotated(cache, q, seq_lens, block_tables, max_seq_len, sm_scale, workspace, sel=sel,
                              stream=stream)
    else:
        qq = q
        if cache.fmt == FMT_TQ4:
            qq = tq4_rotate(cache, q, out=_new((B, Hq, D), torch.float32, q, stream), stream=stream)
        elif q.dtype != torch.float32:
            qq = _new((B, Hq, D), torch.float32, q, stream)
            with torch.cuda.stream(stream):
                qq.copy_(q)
        decode_attn(cache, qq, seq_lens, block_tables, max_seq_len, sm_scale, workspace, sel=sel, stream=stream)
    return merge_diff(cache, workspace, B, Hq, seq_lens, max_seq_len, lam, norm=norm, out_scale=out_scale, out=out,
                      dtype=dtype, n_sel=0 if sel is None else sel.shape[1], stream=stream)


def prefill_diff(cache: Cache, q, q_start, block_table, sm_scale, lam, norm=None, out_scale=1.0, out=None,
                 dtype=torch.float32, status=None, stream=None):
    """Differential prefill of a prompt chunk: prefill_attn() of the Hq query heads,
    then diff_heads(); returns [n, Hq / 2, D]."""
    o = prefill_attn(cache, q, q_start, block_table, sm_scale, out=_new(_three(q, "q"), torch.float32, q, stream),
                     status=status, stream=stream)
    return diff_heads(o, lam, norm=norm, out_scale=out_scale, out=out, dtype=dtype, stream=stream)


def selftest_wait_timeout(d_status, stream=None):
    """Run the bounded-wait diagnostic (about 2 s); KVQ_DEV_TIMEOUT lands in d_status."""
    _check(lib().kvq_selftest_wait_timeout(_ptr(d_status), _stream(stream)), "kvq_selftest_wait_timeout")


def read_status(d_status, stream=None):
    v = ctypes.c_int32(0)
    _check(lib().kvq_read_status(_ptr(d_status), ctypes.byref(v), _stream(stream)), "kvq_read_status")
    return v.value
