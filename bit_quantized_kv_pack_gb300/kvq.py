"""ctypes binding of libkvq.so (include/kvq.h): same names, argument marshalling only.

Every step of the computation runs in the library's CUDA kernels.  Torch supplies
device memory (``KVCache`` allocates the layout's arrays as torch tensors) and the
stream (the current torch stream unless one is given).  The library must be
built (``bit_quantized_kv_pack_gb300._build.build()``); if it is missing, loading
raises: there is no other implementation to fall back to.
"""

from __future__ import annotations

import ctypes
import os
import threading

import torch

from . import _build

# ------------------------------------------------------------------- ABI ----

KVQ_OK = 0
KVQ_ERR_INVALID_ARG = 1
KVQ_ERR_UNSUPPORTED = 2
KVQ_ERR_MISALIGNED = 3
KVQ_ERR_CAPACITY = 4
KVQ_ERR_CUDA = 5
KVQ_ERR_TIMEOUT = 6
KVQ_ERR_EMPTY = 7

KVQ_ERRBIT_CAPACITY = 0x1
KVQ_ERRBIT_EMPTY = 0x2
KVQ_ERRBIT_TIMEOUT = 0x4
KVQ_ERRBIT_BADLEN = 0x8
KVQ_ERRBIT_BADPAGE = 0x10
KVQ_ERRBIT_BADPOS = 0x20

KVQ_ARRAY_CODES = 0
KVQ_ARRAY_PARAMS = 1
KVQ_ARRAY_RESIDUAL = 2
KVQ_ARRAY_SINK = 3
KVQ_ARRAY_MODE = 4

# Every function the header declares (the tests check the library exports them).
EXPORTS = ("kvq_cache_bytes", "kvq_decode_workspace_bytes", "kvq_quantize_pack",
           "kvq_quantize_pack_strided", "kvq_append",
           "kvq_decode_attention", "kvq_decode_step", "kvq_decode_step_host", "kvq_step_io_bytes",
           "kvq_decode_attention_noalloc", "kvq_append_chunk", "kvq_chunk_workspace_bytes",
           "kvq_chunk_attention", "kvq_cross_attention", "kvq_read_tokens",
           "kvq_read_error", "kvq_status_string", "kvq_version", "kvq_testing_wait_fault",
           "kvq_testing_check_arithmetic", "kvq_testing_mma_rounding")


class CacheDesc(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int32), ("num_kv_heads", ctypes.c_int32),
                ("head_dim", ctypes.c_int32), ("bits", ctypes.c_int32), ("group", ctypes.c_int32),
                ("capacity", ctypes.c_int32), ("residual", ctypes.c_int32),
                ("sink", ctypes.c_int32), ("hybrid", ctypes.c_int32),
                ("page_size", ctypes.c_int32), ("num_pages", ctypes.c_int32)]


class CacheView(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in (
        "k_codes", "v_codes", "k_params", "v_params", "k_res", "v_res",
        "packed_len", "res_len", "res_head", "err_word", "k_sink", "v_sink", "sink_len",
        "k_mode", "v_mode", "block_table")]


class AppendArgs(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p),
                ("kv_stride_token", ctypes.c_int64), ("kv_stride_head", ctypes.c_int64),
                ("q", ctypes.c_void_p), ("q_out", ctypes.c_void_p),
                ("q_stride_token", ctypes.c_int64), ("q_stride_head", ctypes.c_int64),
                ("num_q_heads", ctypes.c_int32), ("cu_seqlens", ctypes.c_void_p),
                ("total", ctypes.c_int32), ("max_len", ctypes.c_int32), ("rope", ctypes.c_void_p),
                ("rope_rows", ctypes.c_int32), ("rotary_dim", ctypes.c_int32),
                ("interleaved", ctypes.c_int32), ("positions", ctypes.c_void_p)]


class KvqError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {status_string(status)} ({status})")


_lock = threading.Lock()
_lib = None


def library_path() -> str:
    return _build.LIB


def load(path: str | None = None):
    """Load libkvq.so (raises if it has not been built)."""
    global _lib
    with _lock:
        if _lib is None:
            p = path or library_path()
            if not os.path.exists(p):
                raise RuntimeError(f"libkvq.so not built ({p}); run __graft_entry__.build()")
            lib = ctypes.CDLL(p)
            P, i32, sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_size_t
            DP, VP = ctypes.POINTER(CacheDesc), ctypes.POINTER(CacheView)
            lib.kvq_cache_bytes.argtypes = [DP, ctypes.c_int]
            lib.kvq_cache_bytes.restype = sz
            lib.kvq_decode_workspace_bytes.argtypes = [DP, i32]
            lib.kvq_decode_workspace_bytes.restype = sz
            lib.kvq_quantize_pack.argtypes = [DP, VP, P, P, P, i32, P]
            lib.kvq_quantize_pack.restype = ctypes.c_int
            i64 = ctypes.c_int64
            lib.kvq_quantize_pack_strided.argtypes = [DP, VP, P, P, P, i32, i64, i64, i64, P]
            lib.kvq_quantize_pack_strided.restype = ctypes.c_int
            lib.kvq_append.argtypes = [DP, VP, P, P, P]
            lib.kvq_append.restype = ctypes.c_int
            lib.kvq_decode_attention.argtypes = [DP, VP, P, i32, P, P, sz, ctypes.c_uint32, P]
            lib.kvq_decode_attention.restype = ctypes.c_int
            lib.kvq_decode_step.argtypes = [DP, VP, P, i32, P, P, P, P, sz, ctypes.c_uint32, P]
            lib.kvq_decode_step.restype = ctypes.c_int
            lib.kvq_step_io_bytes.argtypes = [DP, i32]
            lib.kvq_step_io_bytes.restype = sz
            lib.kvq_decode_step_host.argtypes = [DP, VP, P, i32, P, P, sz, P, sz, ctypes.c_uint32, P]
            lib.kvq_decode_step_host.restype = ctypes.c_int
            lib.kvq_decode_attention_noalloc.argtypes = [DP, VP, P, i32, P, ctypes.c_uint32, P]
            lib.kvq_decode_attention_noalloc.restype = ctypes.c_int
            lib.kvq_append_chunk.argtypes = [DP, VP, ctypes.POINTER(AppendArgs), P]
            lib.kvq_append_chunk.restype = ctypes.c_int
            lib.kvq_chunk_workspace_bytes.argtypes = [DP, i32]
            lib.kvq_chunk_workspace_bytes.restype = sz
            for fn in (lib.kvq_chunk_attention, lib.kvq_cross_attention):
                fn.argtypes = [DP, VP, P, i32, P, i32, i32, P, P, sz, ctypes.c_uint32, P]
                fn.restype = ctypes.c_int
            lib.kvq_read_tokens.argtypes = [DP, VP, P, i32, P, P, ctypes.c_uint32, P]
            lib.kvq_read_tokens.restype = ctypes.c_int
            lib.kvq_read_error.argtypes = [VP, ctypes.POINTER(ctypes.c_uint32), P]
            lib.kvq_read_error.restype = ctypes.c_int
            lib.kvq_status_string.argtypes = [ctypes.c_int]
            lib.kvq_status_string.restype = ctypes.c_char_p
            lib.kvq_version.argtypes = []
            lib.kvq_version.restype = i32
            lib.kvq_testing_wait_fault.argtypes = [ctypes.c_uint32]
            lib.kvq_testing_wait_fault.restype = None
            lib.kvq_testing_check_arithmetic.argtypes = [ctypes.POINTER(ctypes.c_uint64),
                                                         ctypes.POINTER(ctypes.c_double)]
            lib.kvq_testing_check_arithmetic.restype = ctypes.c_int
            lib.kvq_testing_mma_rounding.argtypes = [ctypes.POINTER(ctypes.c_float), ctypes.c_int32]
            lib.kvq_testing_mma_rounding.restype = ctypes.c_int
            _lib = lib
    return _lib


def status_string(status: int) -> str:
    return load().kvq_status_string(status).decode()


kvq_status_string = status_string


def _check(status: int, where: str) -> None:
    if status != KVQ_OK:
        raise KvqError(status, where)


def _ptr(t: torch.Tensor | None):
    return ctypes.c_void_p(t.data_ptr()) if t is not None else ctypes.c_void_p(0)


def _stream(stream, device) -> ctypes.c_void_p:
    if stream is None:
        stream = torch.cuda.current_stream(device)
    if isinstance(stream, torch.cuda.Stream):
        stream = stream.cuda_stream
    return ctypes.c_void_p(int(stream))


def _other_stream(stream, device):
    """The stream given to a call as torch's, or None where it is the current one."""
    current = torch.cuda.current_stream(device)
    if not isinstance(stream, torch.cuda.Stream):
        handle = stream.value or 0 if isinstance(stream, ctypes.c_void_p) else int(stream)
        stream = (torch.cuda.ExternalStream(handle, device=device) if handle
                  else torch.cuda.default_stream(device))
    return None if stream.cuda_stream == current.cuda_stream else stream


# A call's own tensors come from the stream that it runs on.  The allocator hands memory
# on in the order of that stream, so what a call drops when it returns (a workspace) is
# not another's before its kernels are done, and what they write was not in use before.


def _scratch(make, device, stream):
    """make(), a workspace that the call drops, on the call's stream."""
    other = None if stream is None else _other_stream(stream, device)
    if other is None:
        return make()
    with torch.cuda.stream(other):
        return make()


def _empty(shape, dtype, device, stream):
    """An output, from the call's stream; it is the caller's on the current one, and
    recorded there."""
    other = None if stream is None else _other_stream(stream, device)
    if other is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(other):
        t = torch.empty(shape, dtype=dtype, device=device)
    t.record_stream(torch.cuda.current_stream(device))
    return t


def _f16(t: torch.Tensor, name: str) -> torch.Tensor:
    if t.dtype != torch.float16 or not t.is_cuda or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous float16 CUDA tensor")
    return t


KVQ_OUT_F32 = 2


def _out(q: torch.Tensor, out: torch.Tensor | None, flags: int, stream=None):
    """The output tensor and the flags that match its dtype: float16, or float32
    (KVQ_OUT_F32).  Without `out`, the dtype follows KVQ_OUT_F32 in flags."""
    if out is None:
        dtype = torch.float32 if flags & KVQ_OUT_F32 else torch.float16
        out = _empty(q.shape, dtype, q.device, stream)
    if out.dtype not in (torch.float16, torch.float32) or not out.is_cuda or not out.is_contiguous():
        raise ValueError("out must be a contiguous float16 or float32 CUDA tensor")
    if out.dtype == torch.float32:
        flags |= KVQ_OUT_F32
    else:
        flags &= ~KVQ_OUT_F32
    return out, flags


# --------------------------------------------------------------- caches ----


class KVCache:
    """One layer's packed cache in device memory (torch tensors in the layout of
    include/kvq.h).  Holds the description and the view the calls take.
    ``sink`` > 0 keeps the first ``sink`` tokens of each sequence in fp16 (the
    attention-sink window, fixed after the prefill); ``hybrid=1`` quantizes each
    group symmetrically or asymmetrically, whichever reconstructs it better, and
    keeps a mode byte per packed row.  ``page_size=32`` keeps the packed rows in
    a pool of ``num_pages`` pages [page][head][32] found through ``block_table``
    [B][capacity / 32] (filled with pages b * capacity / 32 + j when the pool has
    room, for the caller to rewrite)."""

    def __init__(self, batch, num_kv_heads, head_dim, bits, capacity, residual, device="cuda",
                 sink=0, hybrid=0, page_size=0, num_pages=0):
        self.desc = CacheDesc(batch, num_kv_heads, head_dim, bits, 32, capacity, residual, sink,
                              hybrid, page_size, num_pages)
        self.device = torch.device(device)
        B, H, d = batch, num_kv_heads, head_dim
        rb, ng = d * bits // 8, d // 32
        kw = dict(device=self.device)
        rows = (num_pages, H, page_size) if page_size else (B, H, capacity)
        self.k_codes = torch.zeros(*rows, rb, dtype=torch.uint8, **kw)
        self.v_codes = torch.zeros(*rows, rb, dtype=torch.uint8, **kw)
        self.k_params = torch.zeros(*rows, ng, dtype=torch.int32, **kw)
        self.v_params = torch.zeros(*rows, ng, dtype=torch.int32, **kw)
        npb = capacity // page_size if page_size else 0
        self.block_table = (torch.arange(B * npb, dtype=torch.int32, **kw).view(B, npb)
                            % max(num_pages, 1))
        self.k_res = torch.zeros(B, H, residual, d, dtype=torch.float16, **kw)
        self.v_res = torch.zeros(B, H, residual, d, dtype=torch.float16, **kw)
        self.k_sink = torch.zeros(B, H, sink, d, dtype=torch.float16, **kw)
        self.v_sink = torch.zeros(B, H, sink, d, dtype=torch.float16, **kw)
        mrows = rows if hybrid else (0,)
        self.k_mode = torch.zeros(*mrows, dtype=torch.uint8, **kw)
        self.v_mode = torch.zeros(*mrows, dtype=torch.uint8, **kw)
        # packed_len, res_len, res_head, sink_len
        self.counters = torch.zeros(4, B, dtype=torch.int32, **kw)
        self.err = torch.zeros(4, dtype=torch.int32, **kw)
        self.view = self._make_view()

    def _make_view(self) -> CacheView:
        r = lambda t: _ptr(t) if t.numel() else ctypes.c_void_p(0)
        return CacheView(r(self.k_codes), r(self.v_codes), r(self.k_params), r(self.v_params),
                         r(self.k_res), r(self.v_res), _ptr(self.counters[0]),
                         _ptr(self.counters[1]), _ptr(self.counters[2]), _ptr(self.err),
                         r(self.k_sink), r(self.v_sink), _ptr(self.counters[3]),
                         r(self.k_mode), r(self.v_mode), r(self.block_table))

    @property
    def packed_len(self):
        return self.counters[0]

    @property
    def res_len(self):
        return self.counters[1]

    @property
    def res_head(self):
        return self.counters[2]

    @property
    def sink_len(self):
        return self.counters[3]

    def packed_bytes(self) -> int:
        """Code + param bytes of the tokens currently packed (K and V)."""
        D = self.desc
        per_tok = 2 * (D.head_dim * D.bits // 8 + 4 * (D.head_dim // 32))
        return int(self.packed_len.sum().item()) * D.num_kv_heads * per_tok


def kvq_cache_bytes(desc: CacheDesc, which: int) -> int:
    return int(load().kvq_cache_bytes(ctypes.byref(desc), which))


def kvq_decode_workspace_bytes(desc: CacheDesc, num_q_heads: int) -> int:
    return int(load().kvq_decode_workspace_bytes(ctypes.byref(desc), num_q_heads))


def kvq_quantize_pack(cache: KVCache, k: torch.Tensor, v: torch.Tensor, seq_lens: torch.Tensor,
                      stream=None) -> None:
    """Pack a prefill; k, v fp16 [B][Hkv][Lmax][d], seq_lens int32 [B] on the device."""
    _f16(k, "k"), _f16(v, "v")
    if k.shape != v.shape or k.dim() != 4:
        raise ValueError("k and v must both be [B][Hkv][Lmax][d]")
    if seq_lens.dtype != torch.int32 or not seq_lens.is_cuda:
        raise ValueError("seq_lens must be an int32 CUDA tensor")
    st = load().kvq_quantize_pack(ctypes.byref(cache.desc), ctypes.byref(cache.view), _ptr(k),
                                  _ptr(v), _ptr(seq_lens), int(k.shape[2]),
                                  _stream(stream, k.device))
    _check(st, "kvq_quantize_pack")


def kvq_quantize_pack_strided(cache: KVCache, k: torch.Tensor, v: torch.Tensor,
                              seq_lens: torch.Tensor, stream=None) -> None:
    """Pack a prefill from any strided view: k, v fp16 of logical shape
    [B][Hkv][Lmax][d] with head_dim contiguous (for example a permuted view of a
    token-major [B][L][Hkv][d] tensor, or of the key/value columns of a fused
    QKV projection output).  Nothing is copied: the library reads through the
    strides."""
    for t, name in ((k, "k"), (v, "v")):
        if t.dtype != torch.float16 or not t.is_cuda or t.dim() != 4 or t.stride(3) != 1:
            raise ValueError(f"{name} must be a float16 CUDA [B][Hkv][Lmax][d] view with d contiguous")
    if k.shape != v.shape or k.stride() != v.stride():
        raise ValueError("k and v must have the same shape and strides")
    if seq_lens.dtype != torch.int32 or not seq_lens.is_cuda:
        raise ValueError("seq_lens must be an int32 CUDA tensor")
    st = load().kvq_quantize_pack_strided(ctypes.byref(cache.desc), ctypes.byref(cache.view),
                                          _ptr(k), _ptr(v), _ptr(seq_lens), int(k.shape[2]),
                                          int(k.stride(0)), int(k.stride(1)), int(k.stride(2)),
                                          _stream(stream, k.device))
    _check(st, "kvq_quantize_pack_strided")


def kvq_append(cache: KVCache, k_new: torch.Tensor, v_new: torch.Tensor, stream=None) -> None:
    """Append one token per sequence; k_new, v_new fp16 [B][Hkv][d]."""
    _f16(k_new, "k_new"), _f16(v_new, "v_new")
    st = load().kvq_append(ctypes.byref(cache.desc), ctypes.byref(cache.view), _ptr(k_new),
                           _ptr(v_new), _stream(stream, k_new.device))
    _check(st, "kvq_append")


def workspace_for(cache: KVCache, num_q_heads: int) -> torch.Tensor:
    """A zeroed decode workspace (zeroed once; the decode keeps it ready)."""
    n = kvq_decode_workspace_bytes(cache.desc, num_q_heads)
    if n == 0:
        raise KvqError(KVQ_ERR_INVALID_ARG, "kvq_decode_workspace_bytes")
    return torch.zeros(n, dtype=torch.uint8, device=cache.device)


def kvq_decode_attention(cache: KVCache, q: torch.Tensor, out: torch.Tensor | None = None,
                         workspace: torch.Tensor | None = None, stream=None,
                         flags: int = 0) -> torch.Tensor:
    """O = softmax(q K^T / sqrt(d)) V; q fp16 [B][Hq][d] -> out [B][Hq][d], fp16
    or fp32 (an fp32 `out`, or flags=KVQ_OUT_F32)."""
    _f16(q, "q")
    out, flags = _out(q, out, flags, stream)
    if workspace is None:
        workspace = _scratch(lambda: workspace_for(cache, q.shape[1]), cache.device, stream)
    st = load().kvq_decode_attention(ctypes.byref(cache.desc), ctypes.byref(cache.view), _ptr(q),
                                     int(q.shape[1]), _ptr(out), _ptr(workspace),
                                     workspace.numel() * workspace.element_size(), int(flags),
                                     _stream(stream, q.device))
    _check(st, "kvq_decode_attention")
    return out


KVQ_STEP_EARLY_CACHE_READ = 1
KVQ_STEP_HOST_MAPPED = 4


def kvq_decode_step(cache: KVCache, q: torch.Tensor, k_new: torch.Tensor, v_new: torch.Tensor,
                    out: torch.Tensor | None = None, workspace: torch.Tensor | None = None,
                    stream=None, flags: int = 0) -> torch.Tensor:
    """One serving-loop step: append k_new/v_new (fp16 [B][Hkv][d]), then decode
    attention of q over the updated cache; one kernel launch where the tensor-core
    kernel applies.  flags=KVQ_STEP_EARLY_CACHE_READ: the kernel enqueued just
    before does not write this cache (see kvq.h).  An fp32 `out` (or
    KVQ_OUT_F32 in flags) gives fp32 output."""
    _f16(q, "q"), _f16(k_new, "k_new"), _f16(v_new, "v_new")
    out, flags = _out(q, out, flags, stream)
    if workspace is None:
        workspace = _scratch(lambda: workspace_for(cache, q.shape[1]), cache.device, stream)
    st = load().kvq_decode_step(ctypes.byref(cache.desc), ctypes.byref(cache.view), _ptr(q),
                                int(q.shape[1]), _ptr(k_new), _ptr(v_new), _ptr(out),
                                _ptr(workspace), workspace.numel() * workspace.element_size(),
                                int(flags), _stream(stream, q.device))
    _check(st, "kvq_decode_step")
    return out


def kvq_step_io_bytes(cache: KVCache, num_q_heads: int) -> int:
    return int(load().kvq_step_io_bytes(ctypes.byref(cache.desc), int(num_q_heads)))


def step_io_for(cache: KVCache, num_q_heads: int) -> torch.Tensor:
    """Device staging for kvq_decode_step_host (256-byte aligned)."""
    n = kvq_step_io_bytes(cache, num_q_heads)
    if n == 0:
        raise ValueError("invalid cache description or head count")
    buf = torch.empty(n + 256, dtype=torch.uint8, device=cache.device)
    off = (-buf.data_ptr()) % 256
    return buf[off:off + n]


def kvq_decode_step_host(cache: KVCache, in_host: torch.Tensor, num_q_heads: int,
                         out_host: torch.Tensor, dev_io: torch.Tensor | None, workspace: torch.Tensor,
                         stream=None, flags: int = 0) -> None:
    """One step from host memory: in_host = [q | k_new | v_new] fp16 (pinned for
    an asynchronous call), out_host fp16 [B][Hq][d]; copies, step and copy back
    enqueued on the stream by one library call.  An fp32 out_host gives fp32
    output.  flags | KVQ_STEP_HOST_MAPPED (pinned, device-mapped buffers): the
    step reads and writes them in place, no copies, dev_io unused."""
    if in_host.is_cuda or out_host.is_cuda:
        raise ValueError("in_host and out_host must be host tensors")
    flags = (flags | KVQ_OUT_F32) if out_host.dtype == torch.float32 else (flags & ~KVQ_OUT_F32)
    io_ptr = _ptr(dev_io) if dev_io is not None else ctypes.c_void_p(0)
    io_bytes = dev_io.numel() * dev_io.element_size() if dev_io is not None else 0
    st = load().kvq_decode_step_host(ctypes.byref(cache.desc), ctypes.byref(cache.view),
                                     _ptr(in_host), int(num_q_heads), _ptr(out_host), io_ptr,
                                     io_bytes, _ptr(workspace),
                                     workspace.numel() * workspace.element_size(), int(flags),
                                     _stream(stream, workspace.device))
    _check(st, "kvq_decode_step_host")


NOALLOC_SCRATCH_BYTES = 8 << 20


def kvq_decode_attention_noalloc(cache: KVCache, q: torch.Tensor, out: torch.Tensor | None = None,
                                 stream=None) -> torch.Tensor:
    """Decode attention for callers that cannot allocate device scratch: the
    library's own static device array holds the split partials.  Calls that
    overlap on the GPU share that array and race; keep them on one stream."""
    _f16(q, "q")
    out, flags = _out(q, out, 0, stream)
    st = load().kvq_decode_attention_noalloc(ctypes.byref(cache.desc), ctypes.byref(cache.view),
                                             _ptr(q), int(q.shape[1]), _ptr(out), int(flags),
                                             _stream(stream, q.device))
    _check(st, "kvq_decode_attention_noalloc")
    return out


# --------------------------------------------------- runs of several tokens ----


def rope_table(num_positions: int, rotary_dim: int, base: float = 10000.0,
               device="cuda") -> torch.Tensor:
    """Cosine and sine of positions 0 .. num_positions - 1 for kvq_append_chunk, fp32
    [num_positions][rotary_dim / 2][2]: angle = position * base^(-2i / rotary_dim),
    worked out in 64 bits.  Made once; any table of that shape serves (scaled
    frequencies, a magnitude factor)."""
    i = torch.arange(rotary_dim // 2, dtype=torch.float64, device=device)
    angle = (torch.arange(num_positions, dtype=torch.float64, device=device).unsqueeze(1)
             * base ** (-2.0 * i / rotary_dim))
    return torch.stack([angle.cos(), angle.sin()], -1).float()


def _run_int(t: torch.Tensor, n: int, device: torch.device, name: str) -> int:
    if (t.dtype != torch.int32 or not t.is_cuda or t.device != device or not t.is_contiguous()
            or t.numel() != n):
        raise ValueError(f"{name} must be a contiguous int32 CUDA tensor of {n} entries on the cache's device")
    return t.data_ptr()


def _run_tensor(t: torch.Tensor, heads: int, cache: KVCache, device: torch.device, name: str,
                contiguous: bool) -> int:
    d = cache.desc.head_dim
    if (t.dtype != torch.float16 or not t.is_cuda or t.device != device or t.dim() != 3 or t.shape[1] != heads
            or t.shape[2] != d or not (t.is_contiguous() if contiguous else t.stride(2) == 1)):
        raise ValueError(f"{name} must be a float16 CUDA tensor [total][{heads}][{d}] on the cache's device, "
                         f"{'contiguous' if contiguous else 'with head_dim contiguous'}")
    return t.data_ptr()


def _max_len(n: int) -> int:
    """An upper bound as the library's 32 bits hold it (a call has fewer rows than that)."""
    return max(-1, min(int(n), 2 ** 31 - 1))


def _strides(t: torch.Tensor, rows: int, heads: int) -> tuple[int, int]:
    """Strides of rows and heads; of a dimension with one entry (or none) any will do (0),
    and torch keeps whatever it was made with."""
    row, head, _ = t.stride()
    return row if rows > 1 else 0, head if heads > 1 else 0


# The current stream's handle without a Stream object: 2-3 us of a call's 10.
_current_raw = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda index: torch.cuda.current_stream(index).cuda_stream)


def _run_call(fn: str, cache: KVCache, device: torch.device, stream, *args) -> None:
    """One library call on the cache's device, whichever is current."""
    f = getattr(_lib or load(), fn)
    if stream is None:
        stream = _current_raw(device.index)
    elif isinstance(stream, torch.cuda.Stream):
        stream = stream.cuda_stream
    if torch.cuda.current_device() == device.index:
        st = f(ctypes.byref(cache.desc), ctypes.byref(cache.view), *args, stream)
    else:
        with torch.cuda.device(device):
            st = f(ctypes.byref(cache.desc), ctypes.byref(cache.view), *args, stream)
    _check(st, fn)


def kvq_append_chunk(cache: KVCache, k: torch.Tensor, v: torch.Tensor, cu_seqlens: torch.Tensor,
                     max_len: int, q: torch.Tensor | None = None, q_out: torch.Tensor | None = None,
                     rope: torch.Tensor | None = None, interleaved: bool = False,
                     positions: torch.Tensor | None = None, stream=None) -> torch.Tensor | None:
    """Append a run of tokens to each sequence (ragged, concatenated: sequence b's run
    is rows cu_seqlens[b] .. cu_seqlens[b+1]); k, v fp16 [total][Hkv][d] views with d
    contiguous and equal strides.  With ``rope`` (fp32 [rows][rotary_dim / 2][2], see
    rope_table) keys are rotated to their positions first: the tokens the sequence held
    + the place in the run, or ``positions`` (int32 [total]).  ``q`` (fp16 [total][Hq][d])
    is rotated too and returned (in ``q_out``, which may be q itself)."""
    D = cache.desc
    device = cache.counters.device
    total = k.shape[0]
    cu = _run_int(cu_seqlens, D.batch + 1, device, "cu_seqlens")
    a = AppendArgs(k=_run_tensor(k, D.num_kv_heads, cache, device, "k", False),
                   v=_run_tensor(v, D.num_kv_heads, cache, device, "v", False),
                   cu_seqlens=cu, total=total, max_len=_max_len(max_len), interleaved=int(interleaved))
    strides = _strides(k, total, D.num_kv_heads)
    if k.shape != v.shape or strides != _strides(v, total, D.num_kv_heads):
        raise ValueError("k and v must have the same shape and strides")
    a.kv_stride_token, a.kv_stride_head = strides
    if q is not None:
        if q.dim() != 3 or q.shape[0] != total:
            raise ValueError("q must be [total][Hq][d] with k's rows")
        heads = q.shape[1]
        a.q = _run_tensor(q, heads, cache, device, "q", False)
        if q_out is None:
            q_out = _empty(q.shape, torch.float16, device, stream)
        a.q_out = _run_tensor(q_out, heads, cache, device, "q_out", True)
        if q_out.shape != q.shape:
            raise ValueError("q_out must have q's shape")
        if a.q_out == a.q and not q.is_contiguous():
            raise ValueError("q must be contiguous to be rotated in place")
        a.num_q_heads = heads
        a.q_stride_token, a.q_stride_head = _strides(q, total, heads)
    if rope is not None:
        if (rope.dtype != torch.float32 or not rope.is_cuda or rope.device != device
                or rope.dim() != 3 or rope.shape[2] != 2 or not rope.is_contiguous()):
            raise ValueError("rope must be a contiguous float32 CUDA tensor [rows][rotary_dim / 2][2] "
                             "on the cache's device")
        a.rope, a.rope_rows, a.rotary_dim = rope.data_ptr(), rope.shape[0], 2 * rope.shape[1]
    if positions is not None:
        a.positions = _run_int(positions, total, device, "positions")
    _run_call("kvq_append_chunk", cache, device, stream, ctypes.byref(a))
    return q_out


def kvq_chunk_workspace_bytes(desc: CacheDesc, num_q_heads: int) -> int:
    return int(load().kvq_chunk_workspace_bytes(ctypes.byref(desc), int(num_q_heads)))


def chunk_workspace_for(cache: KVCache, num_q_heads: int) -> torch.Tensor:
    """A workspace for kvq_chunk_attention and kvq_cross_attention (any run lengths; one
    call at a time)."""
    device = cache.counters.device
    with torch.cuda.device(device):  # its size follows from the device
        n = kvq_chunk_workspace_bytes(cache.desc, num_q_heads)
    if n == 0:
        raise KvqError(KVQ_ERR_INVALID_ARG, "kvq_chunk_workspace_bytes")
    return torch.empty(n, dtype=torch.uint8, device=device)


def _attend_runs(name: str, cache: KVCache, q, cu_seqlens, max_len, out, workspace, stream, flags):
    if q.dim() != 3:
        raise ValueError("q must be [total][Hq][d]")
    device = cache.counters.device
    total, heads, _ = q.shape
    cu = _run_int(cu_seqlens, cache.desc.batch + 1, device, "cu_seqlens")
    qp = _run_tensor(q, heads, cache, device, "q", True)
    out, flags = _out(q, out, flags, stream)
    if workspace is None:
        workspace = _scratch(lambda: chunk_workspace_for(cache, heads), device, stream)
    if out.shape != q.shape or out.device != device:
        raise ValueError("out must have q's shape, on the cache's device")
    if workspace.device != device or not workspace.is_contiguous():
        raise ValueError("workspace must be contiguous, on the cache's device")
    _run_call(name, cache, device, stream, qp, heads, cu, total, _max_len(max_len), out.data_ptr(),
              workspace.data_ptr(), workspace.numel() * workspace.element_size(), flags)
    return out


def kvq_chunk_attention(cache: KVCache, q: torch.Tensor, cu_seqlens: torch.Tensor, max_len: int,
                        out: torch.Tensor | None = None, workspace: torch.Tensor | None = None,
                        stream=None, flags: int = 0) -> torch.Tensor:
    """Causal attention of each sequence's newest tokens over its cache: q fp16
    [total][Hq][d], sequence b's run (rows cu_seqlens[b] .. cu_seqlens[b+1]) being its
    last tokens, already appended.  out fp16, or fp32 as for kvq_decode_attention."""
    return _attend_runs("kvq_chunk_attention", cache, q, cu_seqlens, max_len, out, workspace, stream,
                        flags)


def kvq_cross_attention(cache: KVCache, q: torch.Tensor, cu_seqlens: torch.Tensor, max_len: int,
                        out: torch.Tensor | None = None, workspace: torch.Tensor | None = None,
                        stream=None, flags: int = 0) -> torch.Tensor:
    """Every row of each sequence's run attends over all its cached tokens (decoder
    tokens over an encoder's states); arguments as for kvq_chunk_attention."""
    return _attend_runs("kvq_cross_attention", cache, q, cu_seqlens, max_len, out, workspace, stream,
                        flags)


def kvq_read_tokens(cache: KVCache, first: torch.Tensor | None, count: int,
                    k_out: torch.Tensor | None = None, v_out: torch.Tensor | None = None,
                    stream=None, flags: int = 0) -> tuple[torch.Tensor, torch.Tensor]:
    """Tokens first[b] .. first[b] + count - 1 of each sequence (sink, packed, residual
    order; first int32 [B] or None for 0) as values: (K, V) [B][Hkv][count][d], fp16 or
    fp32 (KVQ_OUT_F32 in flags, or fp32 outputs).  Rows past the end are zero."""
    D = cache.desc
    device = cache.counters.device
    first_ptr = None if first is None else _run_int(first, D.batch, device, "first")
    shape = (D.batch, D.num_kv_heads, int(count), D.head_dim)
    given = k_out if k_out is not None else v_out
    dtype = given.dtype if given is not None else (
        torch.float32 if flags & KVQ_OUT_F32 else torch.float16)
    if dtype not in (torch.float16, torch.float32):
        raise ValueError("k_out and v_out must be float16 or float32")
    if device.type != "cuda":
        raise ValueError("the cache must be in CUDA memory")
    outs = [_empty(shape, dtype, device, stream) if t is None else t for t in (k_out, v_out)]
    for t in (k_out, v_out):
        if t is not None and (t.shape != shape or t.dtype != dtype or not t.is_cuda or t.device != device
                              or not t.is_contiguous()):
            raise ValueError("k_out and v_out must be contiguous tensors [B][Hkv][count][d] of one type "
                             "on the cache's device")
    flags = (flags | KVQ_OUT_F32) if dtype == torch.float32 else (flags & ~KVQ_OUT_F32)
    _run_call("kvq_read_tokens", cache, device, stream, first_ptr, int(count), outs[0].data_ptr(),
              outs[1].data_ptr(), flags)
    return outs[0], outs[1]


def kvq_read_error(cache: KVCache, stream=None) -> tuple[int, int]:
    """(status, raw error word); synchronizes the stream and clears the word."""
    word = ctypes.c_uint32(0)
    st = load().kvq_read_error(ctypes.byref(cache.view), ctypes.byref(word),
                               _stream(stream, cache.device))
    return st, word.value


def kvq_version() -> int:
    return int(load().kvq_version())


def kvq_testing_wait_fault(limit_us: int) -> None:
    """Testing hook (see kvq.h): limit_us > 0 makes one bounded wait of the next
    tensor-core decode calls, and of the next calls on runs, run out after limit_us microseconds; 0 turns it off."""
    load().kvq_testing_wait_fault(int(limit_us))


def kvq_testing_check_arithmetic():
    """Testing hook (see kvq.h): ([mismatches, in domain] for the divisors 15, 7,
    3, the reciprocal's worst relative error over the fp16 scales)."""
    mm = (ctypes.c_uint64 * 6)()
    worst = ctypes.c_double(0.0)
    _check(load().kvq_testing_check_arithmetic(mm, ctypes.byref(worst)),
           "kvq_testing_check_arithmetic")
    return [(int(mm[2 * i]), int(mm[2 * i + 1])) for i in range(3)], worst.value


def kvq_testing_mma_rounding(n: int = 8):
    """Testing hook (see kvq.h): the eight MMA rounding cases' results."""
    out = (ctypes.c_float * 8)()
    _check(load().kvq_testing_mma_rounding(out, int(n)), "kvq_testing_mma_rounding")
    return [float(out[i]) for i in range(n)]
