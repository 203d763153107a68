"""Thin Python binding of the C ABI in include/splash.h (argument marshalling only).

Every function here forwards torch tensors' device pointers, sizes and the
current CUDA stream to ``libsplash_gb300.so``; every step of the computation
runs in that library's CUDA kernels.  There is no fallback: if the library is
missing or the tensors are not on a CUDA device the call raises.
"""
from __future__ import annotations

import ctypes
import functools
import os
import struct
import threading

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "_build", "libsplash_gb300.so")

SPLASH_OK = 0
SPLASH_ERR_INVALID_ARG = -1
SPLASH_ERR_UNSUPPORTED = -2
SPLASH_ERR_WORKSPACE = -3
SPLASH_ERR_CUDA = -4
SPLASH_DEVICE_TIMEOUT = 1
SPLASH_DEVICE_BAD_INPUT = 2

EXPORTED = ("splash_decode_workspace_size", "splash_decode_attn", "splash_decode_attn_ex",
            "splash_decode_attn_noalloc", "splash_noalloc_status",
            "splash_lse_merge", "splash_kv_migrate", "splash_rope", "splash_kv_append",
            "splash_kv_unpack", "splash_chunk_workspace_size", "splash_chunk_attn",
            "splash_batch_tables", "splash_batch_release", "splash_norm_rope",
            "splash_chunk_workspace_size_ex", "splash_chunk_attn_ex",
            "splash_workspace_status", "splash_status_string")

SPLASH_BF16, SPLASH_F16, SPLASH_F32 = 0, 1, 2
SPLASH_ROPE_PLAIN, SPLASH_ROPE_LINEAR, SPLASH_ROPE_YARN = 0, 1, 2
SPLASH_KV_BF16, SPLASH_KV_MXFP8 = 0, 1
MXFP8_ROW_BYTES = 656     # a token of an MXFP8 pool: 512 e4m3, 16 scale bytes, 64 bf16
_DTYPES = {torch.bfloat16: SPLASH_BF16, torch.float16: SPLASH_F16, torch.float32: SPLASH_F32}
_SCALINGS = {"none": SPLASH_ROPE_PLAIN, "linear": SPLASH_ROPE_LINEAR, "yarn": SPLASH_ROPE_YARN}


class SplashError(RuntimeError):
    def __init__(self, code: int, where: str):
        self.code = code
        super().__init__(f"{where}: {splash_status_string(code)} ({code})")


class SplashAttnDesc(ctypes.Structure):
    _fields_ = [("num_reqs", ctypes.c_int32), ("num_heads", ctypes.c_int32),
                ("d_qk", ctypes.c_int32), ("d_v", ctypes.c_int32), ("page_size", ctypes.c_int32),
                ("num_pages", ctypes.c_int32), ("max_pages_per_req", ctypes.c_int32),
                ("scale", ctypes.c_float)]


class SplashDecodeExt(ctypes.Structure):
    _fields_ = [("tok_lo", ctypes.c_void_p), ("tok_hi", ctypes.c_void_p),
                ("rows", ctypes.c_void_p), ("num_rows", ctypes.c_int32),
                ("max_sms", ctypes.c_int32), ("num_kv_heads", ctypes.c_int32)]


class SplashRopeDesc(ctypes.Structure):
    _fields_ = [("dims", ctypes.c_int32), ("interleaved", ctypes.c_int32),
                ("scaling", ctypes.c_int32), ("reserved", ctypes.c_int32),
                ("base", ctypes.c_double), ("factor", ctypes.c_double),
                ("orig_ctx", ctypes.c_double), ("beta_fast", ctypes.c_double),
                ("beta_slow", ctypes.c_double), ("amplitude", ctypes.c_double)]


class SplashNormDesc(ctypes.Structure):
    _fields_ = [("width", ctypes.c_int32), ("norm_dims", ctypes.c_int32), ("rope_lo", ctypes.c_int32),
                ("weight_dtype", ctypes.c_int32), ("eps", ctypes.c_float), ("weight_offset", ctypes.c_float)]


# Structs that hold a call's pointers, packed (a ctypes structure takes five times as long to fill).
_BATCH = struct.Struct("@6i10P")          # splash_batch
_BATCH_DROP = struct.Struct("@6i5P")      # splash_batch_drop
_NORM_ROWS = struct.Struct("@PqqPqqPii")  # splash_norm_rows


class SplashChunkExt(ctypes.Structure):
    _fields_ = [("window", ctypes.c_int32), ("sinks", ctypes.c_int32), ("cu_groups", ctypes.c_void_p),
                ("prefix_lens", ctypes.c_void_p), ("num_groups", ctypes.c_int32), ("reserved", ctypes.c_int32)]


_lock = threading.Lock()
_lib = None


def load_library(path: str | None = None):
    """Loads (once) and returns the ctypes handle; raises if the library is missing."""
    global _lib
    with _lock:
        if _lib is not None:
            return _lib
        p = path or LIB_PATH
        if not os.path.exists(p):
            raise RuntimeError(f"{p} is missing: build it with layout_agnostic_paged_gb300.build.build()")
        lib = ctypes.CDLL(p)
        vp, i32, i64, sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_size_t
        dp = ctypes.POINTER(SplashAttnDesc)
        lib.splash_decode_workspace_size.argtypes = [dp, i32, i32]
        lib.splash_decode_workspace_size.restype = sz
        lib.splash_decode_attn.argtypes = [dp, vp, vp, vp, vp, i32, i32, i64, i64, vp, vp, vp, sz, vp]
        lib.splash_decode_attn.restype = i32
        lib.splash_decode_attn_ex.argtypes = [dp, ctypes.POINTER(SplashDecodeExt), vp, vp, vp, vp,
                                              i32, i32, i64, i64, vp, vp, vp, sz, vp]
        lib.splash_decode_attn_ex.restype = i32
        lib.splash_decode_attn_noalloc.argtypes = [dp, vp, vp, vp, vp, i32, i32, i64, i64, vp, vp, vp]
        lib.splash_decode_attn_noalloc.restype = i32
        lib.splash_noalloc_status.argtypes = [ctypes.POINTER(ctypes.c_uint32), vp]
        lib.splash_noalloc_status.restype = i32
        lib.splash_lse_merge.argtypes = [vp, vp, i32, i32, i32, i32, vp, vp, vp]
        lib.splash_lse_merge.restype = i32
        lib.splash_kv_migrate.argtypes = [vp, vp, sz, vp, vp, i32, ctypes.c_int32, ctypes.c_int32, vp]
        lib.splash_kv_migrate.restype = i32
        rp = ctypes.POINTER(SplashRopeDesc)
        lib.splash_rope.argtypes = [rp, i32, vp, i64, i64, vp, i64, i64, vp, i32, i32, vp]
        lib.splash_rope.restype = i32
        lib.splash_norm_rope.argtypes = [ctypes.POINTER(SplashNormDesc), rp, i32, vp, vp, vp, i32, vp]
        lib.splash_norm_rope.restype = i32
        lib.splash_kv_append.argtypes = [dp, rp, i32, vp, i64, vp, i64, vp, i32, vp, vp, vp, vp]
        lib.splash_kv_append.restype = i32
        lib.splash_kv_unpack.argtypes = [vp, vp, i32, vp, vp, i32, ctypes.c_int32, ctypes.c_int32, vp]
        lib.splash_kv_unpack.restype = i32
        lib.splash_chunk_workspace_size.argtypes = [dp, i32, i32, i32]
        lib.splash_chunk_workspace_size.restype = sz
        lib.splash_chunk_attn.argtypes = [dp, vp, vp, vp, i32, vp, vp, i32, i32, i64, i64, i32, vp, vp,
                                          vp, sz, vp]
        lib.splash_chunk_attn.restype = i32
        ep = ctypes.POINTER(SplashChunkExt)
        lib.splash_chunk_workspace_size_ex.argtypes = [dp, ep, i32, i32, i32]
        lib.splash_chunk_workspace_size_ex.restype = sz
        lib.splash_chunk_attn_ex.argtypes = [dp, ep, vp, vp, vp, i32, vp, vp, i32, i32, i64, i64, i32, vp, vp, vp, sz, vp]
        lib.splash_chunk_attn_ex.restype = i32
        lib.splash_batch_tables.argtypes = [vp, vp]
        lib.splash_batch_tables.restype = i32
        lib.splash_batch_release.argtypes = [vp, vp]
        lib.splash_batch_release.restype = i32
        lib.splash_workspace_status.argtypes = [vp, ctypes.POINTER(ctypes.c_uint32), vp]
        lib.splash_workspace_status.restype = i32
        lib.splash_status_string.argtypes = [i32]
        lib.splash_status_string.restype = ctypes.c_char_p
        _lib = lib
        return lib


def splash_status_string(code: int) -> str:
    return load_library().splash_status_string(int(code)).decode()


def _ptr(t: torch.Tensor | None):
    return ctypes.c_void_p(0 if t is None else t.data_ptr())


def _stream(stream) -> ctypes.c_void_p:
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(int(stream.cuda_stream) if hasattr(stream, "cuda_stream") else int(stream))


def _check_cuda(*ts):
    for t in ts:
        if not t.is_cuda:
            raise ValueError("splash: tensors must live on a CUDA device")
        if not t.is_contiguous():
            raise ValueError("splash: tensors must be contiguous")


def make_desc(q: torch.Tensor, kv_pool: torch.Tensor, block_table: torch.Tensor,
              scale: float) -> SplashAttnDesc:
    B, H, d_qk = q.shape
    if kv_pool.dim() == 4:   # [num_pages][Hkv][P][576]: several KV heads
        num_pages, _, P, d_qk2 = kv_pool.shape
    else:
        num_pages, P, d_qk2 = kv_pool.shape
    if d_qk2 != d_qk:
        raise ValueError("q and kv_pool disagree on the key width")
    return SplashAttnDesc(B, H, d_qk, 512, P, num_pages, block_table.shape[1], float(scale))


def splash_decode_workspace_size(desc: SplashAttnDesc, head_lo: int, head_hi: int) -> int:
    return int(load_library().splash_decode_workspace_size(ctypes.byref(desc), int(head_lo),
                                                           int(head_hi)))


def decode_workspace(q, kv_pool, block_table, scale, head_lo=0, head_hi=None,
                     num_reqs=None) -> torch.Tensor:
    """Allocates (with torch, on q's device) a workspace large enough for the slice
    (num_reqs: requests in the call, when they are a subset of q's rows)."""
    desc = make_desc(q, kv_pool, block_table, scale)
    if num_reqs is not None:
        desc.num_reqs = int(num_reqs)
    head_hi = q.shape[1] if head_hi is None else head_hi
    with torch.cuda.device(q.device):
        n = splash_decode_workspace_size(desc, head_lo, head_hi)
    if n == 0:
        raise SplashError(SPLASH_ERR_UNSUPPORTED, "splash_decode_workspace_size")
    return torch.empty(n, dtype=torch.uint8, device=q.device)


def splash_decode_attn(q: torch.Tensor, kv_pool: torch.Tensor, block_table: torch.Tensor,
                       ctx_lens: torch.Tensor, head_lo: int, head_hi: int, tok_lo: int,
                       tok_hi: int, out: torch.Tensor, lse: torch.Tensor,
                       workspace: torch.Tensor, scale: float, stream=None) -> None:
    """Paged decode attention of one ownership slice (see splash.h); writes out / lse rows."""
    _check_cuda(q, kv_pool, block_table, ctx_lens, out, lse, workspace)
    if kv_pool.dim() != 3:
        raise ValueError("splash_decode_attn: one shared KV head [num_pages][P][576]; "
                         "use splash_decode_attn_ex for several KV heads")
    if (q.dtype != torch.bfloat16 or kv_pool.dtype != torch.bfloat16 or out.dtype != torch.float32
            or lse.dtype != torch.float32 or block_table.dtype != torch.int32
            or ctx_lens.dtype != torch.int32):
        raise ValueError("splash_decode_attn: dtype mismatch")
    B, H, _ = q.shape
    if out.shape != (B, H, 512) or lse.shape != (B, H) or ctx_lens.shape != (B,):
        raise ValueError("splash_decode_attn: shape mismatch")
    desc = make_desc(q, kv_pool, block_table, scale)
    with torch.cuda.device(q.device):
        rc = load_library().splash_decode_attn(
            ctypes.byref(desc), _ptr(q), _ptr(kv_pool), _ptr(block_table), _ptr(ctx_lens),
            int(head_lo), int(head_hi), int(tok_lo), int(tok_hi), _ptr(out), _ptr(lse),
            _ptr(workspace), workspace.numel() * workspace.element_size(), _stream(stream))
    if rc != SPLASH_OK:
        raise SplashError(rc, "splash_decode_attn")


def splash_decode_attn_ex(q: torch.Tensor, kv_pool: torch.Tensor, block_table: torch.Tensor,
                          ctx_lens: torch.Tensor, head_lo: int, head_hi: int, tok_lo: int,
                          tok_hi: int, out: torch.Tensor, lse: torch.Tensor,
                          workspace: torch.Tensor, scale: float, tok_lo_r=None, tok_hi_r=None,
                          rows=None, max_sms: int = 0, stream=None) -> None:
    """splash_decode_attn with optional per-request token ranges (int32 [B] tensors
    tok_lo_r / tok_hi_r), storage rows (int32 [B] tensor `rows` into q, block_table,
    ctx_lens, out and lse; B is len(rows) when rows is given, else q's rows) and an SM
    budget for the decode grid (max_sms, 0 = all).  A kv_pool of shape
    [num_pages][Hkv][P][576] selects grouped-query attention over Hkv KV heads."""
    opt = [t for t in (tok_lo_r, tok_hi_r, rows) if t is not None]
    _check_cuda(q, kv_pool, block_table, ctx_lens, out, lse, workspace, *opt)
    if (q.dtype != torch.bfloat16 or kv_pool.dtype != torch.bfloat16 or out.dtype != torch.float32
            or lse.dtype != torch.float32 or block_table.dtype != torch.int32
            or ctx_lens.dtype != torch.int32 or any(t.dtype != torch.int32 for t in opt)):
        raise ValueError("splash_decode_attn_ex: dtype mismatch")
    R, H, _ = q.shape
    if out.shape != (R, H, 512) or lse.shape != (R, H) or ctx_lens.shape != (R,):
        raise ValueError("splash_decode_attn_ex: shape mismatch")
    B = int(rows.numel()) if rows is not None else R
    if any(t.shape != (B,) for t in opt):
        raise ValueError("splash_decode_attn_ex: per-request arrays must have one entry per request")
    desc = make_desc(q, kv_pool, block_table, scale)
    desc.num_reqs = B
    ext = SplashDecodeExt(tok_lo_r.data_ptr() if tok_lo_r is not None else None,
                          tok_hi_r.data_ptr() if tok_hi_r is not None else None,
                          rows.data_ptr() if rows is not None else None,
                          R if rows is not None else 0, int(max_sms),
                          int(kv_pool.shape[1]) if kv_pool.dim() == 4 else 0)
    with torch.cuda.device(q.device):
        rc = load_library().splash_decode_attn_ex(
            ctypes.byref(desc), ctypes.byref(ext), _ptr(q), _ptr(kv_pool), _ptr(block_table),
            _ptr(ctx_lens), int(head_lo), int(head_hi), int(tok_lo), int(tok_hi), _ptr(out),
            _ptr(lse), _ptr(workspace), workspace.numel() * workspace.element_size(),
            _stream(stream))
    if rc != SPLASH_OK:
        raise SplashError(rc, "splash_decode_attn_ex")


def splash_decode_attn_noalloc(q: torch.Tensor, kv_pool: torch.Tensor, block_table: torch.Tensor,
                               ctx_lens: torch.Tensor, head_lo: int, head_hi: int, tok_lo: int,
                               tok_hi: int, out: torch.Tensor, lse: torch.Tensor, scale: float,
                               stream=None) -> None:
    """splash_decode_attn with the library's own fixed scratch instead of a caller
    workspace (for callers that cannot allocate device memory where they decode,
    e.g. under stream capture); see splash.h for its size limit and sharing rules."""
    _check_cuda(q, kv_pool, block_table, ctx_lens, out, lse)
    if (q.dtype != torch.bfloat16 or kv_pool.dtype != torch.bfloat16 or out.dtype != torch.float32
            or lse.dtype != torch.float32 or block_table.dtype != torch.int32
            or ctx_lens.dtype != torch.int32):
        raise ValueError("splash_decode_attn_noalloc: dtype mismatch")
    B, H, _ = q.shape
    if out.shape != (B, H, 512) or lse.shape != (B, H) or ctx_lens.shape != (B,):
        raise ValueError("splash_decode_attn_noalloc: shape mismatch")
    desc = make_desc(q, kv_pool, block_table, scale)
    with torch.cuda.device(q.device):
        rc = load_library().splash_decode_attn_noalloc(
            ctypes.byref(desc), _ptr(q), _ptr(kv_pool), _ptr(block_table), _ptr(ctx_lens),
            int(head_lo), int(head_hi), int(tok_lo), int(tok_hi), _ptr(out), _ptr(lse),
            _stream(stream))
    if rc != SPLASH_OK:
        raise SplashError(rc, "splash_decode_attn_noalloc")


def splash_noalloc_status(device=None, stream=None) -> int:
    """Synchronises the stream and returns the SPLASH_DEVICE_* bits of the last
    splash_decode_attn_noalloc call on the device."""
    flags = ctypes.c_uint32(0)
    dev = torch.device("cuda", torch.cuda.current_device()) if device is None else torch.device(device)
    with torch.cuda.device(dev):
        rc = load_library().splash_noalloc_status(ctypes.byref(flags), _stream(stream))
    if rc != SPLASH_OK:
        raise SplashError(rc, "splash_noalloc_status")
    return int(flags.value)


def splash_lse_merge(part_out: torch.Tensor, part_lse: torch.Tensor, out: torch.Tensor,
                     lse: torch.Tensor, stream=None) -> None:
    """part_out [S][B][H][d_v], part_lse [S][B][H] -> out [B][H][d_v], lse [B][H]."""
    _check_cuda(part_out, part_lse, out, lse)
    S, B, H, d_v = part_out.shape
    if part_lse.shape != (S, B, H) or out.shape != (B, H, d_v) or lse.shape != (B, H):
        raise ValueError("splash_lse_merge: shape mismatch")
    if any(t.dtype != torch.float32 for t in (part_out, part_lse, out, lse)):
        raise ValueError("splash_lse_merge: tensors must be float32")
    with torch.cuda.device(out.device):
        rc = load_library().splash_lse_merge(_ptr(part_out), _ptr(part_lse), S, B, H, d_v, _ptr(out),
                                             _ptr(lse), _stream(stream))
    if rc != SPLASH_OK:
        raise SplashError(rc, "splash_lse_merge")


def splash_kv_migrate(src_pool: torch.Tensor, dst_pool: torch.Tensor, src_ids: torch.Tensor,
                      dst_ids: torch.Tensor, stream=None) -> None:
    """dst_pool[dst_ids[i]] <- src_pool[src_ids[i]] byte for byte (pages = leading dim)."""
    _check_cuda(src_pool, dst_pool, src_ids, dst_ids)
    if src_ids.dtype != torch.int32 or dst_ids.dtype != torch.int32 or src_ids.shape != dst_ids.shape:
        raise ValueError("splash_kv_migrate: ids must be int32 of equal length")
    page_bytes = src_pool[0].numel() * src_pool.element_size() if src_pool.shape[0] else 0
    if dst_pool.shape[0] and dst_pool[0].numel() * dst_pool.element_size() != page_bytes:
        raise ValueError("splash_kv_migrate: pools disagree on the page size")
    with torch.cuda.device(dst_pool.device):
        rc = load_library().splash_kv_migrate(_ptr(src_pool), _ptr(dst_pool), page_bytes,
                                              _ptr(src_ids), _ptr(dst_ids), src_ids.numel(),
                                              src_pool.shape[0], dst_pool.shape[0], _stream(stream))
    if rc != SPLASH_OK:
        raise SplashError(rc, "splash_kv_migrate")


# The functions below serve single decode steps, whose kernels take a few microseconds: they
# look each attribute up once and ask for the raw stream handle.

def _call(dev: int, stream, where: str, fn, *args):
    """fn(*args, stream) with device `dev` current; stream None is the device's current stream."""
    if torch._C._cuda_getDevice() == dev:          # (torch is set up: there are tensors on the GPU)
        rc = fn(*args, torch._C._cuda_getCurrentRawStream(dev) if stream is None else _stream(stream))
    else:
        with torch.cuda.device(dev):
            rc = fn(*args, torch._C._cuda_getCurrentRawStream(dev) if stream is None else _stream(stream))
    if rc != SPLASH_OK:
        raise SplashError(rc, where)


def _device_of(where: str, *ts) -> int:
    """Index of the CUDA device that all the tensors live on."""
    dev = ts[0].get_device()
    for t in ts[1:]:
        if t.get_device() != dev:
            dev = -1
    if dev < 0:
        raise ValueError(f"{where}: tensors must live on one CUDA device")
    return dev


def _index_arrays(where: str, cu_q, block_table, ctx_lens) -> tuple[int, int]:
    """(requests, pages per request) of the three arrays of a ragged batch."""
    i32 = torch.int32
    if cu_q.dtype != i32 or block_table.dtype != i32 or ctx_lens.dtype != i32 or not (
            cu_q.is_contiguous() and block_table.is_contiguous() and ctx_lens.is_contiguous()):
        raise ValueError(f"{where}: cu_q, block_table and ctx_lens must be contiguous int32")
    shape, n = block_table.shape, ctx_lens.shape
    if len(shape) != 2 or n != shape[:1] or cu_q.dim() != 1 or cu_q.numel() != shape[0] + 1:
        raise ValueError(f"{where}: cu_q [B + 1], block_table [B][max_pages] and ctx_lens [B] disagree")
    return shape[0], shape[1]


@functools.lru_cache(maxsize=1024)
def _shape_desc(B: int, H: int, P: int, num_pages: int, max_pages: int, scale: float) -> SplashAttnDesc:
    """The description of a shape (read-only; the library reads it during the call)."""
    return SplashAttnDesc(B, H, 576, 512, P, num_pages, max_pages, scale)


def _int32(where: str, name: str, v) -> int:
    """v as an int32 argument of the library (ctypes would take its low 32 bits)."""
    v = int(v)
    if not -2 ** 31 <= v < 2 ** 31:
        raise ValueError(f"{where}: {name} must fit 32 bits")
    return v


def _packed(where: str, fmt: struct.Struct, *values) -> bytes:
    """The packed struct of a call."""
    try:
        return fmt.pack(*values)
    except struct.error as e:
        raise ValueError(f"{where}: sizes must be whole numbers of 32 bits ({e})") from None


def _int32_arrays(where: str, dev: int, arrays) -> None:
    """Each (name, tensor, entries): contiguous int32 of so many entries on device `dev`."""
    i32 = torch.int32
    for name, t, n in arrays:
        if t.dtype is not i32 or t.numel() != n or not t.is_contiguous():
            raise ValueError(f"{where}: {name} must be contiguous int32 of {n} entries")
        if t.get_device() != dev:
            raise ValueError(f"{where}: tensors must live on one CUDA device")


def splash_batch_tables(past_lens: torch.Tensor, new_lens: torch.Tensor, block_table: torch.Tensor, page_size: int,
                        free_pages: torch.Tensor, free_count: torch.Tensor, cu_q: torch.Tensor,
                        ctx_lens: torch.Tensor, positions: torch.Tensor, slots: torch.Tensor, left: torch.Tensor,
                        stream=None) -> None:
    """A step's arrays from its requests' lengths (all int32): takes pages for the new tokens from the top of
    the stack free_pages [num_pages] (free_count [1] entries) into block_table [B][max_pages], and writes cu_q
    [B + 1], ctx_lens [B], positions and slots [N rows] and left [2] = (free pages left, requests served).
    ctx_lens may be past_lens, and free_count left (its first entry is the count); see splash.h for batches that do not fit."""
    where = "splash_batch_tables"
    dev = _device_of(where, block_table)
    count = free_count.numel()
    if block_table.dim() != 2 or not 1 <= count <= 2:
        raise ValueError(f"{where}: block_table must be [B][max_pages], free_count [1] (or left [2])")
    B, pages = block_table.shape
    N, F = positions.numel(), free_pages.numel()
    _int32_arrays(where, dev, (
        ("past_lens", past_lens, B), ("new_lens", new_lens, B), ("block_table", block_table, B * pages),
        ("free_pages", free_pages, F), ("free_count", free_count, count), ("cu_q", cu_q, B + 1), ("ctx_lens", ctx_lens, B),
        ("positions", positions, N), ("slots", slots, N), ("left", left, 2)))
    _call(dev, stream, where, (_lib or load_library()).splash_batch_tables, _packed(
        where, _BATCH, B, page_size, F, pages, N, 0, past_lens.data_ptr(), new_lens.data_ptr(), free_pages.data_ptr(),
        free_count.data_ptr(), block_table.data_ptr(), cu_q.data_ptr(), ctx_lens.data_ptr(), positions.data_ptr(),
        slots.data_ptr(), left.data_ptr()))


def splash_batch_release(ctx_lens: torch.Tensor, keep_lens: torch.Tensor | None, block_table: torch.Tensor,
                         page_size: int, free_pages: torch.Tensor, free_count: torch.Tensor, window: int = 0,
                         sinks: int = 0, stream=None) -> None:
    """Drops all but the first keep_lens [B] tokens of each request (None: drops none), and with a window also
    the tokens that no later one sees: their pages go back on the stack free_pages (free_count [1] entries, or left
    of splash_batch_tables, whose first entry is the count), their entries of block_table become -1, and ctx_lens [B]
    the tokens that are left."""
    where = "splash_batch_release"
    dev = _device_of(where, block_table)
    count = free_count.numel()
    if block_table.dim() != 2 or not 1 <= count <= 2:
        raise ValueError(f"{where}: block_table must be [B][max_pages], free_count [1] (or left [2])")
    B, pages = block_table.shape
    F = free_pages.numel()
    _int32_arrays(where, dev, (
        ("ctx_lens", ctx_lens, B), ("keep_lens", ctx_lens if keep_lens is None else keep_lens, B),
        ("block_table", block_table, B * pages), ("free_pages", free_pages, F), ("free_count", free_count, count)))
    _call(dev, stream, where, (_lib or load_library()).splash_batch_release, _packed(
        where, _BATCH_DROP, B, page_size, F, pages, window, sinks, ctx_lens.data_ptr(), 0 if keep_lens is None else keep_lens.data_ptr(),
        block_table.data_ptr(), free_pages.data_ptr(), free_count.data_ptr()))


def make_rope_desc(dims: int, base: float = 10000.0, interleaved: bool = True, scaling: str = "none",
                   factor: float = 1.0, orig_ctx: float = 4096.0, beta_fast: float = 32.0,
                   beta_slow: float = 1.0, amplitude: float = 1.0) -> SplashRopeDesc:
    """Rotary positions of a model (see splash_rope_desc in splash.h); scaling is "none",
    "linear" or "yarn"."""
    if scaling not in _SCALINGS:
        raise ValueError(f"make_rope_desc: scaling must be one of {sorted(_SCALINGS)}")
    return SplashRopeDesc(int(dims), int(bool(interleaved)), _SCALINGS[scaling], 0, float(base), float(factor),
                          float(orig_ctx), float(beta_fast), float(beta_slow), float(amplitude))


def splash_rope(x: torch.Tensor, positions: torch.Tensor, out: torch.Tensor, rope: SplashRopeDesc,
                stream=None) -> None:
    """out [T][H][d] <- x [T][H][d] rotated by positions int32 [T] (d = rope.dims).  Both are
    views with dense head rows and any token and head strides, e.g. q[..., 512:]; out may
    be x, and elements outside the views are not touched."""
    dev = _device_of("splash_rope", x, positions, out)
    dtype, shape = _DTYPES.get(x.dtype), x.shape
    if dtype is None or out.dtype != x.dtype or positions.dtype != torch.int32:
        raise ValueError("splash_rope: x and out must share bfloat16, float16 or float32; positions int32")
    if len(shape) != 3 or out.shape != shape or shape[2] != rope.dims or positions.shape != shape[:1]:
        raise ValueError("splash_rope: x and out must be [T][H][rope.dims], positions [T]")
    T, H, _ = shape
    xt, xh, x1 = x.stride()
    yt, yh, y1 = out.stride()
    if (x1 != 1 or y1 != 1 or not positions.is_contiguous()) and T and H:
        raise ValueError("splash_rope: head rows and positions must be dense")
    _call(dev, stream, "splash_rope", (_lib or load_library()).splash_rope, rope, dtype, x.data_ptr(), xt, xh,
          out.data_ptr(), yt, yh, positions.data_ptr(), T, H)


@functools.lru_cache(maxsize=1024)
def _norm_desc(width: int, norm_dims: int, rope_lo: int, weight_dtype: int, eps: float, offset: float) -> SplashNormDesc:
    """The description of a norm (read-only; the library reads it during the call)."""
    where = "splash_norm_rope"
    return SplashNormDesc(width, _int32(where, "norm_dims", norm_dims), _int32(where, "rope_lo", rope_lo), weight_dtype, eps, offset)


def _norm_rows(where: str, dev: int, x, weight, out, T: int, D: int, n: int, dtype, weight_dtype) -> bytes:
    shape = x.shape
    if len(shape) != 3 or shape[0] != T or shape[2] != D or out.shape != shape:
        raise ValueError(f"{where}: rows and their results must be [T][heads][D], q's and k's with the same T and D")
    if x.dtype is not dtype or out.dtype is not dtype:
        raise ValueError(f"{where}: rows and results must share one dtype")
    if x.get_device() != dev or out.get_device() != dev or (weight is not None and weight.get_device() != dev):
        raise ValueError(f"{where}: tensors must live on one CUDA device")
    xt, xh, x1 = x.stride()
    yt, yh, y1 = out.stride()
    H = shape[1]
    if (x1 != 1 or y1 != 1) and D > 1 and T and H:
        raise ValueError(f"{where}: rows must be dense")
    w = 0
    if weight is not None:
        if weight.dtype is not weight_dtype or weight.numel() != n or not weight.is_contiguous():
            raise ValueError(f"{where}: weights must be dense [norm_dims] of one floating dtype")
        w = weight.data_ptr()
    return _NORM_ROWS.pack(x.data_ptr(), xt, xh, out.data_ptr(), yt, yh, w, H, 0)


def splash_norm_rope(q: torch.Tensor, q_weight: torch.Tensor | None, q_out: torch.Tensor, k: torch.Tensor | None,
                     k_weight: torch.Tensor | None, k_out: torch.Tensor | None, positions: torch.Tensor | None,
                     rope: SplashRopeDesc | None, eps: float, norm_dims: int | None = None, rope_lo: int = 0,
                     weight_offset: float = 0.0, stream=None) -> None:
    """RMS norm (weights [norm_dims], None: ones) of the first norm_dims dims (None: all) of every row of q
    [T][Hq][D] and k [T][Hk][D] (None: q alone), and the rotation of dims [rope_lo, rope_lo + rope.dims) by positions
    int32 [T] (rope None: no rotation).  All are views with dense rows and any token and head strides; an output
    may be its input."""
    where = "splash_norm_rope"
    dev = _device_of(where, q)
    if (k is None) != (k_out is None):
        raise ValueError(f"{where}: k and k_out belong together")
    shape, dt = q.shape, q.dtype
    if len(shape) != 3:
        raise ValueError(f"{where}: q must be [T][heads][D]")
    T, _, D = shape
    n = D if norm_dims is None else int(norm_dims)
    weight = q_weight if q_weight is not None else k_weight
    wt = torch.float32 if weight is None else weight.dtype
    dtype, weight_dtype = _DTYPES.get(dt), _DTYPES.get(wt)
    if dtype is None or weight_dtype is None:
        raise ValueError(f"{where}: rows and weights must be bfloat16, float16 or float32")
    at = None
    if rope is not None:
        if (positions is None or positions.dtype is not torch.int32 or positions.numel() != T or positions.dim() != 1
                or not positions.is_contiguous() or positions.get_device() != dev):
            raise ValueError(f"{where}: positions must be contiguous int32 [T] on q's device")
        at = positions.data_ptr()
    a = _norm_rows(where, dev, q, q_weight, q_out, T, D, n, dt, wt)
    b = None if k is None else _norm_rows(where, dev, k, k_weight, k_out, T, D, n, dt, wt)
    _call(dev, stream, where, (_lib or load_library()).splash_norm_rope,
          _norm_desc(D, n, rope_lo, weight_dtype, eps, weight_offset), rope, dtype, a, b, at, T)


def splash_kv_append(latent: torch.Tensor, k_rope: torch.Tensor, cu_q: torch.Tensor,
                     block_table: torch.Tensor, ctx_lens: torch.Tensor, kv_pool: torch.Tensor,
                     rope: SplashRopeDesc | None = None, stream=None) -> None:
    """Writes new tokens (latent [N][512] and k_rope [N][64], bf16 with dense rows) to their slots
    of kv_pool: bf16 [num_pages][P][576], or uint8 [num_pages][P][656] for MXFP8.  cu_q, block_table and
    ctx_lens (the new tokens included) say where; rope rotates k_rope by the tokens' positions."""
    where = "splash_kv_append"
    dev = _device_of(where, latent, k_rope, cu_q, block_table, ctx_lens, kv_pool)
    if latent.dtype != torch.bfloat16 or k_rope.dtype != torch.bfloat16:
        raise ValueError("splash_kv_append: latent and k_rope must be bfloat16")
    lat, kr = latent.shape, k_rope.shape
    if len(lat) != 2 or lat[1] != 512 or kr != (lat[0], 64):
        raise ValueError("splash_kv_append: latent [N][512] and k_rope [N][64]")
    N = lat[0]
    lt, l1 = latent.stride()
    kt, k1 = k_rope.stride()
    if N and (l1 != 1 or k1 != 1):
        raise ValueError("splash_kv_append: latent and k_rope must have dense rows")
    if kv_pool.dtype == torch.bfloat16:
        fmt, width = SPLASH_KV_BF16, 576
    elif kv_pool.dtype == torch.uint8:
        fmt, width = SPLASH_KV_MXFP8, MXFP8_ROW_BYTES
    else:
        raise ValueError("splash_kv_append: kv_pool must be bfloat16 or uint8 (MXFP8)")
    pool = kv_pool.shape
    if len(pool) != 3 or pool[2] != width or not kv_pool.is_contiguous():
        raise ValueError(f"splash_kv_append: kv_pool must be contiguous [num_pages][P][{width}]")
    B, pages = _index_arrays(where, cu_q, block_table, ctx_lens)
    _call(dev, stream, where, (_lib or load_library()).splash_kv_append,
          _shape_desc(B, 1, pool[1], pool[0], pages, 1.0), rope, fmt, latent.data_ptr(), lt, k_rope.data_ptr(), kt,
          cu_q.data_ptr(), N, block_table.data_ptr(), ctx_lens.data_ptr(), kv_pool.data_ptr())


def splash_kv_unpack(src_pool: torch.Tensor, dst_pool: torch.Tensor, src_ids: torch.Tensor,
                     dst_ids: torch.Tensor, stream=None) -> None:
    """bf16 dst_pool[dst_ids[i]] <- the values of MXFP8 src_pool[src_ids[i]] (uint8 [num_pages][P][656])."""
    where = "splash_kv_unpack"
    dev = _device_of(where, src_pool, dst_pool, src_ids, dst_ids)
    if src_ids.dtype != torch.int32 or dst_ids.dtype != torch.int32 or src_ids.shape != dst_ids.shape:
        raise ValueError("splash_kv_unpack: ids must be int32 of equal length")
    s, d = src_pool.shape, dst_pool.shape
    if (src_pool.dtype != torch.uint8 or dst_pool.dtype != torch.bfloat16 or len(s) != 3 or len(d) != 3
            or s[2] != MXFP8_ROW_BYTES or d[2] != 576 or s[1] != d[1]):
        raise ValueError("splash_kv_unpack: src uint8 [num_pages][P][656], dst bfloat16 [num_pages][P][576]")
    if not (src_pool.is_contiguous() and dst_pool.is_contiguous() and src_ids.is_contiguous() and dst_ids.is_contiguous()):
        raise ValueError("splash_kv_unpack: tensors must be contiguous")
    if not d[1]:
        return
    _call(dev, stream, where, (_lib or load_library()).splash_kv_unpack, src_pool.data_ptr(), dst_pool.data_ptr(),
          s[1], src_ids.data_ptr(), dst_ids.data_ptr(), src_ids.numel(), s[0], d[0])


def _chunk_desc(where: str, q, kv_pool, B: int, pages: int, scale) -> SplashAttnDesc:
    shape, pool = q.shape, kv_pool.shape
    if q.dtype != torch.bfloat16 or kv_pool.dtype != torch.bfloat16:
        raise ValueError(f"{where}: q and kv_pool must be bfloat16")
    if len(shape) != 3 or len(pool) != 3 or shape[2] != 576 or pool[2] != 576:
        raise ValueError(f"{where}: q [N][H][576] and kv_pool [num_pages][P][576]")
    return _shape_desc(B, shape[1], pool[1], pool[0], pages, float(scale))


def chunk_workspace(q: torch.Tensor, kv_pool: torch.Tensor, block_table: torch.Tensor, scale: float,
                    head_lo: int = 0, head_hi: int | None = None, num_groups: int = 0) -> torch.Tensor:
    """Allocates (with torch, on q's device) a workspace for splash_chunk_attn and splash_chunk_attn_ex on q's
    rows; it serves every later call with no more new tokens, requests, pages per request and groups."""
    where = "splash_chunk_workspace_size"
    dev = _device_of(where, q, kv_pool, block_table)
    if block_table.dim() != 2:
        raise ValueError(f"{where}: block_table must be [B][max_pages]")
    desc = _chunk_desc(where, q, kv_pool, *block_table.shape, scale)
    head_hi = q.shape[1] if head_hi is None else head_hi
    with torch.cuda.device(dev):
        n = int(load_library().splash_chunk_workspace_size_ex(
            desc, SplashChunkExt(num_groups=_int32(where, "num_groups", num_groups)), q.shape[0], int(head_lo), int(head_hi)))
    if n == 0:
        raise SplashError(SPLASH_ERR_UNSUPPORTED, where)
    return torch.empty(n, dtype=torch.uint8, device=q.device)


def splash_chunk_attn(q: torch.Tensor, kv_pool: torch.Tensor, cu_q: torch.Tensor, block_table: torch.Tensor,
                      ctx_lens: torch.Tensor, head_lo: int, head_hi: int, tok_lo: int, tok_hi: int,
                      out: torch.Tensor, lse: torch.Tensor, workspace: torch.Tensor, scale: float,
                      stream=None) -> None:
    """Causal attention of new tokens q [N][H][576] over the paged cache that holds them (see
    splash.h); writes heads [head_lo, head_hi) of out [N][H][512] (bf16 or fp32) and lse [N][H]."""
    args, dev = _chunk_args("splash_chunk_attn", q, kv_pool, cu_q, block_table, ctx_lens, head_lo, head_hi, tok_lo,
                            tok_hi, out, lse, workspace, scale)
    _call(dev, stream, "splash_chunk_attn", (_lib or load_library()).splash_chunk_attn, *args)


@functools.lru_cache(maxsize=256)
def _window_ext(window: int, sinks: int) -> SplashChunkExt:
    """A window without groups (read-only; the library reads it during the call)."""
    where = "splash_chunk_attn_ex"
    return SplashChunkExt(_int32(where, "window", window), _int32(where, "sinks", sinks))


def splash_chunk_attn_ex(q: torch.Tensor, kv_pool: torch.Tensor, cu_q: torch.Tensor, block_table: torch.Tensor,
                         ctx_lens: torch.Tensor, head_lo: int, head_hi: int, tok_lo: int, tok_hi: int,
                         out: torch.Tensor, lse: torch.Tensor, workspace: torch.Tensor, scale: float, window: int = 0,
                         sinks: int = 0, cu_groups: torch.Tensor | None = None,
                         prefix_lens: torch.Tensor | None = None, stream=None) -> None:
    """splash_chunk_attn whose new tokens see, with window > 0, the last `window` positions up to their own and the
    first `sinks` ones; or where the requests [cu_groups[g], cu_groups[g + 1]) (int32 [G + 1]) share the pages of their
    first prefix_lens[g] (int32 [G]) tokens, which gives the same results with fewer reads and products."""
    where = "splash_chunk_attn_ex"
    args, dev = _chunk_args(where, q, kv_pool, cu_q, block_table, ctx_lens, head_lo, head_hi, tok_lo, tok_hi, out, lse,
                            workspace, scale)
    if (cu_groups is None) != (prefix_lens is None):
        raise ValueError(f"{where}: cu_groups and prefix_lens belong together")
    if cu_groups is None:
        ext = _window_ext(int(window), int(sinks))
    else:
        G = prefix_lens.numel()
        _int32_arrays(where, dev, (("cu_groups", cu_groups, G + 1), ("prefix_lens", prefix_lens, G)))
        ext = SplashChunkExt(_int32(where, "window", window), _int32(where, "sinks", sinks), cu_groups.data_ptr(),
                             prefix_lens.data_ptr(), G)
    _call(dev, stream, where, (_lib or load_library()).splash_chunk_attn_ex, args[0], ext, *args[1:])


def _chunk_args(where: str, q, kv_pool, cu_q, block_table, ctx_lens, head_lo, head_hi, tok_lo, tok_hi, out, lse, workspace,
                scale):
    """The C arguments of a chunk call (ext and stream aside) and the device."""
    dev = _device_of(where, q, kv_pool, cu_q, block_table, ctx_lens, out, lse, workspace)
    B, pages = _index_arrays(where, cu_q, block_table, ctx_lens)
    desc = _chunk_desc(where, q, kv_pool, B, pages, scale)
    N, H, _ = q.shape
    out_dtype = _DTYPES.get(out.dtype)
    if out_dtype not in (SPLASH_BF16, SPLASH_F32) or lse.dtype != torch.float32:
        raise ValueError(f"{where}: out must be bfloat16 or float32, lse float32")
    if out.shape != (N, H, 512) or lse.shape != (N, H):
        raise ValueError(f"{where}: out must be [N][H][512], lse [N][H]")
    if not (q.is_contiguous() and kv_pool.is_contiguous() and out.is_contiguous() and lse.is_contiguous()
            and workspace.is_contiguous()):
        raise ValueError(f"{where}: tensors must be contiguous")
    return (desc, q.data_ptr(), kv_pool.data_ptr(), cu_q.data_ptr(), N, block_table.data_ptr(), ctx_lens.data_ptr(),
            int(head_lo), int(head_hi), int(tok_lo), int(tok_hi), out_dtype, out.data_ptr(), lse.data_ptr(),
            workspace.data_ptr(), workspace.numel() * workspace.element_size()), dev


def splash_workspace_status(workspace: torch.Tensor, stream=None) -> int:
    """Synchronises the stream and returns the SPLASH_DEVICE_* bits of the workspace's last decode or chunk call."""
    flags = ctypes.c_uint32(0)
    with torch.cuda.device(workspace.device):
        rc = load_library().splash_workspace_status(_ptr(workspace), ctypes.byref(flags),
                                                    _stream(stream))
    if rc != SPLASH_OK:
        raise SplashError(rc, "splash_workspace_status")
    return int(flags.value)
