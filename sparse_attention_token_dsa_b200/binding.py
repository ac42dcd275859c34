"""Thin ctypes binding of libdsaidx.so (C ABI declared in include/dsaidx.h).

Argument marshalling only: PyTorch provides device memory and the current
stream; every step of the computation runs in the library's CUDA kernels.
There is no CPU fallback — importing this module without the built library
raises.
"""
from __future__ import annotations

import ctypes as C
import os

import torch

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libdsaidx.so")

DSA_OK, DSA_ERR_INVALID, DSA_ERR_UNSUPPORTED, DSA_ERR_WORKSPACE = 0, -1, -2, -3
DSA_ERR_CUDA, DSA_ERR_NONFINITE, DSA_ERR_TIMEOUT, DSA_ERR_INTERNAL = -4, -5, -6, -7
DSA_F32, DSA_BF16, DSA_E4M3 = 0, 1, 2
DSA_ALGO_DSA, DSA_ALGO_MISA, DSA_ALGO_MISA_DAGGER, DSA_ALGO_HISA = 0, 1, 2, 3
DSA_ALGO_LISA, DSA_ALGO_RESMISA = 4, 5
DSA_FLAG_CHECK = 1
DSA_FLAG_SORTED = 2
DSA_FLAG_BY_POSITION = 4
DSA_FLAG_DOSA = 8                    # exact bound pruning of the dense scan
DSA_FLAG_INTERLEAVED = 16            # rotary pairs side by side (default: two halves)
DSA_FLAG_INVERSE = 32                # rotary positions: the transpose
DSA_FLAG_POW2_SCALE = 64             # cache write: scales are powers of two
DSA_ROPE_PLAIN, DSA_ROPE_LINEAR, DSA_ROPE_YARN = 0, 1, 2
DSA_FLAG_TEST_STALL = 0x80000000   # tests of the timeout path only (see include/dsaidx.h)


class DsaProblem(C.Structure):
    _fields_ = [("batch", C.c_int32), ("n_q", C.c_int32), ("n_k", C.c_int32),
                ("heads", C.c_int32), ("dim", C.c_int32), ("topk", C.c_int32),
                ("q_dtype", C.c_int32), ("k_dtype", C.c_int32), ("q_pos0", C.c_void_p),
                ("k_len", C.c_void_p), ("flags", C.c_uint32)]


class DsaRouteParams(C.Structure):
    _fields_ = [("misa_block", C.c_int32), ("misa_h", C.c_int32), ("k_prime", C.c_int32),
                ("hisa_block", C.c_int32), ("hisa_r", C.c_int32), ("lisa_pool", C.c_int32),
                ("res_block", C.c_int32), ("res_r", C.c_int32)]


class DsaMlaProblem(C.Structure):
    _fields_ = [("batch", C.c_int32), ("tokens_per_seq", C.c_int32), ("n_k", C.c_int32),
                ("heads", C.c_int32), ("dim_qk", C.c_int32), ("dim_v", C.c_int32),
                ("topk", C.c_int32), ("scale", C.c_float), ("flags", C.c_uint32)]


class DsaRopeProblem(C.Structure):
    _fields_ = [("n_tokens", C.c_int64), ("heads", C.c_int32), ("dim", C.c_int32),
                ("offset", C.c_int32), ("rot_dim", C.c_int32), ("dtype", C.c_int32),
                ("mscale", C.c_float), ("x_token_stride", C.c_int64),
                ("x_head_stride", C.c_int64), ("out_token_stride", C.c_int64),
                ("out_head_stride", C.c_int64), ("flags", C.c_uint32)]


class DsaCache(C.Structure):
    _fields_ = [("n_pages", C.c_int32), ("page_size", C.c_int32), ("dim_q", C.c_int32),
                ("dim_raw", C.c_int32), ("codes", C.c_void_p), ("scale", C.c_void_p),
                ("raw", C.c_void_p), ("codes_page_stride", C.c_int64),
                ("scale_page_stride", C.c_int64), ("raw_page_stride", C.c_int64)]


class DsaPagedMlaProblem(C.Structure):
    _fields_ = [("batch", C.c_int32), ("n_q", C.c_int32), ("heads", C.c_int32),
                ("dim_qk", C.c_int32), ("dim_v", C.c_int32), ("max_pages", C.c_int32),
                ("page_size", C.c_int32), ("scale", C.c_float), ("flags", C.c_uint32)]


class DsaError(RuntimeError):
    def __init__(self, status: int, what: str):
        super().__init__(f"{what}: {status_string(status)} ({status})")
        self.status = status


def _load():
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"{LIB_PATH} is missing: build it with "
                          "`python -m sparse_attention_token_dsa_b200.build`")
    lib = C.CDLL(LIB_PATH)
    vp, i32, i64, sz = C.c_void_p, C.c_int32, C.c_int64, C.c_size_t
    P = C.POINTER(DsaProblem)
    R = C.POINTER(DsaRouteParams)
    lib.dsa_status_string.restype = C.c_char_p
    lib.dsa_status_string.argtypes = [i32]
    lib.dsa_read_status.argtypes = [vp, vp]
    lib.dsa_read_pruned.argtypes = [vp, vp, C.POINTER(C.c_ulonglong)]
    lib.dsa_host_staging_size.argtypes = [P, i32, C.POINTER(sz)]
    lib.dsa_dosa_bounds.argtypes = [P, vp, vp, vp, vp, vp, vp, sz, vp]
    lib.dsa_index_host.argtypes = [P, vp, vp, vp, vp, vp, vp, vp, i32, vp, sz, vp]
    lib.dsa_workspace_size.argtypes = [P, i32, R, C.POINTER(sz)]
    lib.dsa_index.argtypes = [P, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp]
    lib.dsa_route_chunk_rows.argtypes = [P, i32, R, C.POINTER(i32)]
    lib.dsa_index_noalloc.argtypes = [P, vp, vp, vp, vp, vp, vp, vp, vp]
    lib.dsa_index_scan.argtypes = [P, vp, vp, vp, vp, vp, vp, sz, vp]
    lib.dsa_index_select.argtypes = [P, vp, vp, vp, sz, vp]
    lib.misa_index.argtypes = [P, R, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp]
    lib.misa_dagger_index.argtypes = [P, R, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp]
    lib.hisa_index.argtypes = [P, R, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp]
    lib.lisa_index.argtypes = [P, R, vp, vp, vp, vp, vp, vp, vp, sz, vp]
    lib.resmisa_index.argtypes = [P, R, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp]
    lib.dsa_quantize_e4m3.argtypes = [vp, i32, i64, i32, vp, vp, vp]
    lib.dsa_sparse_mla.argtypes = [C.POINTER(DsaMlaProblem), vp, vp, vp, vp, vp, vp, sz, vp]
    lib.dsa_indexer_backward.argtypes = [P, vp, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp]
    f64, K, Z = C.c_double, C.POINTER(DsaCache), C.POINTER(DsaRopeProblem)
    lib.dsa_rope_frequencies.argtypes = [i32, f64, i32, f64, f64, f64, f64, C.POINTER(f64)]
    lib.dsa_rope.argtypes = [Z, vp, vp, vp, vp, vp]
    lib.dsa_cache_write.argtypes = [K, vp, i32, i64, i64, vp, Z, vp, vp, C.c_uint32, vp]
    lib.dsa_cache_read.argtypes = [K, vp, i32, i32, i32, vp, vp, i32, vp]
    lib.dsa_cache_read_codes.argtypes = [K, vp, i32, i32, i32, vp, vp, vp, vp]
    A = C.POINTER(DsaPagedMlaProblem)
    lib.dsa_paged_mla_workspace_size.argtypes = [A, C.POINTER(sz)]
    lib.dsa_paged_mla.argtypes = [A, K, vp, vp, vp, vp, vp, vp, vp, sz, vp]
    for f in ("dsa_paged_mla_workspace_size", "dsa_paged_mla", "dsa_rope_frequencies", "dsa_rope", "dsa_cache_write", "dsa_cache_read",
              "dsa_cache_read_codes",
              "dsa_read_status", "dsa_read_pruned", "dsa_host_staging_size", "dsa_index_host",
              "dsa_dosa_bounds",
              "dsa_workspace_size", "dsa_route_chunk_rows", "dsa_index",
              "dsa_index_noalloc",
              "dsa_index_scan",
              "dsa_index_select", "misa_index",
              "misa_dagger_index", "hisa_index", "lisa_index", "resmisa_index",
              "dsa_quantize_e4m3", "dsa_sparse_mla", "dsa_indexer_backward"):
        getattr(lib, f).restype = C.c_int
    return lib


lib = _load()


def status_string(s: int) -> str:
    return lib.dsa_status_string(s).decode()


def _check(rc: int, what: str):
    if rc != DSA_OK:
        raise DsaError(rc, what)


def _dtype_code(t: torch.Tensor) -> int:
    if t.dtype == torch.float32:
        return DSA_F32
    if t.dtype == torch.bfloat16:
        return DSA_BF16
    if t.dtype in (torch.uint8, torch.float8_e4m3fn):
        return DSA_E4M3
    raise TypeError(f"unsupported operand dtype {t.dtype}")


def _ptr(t):
    return None if t is None else C.c_void_p(t.data_ptr())


_OPERAND = (torch.float32, torch.bfloat16, torch.uint8, torch.float8_e4m3fn)
_F32 = (torch.float32,)
_I32 = (torch.int32,)
_U8 = (torch.uint8,)


def _args(**named):
    """Check tensor arguments before any library call: dtype, C-contiguous
    layout and a CUDA device (the kernels take raw device pointers, so a host or
    strided tensor would be misread).  Each value is (tensor or None, dtypes)."""
    given = [(name, t, dtypes) for name, (t, dtypes) in named.items() if t is not None]
    for name, t, dtypes in given:
        if not isinstance(t, torch.Tensor):
            raise TypeError(f"{name}: expected a torch.Tensor, got {type(t).__name__}")
        if t.dtype not in dtypes:
            raise TypeError(f"{name}: dtype {t.dtype}, expected one of {dtypes}")
        if not t.is_contiguous():
            raise ValueError(f"{name}: must be contiguous")
    for name, t, _ in given:
        if t.device.type != "cuda":
            raise ValueError(f"{name}: must be on a CUDA device, not {t.device}")


def _common_args(q, k, w, q_scale=None, k_scale=None, q_pos0=None, k_len=None, out=None,
                 workspace=None, **extra):
    idx, sc = (None, None) if out is None else out
    _args(q=(q, _OPERAND), k=(k, _OPERAND), w=(w, _F32), q_scale=(q_scale, _F32),
          k_scale=(k_scale, _F32), q_pos0=(q_pos0, _I32), k_len=(k_len, _I32),
          out_idx=(idx, _I32), out_score=(sc, _F32), workspace=(workspace, _U8), **extra)


def _stream(stream):
    if stream is None:
        stream = torch.cuda.current_stream()
    return C.c_void_p(stream.cuda_stream)


def problem(q: torch.Tensor, k: torch.Tensor, topk: int, q_pos0=None, k_len=None,
            flags: int = 0) -> DsaProblem:
    """q [batch, n_q, heads, dim], k [batch, n_k, dim]."""
    B, nq, H, d = q.shape
    nk = k.shape[1]
    return DsaProblem(B, nq, nk, H, d, topk, _dtype_code(q), _dtype_code(k), _ptr(q_pos0),
                      _ptr(k_len), flags)


def route_params(misa_block=0, misa_h=0, k_prime=0, hisa_block=0, hisa_r=0, lisa_pool=0,
                 res_block=0, res_r=0) -> DsaRouteParams:
    return DsaRouteParams(misa_block, misa_h, k_prime, hisa_block, hisa_r, lisa_pool, res_block,
                          res_r)


def dsa_workspace_size(p: DsaProblem, algo: int = DSA_ALGO_DSA, rp: DsaRouteParams | None = None) -> int:
    n = C.c_size_t(0)
    _check(lib.dsa_workspace_size(C.byref(p), algo, None if rp is None else C.byref(rp),
                                  C.byref(n)), "dsa_workspace_size")
    return n.value


def dsa_route_chunk_rows(p: DsaProblem, algo: int, rp: DsaRouteParams) -> int:
    """Query rows per sequence of one row chunk of a routed entry point."""
    n = C.c_int32(0)
    _check(lib.dsa_route_chunk_rows(C.byref(p), algo, C.byref(rp), C.byref(n)),
           "dsa_route_chunk_rows")
    return n.value


def _workspace(nbytes: int, device, workspace):
    if workspace is not None and workspace.numel() >= nbytes:
        return workspace
    return torch.empty(max(nbytes, 256), dtype=torch.uint8, device=device)


def _outputs(B, nq, topk, device, out):
    if out is not None:
        return out
    return (torch.empty((B, nq, topk), dtype=torch.int32, device=device),
            torch.empty((B, nq, topk), dtype=torch.float32, device=device))


def dsa_index(q, k, w, topk, q_scale=None, k_scale=None, q_pos0=None, k_len=None, flags=0,
              out=None, workspace=None, stream=None):
    """DSA indexer top-k.  Returns (idx int32 [B,n_q,k], score fp32 [B,n_q,k])."""
    _common_args(q, k, w, q_scale, k_scale, q_pos0, k_len, out, workspace)
    p = problem(q, k, topk, q_pos0, k_len, flags)
    ws = _workspace(dsa_workspace_size(p), q.device, workspace)
    idx, sc = _outputs(q.shape[0], q.shape[1], topk, q.device, out)
    _check(lib.dsa_index(C.byref(p), _ptr(q), _ptr(q_scale), _ptr(k), _ptr(k_scale), _ptr(w),
                         _ptr(idx), _ptr(sc), _ptr(ws), ws.numel(), _stream(stream)), "dsa_index")
    return idx, sc


def dsa_index_noalloc(q, k, w, topk, q_scale=None, k_scale=None, q_pos0=None, k_len=None,
                      flags=0, out=None, stream=None):
    """dsa_index on the library's fixed internal scratch (no workspace argument).

    For callers that cannot allocate device memory at call time; problems that
    need more than the library's 64 MiB scratch raise DsaError(DSA_ERR_WORKSPACE),
    and calls that overlap on the GPU race on the shared scratch."""
    _common_args(q, k, w, q_scale, k_scale, q_pos0, k_len, out)
    p = problem(q, k, topk, q_pos0, k_len, flags)
    idx, sc = _outputs(q.shape[0], q.shape[1], topk, q.device, out)
    _check(lib.dsa_index_noalloc(C.byref(p), _ptr(q), _ptr(q_scale), _ptr(k), _ptr(k_scale),
                                 _ptr(w), _ptr(idx), _ptr(sc), _stream(stream)),
           "dsa_index_noalloc")
    return idx, sc


def _host_args(**named):
    """Host-side tensors of dsa_index_host: dtype, C-contiguous, on the CPU."""
    for name, (t, dtypes) in named.items():
        if t is None:
            continue
        if not isinstance(t, torch.Tensor):
            raise TypeError(f"{name}: expected a torch.Tensor, got {type(t).__name__}")
        if t.dtype not in dtypes:
            raise TypeError(f"{name}: dtype {t.dtype}, expected one of {dtypes}")
        if not t.is_contiguous():
            raise ValueError(f"{name}: must be contiguous")
        if t.device.type != "cpu":
            raise ValueError(f"{name}: must be in host memory, not {t.device}")


def dsa_host_staging_size(p: DsaProblem, chunk_rows: int) -> int:
    n = C.c_size_t(0)
    _check(lib.dsa_host_staging_size(C.byref(p), chunk_rows, C.byref(n)), "dsa_host_staging_size")
    return n.value


def dsa_index_host(q_host, k, w_host, topk, q_scale_host=None, k_scale=None, q_pos0=None,
                   k_len=None, flags=0, chunk_rows=16384, out=None, staging=None, stream=None):
    """dsa_index with q, w (and q_scale) in (page-locked) host memory and the
    results written to host tensors; the rows stream in chunks so the copies
    overlap the scan.  k, k_scale, q_pos0, k_len on the GPU.  Returns host
    (idx int32 [B, n_q, k], score fp32 [B, n_q, k]); with `out` given, writes there."""
    _host_args(q_host=(q_host, _OPERAND), w_host=(w_host, _F32), q_scale_host=(q_scale_host, _F32))
    _args(k=(k, _OPERAND), k_scale=(k_scale, _F32), q_pos0=(q_pos0, _I32), k_len=(k_len, _I32),
          staging=(staging, _U8))
    p = problem(q_host, k, topk, q_pos0, k_len, flags)
    B, nq = q_host.shape[0], q_host.shape[1]
    if out is None:
        out = (torch.empty((B, nq, topk), dtype=torch.int32).pin_memory(),
               torch.empty((B, nq, topk), dtype=torch.float32).pin_memory())
    idx, sc = out
    _host_args(out_idx=(idx, _I32), out_score=(sc, _F32))
    nbytes = dsa_host_staging_size(p, chunk_rows)
    if staging is None or staging.numel() < nbytes:
        staging = torch.empty(nbytes, dtype=torch.uint8, device=k.device)
    _check(lib.dsa_index_host(C.byref(p), _ptr(q_host), _ptr(q_scale_host), _ptr(k), _ptr(k_scale),
                              _ptr(w_host), _ptr(idx), _ptr(sc), chunk_rows, _ptr(staging),
                              staging.numel(), _stream(stream)), "dsa_index_host")
    return idx, sc


def dsa_index_scan(p: DsaProblem, q, k, w, workspace, q_scale=None, k_scale=None, stream=None):
    """First stage of dsa_index (scores + candidate logs in `workspace`)."""
    _common_args(q, k, w, q_scale, k_scale, workspace=workspace)
    _check(lib.dsa_index_scan(C.byref(p), _ptr(q), _ptr(q_scale), _ptr(k), _ptr(k_scale), _ptr(w),
                              _ptr(workspace), workspace.numel(), _stream(stream)), "dsa_index_scan")


def dsa_index_select(p: DsaProblem, idx, score, workspace, stream=None):
    """Second stage of dsa_index (exact top-k per row from the logs)."""
    _args(idx=(idx, _I32), score=(score, _F32), workspace=(workspace, _U8))
    _check(lib.dsa_index_select(C.byref(p), _ptr(idx), _ptr(score), _ptr(workspace),
                                workspace.numel(), _stream(stream)), "dsa_index_select")


def misa_index(q, k, w, topk, block, h, q_pos0=None, k_len=None, flags=0, out=None,
               out_heads=None, out_E=None, workspace=None, stream=None):
    _common_args(q, k, w, None, None, q_pos0, k_len, out, workspace,
                 out_heads=(out_heads, _I32), out_E=(out_E, _F32))
    p = problem(q, k, topk, q_pos0, k_len, flags)
    rp = route_params(misa_block=block, misa_h=h)
    ws = _workspace(dsa_workspace_size(p, DSA_ALGO_MISA, rp), q.device, workspace)
    idx, sc = _outputs(q.shape[0], q.shape[1], topk, q.device, out)
    _check(lib.misa_index(C.byref(p), C.byref(rp), _ptr(q), _ptr(k), _ptr(w), _ptr(idx), _ptr(sc),
                          _ptr(out_heads), _ptr(out_E), _ptr(ws), ws.numel(), _stream(stream)),
           "misa_index")
    return idx, sc


def misa_dagger_index(q, k, w, topk, block, h, k_prime, q_pos0=None, k_len=None, flags=0,
                      out=None, out_heads=None, out_pool=None, workspace=None, stream=None):
    _common_args(q, k, w, None, None, q_pos0, k_len, out, workspace,
                 out_heads=(out_heads, _I32), out_pool=(out_pool, _I32))
    p = problem(q, k, topk, q_pos0, k_len, flags)
    rp = route_params(misa_block=block, misa_h=h, k_prime=k_prime)
    ws = _workspace(dsa_workspace_size(p, DSA_ALGO_MISA_DAGGER, rp), q.device, workspace)
    idx, sc = _outputs(q.shape[0], q.shape[1], topk, q.device, out)
    _check(lib.misa_dagger_index(C.byref(p), C.byref(rp), _ptr(q), _ptr(k), _ptr(w), _ptr(idx),
                                 _ptr(sc), _ptr(out_heads), _ptr(out_pool), _ptr(ws), ws.numel(),
                                 _stream(stream)), "misa_dagger_index")
    return idx, sc


def hisa_index(q, k, w, topk, block, r, route_h=0, route_block=1024, q_pos0=None, k_len=None,
               flags=0, out=None, out_blocks=None, out_heads=None, workspace=None, stream=None):
    _common_args(q, k, w, None, None, q_pos0, k_len, out, workspace,
                 out_blocks=(out_blocks, _I32), out_heads=(out_heads, _I32))
    p = problem(q, k, topk, q_pos0, k_len, flags)
    rp = route_params(misa_block=route_block if route_h else 0, misa_h=route_h, hisa_block=block,
                      hisa_r=r)
    ws = _workspace(dsa_workspace_size(p, DSA_ALGO_HISA, rp), q.device, workspace)
    idx, sc = _outputs(q.shape[0], q.shape[1], topk, q.device, out)
    _check(lib.hisa_index(C.byref(p), C.byref(rp), _ptr(q), _ptr(k), _ptr(w), _ptr(idx), _ptr(sc),
                          _ptr(out_blocks), _ptr(out_heads), _ptr(ws), ws.numel(), _stream(stream)),
           "hisa_index")
    return idx, sc


def lisa_index(q, k, w, topk, pool=0, q_pos0=None, k_len=None, flags=0, out=None,
               out_pool=None, workspace=None, stream=None):
    """Indexer LISA (pool == 0: top-k by the linear term g . k) or LISA-dagger
    (pool = M: the top-M by g . k reranked by the full score over every head)."""
    _common_args(q, k, w, None, None, q_pos0, k_len, out, workspace, out_pool=(out_pool, _I32))
    p = problem(q, k, topk, q_pos0, k_len, flags)
    rp = route_params(lisa_pool=pool)
    ws = _workspace(dsa_workspace_size(p, DSA_ALGO_LISA, rp), q.device, workspace)
    idx, sc = _outputs(q.shape[0], q.shape[1], topk, q.device, out)
    _check(lib.lisa_index(C.byref(p), C.byref(rp), _ptr(q), _ptr(k), _ptr(w), _ptr(idx), _ptr(sc),
                          _ptr(out_pool), _ptr(ws), ws.numel(), _stream(stream)), "lisa_index")
    return idx, sc


def resmisa_index(q, k, w, topk, block, r, q_pos0=None, k_len=None, flags=0, out=None,
                  out_heads=None, out_S=None, workspace=None, stream=None):
    """ResMiSA: the linear term of every head plus r routed residual heads."""
    _common_args(q, k, w, None, None, q_pos0, k_len, out, workspace,
                 out_heads=(out_heads, _I32), out_S=(out_S, _F32))
    p = problem(q, k, topk, q_pos0, k_len, flags)
    rp = route_params(res_block=block, res_r=r)
    ws = _workspace(dsa_workspace_size(p, DSA_ALGO_RESMISA, rp), q.device, workspace)
    idx, sc = _outputs(q.shape[0], q.shape[1], topk, q.device, out)
    _check(lib.resmisa_index(C.byref(p), C.byref(rp), _ptr(q), _ptr(k), _ptr(w), _ptr(idx),
                             _ptr(sc), _ptr(out_heads), _ptr(out_S), _ptr(ws), ws.numel(),
                             _stream(stream)), "resmisa_index")
    return idx, sc


def sparse_mla(q, kv, idx, scale, tokens_per_seq=None, flags=0, out=None, out_lse=None,
               workspace=None, stream=None):
    """Sparse MLA over fixed selected positions.  q [T, heads, 576] bf16,
    kv [batch, n_k, 576] bf16, idx [T, k] int32 (-1 empty).  Returns (out
    [T, heads, 512] bf16, lse [T, heads] fp32)."""
    _args(q=(q, (torch.bfloat16,)), kv=(kv, (torch.bfloat16,)), idx=(idx, _I32),
          out=(out, (torch.bfloat16,)), out_lse=(out_lse, _F32), workspace=(workspace, _U8))
    T, H, dqk = q.shape
    B, n_k, _ = kv.shape
    tps = T // B if tokens_per_seq is None else tokens_per_seq
    p = DsaMlaProblem(B, tps, n_k, H, dqk, 512, idx.shape[1], float(scale), flags)
    if out is None:
        out = torch.empty((T, H, 512), dtype=torch.bfloat16, device=q.device)
    if out_lse is None:
        out_lse = torch.empty((T, H), dtype=torch.float32, device=q.device)
    ws = _workspace(256, q.device, workspace)
    _check(lib.dsa_sparse_mla(C.byref(p), _ptr(q), _ptr(kv), _ptr(idx), _ptr(out), _ptr(out_lse),
                              _ptr(ws), ws.numel(), _stream(stream)), "dsa_sparse_mla")
    return out, out_lse


def indexer_backward(q, k, w, sel, grad, dk=None, flags=0, workspace=None, stream=None):
    """Gradients of sum g I over the selected positions: returns (dq [B, n_q, H, d],
    dk [B, n_k, d], dw [B, n_q, H]) in fp32; dk is added to when given."""
    _args(q=(q, (torch.bfloat16,)), k=(k, (torch.bfloat16,)), w=(w, _F32), sel=(sel, _I32),
          grad=(grad, _F32), dk=(dk, _F32), workspace=(workspace, _U8))
    p = problem(q, k, sel.shape[-1], flags=flags)
    dq = torch.empty(q.shape, dtype=torch.float32, device=q.device)
    dw = torch.empty(w.shape, dtype=torch.float32, device=q.device)
    if dk is None:
        dk = torch.zeros(k.shape, dtype=torch.float32, device=q.device)
    ws = _workspace(256, q.device, workspace)
    _check(lib.dsa_indexer_backward(C.byref(p), _ptr(q), _ptr(k), _ptr(w), _ptr(sel), _ptr(grad),
                                    _ptr(dq), _ptr(dk), _ptr(dw), _ptr(ws), ws.numel(),
                                    _stream(stream)), "dsa_indexer_backward")
    return dq, dk, dw


def dsa_quantize_e4m3(x: torch.Tensor, stream=None):
    """Per-row e4m3 codes (uint8, same shape) and fp32 scales (shape[:-1])."""
    _args(x=(x, (torch.float32, torch.bfloat16)))
    cols = x.shape[-1]
    rows = x.numel() // cols
    out = torch.empty(x.shape, dtype=torch.uint8, device=x.device)
    sc = torch.empty(x.shape[:-1], dtype=torch.float32, device=x.device)
    _check(lib.dsa_quantize_e4m3(_ptr(x), _dtype_code(x), rows, cols, _ptr(out), _ptr(sc),
                                 _stream(stream)), "dsa_quantize_e4m3")
    return out, sc


# ------------------------------------------------------ a cached DSA layer --
# A call of a decode step takes a few microseconds on the GPU, so what is right is found
# out in a few attribute reads (numbers rather than objects for devices and streams).

_F64, _I64 = (torch.float64,), (torch.int64,)
_ROWS = (torch.bfloat16, torch.float32)
_CODES = (torch.uint8, torch.float8_e4m3fn)
_BF16 = (torch.bfloat16,)
_ROW_CODE = {torch.bfloat16: DSA_BF16, torch.float32: DSA_F32}
_Tensor = torch.Tensor


def _need(name, t, dtypes, device, strided=False):
    """Raise for the first thing that is wrong with a tensor; `device`: its index."""
    if not isinstance(t, _Tensor):
        raise TypeError(f"{name}: expected a torch.Tensor, got {type(t).__name__}")
    if t.dtype not in dtypes:
        raise TypeError(f"{name}: dtype {t.dtype}, expected one of {dtypes}")
    if t.get_device() != device:
        raise ValueError(f"{name}: must be on cuda:{device}, not {t.device}")
    if not strided and not t.is_contiguous():
        raise ValueError(f"{name}: must be contiguous")


def _cuda_index(name, t):
    """Index of a tensor's CUDA device."""
    if not isinstance(t, _Tensor):
        raise TypeError(f"{name}: expected a torch.Tensor, got {type(t).__name__}")
    if not t.is_cuda:
        raise ValueError(f"{name}: must be on a CUDA device, not {t.device}")
    return t.get_device()


# The current stream and device as numbers (torch.cuda.current_stream() makes an object,
# which takes longer than the launch it is for).
_current_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda index: torch.cuda.current_stream(index).cuda_stream)
_current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device


def _on(index, stream, what, call, *args):
    """call(*args, stream) with device `index` current, on `stream` (default: that device's
    current one); raises DsaError for a status other than DSA_OK."""
    raw = _current_stream(index) if stream is None else stream.cuda_stream
    if index == _current_device():
        rc = call(*args, raw)
    else:
        with torch.cuda.device(index):
            rc = call(*args, raw)
    if rc != DSA_OK:
        raise DsaError(rc, what)


def _new(stream, make):
    """make() with its memory (and fill) on the stream that the call runs on."""
    if stream is None:
        return make()
    with torch.cuda.stream(stream):
        return make()


def rope_frequencies(rot_dim, base=10000.0, scaling="plain", factor=1.0, original_len=4096,
                     beta_fast=32.0, beta_slow=1.0, device="cuda"):
    """Table of rotary frequencies (radians a position, float64 [rot_dim / 2]) to keep
    beside the weights.  scaling: "plain", "linear" or "yarn" (see include/dsaidx.h)."""
    kinds = {"plain": DSA_ROPE_PLAIN, "linear": DSA_ROPE_LINEAR, "yarn": DSA_ROPE_YARN}
    if scaling not in kinds:
        raise ValueError(f"scaling: {scaling!r}, expected one of {tuple(kinds)}")
    out = torch.empty(max(rot_dim, 0) // 2, dtype=torch.float64)
    _check(lib.dsa_rope_frequencies(rot_dim, base, kinds[scaling], factor, original_len, beta_fast,
                                    beta_slow, C.cast(out.data_ptr(), C.POINTER(C.c_double))),
           "dsa_rope_frequencies")
    return out.to(device)


def _rope(x, pos, freq, offset, interleaved, mscale, out, stream, flags, what):
    dev = _cuda_index("x", x)
    code = _ROW_CODE.get(x.dtype)
    if code is None:
        _need("x", x, _ROWS, dev, strided=True)
    shape = x.shape
    if len(shape) != 3:
        raise ValueError("x: must be [tokens, heads, dim] with contiguous values")
    n, heads, dim = shape
    xt, xh, xv = x.stride()
    if xv != 1 and dim > 1:
        raise ValueError("x: must be [tokens, heads, dim] with contiguous values")
    _need("pos", pos, _I32, dev)
    _need("freq", freq, _F64, dev)
    if pos.numel() != n:
        raise ValueError(f"pos: {pos.numel()} positions for {n} tokens")
    if out is None:
        out = _new(stream, lambda: torch.empty((n, heads, dim), dtype=x.dtype, device=x.device))
        ot, oh = heads * dim, dim
    else:
        _need("out", out, (x.dtype,), dev, strided=True)
        if out.shape != shape:
            raise ValueError("out: must have x's shape and contiguous values")
        ot, oh, ov = out.stride()
        if ov != 1 and dim > 1:
            raise ValueError("out: must have x's shape and contiguous values")
    if n == 0 or heads == 0:
        return out
    p = DsaRopeProblem(n, heads, dim, offset, 2 * freq.numel(), code, mscale, xt, xh, ot, oh,
                       flags | DSA_FLAG_INTERLEAVED if interleaved else flags)
    _on(dev, stream, what, lib.dsa_rope, C.byref(p), x.data_ptr(), pos.data_ptr(),
        freq.data_ptr(), out.data_ptr())
    return out


def rope(x, pos, freq, offset=0, interleaved=False, mscale=1.0, out=None, stream=None):
    """Rotary positions on the 2 * len(freq) values of each head that start at `offset`.
    x [tokens, heads, dim] bf16 or fp32 (any token and head strides), pos [tokens] int32,
    freq as from rope_frequencies.  out=x works in place."""
    return _rope(x, pos, freq, offset, interleaved, mscale, out, stream, 0, "rope")


def rope_backward(grad, pos, freq, offset=0, interleaved=False, mscale=1.0, out=None, stream=None):
    """Gradient of rope: the transpose of the same rotation applied to `grad`."""
    return _rope(grad, pos, freq, offset, interleaved, mscale, out, stream, DSA_FLAG_INVERSE,
                 "rope_backward")


def _page_stride(name, t, dtypes, dev, pages, page, width):
    """Page stride of a plane of rows of `width`."""
    _need(name, t, dtypes, dev, strided=True)
    if t.shape != (pages, page, width):
        raise ValueError(f"{name}: shape {tuple(t.shape)}, expected {(pages, page, width)}")
    ps, rs, vs = t.stride()
    if (vs != 1 and width > 1) or (rs != width and page > 1):
        raise ValueError(f"{name}: the rows of a page must be contiguous")
    return page * width if pages == 1 else ps


class PagedCache:
    """The planes of a paged cache (dsa_cache of include/dsaidx.h): codes [pages, page,
    dim_q] e4m3 (or uint8), scale [pages, page, dim_q / 128] fp32, raw [pages, page,
    dim_raw] bf16; codes and scale, or raw, may be None.  The pages of a plane may be
    strided (a layer of a larger block); the rest of it is contiguous."""

    __slots__ = ("codes", "scale", "raw", "c", "index")

    def __init__(self, codes=None, scale=None, raw=None):
        if codes is None and raw is None:
            raise ValueError("codes, raw: at least one plane is needed")
        if (codes is None) != (scale is None):
            raise ValueError("codes and scale come together")
        first = raw if codes is None else codes
        dev = self.index = _cuda_index("raw" if codes is None else "codes", first)
        self.codes, self.scale, self.raw = codes, scale, raw
        if first.dim() != 3:
            raise ValueError("planes: must be [pages, page, width]")
        pages, page, dim_q = first.shape
        dim_raw = codes_ps = scale_ps = raw_ps = 0
        codes_p = scale_p = raw_p = None
        if codes is None:
            dim_q = 0
        else:
            codes_ps = _page_stride("codes", codes, _CODES, dev, pages, page, dim_q)
            scale_ps = _page_stride("scale", scale, _F32, dev, pages, page, dim_q // 128)
            codes_p, scale_p = codes.data_ptr(), scale.data_ptr()
        if raw is not None:
            _need("raw", raw, _BF16, dev, strided=True)
            dim_raw = raw.shape[-1] if raw.dim() else 0
            raw_ps = _page_stride("raw", raw, _BF16, dev, pages, page, dim_raw)
            raw_p = raw.data_ptr()
        self.c = DsaCache(pages, page, dim_q, dim_raw, codes_p, scale_p, raw_p, codes_ps, scale_ps,
                          raw_ps)

    @staticmethod
    def empty(n_pages, page_size, dim_q, dim_raw, device="cuda"):
        """A cache of zeros (e4m3 codes 0, scale 1)."""
        codes = scale = raw = None
        if dim_q:
            codes = torch.zeros((n_pages, page_size, dim_q), dtype=torch.uint8, device=device)
            codes = codes.view(torch.float8_e4m3fn)
            scale = torch.ones((n_pages, page_size, dim_q // 128), device=device)
        if dim_raw:
            raw = torch.zeros((n_pages, page_size, dim_raw), dtype=torch.bfloat16, device=device)
        return PagedCache(codes, scale, raw)


def cache_write(cache, x, slots, pow2=False, freq=None, pos=None, offset=0, interleaved=False,
                mscale=1.0, stream=None):
    """Write rows x [tokens, dim_q + dim_raw] (bf16 or fp32, rows may be strided) at slots
    [tokens] int64 (page * page_size + row; -1 skips).  With freq and pos the values at
    `offset` are rotated first.  pow2: scales that are powers of two (for paged_mla)."""
    dev, c = cache.index, cache.c
    _need("x", x, _ROWS, dev, strided=True)
    _need("slots", slots, _I64, dev)
    width = c.dim_q + c.dim_raw
    if x.dim() != 2 or x.shape[1] != width:
        raise ValueError(f"x: must be [tokens, {width}] with contiguous rows")
    n, (xt, xv) = x.shape[0], x.stride()
    if xv != 1 and width > 1:
        raise ValueError(f"x: must be [tokens, {width}] with contiguous rows")
    if slots.numel() != n:
        raise ValueError(f"slots: {slots.numel()} slots for {n} tokens")
    turn = pos_p = freq_p = None
    if freq is not None and pos is not None:
        _need("freq", freq, _F64, dev)
        _need("pos", pos, _I32, dev)
        if pos.numel() != n:
            raise ValueError(f"pos: {pos.numel()} positions for {n} tokens")
        turn = C.byref(DsaRopeProblem(n, 1, width, offset, 2 * freq.numel(), 0, mscale, 0, 0, 0, 0,
                                      DSA_FLAG_INTERLEAVED if interleaved else 0))
        pos_p, freq_p = pos.data_ptr(), freq.data_ptr()
    elif freq is not None or pos is not None:
        raise ValueError("freq and pos come together")
    _on(dev, stream, "dsa_cache_write", lib.dsa_cache_write, C.byref(c), x.data_ptr(),
        _ROW_CODE[x.dtype], xt, n, slots.data_ptr(), turn, pos_p, freq_p,
        DSA_FLAG_POW2_SCALE if pow2 else 0)


def _table(cache, block_table, k_len):
    """Sequences and pages of a block table; pointer of the lengths."""
    _need("block_table", block_table, _I32, cache.index)
    if block_table.dim() != 2:
        raise ValueError("block_table: must be [batch, max_pages]")
    batch, pages = block_table.shape
    if k_len is None:
        return batch, pages, None
    _need("k_len", k_len, _I32, cache.index)
    if k_len.numel() != batch:
        raise ValueError(f"k_len: {k_len.numel()} lengths for {batch} sequences")
    return batch, pages, k_len.data_ptr()


def cache_read(cache, block_table, n_k, k_len=None, dtype=torch.bfloat16, out=None, stream=None):
    """Positions [0, n_k) of each sequence as rows [batch, n_k, dim_q + dim_raw] of bf16
    (the kv of sparse_mla) or fp32.  Rows at or behind k_len[b] are left as they were
    (zeros in a new tensor)."""
    dev, c = cache.index, cache.c
    batch, pages, lens = _table(cache, block_table, k_len)
    shape = (batch, n_k, c.dim_q + c.dim_raw)
    if out is None:
        out = _new(stream, lambda: torch.zeros(shape, dtype=dtype, device=block_table.device))
    _need("out", out, _ROWS, dev)
    if out.shape != shape:
        raise ValueError(f"out: shape {tuple(out.shape)}, expected {shape}")
    _on(dev, stream, "dsa_cache_read", lib.dsa_cache_read, C.byref(c), block_table.data_ptr(),
        batch, pages, n_k, lens, out.data_ptr(), _ROW_CODE[out.dtype])
    return out


def cache_read_codes(cache, block_table, n_k, k_len=None, out=None, stream=None):
    """Positions [0, n_k) of each sequence as they are held: (codes [batch, n_k, dim_q],
    scale [batch, n_k] or [batch, n_k, dim_q / 128]), with dim_q = 128 the k and k_scale of
    dsa_index.  Rows at or behind k_len[b] are left as they were (codes 0, scale 1 in new
    tensors)."""
    dev, c = cache.index, cache.c
    batch, pages, lens = _table(cache, block_table, k_len)
    dim_q = c.dim_q
    groups = dim_q // 128
    if out is None:
        per_row = (batch, n_k) if groups == 1 else (batch, n_k, groups)
        out = _new(stream, lambda: (
            torch.zeros((batch, n_k, dim_q), dtype=torch.uint8, device=block_table.device)
            .view(torch.float8_e4m3fn), torch.ones(per_row, device=block_table.device)))
    codes, scale = out
    _need("codes", codes, _CODES, dev)
    _need("scale", scale, _F32, dev)
    if codes.shape != (batch, n_k, dim_q) or scale.numel() != batch * n_k * groups:
        raise ValueError(f"out: shapes {tuple(codes.shape)}, {tuple(scale.shape)}")
    _on(dev, stream, "dsa_cache_read_codes", lib.dsa_cache_read_codes, C.byref(c),
        block_table.data_ptr(), batch, pages, n_k, lens, codes.data_ptr(), scale.data_ptr())
    return codes, scale


def paged_mla_workspace_size(batch, n_q, heads, max_pages, page_size) -> int:
    """Bytes of workspace of a paged_mla call (q [batch, n_q, heads, 576])."""
    p = DsaPagedMlaProblem(batch, n_q, heads, 576, 512, max_pages, page_size, 1.0, 0)
    n = C.c_size_t(0)
    _check(lib.dsa_paged_mla_workspace_size(C.byref(p), C.byref(n)), "dsa_paged_mla_workspace_size")
    return n.value


def paged_mla(q, cache, block_table, k_len, scale, q_len=None, flags=0, out=None, out_lse=None,
              workspace=None, stream=None):
    """Latent attention over every cached position.  q [batch, n_q, heads, 576] bf16, cache a
    PagedCache of 576-wide rows (bf16, or 512 e4m3 + 64 bf16), block_table [batch, max_pages],
    k_len [batch] cached positions (the queries' own included), q_len [batch] query tokens
    (default n_q).  Returns (out [batch, n_q, heads, 512] bf16, lse [batch, n_q, heads] fp32);
    rows of tokens at or behind q_len are left as they were."""
    dev, c = cache.index, cache.c
    _need("q", q, _BF16, dev)
    shape = q.shape
    if len(shape) != 4:
        raise ValueError("q: must be [batch, n_q, heads, 576]")
    batch, n_q, heads, dim = shape
    seqs, pages, lens = _table(cache, block_table, k_len)
    if lens is None or seqs != batch:
        raise ValueError(f"block_table, k_len: {seqs} sequences for {batch} in q")
    q_lens = None
    if q_len is not None:
        _need("q_len", q_len, _I32, dev)
        if q_len.numel() != batch:
            raise ValueError(f"q_len: {q_len.numel()} lengths for {batch} sequences")
        q_lens = q_len.data_ptr()
    p = DsaPagedMlaProblem(batch, n_q, heads, dim, 512, pages, c.page_size, scale, flags)
    rows = batch * n_q * heads
    if out is None:
        out = _new(stream, lambda: torch.empty((batch, n_q, heads, 512), dtype=torch.bfloat16,
                                               device=q.device))
    else:
        _need("out", out, _BF16, dev)
        if out.numel() != rows * 512:
            raise ValueError(f"out: shape {tuple(out.shape)}")
    if out_lse is None:
        out_lse = _new(stream, lambda: torch.empty((batch, n_q, heads), device=q.device))
    else:
        _need("out_lse", out_lse, _F32, dev)
        if out_lse.numel() != rows:
            raise ValueError(f"out_lse: shape {tuple(out_lse.shape)}")
    if workspace is None:
        n = C.c_size_t(0)
        _check(lib.dsa_paged_mla_workspace_size(C.byref(p), C.byref(n)), "dsa_paged_mla")
        workspace = _new(stream, lambda: torch.empty(n.value, dtype=torch.uint8, device=q.device))
    else:
        _need("workspace", workspace, _U8, dev)
    _on(dev, stream, "dsa_paged_mla", lib.dsa_paged_mla, C.byref(p), C.byref(c), q.data_ptr(),
        block_table.data_ptr(), lens, q_lens, out.data_ptr(), out_lse.data_ptr(),
        workspace.data_ptr(), workspace.numel())
    return out, out_lse


def dsa_read_status(workspace: torch.Tensor, stream=None) -> int:
    _args(workspace=(workspace, _U8))
    return lib.dsa_read_status(_ptr(workspace), _stream(stream))


def dsa_read_pruned(workspace: torch.Tensor, stream=None) -> int:
    """(query row, key tile) pairs the last DSA_FLAG_DOSA call on `workspace` skipped."""
    _args(workspace=(workspace, _U8))
    n = C.c_ulonglong(0)
    _check(lib.dsa_read_pruned(_ptr(workspace), _stream(stream), C.byref(n)), "dsa_read_pruned")
    return int(n.value)


def dsa_dosa_bounds(q, k, w, q_pos0=None, k_len=None, flags=0, workspace=None, stream=None):
    """DoSA block upper and lower bounds, each [B * n_q, ceil(n_k / 1024)] fp32
    (see include/dsaidx.h)."""
    _common_args(q, k, w, q_pos0=q_pos0, k_len=k_len, workspace=workspace)
    p = problem(q, k, 1, q_pos0, k_len, flags | DSA_FLAG_DOSA)
    ws = _workspace(dsa_workspace_size(p), q.device, workspace)
    nblk = (k.shape[1] + 1023) // 1024
    ub = torch.empty((q.shape[0] * q.shape[1], nblk), dtype=torch.float32, device=q.device)
    lb = torch.empty_like(ub)
    _check(lib.dsa_dosa_bounds(C.byref(p), _ptr(q), _ptr(k), _ptr(w), _ptr(ub), _ptr(lb),
                               _ptr(ws), ws.numel(), _stream(stream)), "dsa_dosa_bounds")
    return ub, lb
