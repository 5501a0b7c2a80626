"""Thin Python binding of libtsa's C ABI (include/tsa.h), same names.

Argument marshalling only: every step of the decode path runs in the CUDA
kernels behind these calls.  Torch supplies device memory and streams.  There
is no CPU fallback: if libtsa.so is missing or cannot load, importing this
module raises.
"""
from __future__ import annotations

import ctypes
import math
import os

import torch

_LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libtsa.so")
if not os.path.exists(_LIB_PATH):
    raise ImportError(f"libtsa.so is not built ({_LIB_PATH}); run `python -m "
                      "top_sparse_attention_02_b200.build` (or __graft_entry__.build())")
_lib = ctypes.CDLL(_LIB_PATH)

TSA_OK, TSA_ERR_INVALID_ARG, TSA_ERR_UNSUPPORTED, TSA_ERR_WORKSPACE = 0, 1, 2, 3
TSA_ERR_CUDA, TSA_ERR_DEVICE_BOUNDS, TSA_ERR_DEVICE_TIMEOUT = 4, 5, 6
FULL, SELECT, REUSE = 0, 1, 2
STATUS_NAMES = {0: "TSA_OK", 1: "TSA_ERR_INVALID_ARG", 2: "TSA_ERR_UNSUPPORTED", 3: "TSA_ERR_WORKSPACE",
                4: "TSA_ERR_CUDA", 5: "TSA_ERR_DEVICE_BOUNDS", 6: "TSA_ERR_DEVICE_TIMEOUT"}


class tsa_shape(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int32), ("Hq", ctypes.c_int32), ("Hkv", ctypes.c_int32),
                ("Ncap", ctypes.c_int32), ("d", ctypes.c_int32)]


class tsa_step_args(ctypes.Structure):
    _fields_ = [("shape", tsa_shape), ("Q", ctypes.c_void_p), ("K", ctypes.c_void_p),
                ("V", ctypes.c_void_p), ("Kmean", ctypes.c_void_p), ("seq_lens", ctypes.c_void_p),
                ("k_per_seq", ctypes.c_void_p), ("k_max", ctypes.c_int32), ("block", ctypes.c_int32),
                ("mode", ctypes.c_int32), ("scale", ctypes.c_float), ("idx_in", ctypes.c_void_p),
                ("idx_out", ctypes.c_void_p), ("O", ctypes.c_void_p), ("ws", ctypes.c_void_p),
                ("ws_bytes", ctypes.c_size_t), ("flags", ctypes.c_uint32)]


KV_HOST = 1  # tsa_step_args.flags: K and V in mapped page-locked host memory
EARLY_INPUTS = 2  # tsa_step_args.flags: the kernel before the step writes none of lens, k's, K, V, idx_in


_vp, _sz, _i32, _f32 = ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int32, ctypes.c_float
_i64 = ctypes.c_int64
_SIGS = {
    "tsa_workspace_size": (_sz, [tsa_shape, _i32, _i32, _i32]),
    "tsa_workspace_init": (ctypes.c_int, [_vp, _sz, _vp]),
    "tsa_block_summarize": (ctypes.c_int, [_vp, _vp, tsa_shape, _i32, _vp, _vp, _sz, _vp]),
    "sparse_decode_score": (ctypes.c_int, [_vp, _vp, _vp, tsa_shape, _i32, _f32, _vp, _vp, _sz, _vp]),
    "topk_select": (ctypes.c_int, [_vp, _vp, _vp, _i32, tsa_shape, _i32, _vp, _vp, _sz, _vp]),
    "sparse_decode_attn": (ctypes.c_int, [_vp, _vp, _vp, _vp, _vp, _vp, _i32, _i32, tsa_shape, _f32,
                                          _vp, _vp, _sz, _vp]),
    "sparse_decode_attn_noalloc": (ctypes.c_int, [_vp, _vp, _vp, _vp, _vp, _vp, _i32, _i32, tsa_shape,
                                                  _f32, _vp, _vp]),
    "tsa_decode_step": (ctypes.c_int, [ctypes.POINTER(tsa_step_args), _vp]),
    "tsa_index_overlap": (ctypes.c_int, [_vp, _i32, _i32, _i32, _vp, _vp, _vp, _sz, _vp]),
    "tsa_reuse_policy": (ctypes.c_int, [_vp, _i32, ctypes.c_double, _vp, _vp, _vp, _vp]),
    "tsa_shard_workspace_size": (_sz, [tsa_shape, _i32, _i32]),
    "tsa_shard_select": (ctypes.c_int, [_vp, _vp, _vp, tsa_shape, _vp, _i32, _f32, _i32, _vp, _vp, _vp, _sz, _vp]),
    "tsa_shard_merge": (ctypes.c_int, [_vp, _vp, _i32, tsa_shape, _vp, _i32, _vp, _vp, _sz, _vp]),
    "tsa_shard_attend": (ctypes.c_int, [_vp, _vp, _vp, _vp, tsa_shape, _vp, _vp, _i32, _i32, _f32, _vp, _vp, _vp,
                                        _sz, _vp]),
    "tsa_shard_combine": (ctypes.c_int, [_vp, _vp, _i32, tsa_shape, _vp, _vp]),
    "tsa_check_device_status": (ctypes.c_int, [_vp, _vp]),
    "tsa_last_error_string": (ctypes.c_char_p, []),
    "tsa_launch_count": (ctypes.c_uint64, []),
    "tsa_hbm_copy": (ctypes.c_int, [_vp, _vp, _sz, _vp]),
    "tsa_hbm_read": (ctypes.c_int, [_vp, _sz, _vp, _sz, _vp]),
    "tsa_hbm_gather": (ctypes.c_int, [_vp, _sz, _vp, _i32, _vp, _sz, _vp]),
}
for _name, (_res, _args) in _SIGS.items():
    _f = getattr(_lib, _name)
    _f.restype, _f.argtypes = _res, _args


class TsaError(RuntimeError):
    def __init__(self, status: int, msg: str):
        super().__init__(f"{STATUS_NAMES.get(status, status)}: {msg}")
        self.status = status


def lib():
    """The loaded ctypes library (for callers that marshal raw pointers themselves)."""
    return _lib


def last_error() -> str:
    return (_lib.tsa_last_error_string() or b"").decode()


def _ok(st: int):
    if st != TSA_OK:
        raise TsaError(st, last_error())


def _ptr(t):
    if t is None:
        return None
    if isinstance(t, int):
        return t
    return t.data_ptr()


def _stream(stream):
    if stream is None:
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def shape_of(Q: torch.Tensor, K: torch.Tensor) -> tsa_shape:
    B, Hq, d = Q.shape
    _, Hkv, Ncap, _ = K.shape
    return tsa_shape(B, Hq, Hkv, Ncap, d)


def workspace_size(shape: tsa_shape, k_max: int, block: int, mode: int) -> int:
    n = _lib.tsa_workspace_size(shape, k_max, block, mode)
    if n == 0:
        raise TsaError(TSA_ERR_INVALID_ARG, last_error())
    return n


def workspace_init(ws: torch.Tensor, stream=None):
    _ok(_lib.tsa_workspace_init(_ptr(ws), ws.numel() * ws.element_size(), _stream(stream)))


def new_workspace(shape: tsa_shape, k_max: int, block: int, mode: int, device) -> torch.Tensor:
    """Allocate (with torch) and zero a workspace for these arguments."""
    n = workspace_size(shape, k_max, block, mode)
    ws = torch.empty(n, dtype=torch.uint8, device=device)
    workspace_init(ws)
    return ws


def _wsargs(ws):
    return _ptr(ws), ws.numel() * ws.element_size()


def block_summarize(K, seq_lens, block: int, Kmean, ws, stream=None, shape=None):
    s = shape or tsa_shape(K.shape[0], K.shape[1], K.shape[1], K.shape[2], K.shape[3])
    _ok(_lib.tsa_block_summarize(_ptr(K), _ptr(seq_lens), s, block, _ptr(Kmean), *_wsargs(ws),
                                 _stream(stream)))


def sparse_decode_score(Q, keys, seq_lens, shape: tsa_shape, block: int, scale: float, scores, ws,
                        stream=None):
    _ok(_lib.sparse_decode_score(_ptr(Q), _ptr(keys), _ptr(seq_lens), shape, block, scale,
                                 _ptr(scores), *_wsargs(ws), _stream(stream)))


def topk_select(scores, seq_lens, k_per_seq, k_max: int, shape: tsa_shape, block: int, idx, ws,
                stream=None):
    _ok(_lib.topk_select(_ptr(scores), _ptr(seq_lens), _ptr(k_per_seq), k_max, shape, block,
                         _ptr(idx), *_wsargs(ws), _stream(stream)))


def sparse_decode_attn(Q, K, V, seq_lens, idx, k_per_seq, k_max: int, block: int, scale: float, O,
                       ws, stream=None, shape=None):
    s = shape or shape_of(Q, K)
    _ok(_lib.sparse_decode_attn(_ptr(Q), _ptr(K), _ptr(V), _ptr(seq_lens), _ptr(idx),
                                _ptr(k_per_seq), k_max, block, s, scale, _ptr(O), *_wsargs(ws),
                                _stream(stream)))


def sparse_decode_attn_noalloc(Q, K, V, seq_lens, idx, k_per_seq, k_max: int, block: int,
                               scale: float, O, stream=None, shape=None):
    """sparse_decode_attn with the library's fixed internal scratch instead of a workspace
    (for callers that cannot allocate one); calls on one device must not overlap."""
    s = shape or shape_of(Q, K)
    _ok(_lib.sparse_decode_attn_noalloc(_ptr(Q), _ptr(K), _ptr(V), _ptr(seq_lens), _ptr(idx),
                                        _ptr(k_per_seq), k_max, block, s, scale, _ptr(O),
                                        _stream(stream)))


def step_args(Q, K, V, seq_lens, O, ws, *, mode: int, scale: float, k_max: int = 0, block: int = 1,
              k_per_seq=None, Kmean=None, idx_in=None, idx_out=None, flags: int = 0) -> tsa_step_args:
    a = tsa_step_args()
    a.shape = shape_of(Q, K)
    a.Q, a.K, a.V, a.Kmean = _ptr(Q), _ptr(K), _ptr(V), _ptr(Kmean)
    a.seq_lens, a.k_per_seq = _ptr(seq_lens), _ptr(k_per_seq)
    a.k_max, a.block, a.mode, a.scale = k_max, block, mode, scale
    a.idx_in, a.idx_out, a.O = _ptr(idx_in), _ptr(idx_out), _ptr(O)
    a.ws, a.ws_bytes = _wsargs(ws)
    a.flags = flags
    return a


def decode_step(args: tsa_step_args, stream=None):
    _ok(_lib.tsa_decode_step(ctypes.byref(args), _stream(stream)))


def index_overlap(idx, counts, M, ws, stream=None):
    """Overlap of L layers' index lists idx [L, B, Hkv, k_max] (int32, device) into
    counts [L, L, B*Hkv] int32 and M [L, L] float64 (either may be None)."""
    L, units, k_max = idx.shape[0], math.prod(idx.shape[1:-1]), idx.shape[-1]
    _ok(_lib.tsa_index_overlap(_ptr(idx), L, units, k_max, _ptr(counts), _ptr(M), *_wsargs(ws),
                               _stream(stream)))


def reuse_policy(M, theta: float, force_full=None):
    """HyLRA's reuse policy from the similarity matrix M [L, L] (host, float64,
    row = target layer): returns (source [L] int32 numpy array, n_full, total_sim)."""
    import numpy as np

    Mh = np.ascontiguousarray(M.cpu().numpy() if isinstance(M, torch.Tensor) else M, dtype=np.float64)
    L = Mh.shape[0]
    assert Mh.shape == (L, L)
    ff = None if force_full is None else np.ascontiguousarray(np.asarray(force_full, dtype=np.uint8))
    src = np.empty(L, dtype=np.int32)
    nf = ctypes.c_int32()
    sim = ctypes.c_double()
    _ok(_lib.tsa_reuse_policy(Mh.ctypes.data, L, float(theta), None if ff is None else ff.ctypes.data,
                              src.ctypes.data, ctypes.byref(nf), ctypes.byref(sim)))
    return src, nf.value, sim.value


def shard_workspace_size(shard_shape: tsa_shape, k_max: int, n_shards: int) -> int:
    n = _lib.tsa_shard_workspace_size(shard_shape, k_max, n_shards)
    if n == 0:
        raise TsaError(TSA_ERR_INVALID_ARG, last_error())
    return int(n)


def shard_select(Q, K_shard, shard_lens, k_per_seq, k_max: int, scale: float, row0: int, cand_scores, cand_rows,
                 ws, stream=None):
    _ok(_lib.tsa_shard_select(_ptr(Q), _ptr(K_shard), _ptr(shard_lens), shape_of(Q, K_shard), _ptr(k_per_seq),
                              k_max, scale, row0, _ptr(cand_scores), _ptr(cand_rows), *_wsargs(ws), _stream(stream)))


def shard_merge(cand_scores, cand_rows, shape: tsa_shape, k_per_seq, k_max: int, idx, ws, stream=None):
    _ok(_lib.tsa_shard_merge(_ptr(cand_scores), _ptr(cand_rows), cand_scores.shape[0], shape, _ptr(k_per_seq),
                             k_max, _ptr(idx), *_wsargs(ws), _stream(stream)))


def shard_attend(Q, K_shard, V_shard, shard_lens, idx, k_per_seq, k_max: int, row0: int, scale: float, O_part,
                 lse_part, ws, stream=None):
    _ok(_lib.tsa_shard_attend(_ptr(Q), _ptr(K_shard), _ptr(V_shard), _ptr(shard_lens), shape_of(Q, K_shard),
                              _ptr(idx), _ptr(k_per_seq), k_max, row0, scale, _ptr(O_part), _ptr(lse_part),
                              *_wsargs(ws), _stream(stream)))


def shard_combine(O_parts, lse_parts, shape: tsa_shape, O, stream=None):
    _ok(_lib.tsa_shard_combine(_ptr(O_parts), _ptr(lse_parts), O_parts.shape[0], shape, _ptr(O), _stream(stream)))


def check_device_status(ws, stream=None):
    _ok(_lib.tsa_check_device_status(_ptr(ws), _stream(stream)))


def launch_count() -> int:
    return int(_lib.tsa_launch_count())


def hbm_copy(src, dst, nbytes: int, stream=None):
    _ok(_lib.tsa_hbm_copy(_ptr(src), _ptr(dst), nbytes, _stream(stream)))


def hbm_read(src, nbytes: int, ws, stream=None):
    _ok(_lib.tsa_hbm_read(_ptr(src), nbytes, *_wsargs(ws), _stream(stream)))


def hbm_gather(base, rows, ws, stream=None):
    """Gather the 256-byte rows `rows` (int32, device) of `base` (the probe; nothing is kept)."""
    nbytes = base.numel() * base.element_size()
    _ok(_lib.tsa_hbm_gather(_ptr(base), nbytes, _ptr(rows), rows.numel(), *_wsargs(ws), _stream(stream)))


# ------------------------------------------------------------------ paged cache

class tsa_paged_cache(ctypes.Structure):
    _fields_ = [("K", _vp), ("V", _vp), ("page_table", _vp), ("page_stride", _i64), ("head_stride", _i64),
                ("row_stride", _i64), ("num_pages", _i32), ("page_size", _i32), ("max_pages", _i32), ("B", _i32),
                ("Hkv", _i32), ("d", _i32), ("dtype", _i32)]


class tsa_rotation(ctypes.Structure):
    _fields_ = [("inv_freq", _vp), ("rot_dim", _i32), ("interleaved", _i32)]


class tsa_qk_args(ctypes.Structure):
    _fields_ = [("q", _vp), ("k", _vp), ("q_out", _vp), ("k_out", _vp), ("q_stride_t", _i64), ("q_stride_h", _i64),
                ("k_stride_t", _i64), ("k_stride_h", _i64), ("q_out_stride_t", _i64), ("q_out_stride_h", _i64),
                ("k_out_stride_t", _i64), ("k_out_stride_h", _i64), ("q_weight", _vp), ("k_weight", _vp),
                ("positions", _vp), ("rot", tsa_rotation), ("T", _i32), ("Hq", _i32), ("Hkv", _i32), ("d", _i32),
                ("dtype", _i32), ("eps", _f32)]


class tsa_append_args(ctypes.Structure):
    _fields_ = [("cache", tsa_paged_cache), ("K", _vp), ("V", _vp), ("k_stride_t", _i64), ("k_stride_h", _i64),
                ("v_stride_t", _i64), ("v_stride_h", _i64), ("seq", _vp), ("row", _vp), ("positions", _vp),
                ("rot", tsa_rotation), ("T", _i32), ("ws", _vp), ("ws_bytes", _sz)]


class tsa_paged_attn_args(ctypes.Structure):
    _fields_ = [("cache", tsa_paged_cache), ("Q", _vp), ("seq_lens", _vp), ("idx", _vp), ("k_per_seq", _vp),
                ("O", _vp), ("lse", _vp), ("Hq", _i32), ("k_max", _i32), ("prefix_len", _i32), ("scale", _f32),
                ("ws", _vp), ("ws_bytes", _sz)]


for _name, _argtypes, _res in (("tsa_qk_norm_rope", [ctypes.POINTER(tsa_qk_args), _vp], ctypes.c_int),
                               ("tsa_paged_append", [ctypes.POINTER(tsa_append_args), _vp], ctypes.c_int),
                               ("tsa_paged_workspace_size", [ctypes.POINTER(tsa_paged_cache), _i32, _i32], _sz),
                               ("tsa_paged_attn", [ctypes.POINTER(tsa_paged_attn_args), _vp], ctypes.c_int),
                               ("tsa_prefix_attn", [ctypes.POINTER(tsa_paged_attn_args), _vp], ctypes.c_int)):
    _f = getattr(_lib, _name)
    _f.restype, _f.argtypes = _res, _argtypes

_DTYPES = {torch.bfloat16: 0, torch.float16: 1}


def _need(ok: bool, msg: str):
    if not ok:
        raise TsaError(TSA_ERR_INVALID_ARG, msg)


def _tensor(t, what: str, dtype, shape, device, contiguous: bool = True):
    """t is a tensor of this type, shape (None: any size) and device; contiguous, or
    with contiguous elements in its last dimension."""
    _need(isinstance(t, torch.Tensor) and t.dtype == dtype, f"{what} must be a {dtype} tensor")
    _need(t.dim() == len(shape) and all(n is None or n == m for n, m in zip(shape, t.shape)),
          f"{what} must have the shape {list(shape)} (got {list(t.shape)})")
    _need(t.device == device, f"{what} is on {t.device}, not {device}")
    if contiguous:
        _need(t.is_contiguous(), f"{what} must be contiguous")
    else:
        _need(t.shape[-1] == 1 or t.stride(-1) == 1, f"{what}: the last dimension must be contiguous")


def _hold(a, device, *tensors):
    """The arguments keep their tensors alive and remember their device."""
    a._tensors, a._device, a._index = tensors, device, device.index if device.type == "cuda" else None
    return a


def _launch(fn, a, stream):
    """Enqueue on `stream` (None: torch's current stream on the tensors' device), with
    that device current.  (The raw queries below: a decode step makes many such calls of
    a few microseconds each, and torch's stream and device objects cost as much again.)"""
    i = a._index
    _need(i is not None, "the tensors are not on a CUDA device")
    if i == torch._C._cuda_getDevice():
        st = fn(ctypes.byref(a), torch._C._cuda_getCurrentRawStream(i) if stream is None else _stream(stream))
    else:
        with torch.cuda.device(i):
            st = fn(ctypes.byref(a), _stream(stream))
    if st:
        _ok(st)


def paged_cache(K_pages, V_pages, page_table) -> tsa_paged_cache:
    """A cache in pages: K_pages, V_pages [num_pages, Hkv, page_size, 128] bf16 or fp16 with
    the same strides (a pool laid out row by row is passed as pool.permute(0, 2, 1, 3)),
    page_table [B, max_pages] int32."""
    _need(isinstance(K_pages, torch.Tensor) and K_pages.dtype in _DTYPES, "K_pages must be a bf16 or fp16 tensor")
    dev = K_pages.device
    _tensor(K_pages, "K_pages", K_pages.dtype, (None,) * 4, dev, contiguous=False)
    _tensor(V_pages, "V_pages", K_pages.dtype, K_pages.shape, dev, contiguous=False)
    _need(all(n == 1 or a == b for n, a, b in zip(K_pages.shape, K_pages.stride(), V_pages.stride())),
          "K_pages and V_pages must have the same strides")  # (a dimension of one has none)
    _tensor(page_table, "page_table", torch.int32, (None, None), dev)
    c = tsa_paged_cache()
    c.K, c.V, c.page_table = K_pages.data_ptr(), V_pages.data_ptr(), page_table.data_ptr()
    c.page_stride, c.head_stride, c.row_stride = K_pages.stride()[:3]
    c.num_pages, c.Hkv, c.page_size, c.d = K_pages.shape
    c.B, c.max_pages = page_table.shape
    c.dtype = _DTYPES[K_pages.dtype]
    c._torch_dtype = K_pages.dtype
    return _hold(c, dev, K_pages, V_pages, page_table)


def paged_workspace_size(cache: tsa_paged_cache, Hq: int = 0, prefix_len: int = 0) -> int:
    _need(-2 ** 31 <= prefix_len < 2 ** 31, f"prefix_len={prefix_len} does not fit 32 bits")
    n = _lib.tsa_paged_workspace_size(ctypes.byref(cache), Hq, prefix_len)
    if n == 0:
        raise TsaError(TSA_ERR_INVALID_ARG, last_error())
    return int(n)


def new_paged_workspace(cache: tsa_paged_cache, Hq: int = 0, prefix_len: int = 0) -> torch.Tensor:
    """Allocate (with torch) and zero a workspace for paged_attn / prefix_attn with Hq query
    heads (Hq = 0: for paged_append), on the cache's device."""
    ws = torch.empty(paged_workspace_size(cache, Hq, prefix_len), dtype=torch.uint8, device=cache._device)
    with torch.cuda.device(cache._device):
        workspace_init(ws)
    return ws


def _rotation(inv_freq, interleaved: bool, device) -> tsa_rotation:
    r = tsa_rotation()
    if inv_freq is not None:
        _tensor(inv_freq, "inv_freq", torch.float64, (None,), device)
        r.inv_freq, r.rot_dim = inv_freq.data_ptr(), 2 * inv_freq.numel()
    r.interleaved = int(interleaved)
    return r


def qk_norm_rope_args(q, k, q_out, k_out, *, q_weight=None, k_weight=None, eps: float = 1e-6, positions=None,
                      inv_freq=None, interleaved: bool = False) -> tsa_qk_args:
    """Arguments of qk_norm_rope: q [T, Hq, 128], k [T, Hkv, 128] (either may be None) of any
    token and head strides, their outputs (which may be q and k), norm weights [128] fp32
    (None: no norm), positions [T] int32 and inv_freq [rot_dim / 2] float64 (None: no rotation)."""
    some = q if q is not None else k
    _need(isinstance(some, torch.Tensor) and some.dtype in _DTYPES and some.dim() == 3,
          "q or k must be a bf16 or fp16 tensor [T, heads, 128]")
    dev, T, d = some.device, some.shape[0], some.shape[2]
    a = tsa_qk_args()
    for x, out, w, n in ((q, q_out, q_weight, "q"), (k, k_out, k_weight, "k")):
        if x is None:
            _need(out is None and w is None, f"{n} is None, but {n}_out or {n}_weight is not")
            continue
        _tensor(x, n, some.dtype, (T, None, d), dev, contiguous=False)
        _tensor(out, n + "_out", some.dtype, x.shape, dev, contiguous=False)
        if w is not None:
            _tensor(w, n + "_weight", torch.float32, (d,), dev)
        setattr(a, n, x.data_ptr())
        setattr(a, n + "_out", out.data_ptr())
        setattr(a, n + "_weight", _ptr(w))
        for name, t in ((n, x), (n + "_out", out)):
            setattr(a, name + "_stride_t", t.stride(0))
            setattr(a, name + "_stride_h", t.stride(1))
    a.rot = _rotation(inv_freq, interleaved, dev)
    if positions is not None:
        _tensor(positions, "positions", torch.int32, (T,), dev)
        a.positions = positions.data_ptr()
    a.T, a.d, a.dtype, a.eps = T, d, _DTYPES[some.dtype], eps
    a.Hq, a.Hkv = 0 if q is None else q.shape[1], 0 if k is None else k.shape[1]
    return _hold(a, dev, q, k, q_out, k_out, q_weight, k_weight, positions, inv_freq)


def qk_norm_rope(args: tsa_qk_args, stream=None):
    """The norms of each query and key head, and their rotation, in one pass."""
    _launch(_lib.tsa_qk_norm_rope, args, stream)


def paged_append_args(cache: tsa_paged_cache, K, V, row, ws, *, seq=None, positions=None, inv_freq=None,
                      interleaved: bool = False) -> tsa_append_args:
    """Arguments of paged_append: K, V [T, Hkv, 128] of any token and head strides; row,
    seq (None: token t is sequence t's) and positions (None: row) are [T] int32."""
    dev = cache._device
    a = tsa_append_args()
    a.cache = cache
    _tensor(K, "K", cache._torch_dtype, (None, cache.Hkv, cache.d), dev, contiguous=False)
    _tensor(V, "V", cache._torch_dtype, K.shape, dev, contiguous=False)
    T = K.shape[0]
    for n, t in (("row", row), ("seq", seq), ("positions", positions)):
        if t is not None or n == "row":
            _tensor(t, n, torch.int32, (T,), dev)
            setattr(a, n, t.data_ptr())
    _tensor(ws, "ws", torch.uint8, (None,), dev)
    a.K, a.V, a.T = K.data_ptr(), V.data_ptr(), T
    a.k_stride_t, a.k_stride_h, a.v_stride_t, a.v_stride_h = K.stride(0), K.stride(1), V.stride(0), V.stride(1)
    a.rot = _rotation(inv_freq, interleaved, dev)
    a.ws, a.ws_bytes = _wsargs(ws)
    return _hold(a, dev, cache, K, V, row, ws, seq, positions, inv_freq)


def paged_append(args: tsa_append_args, stream=None):
    """New keys, rotated on the way, and values into the cache's pages."""
    _launch(_lib.tsa_paged_append, args, stream)


def paged_attn_args(cache: tsa_paged_cache, Q, seq_lens, O, ws, *, scale: float, idx=None, k_per_seq=None,
                    prefix_len: int = 0, lse=None) -> tsa_paged_attn_args:
    """Arguments of paged_attn and prefix_attn: Q, O [B, Hq, 128] in the cache's type, seq_lens
    [B] int32; idx [B, Hkv, k_max] int32 with k_per_seq [B] (paged_attn), or prefix_len
    (prefix_attn); lse [B, Hq] fp32 or None."""
    dev = cache._device
    a = tsa_paged_attn_args()
    a.cache = cache
    _tensor(Q, "Q", cache._torch_dtype, (cache.B, None, cache.d), dev)
    _tensor(O, "O", cache._torch_dtype, Q.shape, dev)
    _tensor(seq_lens, "seq_lens", torch.int32, (cache.B,), dev)
    if idx is not None:
        _tensor(idx, "idx", torch.int32, (cache.B, cache.Hkv, None), dev)
        a.idx, a.k_max = idx.data_ptr(), idx.shape[2]
    if k_per_seq is not None:
        _tensor(k_per_seq, "k_per_seq", torch.int32, (cache.B,), dev)
        a.k_per_seq = k_per_seq.data_ptr()
    if lse is not None:
        _tensor(lse, "lse", torch.float32, Q.shape[:2], dev)
        a.lse = lse.data_ptr()
    _need(-2 ** 31 <= prefix_len < 2 ** 31, f"prefix_len={prefix_len} does not fit 32 bits")  # (ctypes would cut it)
    _tensor(ws, "ws", torch.uint8, (None,), dev)
    a.Q, a.O, a.seq_lens = Q.data_ptr(), O.data_ptr(), seq_lens.data_ptr()
    a.Hq, a.prefix_len, a.scale = Q.shape[1], prefix_len, scale
    a.ws, a.ws_bytes = _wsargs(ws)
    return _hold(a, dev, cache, Q, seq_lens, O, ws, idx, k_per_seq, lse)


def paged_attn(args: tsa_paged_attn_args, stream=None):
    """One token per sequence over its pages: every row, or the rows of idx."""
    _launch(_lib.tsa_paged_attn, args, stream)


def prefix_attn(args: tsa_paged_attn_args, stream=None):
    """One token per sequence, the rows [0, prefix_len) that the batch shares read once for all.  Over a
    long enough prefix the softmax weights are rounded to the cache's type (include/tsa.h says from
    where on); paged_attn over the same tables keeps 16 bits of them or more."""
    _launch(_lib.tsa_prefix_attn, args, stream)
