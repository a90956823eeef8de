"""Gradient-synchronisation collectives on one MI355X: Python binding of libgc.

A thin ctypes layer over the C ABI declared in include/gc.h.  It only marshals
arguments: it turns lists of tensors (or raw device addresses) into pointer
arrays, maps dtype/op/order names onto the C enums, passes torch's current HIP
stream, and raises GcError for a non-OK status.  Since the library sees only
addresses, a tensor is checked here first (a contiguous device tensor that
holds every byte the call touches, else ValueError; the norm, the 8-bit rows,
the experts, the combine's gradient, the embedding, dropout and log
probabilities also check its type, where integer tensors count as raw bits);
raw addresses and gc_pointers arrays are the caller's responsibility.  Every
collective runs in the
HIP kernels of libgc.so; there is no other implementation to fall back to, and
importing this package fails if the library has not been built
(python collective_communication_reduction_amd/build.py).

The functions carry the C names:
  gc_all_reduce, gc_reduce_scatter, gc_all_gather, gc_all_to_all,
  gc_all_reduce_scratch_bytes, gc_bucket_plan_create / _query / _destroy,
  gc_bucket_pack, gc_bucket_unpack, gc_bucket_all_reduce, gc_status_string,
  gc_version, gc_last_hip_error; the MoE calls gc_moe_route, gc_moe_dispatch,
  gc_moe_combine and its gradient, gc_moe_ffn and its backward; gc_rms_norm and
  its backward; gc_mx8_pack, gc_mx8_unpack; gc_embedding and its backward,
  gc_dropout, gc_token_logprob and its backward
plus BucketPlan, a small owner of a gc_bucket_plan handle; RankArena, which
gives each rank its own region of HBM; gc_rank_buffers, which lays N rank
buffers out in one allocation with a per-rank stagger; and gc_pointers, which
marshals a pointer array once for buffers synchronised every step.
"""

import ctypes
import functools
import os

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libgc.so")

if not os.path.exists(LIB_PATH):
    raise ImportError(
        f"{LIB_PATH} is missing: build the HIP library first "
        "(python collective_communication_reduction_amd/build.py)")

# PyTorch ships its own HIP runtime, which its libraries request as
# "libamdhip64.so"; libgc requests "libamdhip64.so.7".  Importing torch first
# makes libgc bind to the runtime already in the process, so both sides share
# one runtime (and torch's streams and allocations are valid for libgc).
# Loading libgc first would pull in the system runtime as a second copy.
try:
    import torch  # noqa: F401
except ImportError:  # pragma: no cover - the library itself does not need torch
    torch = None

_lib = ctypes.CDLL(LIB_PATH)

GC_MAX_RANKS = 64
GC_OK, GC_ERR_INVALID_ARG, GC_ERR_UNSUPPORTED, GC_ERR_HIP, GC_ERR_NO_MEMORY = range(5)
GC_INT32, GC_FP32, GC_BF16, GC_MX8 = 0, 1, 2, 3
GC_SUM, GC_AVG = 0, 1
GC_ORDER_RING, GC_ORDER_RANK, GC_ORDER_RING_WIRE = 0, 1, 2
GC_AR_FUSED, GC_AR_RS_AG = 0, 1
SIZE_MAX = (1 << 64) - 1

_DTYPE = {"int32": GC_INT32, "fp32": GC_FP32, "bf16": GC_BF16, "mx8": GC_MX8}
_OP = {"sum": GC_SUM, "avg": GC_AVG}
_ORDER = {"ring": GC_ORDER_RING, "rank": GC_ORDER_RANK, "ring_wire": GC_ORDER_RING_WIRE}
_ALGO = {"fused": GC_AR_FUSED, "rs_ag": GC_AR_RS_AG}

_vp, _sz, _int = ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int
_VPP = ctypes.POINTER(ctypes.c_void_p)


def _sig(name, restype, *argtypes):
    f = getattr(_lib, name)
    f.restype = restype
    f.argtypes = list(argtypes)
    return f


_c_rs = _sig("gc_reduce_scatter", _int, _VPP, _VPP, _sz, _int, _int, _int, _int, _int, _vp)
_c_ag = _sig("gc_all_gather", _int, _VPP, _VPP, _sz, _int, _int, _vp)
_c_ar_scratch = _sig("gc_all_reduce_scratch_bytes", _sz, _sz, _int, _int, _int)
_c_ar = _sig("gc_all_reduce", _int, _VPP, _VPP, _sz, _int, _int, _int, _int, _int, _vp, _sz, _vp)
_c_a2a = _sig("gc_all_to_all", _int, _VPP, _VPP, ctypes.POINTER(ctypes.c_int64), _int, _int, _sz, _vp)
_I64P = ctypes.POINTER(ctypes.c_int64)
_SZP = ctypes.POINTER(ctypes.c_size_t)
_c_fsdp2_rs = _sig("gc_fsdp2_reduce_scatter", _int, _VPP, _VPP, _SZP, _SZP, _int, _int, _int, _int, _int, _int, _vp)
_c_hier_ar = _sig("gc_hier_all_reduce", _int, _VPP, _VPP, _sz, _int, _int, _int, _int, _int, _vp)
_c_hsdp_rs = _sig("gc_hsdp_reduce_scatter", _int, _VPP, _VPP, _sz, _int, _int, _int, _int, _int, _int, _vp)
_c_fsdp2_ag = _sig("gc_fsdp2_all_gather", _int, _VPP, _VPP, _SZP, _SZP, _int, _int, _int, _vp)
_c_moe_scratch = _sig("gc_moe_route_scratch_bytes", _sz, _I64P, _int, _int, _int)
_c_moe_route = _sig("gc_moe_route", _int, _VPP, _I64P, _int, _int, _int, _vp, _VPP, _vp, _sz, _vp)
_c_moe_route_noalloc = _sig("gc_moe_route_noalloc", _int, _VPP, _I64P, _int, _int, _int, _vp, _VPP, _vp)
_c_moe_dispatch = _sig("gc_moe_dispatch", _int, _VPP, _I64P, _VPP, _int, _int, _sz, _VPP, _I64P, _vp)
_c_moe_combine = _sig("gc_moe_combine", _int, _VPP, _I64P, _VPP, _VPP, _I64P, _int, _int, _sz, _int, _VPP, _vp)
_c_plan_create = _sig("gc_bucket_plan_create", _int, ctypes.POINTER(ctypes.c_size_t), _int, _int, _sz, _int, _sz,
                      ctypes.POINTER(_vp))
_c_plan_query = _sig("gc_bucket_plan_query", _int, _vp, ctypes.POINTER(_int), ctypes.POINTER(ctypes.c_size_t),
                     ctypes.POINTER(_int), ctypes.POINTER(ctypes.c_size_t))
_c_pack = _sig("gc_bucket_pack", _int, _vp, _int, _VPP, _VPP, _int, _vp)
_c_unpack = _sig("gc_bucket_unpack", _int, _vp, _int, _VPP, _VPP, _int, _vp)
_c_bucket_ar = _sig("gc_bucket_all_reduce", _int, _vp, _int, _VPP, _int, _int, _int, _vp, _vp)
_c_moe_combine_bwd = _sig("gc_moe_combine_backward", _int, _VPP, _VPP, _I64P, _VPP, _VPP, _I64P, _int, _int, _sz, _int,
                          _VPP, _VPP, _vp)
_c_mx8_row = _sig("gc_mx8_row_bytes", _sz, _sz)
_c_mx8_pack = _sig("gc_mx8_pack", _int, _VPP, _I64P, _int, _sz, _int, _VPP, _vp)
_c_mx8_unpack = _sig("gc_mx8_unpack", _int, _VPP, _I64P, _int, _sz, _int, _VPP, _vp)
_c_norm = _sig("gc_rms_norm", _int, _VPP, _VPP, _VPP, _I64P, _int, _sz, ctypes.c_float, _int, _VPP, _VPP, _int, _VPP, _vp)
_c_norm_bwd_scratch = _sig("gc_rms_norm_backward_scratch_bytes", _sz, _I64P, _int, _sz)
_c_norm_bwd = _sig("gc_rms_norm_backward", _int, _VPP, _VPP, _VPP, _VPP, _VPP, _I64P, _int, _sz, _int, _VPP, _VPP, _vp,
                   _sz, _vp)
_c_ffn_scratch = _sig("gc_moe_ffn_scratch_bytes", _sz, _I64P, _int, _int, _sz, _sz, _int, _int)
_c_ffn = _sig("gc_moe_ffn", _int, _VPP, _int, _I64P, _vp, _int, _int, _sz, _sz, _VPP, _VPP, _VPP, _VPP, _int, _VPP, _vp,
              _sz, _vp)
_c_ffn_bwd = _sig("gc_moe_ffn_backward", _int, _VPP, _VPP, _int, _VPP, _int, _I64P, _vp, _int, _int, _sz, _sz, _VPP, _VPP,
                  _VPP, _VPP, _VPP, _VPP, _VPP, _int, _vp, _sz, _vp)
_u64, _f32 = ctypes.c_uint64, ctypes.c_float
_c_embed = _sig("gc_embedding", _int, _VPP, _VPP, _I64P, _int, _sz, _sz, _f32, _int, _VPP, _vp)
_c_embed_bwd_scratch = _sig("gc_embedding_backward_scratch_bytes", _sz, _I64P, _int, _sz, _sz)
_c_embed_bwd = _sig("gc_embedding_backward", _int, _VPP, _VPP, _I64P, _int, _sz, _sz, _f32, _int, _VPP, _int, _int, _vp,
                    _sz, _vp)
_c_dropout = _sig("gc_dropout", _int, _VPP, _VPP, _I64P, _int, _f32, _u64, _u64, _vp, _int, _VPP, _vp)
_c_logprob_scratch = _sig("gc_token_logprob_scratch_bytes", _sz, _I64P, _int, _sz, _int)
_c_logprob = _sig("gc_token_logprob", _int, _VPP, _VPP, _I64P, _int, _sz, _sz, _f32, _int, _VPP, _VPP, _VPP, _int, _VPP,
                  _VPP, _VPP, _VPP, _VPP, _vp, _sz, _vp)
_c_logprob_bwd = _sig("gc_token_logprob_backward", _int, _VPP, _VPP, _VPP, _VPP, _VPP, _VPP, _I64P, _int, _sz, _sz, _f32,
                      _int, _VPP, _vp)
_c_plan_destroy = _sig("gc_bucket_plan_destroy", None, _vp)
_c_status = _sig("gc_status_string", ctypes.c_char_p, _int)
_c_version = _sig("gc_version", _int)
_c_last_hip = _sig("gc_last_hip_error", _int)


class GcError(RuntimeError):
    def __init__(self, status, what):
        self.status = status
        detail = f" (hipError_t {gc_last_hip_error()})" if status == GC_ERR_HIP else ""
        super().__init__(f"{what}: {gc_status_string(status)}{detail}")


def gc_last_hip_error():
    """hipError_t of the last HIP call that failed inside libgc on this thread (0 if none)."""
    return _c_last_hip()


def gc_status_string(status):
    return _c_status(int(status)).decode()


def gc_version():
    return _c_version()


def _check(status, what):
    if status != GC_OK:
        raise GcError(status, what)


# ------------------------------------------------------------------ marshalling

_ES = {GC_INT32: 4, GC_FP32: 4, GC_BF16: 2}


# Tensors that hold values of a type (a code, or int64): its own, or integers as raw bits.  A stand-in
# without a dtype (None) passes.
_RAW = () if torch is None else (torch.uint8, torch.int8, None)
_HOLDS = {} if torch is None else {
    GC_BF16: frozenset((torch.bfloat16, torch.int16, torch.uint16) + _RAW),
    GC_FP32: frozenset((torch.float32, torch.int32, torch.uint32) + _RAW),
    GC_INT32: frozenset((torch.int32, torch.uint32) + _RAW), GC_MX8: frozenset(_RAW),
    "int64": frozenset((torch.int64, torch.uint64) + _RAW)}


def _buf(x, nbytes, what, holds=None):
    """Address of one device buffer that a call reads or writes for nbytes bytes.

    A tensor must be a contiguous device tensor of at least nbytes bytes: the C
    ABI sees only its address, so a host, strided or short tensor would reach the
    kernels as an out-of-bounds access.  A raw integer address (or None) is the
    caller's responsibility and passes unchecked."""
    if x is None or isinstance(x, int):
        return x
    if not x.is_cuda:
        raise ValueError(f"{what}: a device (cuda) tensor is required")
    if not x.is_contiguous():
        raise ValueError(f"{what}: the tensor is not contiguous")
    have = x.numel() * x.element_size()
    if have < nbytes:
        raise ValueError(f"{what}: {have} bytes, the call touches {nbytes}")
    if holds is not None and nbytes and getattr(x, "dtype", None) not in holds:
        names = ", ".join(sorted(str(t).replace("torch.", "") for t in holds if t is not None))
        raise ValueError(f"{what}: a tensor of {x.dtype}, where the call takes one of {names}")
    return x.data_ptr()


def _bufs(xs, n, nbytes, what, t=None):
    """Pointer array of the first n buffers of xs, each checked by _buf.

    nbytes is one size for every buffer or a sequence with one size per buffer.
    A pointer array made by gc_pointers passes unchecked but must hold n
    entries; None passes as NULL (the library rejects it).  t: the type of the
    values, where the tensors' types are checked too."""
    if xs is None:
        return None
    m = len(xs)
    if m < n:
        raise ValueError(f"{what}: {m} buffers, the call needs {n}")
    if isinstance(xs, ctypes.Array):
        return xs
    arr = _ptr_array(m)()
    need = [nbytes] * n if isinstance(nbytes, int) else nbytes
    holds = _HOLDS.get(t)
    if m > n:
        need = [*need[:n], *[0] * (m - n)]
    try:
        # the checks of _buf in line: this loop is most of a short call's time on the host
        for i, x in enumerate(xs):
            if x is None or type(x) is int:
                arr[i] = x
            elif x.is_cuda and x.is_contiguous() and x.nbytes >= need[i] and (holds is None or x.dtype in holds):
                arr[i] = x.data_ptr()
            else:
                arr[i] = _buf(x, need[i], f"{what}[{i}]", holds)
    except AttributeError:      # addresses of another integer type, tensors of another library
        for i, x in enumerate(xs):
            arr[i] = _buf(x, need[i], f"{what}[{i}]", holds)
    return arr


@functools.lru_cache(maxsize=None)
def _ptr_array(n):
    return ctypes.c_void_p * max(1, n)


@functools.lru_cache(maxsize=None)
def _int64_array(n):
    return ctypes.c_int64 * max(1, n)


_TORCH_DTYPE = {}


def _dtype_code(x):
    if isinstance(x, str):
        return _DTYPE[x]
    if isinstance(x, int):
        return x
    if not _TORCH_DTYPE:
        import torch
        _TORCH_DTYPE.update({torch.bfloat16: GC_BF16, torch.float32: GC_FP32, torch.int32: GC_INT32, torch.uint8: GC_MX8})
    return _TORCH_DTYPE[x]


def _enum(table, x):
    return table[x] if isinstance(x, str) else int(x)


def gc_pointers(tensors):
    """Marshal a list of tensors (or addresses, or None) into a pointer array once.

    Every call that takes a list also accepts the returned array, which saves
    rebuilding it when the same buffers are synchronised every step (DDP's
    gradient tensors persist across steps).  Tensors must be contiguous device
    tensors; their sizes are not known here, so the calls that take the array
    trust it."""
    xs = list(tensors)
    return _bufs(xs, len(xs), 0, "gc_pointers")


# The current stream's handle without building a Stream object (2 us of a call).
_raw_stream = getattr(getattr(torch, "_C", None), "_cuda_getCurrentRawStream", None)


def _stream(stream, like=None):
    """HIP stream handle: an explicit int / torch stream, else torch's current stream on like's device."""
    if stream is None:
        dev = like.device if hasattr(like, "device") and like.device.type == "cuda" else None
        if dev is None:
            return torch.cuda.current_stream().cuda_stream if torch.cuda.is_available() else None
        if _raw_stream is not None and dev.index is not None:
            return _raw_stream(dev.index)
        return torch.cuda.current_stream(dev).cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _first(xs):
    """First tensor-like element (its device picks the stream), or None."""
    if xs is None or isinstance(xs, ctypes.Array):
        return None
    for x in xs:
        if x is not None and not isinstance(x, int):
            return x
    return None


def _numel(xs, count):
    if count is not None:
        return int(count)
    return int(xs[0].numel())


def _infer_dtype(xs, dtype):
    if dtype is not None:
        return _dtype_code(dtype)
    return _dtype_code(xs[0].dtype)


# ------------------------------------------------------------------ collectives

def gc_all_reduce(send, recv=None, op="avg", order="ring", algo="fused", scratch=None, scratch_bytes=None,
                  count=None, dtype=None, stream=None):
    """All-reduce N rank buffers; recv defaults to send (in place).  See include/gc.h."""
    recv = send if recv is None else recv
    n = len(send)
    t = _infer_dtype(send, dtype)
    cnt = _numel(send, count)
    a = _enum(_ALGO, algo)
    if scratch_bytes is None:
        scratch_bytes = scratch.numel() * scratch.element_size() if hasattr(scratch, "numel") else 0
    nb = cnt * _ES.get(t, 0)
    _check(_c_ar(_bufs(send, n, nb, "send"), _bufs(recv, n, nb, "recv"), cnt, n, t, _enum(_OP, op),
                 _enum(_ORDER, order), a, _buf(scratch, int(scratch_bytes), "scratch"), int(scratch_bytes),
                 _stream(stream, _first(send))), "gc_all_reduce")
    return recv


def gc_all_reduce_scratch_bytes(count, nranks, dtype, algo="rs_ag"):
    return int(_c_ar_scratch(int(count), int(nranks), _dtype_code(dtype), _enum(_ALGO, algo)))


def gc_reduce_scatter(send, recv, op="avg", order="ring", recv_count=None, in_dtype=None, out_dtype=None,
                      stream=None):
    """Reduce-scatter: recv[j] = op_i send[i][j*recv_count : (j+1)*recv_count]."""
    n = len(send)
    ti = _infer_dtype(send, in_dtype)
    to = _infer_dtype(recv, out_dtype)
    rc = _numel(recv, recv_count)
    _check(_c_rs(_bufs(send, n, n * rc * _ES.get(ti, 0), "send"), _bufs(recv, n, rc * _ES.get(to, 0), "recv"), rc,
                 n, ti, to, _enum(_OP, op), _enum(_ORDER, order), _stream(stream, _first(send))),
           "gc_reduce_scatter")
    return recv


def gc_all_gather(send, recv, count=None, dtype=None, stream=None):
    """All-gather: recv[d][i*count : (i+1)*count] = send[i] for every d."""
    n = len(send)
    t = _infer_dtype(send, dtype)
    cnt = _numel(send, count)
    nb = cnt * _ES.get(t, 0)
    _check(_c_ag(_bufs(send, n, nb, "send"), _bufs(recv, n, n * nb, "recv"), cnt, n, t,
                 _stream(stream, _first(send))), "gc_all_gather")
    return recv


def gc_all_to_all(send, recv, splits, row_bytes, stream=None):
    """All-to-all(v) with experts: splits is an int64 array-like [N][N][E] of rows."""
    import numpy as np
    sp = np.ascontiguousarray(np.asarray(splits, dtype=np.int64))
    if sp.ndim != 3:
        raise ValueError("splits must be [N][N][E]")
    n, _, e = sp.shape
    rb = int(row_bytes)
    rows_out = [max(0, int(x)) * rb for x in sp.clip(min=0).sum(axis=(1, 2))] if n else []
    rows_in = [max(0, int(x)) * rb for x in sp.clip(min=0).sum(axis=(0, 2))] if n else []
    _check(_c_a2a(_bufs(send, n, rows_out, "send"), _bufs(recv, n, rows_in, "recv"),
                  sp.ctypes.data_as(ctypes.POINTER(ctypes.c_int64)), n, e, rb, _stream(stream, _first(send))),
           "gc_all_to_all")
    return recv


def gc_hier_all_reduce(send, recv, group_size, op="avg", order="ring", count=None, dtype=None, stream=None):
    """Two-level all-reduce over len(send) = R * group_size ranks (member i of group g = rank g*group_size + i)."""
    n = len(send)
    t = _infer_dtype(send, dtype)
    cnt = _numel(send, count)
    nb = cnt * _ES.get(t, 0)
    _check(_c_hier_ar(_bufs(send, n, nb, "send"), _bufs(recv, n, nb, "recv"), cnt, n, int(group_size), t,
                      _enum(_OP, op), _enum(_ORDER, order), _stream(stream, _first(send))), "gc_hier_all_reduce")
    return recv


def gc_hsdp_reduce_scatter(send, recv, group_size, op="avg", order="ring", recv_count=None, in_dtype=None,
                           out_dtype=None, stream=None):
    """HSDP gradient reduce-scatter: recv[r] = chunk (r mod group_size) of the reduction over all ranks."""
    n = len(send)
    rc = int(recv_count) if recv_count is not None else int(recv[0].numel())
    tin = _infer_dtype(send, in_dtype)
    tout = _infer_dtype(recv, out_dtype)
    g = max(0, int(group_size))
    _check(_c_hsdp_rs(_bufs(send, n, g * rc * _ES.get(tin, 0), "send"), _bufs(recv, n, rc * _ES.get(tout, 0), "recv"),
                      rc, n, int(group_size), tin, tout, _enum(_OP, op), _enum(_ORDER, order),
                      _stream(stream, _first(send))), "gc_hsdp_reduce_scatter")
    return recv


def _sz_array(xs):
    xs = [int(x) for x in xs]
    return (ctypes.c_size_t * max(1, len(xs)))(*xs)


def _rank_major(xs, nranks, nparams):
    """Accept [rank][param] nested lists or a flat rank-major list (returned flat), or a marshalled array."""
    if isinstance(xs, ctypes.Array):
        return xs
    if len(xs) == nranks and nparams and isinstance(xs[0], (list, tuple)):
        xs = [x for row in xs for x in row]
    if len(xs) != nranks * nparams:
        raise ValueError("need nranks * nparams pointers")
    return xs


def _shard_bytes(rows, cols, nranks, es):
    """Bytes of every (rank, parameter) dim-0 shard, rank-major (torch.chunk's rule)."""
    out = []
    for r in range(nranks):
        for nr, nc in zip(rows, cols):
            c = -(-int(nr) // nranks)
            out.append((min(int(nr), (r + 1) * c) - min(int(nr), r * c)) * int(nc) * es)
    return out


def gc_fsdp2_reduce_scatter(grads, shards, rows, cols, nranks, in_dtype, out_dtype=None, op="avg", order="ring",
                            stream=None):
    """Per-parameter Shard(0) reduce-scatter; grads / shards as [rank][param] (or flat rank-major)."""
    P, N = len(rows), int(nranks)
    out_dtype = in_dtype if out_dtype is None else out_dtype
    ti, to = _dtype_code(in_dtype), _dtype_code(out_dtype)
    g = _rank_major(grads, N, P)
    sh = _rank_major(shards, N, P)
    full = [int(nr) * int(nc) * _ES.get(ti, 0) for nr, nc in zip(rows, cols)] * max(N, 0)
    part = _shard_bytes(rows, cols, N, _ES.get(to, 0)) if N > 0 else []
    like = None if isinstance(g, ctypes.Array) else _first(g)
    _check(_c_fsdp2_rs(_bufs(g, N * P, full, "grads"), _bufs(sh, N * P, part, "shards"), _sz_array(rows),
                       _sz_array(cols), P, N, ti, to, _enum(_OP, op), _enum(_ORDER, order), _stream(stream, like)),
           "gc_fsdp2_reduce_scatter")
    return shards


def gc_fsdp2_all_gather(shards, params, rows, cols, nranks, dtype, stream=None):
    """Per-parameter Shard(0) all-gather; shards / params as [rank][param] (or flat rank-major)."""
    P, N = len(rows), int(nranks)
    t = _dtype_code(dtype)
    sh = _rank_major(shards, N, P)
    pa = _rank_major(params, N, P)
    full = [int(nr) * int(nc) * _ES.get(t, 0) for nr, nc in zip(rows, cols)] * max(N, 0)
    part = _shard_bytes(rows, cols, N, _ES.get(t, 0)) if N > 0 else []
    like = None if isinstance(pa, ctypes.Array) else _first(pa)
    _check(_c_fsdp2_ag(_bufs(sh, N * P, part, "shards"), _bufs(pa, N * P, full, "params"), _sz_array(rows),
                       _sz_array(cols), P, N, t, _stream(stream, like)), "gc_fsdp2_all_gather")
    return params


def _i64_array(xs):
    xs = [int(x) for x in xs]
    return _int64_array(len(xs))(*xs)


def gc_moe_route_scratch_bytes(ntokens, topk, experts_per_rank):
    """Scratch bytes gc_moe_route needs for these per-source token counts (0 if the sizes are invalid)."""
    return int(_c_moe_scratch(_i64_array(ntokens), len(ntokens), int(topk), int(experts_per_rank)))


def _per_route(ntokens, topk, nbytes):
    return [max(0, int(t)) * max(0, int(topk)) * nbytes for t in ntokens]


def gc_moe_route(experts, ntokens, topk, experts_per_rank, splits, dest, scratch, scratch_bytes=None, stream=None):
    """MoE routing plan on the device.  experts[s]: int32 [ntokens[s] * topk] global expert ids;
    splits: int64 [N*N*E] out; dest[s]: int32 [ntokens[s] * topk * 2] (rank, row) out."""
    n = len(ntokens)
    if scratch_bytes is None:
        scratch_bytes = scratch.numel() * scratch.element_size()
    nsplit = n * n * max(0, int(experts_per_rank)) * 8
    _check(_c_moe_route(_bufs(experts, n, _per_route(ntokens, topk, 4), "experts"), _i64_array(ntokens), n,
                        int(topk), int(experts_per_rank), _buf(splits, nsplit, "splits"),
                        _bufs(dest, n, _per_route(ntokens, topk, 8), "dest"),
                        _buf(scratch, int(scratch_bytes), "scratch"), int(scratch_bytes), _stream(stream, splits)),
           "gc_moe_route")
    return splits, dest


GC_MOE_ROUTE_NOALLOC_SCRATCH_BYTES = 4 << 20


def gc_moe_route_noalloc(experts, ntokens, topk, experts_per_rank, splits, dest, stream=None):
    """gc_moe_route without a scratch argument, for callers that cannot allocate device
    memory: the plan uses the library's static per-GPU scratch (at most
    GC_MOE_ROUTE_NOALLOC_SCRATCH_BYTES; larger plans raise GcError with GC_ERR_UNSUPPORTED).
    Calls that overlap on one GPU share that scratch and race."""
    n = len(ntokens)
    nsplit = n * n * max(0, int(experts_per_rank)) * 8
    st = _c_moe_route_noalloc(_bufs(experts, n, _per_route(ntokens, topk, 4), "experts"), _i64_array(ntokens), n,
                              int(topk), int(experts_per_rank), _buf(splits, nsplit, "splits"),
                              _bufs(dest, n, _per_route(ntokens, topk, 8), "dest"), _stream(stream, splits))
    if st == GC_ERR_UNSUPPORTED:
        need = gc_moe_route_scratch_bytes(ntokens, topk, experts_per_rank)
        if need > GC_MOE_ROUTE_NOALLOC_SCRATCH_BYTES:
            raise GcError(st, f"gc_moe_route_noalloc (the plan needs {need} bytes of scratch, the static scratch "
                              f"holds {GC_MOE_ROUTE_NOALLOC_SCRATCH_BYTES}; use gc_moe_route with a scratch buffer)")
    _check(st, "gc_moe_route_noalloc")
    return splits, dest


def gc_moe_dispatch(tokens, ntokens, dest, topk, row_bytes, recv, recv_rows, stream=None):
    """Copy every token row of every source to the receive rows its routes name."""
    n, rb = len(ntokens), int(row_bytes)
    _check(_c_moe_dispatch(_bufs(tokens, n, [max(0, int(t)) * rb for t in ntokens], "tokens"), _i64_array(ntokens),
                           _bufs(dest, n, _per_route(ntokens, topk, 8), "dest"), n, int(topk), rb,
                           _bufs(recv, n, [max(0, int(r)) * rb for r in recv_rows], "recv"), _i64_array(recv_rows),
                           _stream(stream, _first(recv))), "gc_moe_dispatch")
    return recv


def gc_moe_combine(expert_out, expert_rows, dest, weights, ntokens, topk, hidden, dtype, out, stream=None):
    """out[s][t] = sum_k weights[s][t*topk + k] * expert_out[rank][row] over the routes of token t."""
    n, t = len(ntokens), _dtype_code(dtype)
    rb = max(0, int(hidden)) * _ES.get(t, 0)
    _check(_c_moe_combine(_bufs(expert_out, n, [max(0, int(r)) * rb for r in expert_rows], "expert_out"),
                          _i64_array(expert_rows), _bufs(dest, n, _per_route(ntokens, topk, 8), "dest"),
                          _bufs(weights, n, _per_route(ntokens, topk, 4), "weights"), _i64_array(ntokens), n,
                          int(topk), int(hidden), t, _bufs(out, n, [max(0, int(x)) * rb for x in ntokens], "out"),
                          _stream(stream, _first(out))), "gc_moe_combine")
    return out


def gc_moe_combine_backward(dout, expert_out, expert_rows, dest, weights, ntokens, topk, hidden, dtype, dexpert, dweights,
                            stream=None):
    """Gradient of gc_moe_combine: dexpert rows = weights * dout, dweights = the rows' dot products (fp32)."""
    n, t = len(ntokens), _dtype_code(dtype)
    rb = max(0, int(hidden)) * _ES.get(t, 0)
    rows = [max(0, int(r)) * rb for r in expert_rows]
    _check(_c_moe_combine_bwd(_bufs(dout, n, [max(0, int(x)) * rb for x in ntokens], "dout", t),
                              _bufs(expert_out, n, rows, "expert_out", t), _i64_array(expert_rows),
                              _bufs(dest, n, _per_route(ntokens, topk, 8), "dest", GC_INT32),
                              _bufs(weights, n, _per_route(ntokens, topk, 4), "weights", GC_FP32), _i64_array(ntokens), n,
                              int(topk), int(hidden), t, _bufs(dexpert, n, rows, "dexpert", t),
                              _bufs(dweights, n, _per_route(ntokens, topk, 4), "dweights", GC_FP32),
                              _stream(stream, _first(dexpert))), "gc_moe_combine_backward")
    return dexpert, dweights


# ------------------------------------------------------------------ 8-bit rows and norm

def gc_mx8_row_bytes(n):
    """Bytes of an 8-bit row of n values: e4m3 codes, a scale byte per 32 values, zeros to a multiple of 16."""
    return int(_c_mx8_row(max(0, int(n))))


def _row_bytes(n, t):
    return gc_mx8_row_bytes(n) if t == GC_MX8 else max(0, int(n)) * _ES.get(t, 0)


def _rows_of(counts, row):
    return [max(0, int(c)) * row for c in counts]


def gc_mx8_pack(x, rows, n, packed, dtype=None, stream=None):
    """x[r]: rows[r] rows of n bf16 or fp32 values -> packed[r]: as many 8-bit rows (uint8)."""
    N, t = len(rows), _infer_dtype(x, dtype)
    _check(_c_mx8_pack(_bufs(x, N, _rows_of(rows, _row_bytes(n, t)), "x", t), _i64_array(rows), N, int(n), t,
                       _bufs(packed, N, _rows_of(rows, _row_bytes(n, GC_MX8)), "packed", GC_MX8),
                       _stream(stream, _first(packed))), "gc_mx8_pack")
    return packed


def gc_mx8_unpack(packed, rows, n, out, dtype=None, stream=None):
    """Inverse of gc_mx8_pack: the values that 8-bit rows stand for, exact in bf16 and fp32."""
    N, t = len(rows), _infer_dtype(out, dtype)
    _check(_c_mx8_unpack(_bufs(packed, N, _rows_of(rows, _row_bytes(n, GC_MX8)), "packed", GC_MX8), _i64_array(rows), N,
                         int(n), t, _bufs(out, N, _rows_of(rows, _row_bytes(n, t)), "out", t),
                         _stream(stream, _first(out))), "gc_mx8_unpack")
    return out


def gc_rms_norm(x, weight, ntokens, hidden, y, residual=None, sum_out=None, rstd=None, eps=1e-6, dtype=None,
                y_dtype=None, stream=None):
    """s = x + residual; y = s / sqrt(mean(s^2) + eps) * weight, per row.  y: rows of x's type, or uint8 buffers
    for 8-bit rows.  sum_out (may be x or residual) takes s, rstd [ntokens] fp32 what the backward needs."""
    N, t = len(ntokens), _infer_dtype(x, dtype)
    yt = _infer_dtype(y, y_dtype)
    full = _rows_of(ntokens, _row_bytes(hidden, t))
    one = [_row_bytes(hidden, t) if int(c) > 0 else 0 for c in ntokens]
    _check(_c_norm(_bufs(x, N, full, "x", t), _bufs(residual, N, full, "residual", t), _bufs(weight, N, one, "weight", t),
                   _i64_array(ntokens), N, int(hidden), float(eps), t, _bufs(sum_out, N, full, "sum_out", t),
                   _bufs(y, N, _rows_of(ntokens, _row_bytes(hidden, yt)), "y", yt), yt,
                   _bufs(rstd, N, _rows_of(ntokens, 4), "rstd", GC_FP32), _stream(stream, _first(y))), "gc_rms_norm")
    return y


def gc_rms_norm_backward_scratch_bytes(ntokens, hidden):
    """Scratch bytes gc_rms_norm_backward needs (0 if the sizes are invalid)."""
    return int(_c_norm_bwd_scratch(_i64_array(ntokens), len(ntokens), max(0, int(hidden))))


def gc_rms_norm_backward(dy, sum, weight, rstd, ntokens, hidden, dx, dweight, scratch, dsum=None, scratch_bytes=None,
                         dtype=None, stream=None):
    """dx (of x and residual alike; may be dy or dsum) and dweight[r] (fp32 [hidden], one per rank) from dy and,
    optionally, dsum, the gradient arriving at the forward's sum_out."""
    N, t = len(ntokens), _infer_dtype(dy, dtype)
    if scratch_bytes is None:
        scratch_bytes = scratch.numel() * scratch.element_size()
    full = _rows_of(ntokens, _row_bytes(hidden, t))
    one = [_row_bytes(hidden, t) if int(c) > 0 else 0 for c in ntokens]
    _check(_c_norm_bwd(_bufs(dy, N, full, "dy", t), _bufs(dsum, N, full, "dsum", t), _bufs(sum, N, full, "sum", t),
                       _bufs(weight, N, one, "weight", t), _bufs(rstd, N, _rows_of(ntokens, 4), "rstd", GC_FP32),
                       _i64_array(ntokens), N, int(hidden), t, _bufs(dx, N, full, "dx", t),
                       _bufs(dweight, N, max(0, int(hidden)) * 4, "dweight", GC_FP32),
                       _buf(scratch, int(scratch_bytes), "scratch"), int(scratch_bytes), _stream(stream, _first(dx))),
           "gc_rms_norm_backward")
    return dx, dweight


# ------------------------------------------------------------------ experts

def gc_moe_ffn_scratch_bytes(rows, experts_per_rank, hidden, inter, x_dtype="bf16", backward=False):
    """Scratch bytes gc_moe_ffn (or gc_moe_ffn_backward) needs for these row counts (0 if the sizes are invalid)."""
    return int(_c_ffn_scratch(_i64_array(rows), len(rows), int(experts_per_rank), max(0, int(hidden)),
                              max(0, int(inter)), _dtype_code(x_dtype), int(bool(backward))))


def _ffn_common(rows, splits, experts_per_rank, hidden, inter, w_gate, w_up, w_down, scratch, scratch_bytes):
    N, E = len(rows), max(0, int(experts_per_rank))
    w = E * max(0, int(hidden)) * max(0, int(inter))
    if scratch_bytes is None:
        scratch_bytes = scratch.numel() * scratch.element_size()
    return (N, w, _buf(splits, N * N * E * 8, "splits", _HOLDS.get("int64")),
            [_bufs(p, N, 2 * w, k, GC_BF16) for p, k in ((w_gate, "w_gate"), (w_up, "w_up"), (w_down, "w_down"))],
            _buf(scratch, int(scratch_bytes), "scratch"), int(scratch_bytes))


def gc_moe_ffn(x, rows, splits, experts_per_rank, hidden, inter, w_gate, w_up, w_down, y, scratch, saved=None,
               x_dtype=None, saved_dtype=None, scratch_bytes=None, stream=None):
    """The experts' gated feed-forward on the receive layout: y = (silu(x Wg^T) * (x Wu^T)) Wd^T per expert block.
    x[d], y[d]: rows[d] rows of hidden (x: bf16, or uint8 8-bit rows); splits: the device table of gc_moe_route;
    w_gate[d], w_up[d] [E][inter][hidden] and w_down[d] [E][hidden][inter] bf16; saved[d]: rows of 2 * inter values
    (gate then up, bf16 or 8-bit rows) for the backward, or None."""
    N, _w, sp, ws, sc, scb = _ffn_common(rows, splits, experts_per_rank, hidden, inter, w_gate, w_up, w_down, scratch,
                                         scratch_bytes)
    xt = _infer_dtype(x, x_dtype)
    st = GC_BF16 if saved is None else _infer_dtype(saved, saved_dtype)
    _check(_c_ffn(_bufs(x, N, _rows_of(rows, _row_bytes(hidden, xt)), "x", xt), xt, _i64_array(rows), sp, N,
                  int(experts_per_rank), int(hidden), int(inter), *ws,
                  _bufs(saved, N, _rows_of(rows, _row_bytes(2 * int(inter), st)), "saved", st), st,
                  _bufs(y, N, _rows_of(rows, 2 * max(0, int(hidden))), "y", GC_BF16), sc, scb, _stream(stream, _first(y))),
           "gc_moe_ffn")
    return y


def gc_moe_ffn_backward(dy, x, saved, rows, splits, experts_per_rank, hidden, inter, w_gate, w_up, w_down, dx, dw_gate,
                        dw_up, dw_down, scratch, x_dtype=None, saved_dtype=None, dw_dtype=None, scratch_bytes=None,
                        stream=None):
    """Backward of gc_moe_ffn from its checkpoints: dx rows and the three weight gradients (bf16 or fp32)."""
    N, w, sp, ws, sc, scb = _ffn_common(rows, splits, experts_per_rank, hidden, inter, w_gate, w_up, w_down, scratch,
                                        scratch_bytes)
    xt, st, wt = _infer_dtype(x, x_dtype), _infer_dtype(saved, saved_dtype), _infer_dtype(dw_gate, dw_dtype)
    row = _rows_of(rows, 2 * max(0, int(hidden)))
    dws = [_bufs(p, N, w * _ES.get(wt, 0), k, wt) for p, k in ((dw_gate, "dw_gate"), (dw_up, "dw_up"), (dw_down, "dw_down"))]
    _check(_c_ffn_bwd(_bufs(dy, N, row, "dy", GC_BF16), _bufs(x, N, _rows_of(rows, _row_bytes(hidden, xt)), "x", xt), xt,
                      _bufs(saved, N, _rows_of(rows, _row_bytes(2 * int(inter), st)), "saved", st), st, _i64_array(rows), sp,
                      N, int(experts_per_rank), int(hidden), int(inter), *ws, _bufs(dx, N, row, "dx", GC_BF16), *dws, wt, sc, scb,
                      _stream(stream, _first(dx))), "gc_moe_ffn_backward")
    return dx, dw_gate, dw_up, dw_down


# ------------------------------------------------------------------ the two ends of a training step

def gc_embedding(weight, tokens, ntokens, vocab, hidden, out, scale=1.0, dtype=None, stream=None):
    """out[r][t] = scale * weight[r][tokens[r][t]], per rank; a token outside [0, vocab) gives a zero row.
    tokens[r]: int32 [ntokens[r]]; weight[r]: [vocab][hidden] bf16 or fp32; out[r]: [ntokens[r]][hidden]."""
    N, t = len(ntokens), _infer_dtype(weight, dtype)
    row = _row_bytes(hidden, t)
    full = [max(0, int(vocab)) * row if int(c) > 0 else 0 for c in ntokens]
    _check(_c_embed(_bufs(weight, N, full, "weight", t), _bufs(tokens, N, _rows_of(ntokens, 4), "tokens", GC_INT32),
                    _i64_array(ntokens), N, max(0, int(vocab)), max(0, int(hidden)), float(scale), t,
                    _bufs(out, N, _rows_of(ntokens, row), "out", t), _stream(stream, _first(out))), "gc_embedding")
    return out


def gc_embedding_backward_scratch_bytes(ntokens, vocab, hidden):
    """Scratch bytes gc_embedding_backward needs (0 if the sizes are invalid)."""
    return int(_c_embed_bwd_scratch(_i64_array(ntokens), len(ntokens), max(0, int(vocab)), max(0, int(hidden))))


def gc_embedding_backward(dout, tokens, ntokens, vocab, hidden, dweight, scratch, scale=1.0, accumulate=False,
                          scratch_bytes=None, dtype=None, dw_dtype=None, stream=None):
    """dweight[r][v] = scale * (sum of dout[r][t] over the tokens t equal to v), zeros for other rows; with accumulate
    the sums are added to dweight, whose other rows stay.  dout and dweight: bf16 or fp32 each."""
    N, t, wt = len(ntokens), _infer_dtype(dout, dtype), _infer_dtype(dweight, dw_dtype)
    if scratch_bytes is None:
        scratch_bytes = scratch.numel() * scratch.element_size()
    _check(_c_embed_bwd(_bufs(dout, N, _rows_of(ntokens, _row_bytes(hidden, t)), "dout", t),
                        _bufs(tokens, N, _rows_of(ntokens, 4), "tokens", GC_INT32), _i64_array(ntokens), N,
                        max(0, int(vocab)), max(0, int(hidden)), float(scale), t,
                        _bufs(dweight, N, max(0, int(vocab)) * _row_bytes(hidden, wt), "dweight", wt), wt,
                        int(bool(accumulate)), _buf(scratch, int(scratch_bytes), "scratch"), int(scratch_bytes),
                        _stream(stream, _first(dweight))), "gc_embedding_backward")
    return dweight


def gc_dropout(x, counts, p, seed, y, offset=0, step=None, residual=None, dtype=None, stream=None):
    """y = residual + dropout(x) of each rank's counts[r] elements; y may be x or residual.  The mask follows from
    (seed, offset + step, rank, element) alone, so the gradient is the same call on y's gradient without residual.
    step: an int64 device tensor of one value that a replayed graph may count up, or None.  Dropouts with the same sum of
    offset and step share a mask: give the l-th one of a step the offset l << 40 where steps count by one."""
    N, t = len(counts), _infer_dtype(x, dtype)
    nb = _rows_of(counts, _ES.get(t, 0))
    _check(_c_dropout(_bufs(x, N, nb, "x", t), _bufs(residual, N, nb, "residual", t), _i64_array(counts), N, float(p),
                      int(seed) & SIZE_MAX, int(offset) & SIZE_MAX, _buf(step, 8, "step", _HOLDS.get("int64")), t,
                      _bufs(y, N, nb, "y", t), _stream(stream, _first(y))), "gc_dropout")
    return y


def gc_token_logprob_scratch_bytes(ntokens, vocab, top=0):
    """Scratch bytes gc_token_logprob needs (0 if the sizes are invalid)."""
    return int(_c_logprob_scratch(_i64_array(ntokens), len(ntokens), max(0, int(vocab)), int(top)))


def gc_token_logprob(logits, ntokens, vocab, scratch, targets=None, logprob=None, entropy=None, lse=None, top=0,
                     top_ids=None, top_logprob=None, dlogprob=None, dentropy=None, dlogits=None, stride=None, scale=1.0,
                     scratch_bytes=None, dtype=None, stream=None):
    """Per row of scale * logits[r] ([ntokens[r]] rows of stride elements, vocab of them read): the log probability of
    the row's target, the entropy, the log of the sum of exponentials and the `top` most likely tokens with their log
    probabilities, each where a buffer is given.  With dlogprob (and dentropy) the gradient is written to dlogits in
    the same pass, as gc_token_logprob_backward would."""
    N, t = len(ntokens), _infer_dtype(logits, dtype)
    stride, vocab = int(vocab if stride is None else stride), max(0, int(vocab))
    if scratch_bytes is None:
        scratch_bytes = scratch.numel() * scratch.element_size()
    rows, each, tops = (_rows_of(ntokens, k) for k in (_row_bytes(stride, t), 4, 4 * max(0, int(top))))
    f = lambda xs, what: _bufs(xs, N, each, what, GC_FP32)  # noqa: E731
    _check(_c_logprob(_bufs(logits, N, rows, "logits", t), _bufs(targets, N, each, "targets", GC_INT32), _i64_array(ntokens),
                      N, vocab, max(0, stride), float(scale), t, f(logprob, "logprob"), f(entropy, "entropy"), f(lse, "lse"),
                      int(top), _bufs(top_ids, N, tops, "top_ids", GC_INT32), _bufs(top_logprob, N, tops, "top_logprob", GC_FP32),
                      f(dlogprob, "dlogprob"), f(dentropy, "dentropy"), _bufs(dlogits, N, rows, "dlogits", t),
                      _buf(scratch, int(scratch_bytes), "scratch"), int(scratch_bytes), _stream(stream, _first(logits))),
           "gc_token_logprob")
    return logprob


def gc_token_logprob_backward(logits, ntokens, vocab, lse, targets, dlogprob, dlogits, entropy=None, dentropy=None,
                              stride=None, scale=1.0, dtype=None, stream=None):
    """dlogits (may be logits) from dlogprob and, with the forward's entropy, dentropy; zeros in the padding columns."""
    N, t = len(ntokens), _infer_dtype(logits, dtype)
    stride, vocab = int(vocab if stride is None else stride), max(0, int(vocab))
    rows, each = _rows_of(ntokens, _row_bytes(stride, t)), _rows_of(ntokens, 4)
    f = lambda xs, what: _bufs(xs, N, each, what, GC_FP32)  # noqa: E731
    _check(_c_logprob_bwd(_bufs(logits, N, rows, "logits", t), _bufs(targets, N, each, "targets", GC_INT32), f(lse, "lse"),
                          f(entropy, "entropy"), f(dlogprob, "dlogprob"), f(dentropy, "dentropy"), _i64_array(ntokens), N,
                          vocab, max(0, stride), float(scale), t, _bufs(dlogits, N, rows, "dlogits", t),
                          _stream(stream, _first(dlogits))), "gc_token_logprob_backward")
    return dlogits


# ------------------------------------------------------------------ HBM layout

def gc_rank_buffers(nranks, count, dtype, device="cuda", stagger_bytes=4096, slot_align=2 << 20):
    """N rank buffers of `count` elements carved from one device allocation.

    Rank r starts at r * (slot + stagger_bytes) bytes, slot = the buffer size
    rounded up to slot_align.  Every element offset then sits at a different
    position modulo slot_align on each rank, so the N same-offset accesses a
    reduction makes at once fall into different HBM channels and banks instead
    of piling onto one.  On MI355X a 4 KiB stagger raised the 8 x 64 MiB bf16
    all-reduce from about 5.6 to 5.8 TB/s.  Returns a list of 1-D views.
    """
    import torch
    tdt = {"bf16": torch.bfloat16, "fp32": torch.float32, "int32": torch.int32}.get(dtype, dtype)
    es = torch.empty((), dtype=tdt).element_size()
    slot = -(-count * es // slot_align) * slot_align
    step = slot + stagger_bytes
    if step % es:
        raise ValueError("stagger_bytes must be a multiple of the element size")
    total = (nranks - 1) * step + count * es
    slab = torch.empty(max(1, total // es), dtype=tdt, device=device)
    return [slab[r * step // es: r * step // es + count] for r in range(nranks)]


class RankArena:
    """Per-rank HBM regions for N ranks on one GPU: every rank owns one region,
    as a real rank owns its GPU's memory, and all of a rank's buffers are
    bump-allocated inside it at the same offset on every rank.

    The regions are carved from one allocation; rank r's region starts at
    r * (region_bytes + stagger_bytes).  A collective reads and writes the same
    offset on all N ranks at once; regions a large power of two apart plus a
    small stagger spread those N streams over HBM's channels and stacks.  On
    MI355X, 16 GiB regions raised the 8 x 64 MiB bf16 all-reduce from about 5.8
    to 6.2 TB/s and 32 GiB regions by up to 1.7 % more (every 8-rank workload
    gained 0.4-1.1 %); 4 GiB regions raised the 64-rank all-gather from about
    5.4 to 6.7 TB/s.

    region_bytes=None picks the largest power of two up to max_region for which
    all N regions fit in free device memory (keeping reserve_bytes free), and at
    least min_bytes.
    """

    def __init__(self, nranks, region_bytes=None, stagger_bytes=4096, min_bytes=0, device="cuda",
                 reserve_bytes=4 << 30, max_region=32 << 30):
        import torch
        self.nranks = int(nranks)
        self.stagger = int(stagger_bytes)
        if region_bytes is None:
            free = torch.cuda.mem_get_info(torch.device(device))[0] if str(device).startswith("cuda") else 1 << 40
            region_bytes = 1 << 21
            while (region_bytes * 2 <= max_region and
                   self.nranks * (region_bytes * 2 + self.stagger) <= free - reserve_bytes):
                region_bytes *= 2
            while region_bytes < min_bytes:
                region_bytes *= 2
        self.region = int(region_bytes)
        self.step = self.region + self.stagger
        self.slab = torch.empty(self.nranks * self.step, dtype=torch.uint8, device=device)
        self.used = 0

    def alloc(self, count, dtype):
        """One buffer of `count` elements per rank, at the same offset of every region."""
        import torch
        tdt = {"bf16": torch.bfloat16, "fp32": torch.float32, "int32": torch.int32}.get(dtype, dtype)
        es = torch.empty((), dtype=tdt).element_size()
        nbytes = int(count) * es
        if self.used + nbytes > self.region:
            raise MemoryError(f"rank region of {self.region} bytes is full")
        out = [self.slab[r * self.step + self.used: r * self.step + self.used + nbytes].view(tdt)
               for r in range(self.nranks)]
        self.used += -(-nbytes // 256) * 256
        return out


# ------------------------------------------------------------------ bucket plan

def gc_bucket_plan_create(numels, dtype, cap_bytes, reverse=True, pad_to=1):
    arr = (ctypes.c_size_t * max(1, len(numels)))(*[int(x) for x in numels])
    out = ctypes.c_void_p()
    _check(_c_plan_create(arr, len(numels), _dtype_code(dtype), int(cap_bytes), int(bool(reverse)), int(pad_to),
                          ctypes.byref(out)), "gc_bucket_plan_create")
    return out.value


def gc_bucket_plan_query(plan, ntensors):
    nb = ctypes.c_int()
    _check(_c_plan_query(plan, ctypes.byref(nb), None, None, None), "gc_bucket_plan_query")
    bucket_numel = (ctypes.c_size_t * max(1, nb.value))()
    tb = (ctypes.c_int * max(1, ntensors))()
    to = (ctypes.c_size_t * max(1, ntensors))()
    _check(_c_plan_query(plan, ctypes.byref(nb), bucket_numel, tb, to), "gc_bucket_plan_query")
    return (nb.value, [bucket_numel[i] for i in range(nb.value)], [tb[i] for i in range(ntensors)],
            [to[i] for i in range(ntensors)])


def gc_bucket_plan_destroy(plan):
    _c_plan_destroy(plan)


def gc_bucket_pack(plan, bucket, tensors, bucket_bufs, nranks, stream=None):
    """tensors: flat rank-major list of nranks*ntensors tensors (or None for tensors outside the bucket).
    The plan handle does not carry the tensor sizes, so only device and layout are checked here
    (BucketPlan.pack checks sizes too)."""
    _check(_c_pack(plan, int(bucket), _bufs(tensors, 0, 0, "tensors"), _bufs(bucket_bufs, 0, 0, "bucket_bufs"),
                   int(nranks), _stream(stream, _first(bucket_bufs))), "gc_bucket_pack")


def gc_bucket_unpack(plan, bucket, bucket_bufs, tensors, nranks, stream=None):
    _check(_c_unpack(plan, int(bucket), _bufs(bucket_bufs, 0, 0, "bucket_bufs"), _bufs(tensors, 0, 0, "tensors"),
                     int(nranks), _stream(stream, _first(bucket_bufs))), "gc_bucket_unpack")


def gc_bucket_all_reduce(plan, bucket, tensors, nranks, op="avg", order="ring", sumsq=None, stream=None):
    """Zero-copy all-reduce of one bucket, in place over the tensors (rank-major flat list).
    sumsq: optional CUDA float64 tensor (one element) that receives += sum of squared results."""
    _check(_c_bucket_ar(plan, int(bucket), _bufs(tensors, 0, 0, "tensors"), int(nranks), _enum(_OP, op),
                        _enum(_ORDER, order), _buf(sumsq, 8, "sumsq"), _stream(stream, _first(tensors))),
           "gc_bucket_all_reduce")


class BucketPlan:
    """Owns a gc_bucket_plan handle and caches its query results.  Its calls
    check every tensor and bucket buffer against the plan's sizes before the
    library sees the pointers."""

    def __init__(self, numels, dtype, cap_bytes, reverse=True, pad_to=1):
        self.numels = [int(x) for x in numels]
        self.reverse = bool(reverse)
        self.es = _ES.get(_dtype_code(dtype), 0)
        self.handle = gc_bucket_plan_create(self.numels, dtype, cap_bytes, reverse, pad_to)
        self.nbuckets, self.bucket_numel, self.tensor_bucket, self.tensor_offset = gc_bucket_plan_query(
            self.handle, len(self.numels))

    def bucket_tensors(self, b):
        """Tensor indices of bucket b in packing order (an empty tensor shares its
        offset with the next one, so ties follow the visiting order)."""
        ts = [t for t in range(len(self.numels)) if self.tensor_bucket[t] == b]
        return sorted(ts, key=lambda t: (self.tensor_offset[t], -t if self.reverse else t))

    def _tensors(self, bucket, tensors, nranks):
        """Checked pointer array of the rank-major tensor list: bucket members need their full size."""
        if isinstance(tensors, ctypes.Array):        # marshalled once by gc_pointers: only its length is checked
            return _bufs(tensors, max(0, nranks) * len(self.numels), 0, "tensors")
        need = [n * self.es if self.tensor_bucket[t] == bucket else 0 for t, n in enumerate(self.numels)]
        return _bufs(tensors, max(0, nranks) * len(need), need * max(0, nranks), "tensors")

    def _bucket_bufs(self, bucket, bufs, nranks):
        nb = self.bucket_numel[bucket] * self.es if 0 <= bucket < self.nbuckets else 0
        return _bufs(bufs, max(0, nranks), nb, "bucket_bufs")

    def pack(self, bucket, tensors, bucket_bufs, nranks, stream=None):
        stream = _stream(stream, _first(bucket_bufs))
        gc_bucket_pack(self.handle, bucket, self._tensors(bucket, tensors, nranks),
                       self._bucket_bufs(bucket, bucket_bufs, nranks), nranks, stream)

    def unpack(self, bucket, bucket_bufs, tensors, nranks, stream=None):
        stream = _stream(stream, _first(bucket_bufs))
        gc_bucket_unpack(self.handle, bucket, self._bucket_bufs(bucket, bucket_bufs, nranks),
                         self._tensors(bucket, tensors, nranks), nranks, stream)

    def all_reduce(self, bucket, tensors, nranks, op="avg", order="ring", sumsq=None, stream=None):
        stream = _stream(stream, _first(tensors))
        gc_bucket_all_reduce(self.handle, bucket, self._tensors(bucket, tensors, nranks), nranks, op, order, sumsq,
                             stream)

    def close(self):
        if self.handle:
            gc_bucket_plan_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass
