"""ctypes binding of libtps_ar.so, one Python function per C entry point.

Argument marshalling only: tensors become device pointers, Python lists
become pointer arrays, torch streams become ``cudaStream_t`` handles, and a
non-zero status becomes an ``ARError``.  Every step of the reduction runs in
the library's CUDA kernels; there is no other implementation to fall back to.
"""
from __future__ import annotations

import ctypes
import os
import struct

_HERE = os.path.dirname(os.path.abspath(__file__))
_LIB_PATH = os.path.join(_HERE, "libtps_ar.so")

AR_F32, AR_F16, AR_BF16 = 0, 1, 2
DTYPE_CODES = {"f32": AR_F32, "f16": AR_F16, "bf16": AR_BF16}

AR_OK = 0
STATUS_NAMES = {0: "AR_OK", 1: "AR_ERR_INVALID_ARG", 2: "AR_ERR_UNSUPPORTED", 3: "AR_ERR_TOO_LARGE",
                4: "AR_ERR_NOT_INITIALIZED", 5: "AR_ERR_OVERLAP", 6: "AR_ERR_CUDA"}
VARIANTS = {"auto": 0, "naive": 1, "latency": 2, "bandwidth": 3, "scalar": 4, "tma": 5}
KEYS = {"ranks": 0, "max_elems": 1, "device": 2, "sm_count": 3, "latency_max_bytes": 4,
        "forced_variant": 5, "last_variant": 6, "fault_inject": 7, "bw_blocks_per_sm": 8,
        "host_chunk_bytes": 9, "device_status": 10, "tma_drop_tile": 11}

_lib = None


class ArLayout(ctypes.Structure):
    """ar_layout of include/ar.h."""
    _fields_ = [("ne0", ctypes.c_size_t), ("ne1", ctypes.c_size_t),
                ("src_row_bytes", ctypes.POINTER(ctypes.c_int64)),
                ("dst_row_bytes", ctypes.POINTER(ctypes.c_int64)),
                ("residual", ctypes.c_void_p), ("residual_row_bytes", ctypes.c_int64),
                ("inactive_mask", ctypes.c_uint32)]


class ArDropout(ctypes.Structure):
    """ar_dropout of include/ar.h."""
    _fields_ = [("seed", ctypes.c_uint64), ("offset", ctypes.c_uint64), ("p", ctypes.c_float),
                ("bias", ctypes.c_void_p)]


class ArVocab(ctypes.Structure):
    """ar_vocab of include/ar.h."""
    _fields_ = [("rows", ctypes.c_size_t), ("dim", ctypes.c_size_t), ("hidden", ctypes.c_void_p),
                ("hidden_row_bytes", ctypes.c_int64), ("n_pieces", ctypes.c_int),
                ("piece_rows", ctypes.POINTER(ctypes.c_size_t)), ("weights", ctypes.c_char_p),
                ("weight_row_bytes", ctypes.POINTER(ctypes.c_int64)), ("targets", ctypes.c_void_p),
                ("ignore_index", ctypes.c_int64), ("dtype", ctypes.c_int)]


class ARError(RuntimeError):
    def __init__(self, status: int, call: str):
        self.status = status
        super().__init__(f"{call}: {STATUS_NAMES.get(status, status)} ({ar_status_string(status)})")


def library_path() -> str:
    return _LIB_PATH


def lib() -> ctypes.CDLL:
    global _lib
    if _lib is None:
        if not os.path.exists(_LIB_PATH):
            raise RuntimeError(f"{_LIB_PATH} is not built: run `python -m tensor_partial_sum_gb300.build`")
        L = ctypes.CDLL(_LIB_PATH)
        vp, sz, i, i64 = ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int, ctypes.c_int64
        # pointer arrays travel as packed bytes (see _ptrs): the C side reads
        # R or n_dsts 64-bit addresses from the buffer
        pp = ctypes.c_char_p
        L.ar_init.argtypes = [i, sz]
        L.ar_init.restype = i
        L.ar_reduce.argtypes = [pp, pp, i, sz, i, i, vp]
        L.ar_reduce.restype = i
        L.ar_free.argtypes = []
        L.ar_free.restype = None
        L.ar_status_string.argtypes = [i]
        L.ar_status_string.restype = ctypes.c_char_p
        L.ar_check_args.argtypes = [i, pp, pp, i, sz, sz, i, i]
        L.ar_check_args.restype = i
        L.ar_reduce_variant.argtypes = [pp, pp, i, sz, i, i, i, i, vp]
        L.ar_reduce_variant.restype = i
        L.ar_query.argtypes = [i, ctypes.POINTER(i64)]
        L.ar_query.restype = i
        L.ar_set_option.argtypes = [i, i64]
        L.ar_set_option.restype = i
        L.ar_reduce_host.argtypes = [pp, pp, i, sz, i, i, pp, pp, vp]
        L.ar_reduce_host.restype = i
        lp = ctypes.POINTER(ArLayout)
        L.ar_reduce_ex.argtypes = [pp, pp, i, lp, i, i, vp]
        L.ar_reduce_ex.restype = i
        L.ar_check_layout.argtypes = [i, pp, pp, i, lp, sz, i, i]
        L.ar_check_layout.restype = i
        L.ar_wire_pack.argtypes = [vp, vp, sz, i, i, vp]
        L.ar_wire_pack.restype = i
        L.ar_reduce_host_noalloc.argtypes = [pp, pp, i, sz, i, i, vp]
        L.ar_reduce_host_noalloc.restype = i
        dp, szp = ctypes.POINTER(ArDropout), ctypes.POINTER(sz)
        L.ar_reduce_dropout.argtypes = [pp, pp, i, lp, dp, i, i, vp]
        L.ar_reduce_dropout.restype = i
        L.ar_check_dropout.argtypes = [i, pp, pp, i, lp, dp, sz, i, i]
        L.ar_check_dropout.restype = i
        L.ar_reduce_dropout_grad.argtypes = [vp, pp, i, lp, dp, vp, vp, vp, sz, i, vp]
        L.ar_reduce_dropout_grad.restype = i
        L.ar_reduce_dropout_grad_workspace.argtypes = [lp, i, szp]
        L.ar_reduce_dropout_grad_workspace.restype = i
        vcp, i64p = ctypes.POINTER(ArVocab), ctypes.POINTER(i64)
        L.ar_vocab_loss.argtypes = [vcp, vp, vp, vp, sz, vp]
        L.ar_vocab_loss.restype = i
        L.ar_vocab_loss_grad.argtypes = [vcp, vp, vp, pp, i64p, pp, i64p, vp, sz, vp]
        L.ar_vocab_loss_grad.restype = i
        L.ar_check_vocab.argtypes = [vcp, sz]
        L.ar_check_vocab.restype = i
        L.ar_vocab_workspace.argtypes = [vcp, i, szp]
        L.ar_vocab_workspace.restype = i
        _lib = L
    return _lib


# ---- marshalling helpers -------------------------------------------------

def _ptr(x) -> int | None:
    if x is None:
        return None
    if isinstance(x, int):
        return x
    if hasattr(x, "data_ptr"):
        return x.data_ptr()
    if hasattr(x, "ctypes"):  # numpy array (host buffers)
        return x.ctypes.data
    raise TypeError(f"cannot take a pointer of {type(x).__name__}")


AR_MAX_RANKS = 16


_PTR_ARRAY = struct.Struct(f"={AR_MAX_RANKS}Q")


def _ptrs(xs):
    """Pointer array (packed native 64-bit addresses, 0 for None) padded to
    at least AR_MAX_RANKS entries, so a list shorter than the context's R is
    rejected (NULL source) instead of being read past its end.  Packing with
    struct costs a fraction of building a ctypes array of c_void_p."""
    if xs is None:
        return None
    return _packed([_ptr(x) or 0 for x in xs])


def _packed(ptrs):
    if len(ptrs) <= AR_MAX_RANKS:
        return _PTR_ARRAY.pack(*ptrs, *([0] * (AR_MAX_RANKS - len(ptrs))))
    return struct.pack(f"={len(ptrs)}Q", *ptrs)


ESIZE = {AR_F32: 4, AR_F16: 2, AR_BF16: 2}
STORAGE_NAMES = {AR_F32: "float32", AR_F16: "float16", AR_BF16: "bfloat16"}


def _checked(xs, nelem, dcode, where, call):
    """Check the buffers of a 1-D call before their addresses reach the
    library: torch tensors and numpy arrays must be contiguous, hold at
    least ``nelem`` elements of the call's type, and live where the entry
    point reads them (``where`` = "device" or "host").  Plain integers are
    addresses the caller vouches for.  A wrong buffer would otherwise be
    read or written past its end by a kernel."""
    if xs is None:
        return xs
    need = nelem * ESIZE.get(dcode, 1)
    for k, x in enumerate(xs):
        if x is None or isinstance(x, int):
            continue
        if hasattr(x, "data_ptr"):
            if (x.device.type == "cuda") != (where == "device"):
                raise TypeError(f"{call}: buffer {k} is a {x.device.type} tensor, a {where} buffer is needed")
            if not x.is_contiguous():
                raise ValueError(f"{call}: buffer {k} is not contiguous")
            have = x.numel() * x.element_size()
        elif hasattr(x, "ctypes"):
            if where != "host":
                raise TypeError(f"{call}: buffer {k} is a numpy array, a device buffer is needed")
            if not x.flags["C_CONTIGUOUS"]:
                raise ValueError(f"{call}: buffer {k} is not contiguous")
            have = x.nbytes
        else:
            continue
        if have < need:
            raise ValueError(f"{call}: buffer {k} holds {have} bytes, the call needs {need}")
    return xs


def _reach(x) -> int | None:
    """Bytes a kernel may touch from a CUDA tensor's first element to the end
    of its storage (None for raw addresses); a non-CUDA tensor is refused."""
    if x is None or isinstance(x, int) or not hasattr(x, "data_ptr"):
        return None
    if x.device.type != "cuda":
        raise TypeError(f"a {x.device.type} tensor where a device buffer is needed")
    st = x.untyped_storage()
    return st.data_ptr() + st.nbytes() - x.data_ptr()


def _layout_pointers(xs, rows, row, ne1, kind, call):
    """Packed addresses of an ar_layout call's buffers, after checking that the
    rows of each tensor lie inside its storage (raw addresses are the
    caller's).  One pass: a small call's time is mostly spent here."""
    ptrs = []
    more = ne1 - 1
    n = more * row + row
    empty = not (ne1 and row)  # such a call touches no buffer
    for k, x in enumerate(xs):
        if x is None:
            ptrs.append(0)
            continue
        if type(x) is int:
            ptrs.append(x)
            continue
        if empty or not getattr(x, "is_cuda", False):
            if not empty:
                _reach(x)  # refuses host tensors
            ptrs.append(_ptr(x) or 0)
            continue
        if rows is not None:
            n = more * rows[k] + row
        if x.nbytes < n or not x.is_contiguous():
            st = x.untyped_storage()
            reach = st.nbytes() - x.storage_offset() * x.element_size()
            if reach < n:
                raise ValueError(f"{call}: {kind} {k} reaches {reach} bytes, its rows span {n}")
        ptrs.append(x.data_ptr())
    return _packed(ptrs)


_TORCH_CODES = None


def _dtype_code(d) -> int:
    if isinstance(d, int):
        return d
    if isinstance(d, str):
        return DTYPE_CODES[d]
    global _TORCH_CODES
    if _TORCH_CODES is None:
        import torch
        _TORCH_CODES = {torch.float32: AR_F32, torch.float16: AR_F16, torch.bfloat16: AR_BF16}
    return _TORCH_CODES[d]


_raw_stream = None


def _current_stream() -> int | None:
    """Handle of torch's current stream.  torch.cuda.current_stream() builds a
    Stream object each time, several microseconds of a small call."""
    global _raw_stream
    if _raw_stream is None:
        import torch
        get, dev = getattr(torch._C, "_cuda_getCurrentRawStream", None), getattr(torch._C, "_cuda_getDevice", None)
        if get is None or dev is None or not torch.cuda.is_initialized():
            return torch.cuda.current_stream().cuda_stream or None
        _raw_stream = lambda: get(dev())  # noqa: E731
    return _raw_stream() or None


def _stream(s) -> int | None:
    if s is None:
        return _current_stream()
    if isinstance(s, int):
        return s or None
    return s.cuda_stream or None


def _infer(srcs, nelem, dst_dtype):
    """nelem and dtype code from the first buffer unless given: torch tensors
    and numpy arrays (float32 -> f32, float16 -> f16; uint16 bit patterns are
    ambiguous between f16 and bf16 and need an explicit dst_dtype)."""
    t = srcs[0] if srcs else None
    if nelem is None:
        nelem = t.numel() if hasattr(t, "numel") else int(t.size)
    if dst_dtype is None:
        if hasattr(t, "numel"):
            dst_dtype = t.dtype
        else:
            name = {"float32": "f32", "float16": "f16"}.get(str(t.dtype))
            if name is None:
                raise TypeError(f"cannot tell the element type of a {t.dtype} array: pass dst_dtype")
            dst_dtype = name
    return nelem, _dtype_code(dst_dtype)


def _check(status: int, call: str) -> int:
    if status != AR_OK:
        raise ARError(status, call)
    return status


# ---- entry points ----------------------------------------------------------

def ar_status_string(status: int) -> str:
    return lib().ar_status_string(status).decode()


def ar_init(R: int, max_elems: int) -> None:
    _check(lib().ar_init(R, max_elems), "ar_init")


def ar_free() -> None:
    lib().ar_free()


def ar_reduce(srcs, dsts, nelem=None, dst_dtype=None, wire_dtype="bf16", stream=None) -> None:
    """Enqueue one reduction of ``srcs`` (R tensors or device pointers) into
    every tensor of ``dsts``.  ``nelem``/``dst_dtype`` default to the first
    source tensor's; ``stream`` defaults to torch's current stream."""
    nelem, dcode = _infer(srcs, nelem, dst_dtype)
    _checked(srcs, nelem, dcode, "device", "ar_reduce")
    _checked(dsts, nelem, dcode, "device", "ar_reduce")
    _check(lib().ar_reduce(_ptrs(srcs), _ptrs(dsts), len(dsts), nelem, dcode, _dtype_code(wire_dtype),
                           _stream(stream)), "ar_reduce")


def ar_reduce_variant(srcs, dsts, variant="auto", grid_blocks=0, nelem=None, dst_dtype=None,
                      wire_dtype="bf16", stream=None) -> None:
    nelem, dcode = _infer(srcs, nelem, dst_dtype)
    _checked(srcs, nelem, dcode, "device", "ar_reduce_variant")
    _checked(dsts, nelem, dcode, "device", "ar_reduce_variant")
    v = VARIANTS[variant] if isinstance(variant, str) else variant
    _check(lib().ar_reduce_variant(_ptrs(srcs), _ptrs(dsts), len(dsts), nelem, dcode, _dtype_code(wire_dtype),
                                   v, grid_blocks, _stream(stream)), "ar_reduce_variant")


class PreparedReduce:
    """One ar_reduce_variant call with its arguments fixed: the buffer
    checks and the pointer arrays are done once, so each call is a single
    C call (for eager code that repeats the same reduction, e.g. every
    decode step; a CUDA graph removes the per-call cost altogether).  Holds
    references to the buffers it was given."""

    def __init__(self, srcs, dsts, nelem=None, dst_dtype=None, wire_dtype="bf16", variant="auto", stream=None):
        nelem, dcode = _infer(srcs, nelem, dst_dtype)
        _checked(srcs, nelem, dcode, "device", "PreparedReduce")
        _checked(dsts, nelem, dcode, "device", "PreparedReduce")
        self._keep = (list(srcs), list(dsts))
        self._args = (_ptrs(srcs), _ptrs(dsts), len(dsts), nelem, dcode, _dtype_code(wire_dtype),
                      VARIANTS[variant] if isinstance(variant, str) else variant, 0)
        self._stream = None if stream is None else _stream(stream)
        self._fn = lib().ar_reduce_variant

    def __call__(self, stream=None):
        """Enqueue the reduction on ``stream`` (default: the one given at
        preparation, else torch's current stream)."""
        s = _stream(stream) if stream is not None else (self._stream if self._stream is not None else _stream(None))
        st = self._fn(*self._args, s)
        if st != AR_OK:
            raise ARError(st, "ar_reduce")


def ar_check_args(R, srcs, dsts, n_dsts, nelem, max_elems, dst_dtype, wire_dtype) -> int:
    """Host-only validation; returns the status code (does not raise)."""
    return lib().ar_check_args(R, _ptrs(srcs), _ptrs(dsts), n_dsts, nelem, max_elems,
                               _dtype_code(dst_dtype), _dtype_code(wire_dtype))


def ar_query(key) -> int:
    k = KEYS[key] if isinstance(key, str) else key
    v = ctypes.c_int64(0)
    _check(lib().ar_query(k, ctypes.byref(v)), "ar_query")
    return v.value


def ar_set_option(key, value: int) -> None:
    k = KEYS[key] if isinstance(key, str) else key
    _check(lib().ar_set_option(k, value), "ar_set_option")


def ar_reduce_host(h_srcs, h_dsts, d_srcs=None, d_dsts=None, nelem=None, dst_dtype=None, wire_dtype="bf16",
                   stream=None) -> None:
    """Host partials in, host results out: through the caller's device
    staging buffers, or (``d_srcs``/``d_dsts`` None) with the kernel reading
    and writing the pinned host buffers directly; ordered on ``stream``."""
    nelem, dcode = _infer(d_srcs if d_srcs is not None else h_srcs, nelem, dst_dtype)
    for xs, where in ((h_srcs, "host"), (h_dsts, "host"), (d_srcs, "device"), (d_dsts, "device")):
        _checked(xs, nelem, dcode, where, "ar_reduce_host")
    _check(lib().ar_reduce_host(_ptrs(h_srcs), _ptrs(h_dsts), len(h_dsts), nelem, dcode, _dtype_code(wire_dtype),
                                _ptrs(d_srcs), _ptrs(d_dsts), _stream(stream)), "ar_reduce_host")


_I64_ARRAYS = {}


def _i64s(values):
    n = len(values)
    kind = _I64_ARRAYS.get(n)
    if kind is None:
        kind = _I64_ARRAYS[n] = ctypes.c_int64 * n
    return kind(*values)


_SIZE_ARRAYS = {}


def _sizes(values):
    n = len(values)
    kind = _SIZE_ARRAYS.get(n)
    if kind is None:
        kind = _SIZE_ARRAYS[n] = ctypes.c_size_t * n
    return kind(*values)


_torch_module = None


def _torch():
    """torch, imported with the first call that needs it."""
    global _torch_module
    if _torch_module is None:
        import torch
        _torch_module = torch
    return _torch_module


def make_layout(ne0, ne1, src_row_bytes=None, dst_row_bytes=None, residual=None, residual_row_bytes=None,
                inactive=()) -> ArLayout:
    """An ar_layout.  With a residual, ``residual_row_bytes`` is its row
    stride in bytes (0: one bias row broadcast to every row; None: packed
    rows, which needs a tensor residual to know the element size);
    ``inactive`` lists rank indices."""
    L = ArLayout()
    L.ne0, L.ne1 = ne0, ne1
    if src_row_bytes is not None:
        L.src_row_bytes = _i64s(src_row_bytes)
    if dst_row_bytes is not None:
        L.dst_row_bytes = _i64s(dst_row_bytes)
    L.residual = _ptr(residual)
    L._residual_obj = residual  # kept for the binding's reach check
    if residual is not None and residual_row_bytes is None:
        residual_row_bytes = ne0 * residual.element_size()
    L.residual_row_bytes = residual_row_bytes or 0
    mask = 0
    for r in inactive:
        mask |= 1 << r
    L.inactive_mask = mask
    return L


def _layout_buffers(srcs, dsts, layout, dcode, call):
    """Checked, packed addresses of the sources and destinations of an
    ar_layout call, whose residual is checked too."""
    ne0, ne1 = layout.ne0, layout.ne1
    row = ne0 * ESIZE[dcode]
    src = _layout_pointers(srcs, layout.src_row_bytes or None, row, ne1, "source", call)
    dst = _layout_pointers(dsts, layout.dst_row_bytes or None, row, ne1, "destination", call)
    res = layout._residual_obj if hasattr(layout, "_residual_obj") else None
    if res is not None and row * ne1:
        reach = _reach(res)
        n = row if layout.residual_row_bytes == 0 else (ne1 - 1) * layout.residual_row_bytes + row
        if reach is not None and reach < n:
            raise ValueError(f"{call}: the residual reaches {reach} bytes, its rows span {n}")
    return src, dst


def ar_reduce_ex(srcs, dsts, layout: ArLayout, dst_dtype, wire_dtype="bf16", stream=None) -> None:
    """Reduction over an ar_layout (row strides, inactive ranks as None
    sources, residual or bias).  The rows of each CUDA tensor must lie inside
    its storage."""
    dcode = _dtype_code(dst_dtype)
    src, dst = _layout_buffers(srcs, dsts, layout, dcode, "ar_reduce_ex")
    _check(lib().ar_reduce_ex(src, dst, len(dsts), ctypes.byref(layout), dcode, _dtype_code(wire_dtype),
                              _stream(stream)), "ar_reduce_ex")


def ar_check_layout(R, srcs, dsts, layout: ArLayout, max_elems, dst_dtype, wire_dtype) -> int:
    """Host-only validation of an ar_reduce_ex call; returns the status."""
    return lib().ar_check_layout(R, _ptrs(srcs), _ptrs(dsts), len(dsts), ctypes.byref(layout), max_elems,
                                 _dtype_code(dst_dtype), _dtype_code(wire_dtype))


def ar_wire_pack(src, wire, nelem=None, dst_dtype=None, wire_dtype="bf16", stream=None) -> None:
    """wire[i] = T_wire(src[i]): the wire copy a transport would send."""
    if nelem is None:
        nelem = src.numel()
    if dst_dtype is None:
        dst_dtype = src.dtype
    dcode, wcode = _dtype_code(dst_dtype), _dtype_code(wire_dtype)
    _checked([src], nelem, dcode, "device", "ar_wire_pack")
    _checked([wire], nelem, wcode, "device", "ar_wire_pack")
    _check(lib().ar_wire_pack(_ptr(src), _ptr(wire), nelem, _dtype_code(dst_dtype), _dtype_code(wire_dtype),
                              _stream(stream)), "ar_wire_pack")


AR_NOALLOC_SCRATCH_BYTES = 64 << 20


def ar_reduce_host_noalloc(h_srcs, h_dsts, nelem=None, dst_dtype=None, wire_dtype="bf16", stream=None) -> None:
    """Host partials in, host results out, staged through the library's own
    fixed device area: for callers that may not allocate device memory.
    At most AR_NOALLOC_SCRATCH_BYTES of staging per call; calls that overlap
    on the GPU share that area and must not run at the same time."""
    nelem, dcode = _infer(h_srcs, nelem, dst_dtype)
    _checked(h_srcs, nelem, dcode, "host", "ar_reduce_host_noalloc")
    _checked(h_dsts, nelem, dcode, "host", "ar_reduce_host_noalloc")
    _check(lib().ar_reduce_host_noalloc(_ptrs(h_srcs), _ptrs(h_dsts), len(h_dsts), nelem, dcode,
                                        _dtype_code(wire_dtype), _stream(stream)), "ar_reduce_host_noalloc")


# ---- training operators ------------------------------------------------------

def _typed_row(x, n, dtype, name, call):
    """A device row (tensor or address) of at least n elements of a torch dtype."""
    if x is None or isinstance(x, int):
        return
    if not x.is_cuda:
        raise TypeError(f"{call}: {name} is a {x.device.type} tensor, a device buffer is needed")
    if _dtype_code(x.dtype) != dtype or not x.is_contiguous() or x.numel() < n:
        raise ValueError(f"{call}: {name} needs {n} contiguous elements of {STORAGE_NAMES[dtype]}")


def _workspace(need, given, stream, like, call):
    """(tensor or address, bytes) of a call's workspace: the caller's, or one
    from torch's allocator, on the device of ``like`` and the stream that will
    use it."""
    if need == 0:
        return None, 0
    if given is not None:
        if isinstance(given, int):
            return given, need
        if not given.is_cuda or not given.is_contiguous():
            raise TypeError(f"{call}: the workspace has to be a contiguous device tensor")
        return given, given.numel() * given.element_size()
    torch = _torch()
    device = like.device if hasattr(like, "device") else "cuda"
    if stream is None:
        return torch.empty(need, dtype=torch.uint8, device=device), need
    s = torch.cuda.ExternalStream(stream) if isinstance(stream, int) else stream
    with torch.cuda.stream(s):
        return torch.empty(need, dtype=torch.uint8, device=device), need


def make_dropout(p, seed, offset=0, bias=None) -> ArDropout:
    """An ar_dropout: probability ``p`` of dropping an element, the 64-bit
    ``seed``, the 64-bit ``offset`` that tells calls under one seed apart, and
    an optional bias row added before the dropout."""
    if not 0 <= seed < 1 << 64 or not 0 <= offset < 1 << 64:
        raise ValueError("make_dropout: seed and offset are unsigned 64-bit numbers")
    d = ArDropout(seed, offset, p, _ptr(bias))
    d._bias_obj = bias  # kept alive, and for the binding's checks
    return d


def ar_reduce_dropout(srcs, dsts, layout: ArLayout, dropout: ArDropout, dst_dtype, wire_dtype="bf16",
                      stream=None) -> None:
    """ar_reduce_ex with bias and dropout between the rank sum and the
    residual; the mask is a function of the dropout's seed and offset."""
    dcode = _dtype_code(dst_dtype)
    src, dst = _layout_buffers(srcs, dsts, layout, dcode, "ar_reduce_dropout")
    _typed_row(getattr(dropout, "_bias_obj", None), layout.ne0, dcode, "the bias", "ar_reduce_dropout")
    _check(lib().ar_reduce_dropout(src, dst, len(dsts), ctypes.byref(layout), ctypes.byref(dropout), dcode,
                                   _dtype_code(wire_dtype), _stream(stream)), "ar_reduce_dropout")


def ar_check_dropout(R, srcs, dsts, layout: ArLayout, dropout: ArDropout, max_elems, dst_dtype, wire_dtype) -> int:
    """Host-only validation of an ar_reduce_dropout call; returns the status."""
    return lib().ar_check_dropout(R, _ptrs(srcs), _ptrs(dsts), len(dsts), ctypes.byref(layout),
                                  ctypes.byref(dropout), max_elems, _dtype_code(dst_dtype), _dtype_code(wire_dtype))


def ar_reduce_dropout_grad_workspace(layout: ArLayout, n_sums: int) -> int:
    """Workspace bytes of an ar_reduce_dropout_grad call with ``n_sums`` of
    dbias and dresidual."""
    n = ctypes.c_size_t(0)
    _check(lib().ar_reduce_dropout_grad_workspace(ctypes.byref(layout), n_sums, ctypes.byref(n)),
           "ar_reduce_dropout_grad_workspace")
    return n.value


def ar_reduce_dropout_grad(dy, dxs, layout: ArLayout, dropout: ArDropout, dst_dtype, dbias=None, dresidual=None,
                           workspace=None, stream=None) -> None:
    """The backward pass of ar_reduce_dropout: the partials' gradient into
    every tensor of ``dxs``, and, where asked for, the float32 gradients of
    the bias row and of a broadcast residual row.  ``workspace`` defaults to
    one from torch's allocator."""
    call = "ar_reduce_dropout_grad"
    dcode = _dtype_code(dst_dtype)
    _, dst = _layout_buffers([dy], dxs, layout, dcode, call)
    _typed_row(dbias, layout.ne0, AR_F32, "dbias", call)
    _typed_row(dresidual, layout.ne0, AR_F32, "dresidual", call)
    n_sums = (dbias is not None) + (dresidual is not None)
    need = ar_reduce_dropout_grad_workspace(layout, n_sums) if n_sums else 0
    ws, ws_bytes = _workspace(need, workspace, stream, dy, call)
    _check(lib().ar_reduce_dropout_grad(_ptr(dy), dst, len(dxs), ctypes.byref(layout), ctypes.byref(dropout),
                                        _ptr(dbias), _ptr(dresidual), _ptr(ws), ws_bytes, dcode, _stream(stream)), call)


def _matrix(x, rows, dim, dtype, name, call):
    """Row stride in bytes of a device matrix [rows, dim] with adjacent columns."""
    if not x.is_cuda:
        raise TypeError(f"{call}: {name} is a {x.device.type} tensor, a device buffer is needed")
    if x.dtype != dtype:
        raise TypeError(f"{call}: {name} is {x.dtype}, the hidden states are {dtype}")
    if tuple(x.shape) != (rows, dim):
        raise ValueError(f"{call}: {name} has to be [{rows}, {dim}] with adjacent columns")
    if x.is_contiguous():
        return dim * x.element_size()
    if dim > 1 and x.stride(1) != 1:
        raise ValueError(f"{call}: {name} has to be [{rows}, {dim}] with adjacent columns")
    if rows > 1 and x.stride(0) < dim:  # an expanded tensor, for one; the library takes a stride of 0 for packed rows
        raise ValueError(f"{call}: the rows of {name} lie over one another")
    return (x.stride(0) if rows > 1 else dim) * x.element_size()


def _vector(x, n, dtype, name, call):
    if not x.is_cuda:
        raise TypeError(f"{call}: {name} is a {x.device.type} tensor, a device buffer is needed")
    if x.dtype != dtype or x.dim() != 1 or x.numel() != n or not x.is_contiguous():
        raise ValueError(f"{call}: {name} has to be {n} contiguous elements of {dtype}")


def make_vocab(hidden, weights, targets, ignore_index=-100, call="make_vocab") -> ArVocab:
    """An ar_vocab of torch tensors: ``hidden`` [tokens, dim], one [rows, dim]
    matrix per vocabulary piece in ``weights``, and int64 ``targets``
    [tokens] that count through the pieces in order."""
    if hidden.dim() != 2:
        raise ValueError(f"{call}: hidden has to be [tokens, dim]")
    T, D = hidden.shape
    dtype = hidden.dtype
    n = len(weights)
    if not 1 <= n <= AR_MAX_RANKS:
        raise ValueError(f"{call}: {n} vocabulary pieces, 1 to {AR_MAX_RANKS} are possible")
    _vector(targets, T, _torch().int64, "targets", call)
    v = ArVocab()
    v.rows, v.dim, v.hidden = T, D, hidden.data_ptr()
    v.hidden_row_bytes = _matrix(hidden, T, D, dtype, "hidden", call)
    v.n_pieces = n
    rows = [w.shape[0] for w in weights]
    v.weight_row_bytes = _i64s([_matrix(w, m, D, dtype, "a piece of weights", call) for w, m in zip(weights, rows)])
    v.piece_rows = _sizes(rows)
    v._pointers = _packed([w.data_ptr() for w in weights])
    v.weights = v._pointers
    v.targets, v.ignore_index = targets.data_ptr(), ignore_index
    v.dtype = _dtype_code(dtype)
    v._keep = (hidden, weights, targets)
    return v


def ar_check_vocab(v: ArVocab, max_elems) -> int:
    """Host-only checks of an ar_vocab; returns the status."""
    return lib().ar_check_vocab(ctypes.byref(v), max_elems)


def ar_vocab_workspace(v: ArVocab, grad: bool) -> int:
    """Workspace bytes of ar_vocab_loss or (``grad``) ar_vocab_loss_grad."""
    n = ctypes.c_size_t(0)
    _check(lib().ar_vocab_workspace(ctypes.byref(v), int(grad), ctypes.byref(n)), "ar_vocab_workspace")
    return n.value


def ar_vocab_loss(hidden, weights, targets, loss, lse, ignore_index=-100, workspace=None, stream=None) -> None:
    """Softmax cross entropy of every token against a vocabulary split into
    the ``weights`` pieces, without keeping the logits: float32 ``loss`` and
    ``lse`` (log-sum-exp) of each token.  ``workspace`` defaults to one from
    torch's allocator."""
    call = "ar_vocab_loss"
    v = make_vocab(hidden, weights, targets, ignore_index, call)
    f32, T = _torch().float32, v.rows
    _vector(loss, T, f32, "loss", call)
    _vector(lse, T, f32, "lse", call)
    ws, ws_bytes = _workspace(ar_vocab_workspace(v, False), workspace, stream, hidden, call)
    _check(lib().ar_vocab_loss(ctypes.byref(v), loss.data_ptr(), lse.data_ptr(), _ptr(ws), ws_bytes, _stream(stream)),
           call)


def ar_vocab_loss_grad(hidden, weights, targets, lse, dloss, dhidden=None, dweights=None, ignore_index=-100,
                       workspace=None, stream=None) -> None:
    """The gradients of ar_vocab_loss: one partial gradient of the hidden
    states per piece into ``dhidden`` (ar_reduce sums them), each piece's
    weight gradient into ``dweights``; either may be None.  ``lse`` is
    ar_vocab_loss's, ``dloss`` the float32 gradient of each token's loss."""
    call = "ar_vocab_loss_grad"
    v = make_vocab(hidden, weights, targets, ignore_index, call)
    f32, T, D, n, dtype = _torch().float32, v.rows, v.dim, v.n_pieces, hidden.dtype
    _vector(lse, T, f32, "lse", call)
    _vector(dloss, T, f32, "dloss", call)
    strides = []
    for name, xs, rows in (("dhidden", dhidden, [T] * n), ("dweights", dweights, [w.shape[0] for w in weights])):
        if xs is not None and len(xs) != n:
            raise ValueError(f"{call}: {len(xs)} tensors in {name}, {n} vocabulary pieces")
        strides.append(None if xs is None else _i64s([_matrix(x, m, D, dtype, name, call) for x, m in zip(xs, rows)]))
    ws, ws_bytes = _workspace(ar_vocab_workspace(v, True), workspace, stream, hidden, call)
    _check(lib().ar_vocab_loss_grad(ctypes.byref(v), lse.data_ptr(), dloss.data_ptr(), _ptrs(dhidden), strides[0],
                                    _ptrs(dweights), strides[1], _ptr(ws), ws_bytes, _stream(stream)), call)
