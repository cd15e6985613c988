"""Products whose stored operand is held in few bits: the binding of
``sgemm_w4*`` (a matrix held in 4 bits) and ``sgemm_kv8*`` (a cache of keys
and values held in 8), and their tensor helpers.

Like the rest of the binding it only marshals arguments: the kernels are
enqueued on the current stream of the operands' device, nothing waits, and a
refused argument raises. The raw entry points take the C ABI's arguments in
its order; ``cache`` and ``batch`` are :class:`KV8Cache` and
:class:`KV8Batch` structures.
"""

from __future__ import annotations

import ctypes

SGEMM_F32 = 0

EXPORTS = ("sgemm_w4", "sgemm_w4_check_args", "sgemm_w4_quantize", "sgemm_w4_dequantize", "sgemm_w4_pack_check_args",
           "sgemm_kv8_write", "sgemm_kv8_read", "sgemm_kv8_check_args", "sgemm_kv8_attend",
           "sgemm_kv8_attend_check_args", "sgemm_kv8_attend_workspace_size")


class KV8Cache(ctypes.Structure):
    """sgemm_kv8_cache."""

    _fields_ = [("K", ctypes.c_void_p), ("V", ctypes.c_void_p), ("Ks", ctypes.c_void_p), ("Vs", ctypes.c_void_p),
                ("pages", ctypes.c_int), ("heads", ctypes.c_int), ("block", ctypes.c_int), ("dim", ctypes.c_int)]


class KV8Batch(ctypes.Structure):
    """sgemm_kv8_batch."""

    _fields_ = [("table", ctypes.c_void_p), ("lens", ctypes.c_void_p), ("starts", ctypes.c_void_p),
                ("seqs", ctypes.c_int), ("table_ld", ctypes.c_int), ("rows", ctypes.c_int), ("max_new", ctypes.c_int)]


def declare(lib) -> None:
    """Argument and result types of this module's entry points."""
    i, f, vp, sz = ctypes.c_int, ctypes.c_float, ctypes.c_void_p, ctypes.c_size_t
    cache, batch = ctypes.POINTER(KV8Cache), ctypes.POINTER(KV8Batch)
    w4 = [i, i, i, i, i, i, f, vp, i, vp, i, vp, i, vp, i, f, vp, i]
    pack = [i, i, i, i, i, vp, i, vp, i, vp, i, vp, i]
    rows = [cache, batch, i, vp, i, i, vp, i, i]
    attend = [cache, batch, i, i, vp, i, i, f, i, i, vp, i, i, vp, sz]
    lib.sgemm_w4.argtypes, lib.sgemm_w4.restype = w4 + [vp], i
    lib.sgemm_w4_check_args.argtypes, lib.sgemm_w4_check_args.restype = w4, i
    lib.sgemm_w4_quantize.argtypes, lib.sgemm_w4_quantize.restype = pack + [vp], i
    lib.sgemm_w4_dequantize.argtypes = [i, i, i, i, i, vp, i, vp, i, vp, i, vp, i, vp]
    lib.sgemm_w4_dequantize.restype = i
    lib.sgemm_w4_pack_check_args.argtypes, lib.sgemm_w4_pack_check_args.restype = pack, i
    lib.sgemm_kv8_write.argtypes, lib.sgemm_kv8_write.restype = rows + [vp], i
    lib.sgemm_kv8_read.argtypes, lib.sgemm_kv8_read.restype = rows + [vp], i
    lib.sgemm_kv8_check_args.argtypes, lib.sgemm_kv8_check_args.restype = rows, i
    lib.sgemm_kv8_attend.argtypes, lib.sgemm_kv8_attend.restype = attend + [vp], i
    lib.sgemm_kv8_attend_check_args.argtypes, lib.sgemm_kv8_attend_check_args.restype = attend, i
    lib.sgemm_kv8_attend_workspace_size.argtypes = [cache, batch, i, i, i]
    lib.sgemm_kv8_attend_workspace_size.restype = sz


def _lib():
    from . import load_library

    return load_library()


def sgemm_w4(*args) -> int:
    return _lib().sgemm_w4(*args)


def sgemm_w4_check_args(*args) -> int:
    return _lib().sgemm_w4_check_args(*args)


def sgemm_w4_quantize(*args) -> int:
    return _lib().sgemm_w4_quantize(*args)


def sgemm_w4_dequantize(*args) -> int:
    return _lib().sgemm_w4_dequantize(*args)


def sgemm_w4_pack_check_args(*args) -> int:
    return _lib().sgemm_w4_pack_check_args(*args)


def sgemm_kv8_write(*args) -> int:
    return _lib().sgemm_kv8_write(*args)


def sgemm_kv8_read(*args) -> int:
    return _lib().sgemm_kv8_read(*args)


def sgemm_kv8_check_args(*args) -> int:
    return _lib().sgemm_kv8_check_args(*args)


def sgemm_kv8_attend(*args) -> int:
    return _lib().sgemm_kv8_attend(*args)


def sgemm_kv8_attend_check_args(*args) -> int:
    return _lib().sgemm_kv8_attend_check_args(*args)


def sgemm_kv8_attend_workspace_size(*args) -> int:
    return int(_lib().sgemm_kv8_attend_workspace_size(*args))


# ------------------------------------------------------------ tensor helpers


_TYPES = None


def _types():
    global _TYPES
    if _TYPES is None:
        import torch

        _TYPES = {torch.float32: SGEMM_F32, torch.bfloat16: 1, torch.float16: 2}
    return _TYPES


def _type_code(dtype, name):
    code = _types().get(dtype)
    if code is None:
        raise TypeError(f"{name} must be float32, bfloat16 or float16, got {dtype}")
    return code


def _need(t, name, dim, dtypes, device=None):
    """t, if it is a GPU tensor of `dim` dimensions and one of `dtypes` on `device`."""
    import torch

    if not isinstance(t, torch.Tensor) or t.dim() != dim:
        raise TypeError(f"{name} must be a {dim}-D torch.Tensor")
    if dtypes is not None and t.dtype not in dtypes:
        raise TypeError(f"{name} must be one of {tuple(str(d) for d in dtypes)}, got {t.dtype}")
    if t.device.type != "cuda":
        raise ValueError(f"{name} must be on a GPU device")
    if device is not None and t.device != device:
        raise ValueError(f"{name} must be on {device}, is on {t.device}")
    return t


def _row_major(t, name):
    """Row stride of a 2-D tensor with unit column stride."""
    rows, cols = t.shape
    if cols > 1 and t.stride(1) != 1:
        raise ValueError(f"{name} must be row-major (unit column stride)")
    ld = t.stride(0) if rows > 1 else max(cols, 1)
    if rows > 1 and ld < cols:
        raise ValueError(f"{name}'s rows overlap (strides {tuple(t.stride())})")
    return max(ld, 1)


def _heads(t, name):
    """Row and head strides of a rows x heads x dim tensor with unit last stride."""
    if t.shape[2] > 1 and t.stride(2) != 1:
        raise ValueError(f"{name}'s components must be adjacent (unit last stride)")
    rows, heads, dim = t.shape
    hs = t.stride(1) if heads > 1 else dim
    ld = t.stride(0) if rows > 1 else max(heads * dim, 1)
    return ld, hs


def _launch(device, call):
    """call(stream) with `device` current, raising on a status."""
    import torch

    from . import SGEMM_OK, SgemmError

    if torch.cuda.current_device() == device.index:
        rc = call(torch.cuda.current_stream(device).cuda_stream or None)
    else:
        with torch.cuda.device(device):
            rc = call(torch.cuda.current_stream(device).cuda_stream or None)
    if rc != SGEMM_OK:
        raise SgemmError(rc)


def _int32(**sizes):
    from . import _check_int32

    _check_int32(**sizes)


class W4:
    """An N x K matrix held in 4 bits: ``codes`` (uint8, N x ceil(K / 2), the
    lower half of a byte first), ``scales`` (float32, bfloat16 or float16, N x
    ceil(K / group)), ``zeros`` (uint8, the same shape, or None: 8
    everywhere), and ``K`` and ``group``. Its value is
    ``scales * (code - zeros)``. Tensors are used in place, without a copy."""

    __slots__ = ("codes", "scales", "zeros", "K", "group")

    def __init__(self, codes, scales, zeros, K, group):
        import torch

        K, group = int(K), int(group)
        if group <= 0 or group % 32:
            raise ValueError(f"group must be a positive multiple of 32, got {group}")
        _need(codes, "codes", 2, (torch.uint8,))
        _need(scales, "scales", 2, tuple(_types()), codes.device)
        groups = -(-K // group)
        if codes.shape[1] != -(-K // 2):
            raise ValueError(f"codes must have ceil(K / 2) = {-(-K // 2)} columns, has {codes.shape[1]}")
        if tuple(scales.shape) != (codes.shape[0], groups):
            raise ValueError(f"scales must be {codes.shape[0]} x {groups}, is {tuple(scales.shape)}")
        if zeros is not None:
            _need(zeros, "zeros", 2, (torch.uint8,), codes.device)
            if zeros.shape != scales.shape:
                raise ValueError(f"zeros must be {tuple(scales.shape)}, is {tuple(zeros.shape)}")
        for name, t in (("codes", codes), ("scales", scales), ("zeros", zeros)):
            if t is not None:
                _row_major(t, name)
        self.codes, self.scales, self.zeros, self.K, self.group = codes, scales, zeros, K, group

    @property
    def shape(self):
        return (self.codes.shape[0], self.K)

    @property
    def device(self):
        return self.codes.device

    def _args(self):
        z = self.zeros
        return (self.codes.data_ptr() or None, _row_major(self.codes, "codes"), self.scales.data_ptr() or None,
                _row_major(self.scales, "scales"), None if z is None else z.data_ptr() or None,
                1 if z is None else _row_major(z, "zeros"))


def quantize_w4(W, group=128, zeros=False, scale_dtype=None):
    """The N x K matrix W (float32, bfloat16 or float16, row-major, on a GPU)
    in the W4 form, one scale (of ``scale_dtype``, W's type by default) and,
    with ``zeros``, one zero point for each ``group`` elements of a row."""
    import torch

    _need(W, "W", 2, tuple(_types()))
    scale_dtype = W.dtype if scale_dtype is None else scale_dtype
    stype = _type_code(scale_dtype, "scale_dtype")
    group = int(group)
    if group <= 0 or group % 32:
        raise ValueError(f"group must be a positive multiple of 32, got {group}")
    N, K = W.shape
    ldb = _row_major(W, "W")
    groups = -(-K // group)
    out = W4(torch.empty((N, -(-K // 2)), dtype=torch.uint8, device=W.device),
             torch.empty((N, groups), dtype=scale_dtype, device=W.device),
             torch.empty((N, groups), dtype=torch.uint8, device=W.device) if zeros else None, K, group)
    _int32(N=N, K=K, group=group, ldb=ldb)
    _launch(W.device, lambda stream: _lib().sgemm_w4_quantize(_types()[W.dtype], stype, N, K, group, W.data_ptr() or None,
                                                              ldb, *out._args(), stream))
    return out


def dequantize_w4(W, dtype=None, out=None):
    """The N x K matrix that ``W`` stands for, in ``dtype`` (float32 by
    default) or into ``out`` (row-major)."""
    import torch

    if not isinstance(W, W4):
        raise TypeError("W must be a W4")
    N, K = W.shape
    if out is None:
        out = torch.empty((N, K), dtype=torch.float32 if dtype is None else dtype, device=W.device)
    elif dtype is not None and out.dtype != dtype:
        raise TypeError(f"out must be {dtype}, is {out.dtype}")
    _need(out, "out", 2, tuple(_types()), W.device)
    if tuple(out.shape) != (N, K):
        raise ValueError(f"out must be {N} x {K}, is {tuple(out.shape)}")
    ldb = _row_major(out, "out")
    _int32(N=N, K=K, ldb=ldb)
    _launch(W.device, lambda stream: _lib().sgemm_w4_dequantize(_types()[out.dtype], _types()[W.scales.dtype], N, K, W.group,
                                                                *W._args(), out.data_ptr() or None, ldb, stream))
    return out


def gemm_w4(A, W, C=None, alpha=1.0, beta=0.0):
    """C = alpha * A @ W^T + beta * C with A (M x K: float32, bfloat16 or
    float16, row-major), ``W`` an N x K :class:`W4` and C float32 (M x N).

    C is updated in place, read only when beta != 0, and allocated when None
    (then beta must be 0).
    """
    import torch

    if not isinstance(W, W4):
        raise TypeError("W must be a W4")
    _need(A, "A", 2, tuple(_types()), W.device)
    M, K = A.shape
    N = W.codes.shape[0]
    if K != W.K:
        raise ValueError(f"inner dimensions differ: {tuple(A.shape)} and {W.shape}")
    if C is None:
        if beta != 0.0:
            raise ValueError("beta != 0 needs C")
        C = torch.empty((M, N), dtype=torch.float32, device=A.device)
    else:
        _need(C, "C", 2, (torch.float32,), A.device)
        if tuple(C.shape) != (M, N):
            raise ValueError(f"C must be {M} x {N}, is {tuple(C.shape)}")
    lda, ldc = _row_major(A, "A"), _row_major(C, "C")
    _int32(M=M, N=N, K=K, group=W.group, lda=lda, ldc=ldc)
    _launch(A.device, lambda stream: _lib().sgemm_w4(_types()[A.dtype], _types()[W.scales.dtype], M, N, K, W.group,
                                                     float(alpha), A.data_ptr() or None, lda, *W._args(), float(beta),
                                                     C.data_ptr() or None, ldc, stream))
    return C


class KV8:
    """A paged cache of keys and values in 8-bit floats: ``K`` and ``V``
    (float8_e4m3fn, pages x heads x block x dim, contiguous) and ``Ks`` and
    ``Vs`` (float32, pages x heads), one scale for each page and head. The
    tensors are used in place. ``block`` is a power of two from 16 to 1024 and
    ``dim`` a multiple of 16 up to 256."""

    __slots__ = ("K", "V", "Ks", "Vs", "_struct")

    def __init__(self, K, V, Ks, Vs):
        import torch

        for name, t in (("K", K), ("V", V)):
            _need(t, name, 4, (torch.float8_e4m3fn,), K.device)
        for name, t in (("Ks", Ks), ("Vs", Vs)):
            _need(t, name, 2, (torch.float32,), K.device)
        if V.shape != K.shape or Ks.shape != K.shape[:2] or Vs.shape != K.shape[:2]:
            raise ValueError("V must have K's shape, Ks and Vs its first two dimensions")
        if not all(t.is_contiguous() for t in (K, V, Ks, Vs)):
            raise ValueError("K, V, Ks and Vs must be contiguous")
        pages, heads, block, dim = K.shape
        if block < 16 or block > 1024 or block & (block - 1):
            raise ValueError(f"block must be a power of two from 16 to 1024, is {block}")
        if dim < 16 or dim > 256 or dim % 16:
            raise ValueError(f"dim must be a multiple of 16 from 16 to 256, is {dim}")
        _int32(pages=pages, heads=heads)
        self.K, self.V, self.Ks, self.Vs = K, V, Ks, Vs
        self._struct = KV8Cache(K.data_ptr(), V.data_ptr(), Ks.data_ptr(), Vs.data_ptr(), pages, heads, block, dim)

    @staticmethod
    def empty(pages, heads, block, dim, device="cuda"):
        """A cache of zeros."""
        import torch

        codes = [torch.zeros((pages, heads, block, dim), dtype=torch.uint8, device=device).view(torch.float8_e4m3fn)
                 for _ in range(2)]
        return KV8(*codes, *[torch.zeros((pages, heads), dtype=torch.float32, device=device) for _ in range(2)])

    @property
    def device(self):
        return self.K.device


def _batch(cache, table, lens, starts, rows, max_new):
    import torch

    if not isinstance(cache, KV8):
        raise TypeError("cache must be a KV8")
    i32, device = (torch.int32,), cache.K.device
    _need(table, "table", 2, i32, device)
    _need(lens, "lens", 1, i32, device)
    _need(starts, "starts", 1, i32, device)
    seqs = lens.shape[0]
    if table.shape[0] != seqs or starts.shape[0] != seqs + 1:
        raise ValueError(f"{seqs} lens need a table of {seqs} rows and {seqs + 1} starts, got {table.shape[0]} and {starts.shape[0]}")
    if not (table.is_contiguous() and lens.is_contiguous() and starts.is_contiguous()):
        raise ValueError("table, lens and starts must be contiguous")
    max_new = rows if max_new is None else int(max_new)
    _int32(rows=rows, max_new=max_new, seqs=seqs, columns=table.shape[1])
    return KV8Batch(table.data_ptr() or None, lens.data_ptr() or None, starts.data_ptr() or None, seqs, table.shape[1], rows, max_new)


def _operand(t, name, cache, heads, dtypes):
    _need(t, name, 3, dtypes, cache.K.device)
    if t.shape[2] != cache.K.shape[3] or (heads is not None and t.shape[1] != heads):
        raise ValueError(f"{name} must be rows x {heads or 'heads'} x {cache.K.shape[3]}, is {tuple(t.shape)}")
    ld, hs = _heads(t, name)
    _int32(**{f"{name}'s row stride": ld, f"{name}'s head stride": hs})
    return ld, hs


def kv8_write(cache, K, V, table, lens, starts, max_new=None):
    """Quantises new keys and values (rows x heads x dim: float32, bfloat16 or
    float16) into ``cache``.

    Sequence b holds ``lens[b]`` tokens, the new ones among them; its rows
    ``starts[b] .. starts[b + 1] - 1`` are the last of them. Token t lives at
    place ``t % block`` of page ``table[b, t // block]``. table (sequences x
    columns), lens and starts are int32 GPU tensors. ``max_new`` says how many
    rows a sequence has at most (all rows by default): a wrong value costs
    time, not correctness.
    """
    if not isinstance(cache, KV8):
        raise TypeError("cache must be a KV8")
    heads = cache.K.shape[1]
    ldk, hsk = _operand(K, "K", cache, heads, tuple(_types()))
    ldv, hsv = _operand(V, "V", cache, heads, (K.dtype,))
    if V.shape[0] != K.shape[0]:
        raise ValueError(f"K and V must have the same rows, have {K.shape[0]} and {V.shape[0]}")
    batch = _batch(cache, table, lens, starts, K.shape[0], max_new)
    _launch(cache.K.device, lambda stream: _lib().sgemm_kv8_write(cache._struct, batch, _types()[K.dtype], K.data_ptr() or None,
                                                                  ldk, hsk, V.data_ptr() or None, ldv, hsv, stream))


def kv8_read(cache, table, lens, starts, rows=None, dtype=None, K=None, V=None, max_new=None):
    """The last ``starts[b + 1] - starts[b]`` tokens of each sequence read
    back: (K, V), each rows x heads x dim of ``dtype`` (float32 by default).
    Either ``rows`` (``starts[-1]``, known to the host) or both outputs have
    to be given."""
    import torch

    if not isinstance(cache, KV8):
        raise TypeError("cache must be a KV8")
    heads, dim = cache.K.shape[1], cache.K.shape[3]
    if (K is None) != (V is None) or (K is None and rows is None):
        raise ValueError("give rows, or both K and V")
    if K is None:
        dtype = torch.float32 if dtype is None else dtype
        _type_code(dtype, "dtype")
        K, V = (torch.empty((int(rows), heads, dim), dtype=dtype, device=cache.K.device) for _ in range(2))
    elif (rows is not None and K.shape[0] != rows) or (dtype is not None and K.dtype != dtype):
        raise ValueError("K is not of the rows and dtype asked for")
    ldk, hsk = _operand(K, "K", cache, heads, tuple(_types()))
    ldv, hsv = _operand(V, "V", cache, heads, (K.dtype,))
    if V.shape[0] != K.shape[0]:
        raise ValueError(f"K and V must have the same rows, have {K.shape[0]} and {V.shape[0]}")
    batch = _batch(cache, table, lens, starts, K.shape[0], max_new)
    _launch(cache.K.device, lambda stream: _lib().sgemm_kv8_read(cache._struct, batch, _types()[K.dtype], K.data_ptr() or None,
                                                                 ldk, hsk, V.data_ptr() or None, ldv, hsv, stream))
    return K, V


def kv8_attend(Q, cache, table, lens, starts, scale=None, causal=True, window=0, out=None, max_new=None, workspace=None):
    """Softmax attention of the queries Q (rows x query heads x dim: float32,
    bfloat16 or float16) over ``cache``: float32, Q's shape.

    Row i of a sequence's n rows stands at position ``lens[b] - n + i`` and
    sees the tokens up to it (``causal``), the last ``window`` of those
    (``window`` > 0), or all of the sequence (not ``causal``). Query heads are
    a multiple of the cache's heads; ``scale`` is 1 / sqrt(dim) by default.
    A row that sees nothing is zero; rows outside the sequences stay as they
    are in ``out``. table, lens, starts and ``max_new`` are as for
    :func:`kv8_write`. ``workspace`` (a contiguous tensor of
    sgemm_kv8_attend_workspace_size() bytes, used by one stream at a time) is
    allocated when None.
    """
    import torch

    if not isinstance(cache, KV8):
        raise TypeError("cache must be a KV8")
    ldq, hsq = _operand(Q, "Q", cache, None, tuple(_types()))
    rows, heads_q, dim = Q.shape
    if out is None:
        out = torch.empty((rows, heads_q, dim), dtype=torch.float32, device=Q.device)
    ldo, hso = _operand(out, "out", cache, heads_q, (torch.float32,))
    if out.shape[0] != rows:
        raise ValueError(f"out must have Q's shape {tuple(Q.shape)}, is {tuple(out.shape)}")
    window = int(window)
    _int32(window=window, heads_q=heads_q)
    batch = _batch(cache, table, lens, starts, rows, max_new)
    lib = _lib()
    if workspace is None:
        need = lib.sgemm_kv8_attend_workspace_size(cache._struct, batch, heads_q, window, _cus(Q.device))
        if need:
            workspace = torch.empty(need, dtype=torch.uint8, device=Q.device)
    elif not isinstance(workspace, torch.Tensor) or workspace.device != Q.device or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous tensor on Q's device")
    ws, ws_bytes = (None, 0) if workspace is None else (workspace.data_ptr() or None, workspace.numel() * workspace.element_size())
    _launch(Q.device, lambda stream: lib.sgemm_kv8_attend(
        cache._struct, batch, _types()[Q.dtype], heads_q, Q.data_ptr() or None, ldq, hsq,
        float(dim ** -0.5 if scale is None else scale), int(bool(causal)), window, out.data_ptr() or None, ldo, hso,
        ws, ws_bytes, stream))
    return out


_CUS = {}


def _cus(device):
    """Compute units of a device (a property of the hardware, asked once)."""
    import torch

    if device.index not in _CUS:
        _CUS[device.index] = torch.cuda.get_device_properties(device).multi_processor_count
    return _CUS[device.index]
