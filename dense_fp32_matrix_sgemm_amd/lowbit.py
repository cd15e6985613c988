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
           "sgemm_kv8_attend_check_args", "sgemm_kv8_attend_workspace_size", "sgemm_w4_shape", "sgemm_kv8_attend_shape")


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
    lib.sgemm_w4_shape.argtypes, lib.sgemm_w4_shape.restype = [i, i, i, i, i, ctypes.POINTER(i)], i
    lib.sgemm_kv8_attend_shape.argtypes = [cache, batch, i, i, i, ctypes.POINTER(i)]
    lib.sgemm_kv8_attend_shape.restype = i


_LIB = None


def _lib():
    global _LIB
    if _LIB is None:
        from . import load_library

        _LIB = load_library()
    return _LIB


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


def _shape(entry, size, *args) -> tuple:
    shape = (ctypes.c_int * size)()
    rc = entry(*args, shape)
    if rc:
        from . import SgemmError

        raise SgemmError(rc)
    return tuple(shape)


def sgemm_w4_shape(dtype, M, N, K, cus=0) -> tuple:
    """Rows and columns of a work-group, waves along N and K, slabs of A."""
    return _shape(_lib().sgemm_w4_shape, 5, dtype, M, N, K, cus)


def sgemm_kv8_attend_shape(cache, batch, heads_q, window=0, cus=0) -> tuple:
    """Rows of a wave's tile, row tiles of a work-group, work-groups along the rows, splits of the tokens."""
    return _shape(_lib().sgemm_kv8_attend_shape, 4, cache, batch, heads_q, window, cus)


# ------------------------------------------------------------ tensor helpers
#
# A serving program makes these calls once per layer and token, so the helpers
# stay short: what a W4 or a KV8 holds is checked and marshalled once, when it
# is made, and the device and stream are asked for as plain numbers.

_INT32_MAX = 2**31 - 1

_TYPES = None


def _types():
    """Type code of each element type."""
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
    """Checks that t is a GPU tensor of `dim` dimensions and one of `dtypes`, on `device`."""
    import torch

    if not isinstance(t, torch.Tensor) or t.dim() != dim:
        raise TypeError(f"{name} must be a {dim}-D torch.Tensor")
    if t.dtype not in dtypes:
        raise TypeError(f"{name} must be one of {tuple(str(d) for d in dtypes)}, got {t.dtype}")
    if not t.is_cuda:
        raise ValueError(f"{name} must be on a GPU device")
    if device is not None and t.device != device:
        raise ValueError(f"{name} must be on {device}, is on {t.device}")


def _row_major(t, name):
    """Row stride of a 2-D tensor with unit column stride."""
    rows, cols = t.shape
    ld, step = t.stride()
    if step != 1 and cols > 1:
        raise ValueError(f"{name} must be row-major (unit column stride)")
    if rows <= 1:
        return cols or 1
    if ld < cols:
        raise ValueError(f"{name}'s rows overlap (strides {(ld, step)})")
    return ld or 1


def _heads(t, name):
    """Row and head strides of a rows x heads x dim tensor with unit last stride."""
    rows, heads, dim = t.shape
    ld, hs, step = t.stride()
    if step != 1 and dim > 1:
        raise ValueError(f"{name}'s components must be adjacent (unit last stride)")
    if heads <= 1:
        hs = dim
    if rows <= 1:
        ld = heads * dim or 1
    if ld > _INT32_MAX or hs > _INT32_MAX:
        _int32(**{f"{name}'s row stride": ld, f"{name}'s head stride": hs})
    return ld, hs


def _launch(index, entry, *args):
    """entry(*args, stream) with device `index` current, on its current stream; raises on a status."""
    import torch

    if torch._C._cuda_getDevice() == index:
        rc = entry(*args, torch._C._cuda_getCurrentRawStream(index))
    else:
        with torch.cuda.device(index):
            rc = entry(*args, torch._C._cuda_getCurrentRawStream(index))
    if rc:
        from . import SgemmError

        raise SgemmError(rc)


def _int32(**sizes):
    from . import _check_int32

    _check_int32(**sizes)


class W4:
    """An N x K matrix held in 4 bits: ``codes`` (uint8, N x ceil(K / 2), the
    lower half of a byte first), ``scales`` (float32, bfloat16 or float16, N x
    ceil(K / group)), ``zeros`` (uint8, the same shape, or None: 8
    everywhere), and ``K`` and ``group``. Its value is
    ``scales * (code - zeros)``. The tensors are used in place, without a
    copy, and belong to the W4 for good (what they hold may change)."""

    __slots__ = ("_codes", "_scales", "_zeros", "_shape", "_group", "_stype", "_args", "_device")

    def __init__(self, codes, scales, zeros, K, group):
        import torch

        K, group = int(K), int(group)
        if group <= 0 or group % 32:
            raise ValueError(f"group must be a positive multiple of 32, got {group}")
        _need(codes, "codes", 2, (torch.uint8,))
        _need(scales, "scales", 2, _types(), codes.device)
        N, groups = codes.shape[0], -(-K // group)
        if K < 0 or codes.shape[1] != -(-K // 2):
            raise ValueError(f"codes must have ceil(K / 2) = {-(-K // 2)} columns, has {codes.shape[1]}")
        if tuple(scales.shape) != (N, groups):
            raise ValueError(f"scales must be {N} x {groups}, is {tuple(scales.shape)}")
        if zeros is not None:
            _need(zeros, "zeros", 2, (torch.uint8,), codes.device)
            if zeros.shape != scales.shape:
                raise ValueError(f"zeros must be {tuple(scales.shape)}, is {tuple(zeros.shape)}")
        ldw, lds = _row_major(codes, "codes"), _row_major(scales, "scales")
        ldz = 1 if zeros is None else _row_major(zeros, "zeros")
        _int32(N=N, K=K, group=group, ldw=ldw, lds=lds, ldz=ldz)
        self._codes, self._scales, self._zeros, self._shape, self._group = codes, scales, zeros, (N, K), group
        self._device, self._stype = codes.device, _types()[scales.dtype]
        self._args = (codes.data_ptr() or None, ldw, scales.data_ptr() or None, lds,
                      None if zeros is None else zeros.data_ptr() or None, ldz)

    codes = property(lambda self: self._codes)
    scales = property(lambda self: self._scales)
    zeros = property(lambda self: self._zeros)
    shape = property(lambda self: self._shape)
    K = property(lambda self: self._shape[1])
    group = property(lambda self: self._group)
    device = property(lambda self: self._device)


def quantize_w4(W, group=128, zeros=False, scale_dtype=None):
    """The N x K matrix W (float32, bfloat16 or float16, row-major, on a GPU)
    in the W4 form, one scale (of ``scale_dtype``, W's type by default) and,
    with ``zeros``, one zero point for each ``group`` elements of a row."""
    import torch

    _need(W, "W", 2, _types())
    scale_dtype = W.dtype if scale_dtype is None else scale_dtype
    _type_code(scale_dtype, "scale_dtype")
    group = int(group)
    if group <= 0 or group % 32:
        raise ValueError(f"group must be a positive multiple of 32, got {group}")
    N, K = W.shape
    ldb = _row_major(W, "W")
    _int32(N=N, K=K, group=group, ldb=ldb)
    groups, device = -(-K // group), W.device
    out = W4(torch.empty((N, -(-K // 2)), dtype=torch.uint8, device=device),
             torch.empty((N, groups), dtype=scale_dtype, device=device),
             torch.empty((N, groups), dtype=torch.uint8, device=device) if zeros else None, K, group)
    _launch(device.index, _lib().sgemm_w4_quantize, _types()[W.dtype], out._stype, N, K, group, W.data_ptr() or None, ldb,
            *out._args)
    return out


def dequantize_w4(W, dtype=None, out=None):
    """The N x K matrix that ``W`` stands for, in ``dtype`` (float32 by
    default) or into ``out`` (row-major)."""
    import torch

    if not isinstance(W, W4):
        raise TypeError("W must be a W4")
    if out is None:
        dtype = torch.float32 if dtype is None else dtype
        _type_code(dtype, "dtype")
        out = torch.empty(W._shape, dtype=dtype, device=W._device)
    elif dtype is not None and out.dtype != dtype:
        raise TypeError(f"out must be {dtype}, is {out.dtype}")
    _need(out, "out", 2, _types(), W._device)
    N, K = W._shape
    if tuple(out.shape) != (N, K):
        raise ValueError(f"out must be {N} x {K}, is {tuple(out.shape)}")
    ldb = _row_major(out, "out")
    if ldb > _INT32_MAX:
        _int32(ldb=ldb)
    _launch(W._device.index, _lib().sgemm_w4_dequantize, _types()[out.dtype], W._stype, N, K, W._group, *W._args,
            out.data_ptr() or None, ldb)
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
    _need(A, "A", 2, _types(), W._device)
    M, K = A.shape
    N = W._shape[0]
    if K != W._shape[1]:
        raise ValueError(f"inner dimensions differ: {tuple(A.shape)} and {W._shape}")
    if C is None:
        if beta != 0.0:
            raise ValueError("beta != 0 needs C")
        C = torch.empty((M, N), dtype=torch.float32, device=W._device)
    else:
        _need(C, "C", 2, (torch.float32,), W._device)
        if tuple(C.shape) != (M, N):
            raise ValueError(f"C must be {M} x {N}, is {tuple(C.shape)}")
    lda, ldc = _row_major(A, "A"), _row_major(C, "C")
    if M > _INT32_MAX or lda > _INT32_MAX or ldc > _INT32_MAX:
        _int32(M=M, lda=lda, ldc=ldc)
    _launch(W._device.index, _lib().sgemm_w4, _types()[A.dtype], W._stype, M, N, K, W._group, alpha, A.data_ptr() or None,
            lda, *W._args, beta, C.data_ptr() or None, ldc)
    return C


class KV8:
    """A paged cache of keys and values in 8-bit floats: ``K`` and ``V``
    (float8_e4m3fn, pages x heads x block x dim, contiguous) and ``Ks`` and
    ``Vs`` (float32, pages x heads), one scale for each page and head. The
    tensors are used in place and belong to the KV8 for good (what they hold
    may change). ``block`` is a power of two from 16 to 1024 and ``dim`` a
    multiple of 16 up to 256. K and V may be one tensor (so may Ks and Vs) to
    read and attend, but not for :func:`kv8_write`."""

    __slots__ = ("_tensors", "_struct", "_device", "_heads", "_dim")

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
        if pages < 1 or heads < 1:
            raise ValueError("a cache needs a page and a head")
        if block < 16 or block > 1024 or block & (block - 1):
            raise ValueError(f"block must be a power of two from 16 to 1024, is {block}")
        if dim < 16 or dim > 256 or dim % 16:
            raise ValueError(f"dim must be a multiple of 16 from 16 to 256, is {dim}")
        _int32(pages=pages, heads=heads)
        self._tensors, self._device, self._heads, self._dim = (K, V, Ks, Vs), K.device, heads, dim
        self._struct = KV8Cache(K.data_ptr(), V.data_ptr(), Ks.data_ptr(), Vs.data_ptr(), pages, heads, block, dim)

    K = property(lambda self: self._tensors[0])
    V = property(lambda self: self._tensors[1])
    Ks = property(lambda self: self._tensors[2])
    Vs = property(lambda self: self._tensors[3])
    device = property(lambda self: self._device)

    @staticmethod
    def empty(pages, heads, block, dim, device="cuda"):
        """A cache of zeros."""
        import torch

        codes = [torch.zeros((pages, heads, block, dim), dtype=torch.uint8, device=device).view(torch.float8_e4m3fn)
                 for _ in range(2)]
        return KV8(*codes, *[torch.zeros((pages, heads), dtype=torch.float32, device=device) for _ in range(2)])


def _batch(cache, table, lens, starts, rows, max_new):
    import torch

    i32, device = (torch.int32,), cache._device
    _need(table, "table", 2, i32, device)
    _need(lens, "lens", 1, i32, device)
    _need(starts, "starts", 1, i32, device)
    seqs, columns = table.shape
    if lens.shape[0] != seqs or starts.shape[0] != seqs + 1:
        raise ValueError(f"a table of {seqs} rows needs {seqs} lens and {seqs + 1} starts, got {lens.shape[0]} and {starts.shape[0]}")
    if not (table.is_contiguous() and lens.is_contiguous() and starts.is_contiguous()):
        raise ValueError("table, lens and starts must be contiguous")
    max_new = rows if max_new is None else int(max_new)
    if not 0 <= max_new <= _INT32_MAX or rows > _INT32_MAX or seqs > _INT32_MAX or columns > _INT32_MAX:
        _int32(rows=rows, max_new=max_new, seqs=seqs, columns=columns)
    return KV8Batch(table.data_ptr() or None, lens.data_ptr() or None, starts.data_ptr() or None, seqs, columns, rows, max_new)


def _operand(t, name, cache, heads, dtypes):
    _need(t, name, 3, dtypes, cache._device)
    if t.shape[2] != cache._dim or (heads is not None and t.shape[1] != heads):
        raise ValueError(f"{name} must be rows x {heads or 'heads'} x {cache._dim}, is {tuple(t.shape)}")
    return _heads(t, name)


def _pair(cache, K, V):
    """Strides of K and V, rows x heads x dim of one type."""
    ldk, hsk = _operand(K, "K", cache, cache._heads, _types())
    ldv, hsv = _operand(V, "V", cache, cache._heads, (K.dtype,))
    if V.shape[0] != K.shape[0]:
        raise ValueError(f"K and V must have the same rows, have {K.shape[0]} and {V.shape[0]}")
    return _types()[K.dtype], K.data_ptr() or None, ldk, hsk, V.data_ptr() or None, ldv, hsv


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
    operand = _pair(cache, K, V)
    batch = _batch(cache, table, lens, starts, K.shape[0], max_new)
    _launch(cache._device.index, _lib().sgemm_kv8_write, cache._struct, batch, *operand)


def kv8_read(cache, table, lens, starts, rows=None, dtype=None, K=None, V=None, max_new=None):
    """The last ``starts[b + 1] - starts[b]`` tokens of each sequence read
    back: (K, V), each rows x heads x dim of ``dtype`` (float32 by default).
    Either ``rows`` (``starts[-1]``, known to the host) or both outputs have
    to be given. Rows outside the sequences, and rows before token 0, stay as
    they are in given outputs; in new ones they hold whatever was in the
    memory."""
    import torch

    if not isinstance(cache, KV8):
        raise TypeError("cache must be a KV8")
    if (K is None) != (V is None) or (K is None and rows is None):
        raise ValueError("give rows, or both K and V")
    if K is None:
        dtype = torch.float32 if dtype is None else dtype
        _type_code(dtype, "dtype")
        shape = (int(rows), cache._heads, cache._dim)
        K, V = torch.empty(shape, dtype=dtype, device=cache._device), torch.empty(shape, dtype=dtype, device=cache._device)
    operand = _pair(cache, K, V)
    if (rows is not None and K.shape[0] != rows) or (dtype is not None and K.dtype != dtype):
        raise ValueError("K is not of the rows and dtype asked for")
    batch = _batch(cache, table, lens, starts, K.shape[0], max_new)
    _launch(cache._device.index, _lib().sgemm_kv8_read, cache._struct, batch, *operand)
    return K, V


def kv8_attend(Q, cache, table, lens, starts, scale=None, causal=True, window=0, out=None, max_new=None, workspace=None):
    """Softmax attention of the queries Q (rows x query heads x dim: float32,
    bfloat16 or float16) over ``cache``: float32, Q's shape.

    Row i of a sequence's n rows stands at position ``lens[b] - n + i`` and
    sees the tokens up to it (``causal``), the last ``window`` of those
    (``window`` > 0), or all of the sequence (not ``causal``). Query heads are
    a multiple of the cache's heads; ``scale`` is 1 / sqrt(dim) by default.
    A row that sees nothing is zero. Rows outside the sequences (a batch
    padded behind ``starts[-1]``) stay as they are in ``out``; in a new output
    they hold whatever was in the memory. table, lens, starts and ``max_new`` are as for
    :func:`kv8_write`. ``workspace`` (a contiguous tensor of
    sgemm_kv8_attend_workspace_size() bytes, used by one stream at a time) is
    allocated when None.
    """
    import torch

    if not isinstance(cache, KV8):
        raise TypeError("cache must be a KV8")
    ldq, hsq = _operand(Q, "Q", cache, None, _types())
    rows, heads_q, dim = Q.shape
    if out is None:
        out = torch.empty((rows, heads_q, dim), dtype=torch.float32, device=cache._device)
    ldo, hso = _operand(out, "out", cache, heads_q, (torch.float32,))
    if out.shape[0] != rows:
        raise ValueError(f"out must have Q's shape {tuple(Q.shape)}, is {tuple(out.shape)}")
    if not 0 <= window <= _INT32_MAX or heads_q > _INT32_MAX:
        _int32(window=window, heads_q=heads_q)
    batch = _batch(cache, table, lens, starts, rows, max_new)
    lib = _lib()
    ws, ws_bytes = None, 0
    if workspace is None:
        ws_bytes = lib.sgemm_kv8_attend_workspace_size(cache._struct, batch, heads_q, window, _cus(cache._device))
        if ws_bytes:
            workspace = torch.empty(ws_bytes, dtype=torch.uint8, device=cache._device)
            ws = workspace.data_ptr()
    elif not isinstance(workspace, torch.Tensor) or workspace.device != cache._device or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous tensor on Q's device")
    else:
        ws, ws_bytes = workspace.data_ptr() or None, workspace.numel() * workspace.element_size()
    _launch(cache._device.index, lib.sgemm_kv8_attend, cache._struct, batch, _types()[Q.dtype], heads_q, Q.data_ptr() or None,
            ldq, hsq, dim**-0.5 if scale is None else scale, 1 if causal else 0, window, out.data_ptr() or None, ldo, hso, ws,
            ws_bytes)
    return out


_CUS = {}


def _cus(device):
    """Compute units of a device (a property of the hardware, asked once)."""
    import torch

    if device.index not in _CUS:
        _CUS[device.index] = torch.cuda.get_device_properties(device).multi_processor_count
    return _CUS[device.index]
