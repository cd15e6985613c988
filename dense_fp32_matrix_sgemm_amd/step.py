"""A serving step over a paged cache: the binding of ``sgemm_kv4*`` (a cache of
keys and values held in 4 bits, attention over it), ``sgemm_rope`` (rotary
positions) and ``sgemm_kv_tables`` (page tables from lengths), and their tensor
helpers.

Like the rest of the binding it only marshals arguments: the kernels are
enqueued on the current stream of the operands' device, nothing waits, and a
refused argument raises. Of the helpers :func:`rope` alone has a gradient.
The raw entry points take the C ABI's arguments in its order; ``cache``,
``batch`` and ``step`` are :class:`KV4Cache`, ``KV8Batch`` and
:class:`KVStep` structures, ``first`` and ``second`` :class:`RopeRows`.
"""

from __future__ import annotations

import ctypes
import math

from . import lowbit
from .lowbit import _INT32_MAX, KV8Batch, _cus, _heads, _int32, _launch, _lib, _need, _shape, _type_code, _types

EXPORTS = ("sgemm_kv4_write", "sgemm_kv4_read", "sgemm_kv4_check_args", "sgemm_kv4_attend", "sgemm_kv4_attend_check_args",
           "sgemm_kv4_attend_workspace_size", "sgemm_kv4_attend_shape", "sgemm_rope", "sgemm_rope_check_args",
           "sgemm_kv_tables", "sgemm_kv_tables_check_args")


class KV4Cache(ctypes.Structure):
    """sgemm_kv4_cache."""

    _fields_ = [("K", ctypes.c_void_p), ("V", ctypes.c_void_p), ("Ks", ctypes.c_void_p), ("Vs", ctypes.c_void_p),
                ("pages", ctypes.c_int), ("heads", ctypes.c_int), ("block", ctypes.c_int), ("dim", ctypes.c_int)]


class RopeRows(ctypes.Structure):
    """sgemm_rope_rows."""

    _fields_ = [("X", ctypes.c_void_p), ("Y", ctypes.c_void_p), ("heads", ctypes.c_int), ("ldx", ctypes.c_int),
                ("hsx", ctypes.c_int), ("ldy", ctypes.c_int), ("hsy", ctypes.c_int)]


class KVStep(ctypes.Structure):
    """sgemm_kv_step."""

    _fields_ = [(n, ctypes.c_void_p) for n in ("lens", "news", "pool", "taken", "table", "starts", "positions", "slots", "taken_after")] + \
               [(n, ctypes.c_int) for n in ("seqs", "table_ld", "block", "pool_size", "rows")]


def declare(lib) -> None:
    """Argument and result types of this module's entry points."""
    i, f, vp, sz = ctypes.c_int, ctypes.c_float, ctypes.c_void_p, ctypes.c_size_t
    cache, batch, rope, step = (ctypes.POINTER(t) for t in (KV4Cache, KV8Batch, RopeRows, KVStep))
    rows = [cache, batch, i, vp, i, i, vp, i, i]
    attend = [cache, batch, i, i, vp, i, i, f, i, i, vp, i, i, vp, sz]
    turn = [i, i, i, i, i, i, i, f, vp, vp, rope, rope]
    for name, args, result in (
            ("sgemm_kv4_write", rows + [vp], i), ("sgemm_kv4_read", rows + [vp], i), ("sgemm_kv4_check_args", rows, i),
            ("sgemm_kv4_attend", attend + [vp], i), ("sgemm_kv4_attend_check_args", attend, i),
            ("sgemm_kv4_attend_workspace_size", [cache, batch, i, i, i], sz),
            ("sgemm_kv4_attend_shape", [cache, batch, i, i, i, ctypes.POINTER(i)], i),
            ("sgemm_rope", turn + [vp], i), ("sgemm_rope_check_args", turn, i),
            ("sgemm_kv_tables", [step, vp], i), ("sgemm_kv_tables_check_args", [step], i)):
        entry = getattr(lib, name)
        entry.argtypes, entry.restype = args, result


def sgemm_kv4_write(*args) -> int:
    return _lib().sgemm_kv4_write(*args)


def sgemm_kv4_read(*args) -> int:
    return _lib().sgemm_kv4_read(*args)


def sgemm_kv4_check_args(*args) -> int:
    return _lib().sgemm_kv4_check_args(*args)


def sgemm_kv4_attend(*args) -> int:
    return _lib().sgemm_kv4_attend(*args)


def sgemm_kv4_attend_check_args(*args) -> int:
    return _lib().sgemm_kv4_attend_check_args(*args)


def sgemm_kv4_attend_workspace_size(*args) -> int:
    return int(_lib().sgemm_kv4_attend_workspace_size(*args))


def sgemm_kv4_attend_shape(cache, batch, heads_q, window=0, cus=0) -> tuple:
    """Rows of a wave's tile, row tiles of a work-group, work-groups along the rows, work-groups that share out the tokens of all sequences (0: none do)."""
    return _shape(_lib().sgemm_kv4_attend_shape, 4, cache, batch, heads_q, window, cus)


def sgemm_rope(*args) -> int:
    return _lib().sgemm_rope(*args)


def sgemm_rope_check_args(*args) -> int:
    return _lib().sgemm_rope_check_args(*args)


def sgemm_kv_tables(*args) -> int:
    return _lib().sgemm_kv_tables(*args)


def sgemm_kv_tables_check_args(*args) -> int:
    return _lib().sgemm_kv_tables_check_args(*args)


# ------------------------------------------------------------ tensor helpers
#
# A serving program makes these calls once per layer and token. The usual
# operands are therefore checked in as few steps as tell that nothing is wrong
# with them; all others go through the checks that say what is.


def _batch(cache, table, lens, starts, rows, max_new):
    """The sequences of a call over `cache`."""
    try:
        seqs, columns = table.shape
        i32, index = table.dtype, cache._index
        if (lens.dtype is i32 and starts.dtype is i32 and i32 is cache._i32 and table.get_device() == index
                and lens.get_device() == index and starts.get_device() == index and lens.shape == (seqs,)
                and starts.shape == (seqs + 1,) and table.is_contiguous() and lens.is_contiguous() and starts.is_contiguous()
                and columns <= _INT32_MAX and 0 <= (rows if max_new is None else max_new) <= _INT32_MAX and rows <= _INT32_MAX):
            return KV8Batch(table.data_ptr() or None, lens.data_ptr() or None, starts.data_ptr() or None, seqs, columns, rows,
                            rows if max_new is None else int(max_new))
    except (AttributeError, TypeError, ValueError):
        pass
    return lowbit._batch(cache, table, lens, starts, rows, max_new)


def _usual(t, index, heads, dim):
    """Row and head strides of a rows x heads x dim tensor on device `index`, or None if it is not one as usual."""
    try:
        rows, h, d = t.shape
        if h == heads and d == dim and t.get_device() == index:
            ld, hs, step = t.stride()
            if step == 1 and ld <= _INT32_MAX and hs <= _INT32_MAX:
                return (ld if rows > 1 else heads * dim or 1), (hs if heads > 1 else dim)
    except (AttributeError, TypeError, ValueError):
        pass
    return None


def _like(t, dtype):
    """A new contiguous tensor of t's shape and device."""
    import torch

    if t.dtype is dtype and t.is_contiguous():
        return torch.empty_like(t)
    return torch.empty(t.shape, dtype=dtype, device=t.device)


def _pair(cache, K, V):
    """Type, places and strides of K and V, rows x heads x dim of one type."""
    k, v = _usual(K, cache._index, cache._heads, cache._dim), _usual(V, cache._index, cache._heads, cache._dim)
    if k is not None and v is not None and K.dtype is V.dtype and K.shape[0] == V.shape[0]:
        code = _types().get(K.dtype)
        if code is not None:
            return code, K.data_ptr() or None, *k, V.data_ptr() or None, *v
    return lowbit._pair(cache, K, V)


def _operand(t, name, cache, heads, dtypes):
    """Row and head strides of a rows x heads x dim tensor of one of `dtypes`."""
    strides = _usual(t, cache._index, heads, cache._dim) if heads is not None else None
    if strides is not None and t.dtype in dtypes:
        return strides
    return lowbit._operand(t, name, cache, heads, dtypes)


class KV4:
    """A paged cache of keys and values in 4-bit floats: ``K`` and ``V``
    (uint8, pages x heads x block x dim / 2, contiguous, the lower half of a
    byte first) and ``Ks`` and ``Vs`` (bfloat16, pages x heads x block), one
    scale for each token and head. A code's lower three bits stand for 0, 0.5,
    1, 1.5, 2, 3, 4, 6, its upper one for the sign. The tensors are used in
    place and belong to the KV4 for good (what they hold may change).
    ``block`` is a power of two from 16 to 1024 and ``dim`` a multiple of 16 up
    to 256. K and V may be one tensor (so may Ks and Vs) to read and attend,
    but not for :func:`kv4_write`."""

    __slots__ = ("_tensors", "_struct", "_device", "_index", "_i32", "_cus", "_heads", "_dim")

    def __init__(self, K, V, Ks, Vs):
        import torch

        for name, t in (("K", K), ("V", V)):
            _need(t, name, 4, (torch.uint8,), K.device)
        for name, t in (("Ks", Ks), ("Vs", Vs)):
            _need(t, name, 3, (torch.bfloat16,), K.device)
        if V.shape != K.shape or Ks.shape != K.shape[:3] or Vs.shape != K.shape[:3]:
            raise ValueError("V must have K's shape, Ks and Vs its first three dimensions")
        if not all(t.is_contiguous() for t in (K, V, Ks, Vs)):
            raise ValueError("K, V, Ks and Vs must be contiguous")
        pages, heads, block, half = K.shape
        dim = 2 * half
        if pages < 1 or heads < 1:
            raise ValueError("a cache needs a page and a head")
        if block < 16 or block > 1024 or block & (block - 1):
            raise ValueError(f"block must be a power of two from 16 to 1024, is {block}")
        if dim < 16 or dim > 256 or dim % 16:
            raise ValueError(f"dim must be a multiple of 16 from 16 to 256, is {dim}")
        if any(t.data_ptr() % 16 for t in (K, V, Ks, Vs)):
            raise ValueError("K, V, Ks and Vs must begin at a multiple of 16 bytes")
        _int32(pages=pages, heads=heads)
        self._tensors, self._device, self._heads, self._dim = (K, V, Ks, Vs), K.device, heads, dim
        self._index, self._i32, self._cus = K.get_device(), torch.int32, _cus(K.device)
        self._struct = KV4Cache(K.data_ptr(), V.data_ptr(), Ks.data_ptr(), Vs.data_ptr(), pages, heads, block, dim)

    K = property(lambda self: self._tensors[0])
    V = property(lambda self: self._tensors[1])
    Ks = property(lambda self: self._tensors[2])
    Vs = property(lambda self: self._tensors[3])
    device = property(lambda self: self._device)

    @staticmethod
    def empty(pages, heads, block, dim, device="cuda"):
        """A cache of zeros."""
        import torch

        if dim % 2:
            raise ValueError(f"dim must be a multiple of 16 from 16 to 256, is {dim}")
        codes = [torch.zeros((pages, heads, block, dim // 2), dtype=torch.uint8, device=device) for _ in range(2)]
        return KV4(*codes, *[torch.zeros((pages, heads, block), dtype=torch.bfloat16, device=device) for _ in range(2)])


def kv4_write(cache, K, V, table, lens, starts, max_new=None):
    """Quantises new keys and values (rows x heads x dim: float32, bfloat16 or
    float16) into ``cache``. The sequences, their rows and ``max_new`` are as
    for :func:`kv8_write`; earlier tokens keep what they hold."""
    if not isinstance(cache, KV4):
        raise TypeError("cache must be a KV4")
    operand = _pair(cache, K, V)
    batch = _batch(cache, table, lens, starts, K.shape[0], max_new)
    _launch(cache._device.index, _lib().sgemm_kv4_write, cache._struct, batch, *operand)


def kv4_read(cache, table, lens, starts, rows=None, dtype=None, K=None, V=None, max_new=None):
    """The last ``starts[b + 1] - starts[b]`` tokens of each sequence read
    back: (K, V), each rows x heads x dim of ``dtype`` (float32 by default), as
    :func:`kv8_read` does from a KV8. Either ``rows`` (``starts[-1]``, known to
    the host) or both outputs have to be given. Rows outside the sequences, and
    rows before token 0, stay as they are in given outputs; in new ones they
    hold whatever was in the memory."""
    import torch

    if not isinstance(cache, KV4):
        raise TypeError("cache must be a KV4")
    if (K is None) != (V is None) or (K is None and rows is None):
        raise ValueError("give rows, or both K and V")
    if K is None:
        dtype = torch.float32 if dtype is None else dtype
        _type_code(dtype, "dtype")
        K = torch.empty((int(rows), cache._heads, cache._dim), dtype=dtype, device=cache._device)
        V = torch.empty_like(K)
    operand = _pair(cache, K, V)
    if (rows is not None and K.shape[0] != rows) or (dtype is not None and K.dtype != dtype):
        raise ValueError("K is not of the rows and dtype asked for")
    batch = _batch(cache, table, lens, starts, K.shape[0], max_new)
    _launch(cache._device.index, _lib().sgemm_kv4_read, cache._struct, batch, *operand)
    return K, V


def kv4_attend(Q, cache, table, lens, starts, scale=None, causal=True, window=0, out=None, max_new=None, workspace=None):
    """Softmax attention of the queries Q (rows x query heads x dim: float32,
    bfloat16 or float16) over a :class:`KV4`: float32, Q's shape. Rows, masks,
    query heads, ``out`` and ``max_new`` are as for :func:`kv8_attend`;
    ``workspace`` (a contiguous tensor of sgemm_kv4_attend_workspace_size()
    bytes, used by one stream at a time) is allocated when None."""
    import torch

    if not isinstance(cache, KV4):
        raise TypeError("cache must be a KV4")
    heads_q = Q.shape[1] if isinstance(Q, torch.Tensor) and Q.dim() == 3 else None
    ldq, hsq = _operand(Q, "Q", cache, heads_q, _types())
    rows, heads_q, dim = Q.shape
    if out is None:
        out = _like(Q, torch.float32)
        ldo, hso = heads_q * dim or 1, dim
    else:
        ldo, hso = _operand(out, "out", cache, heads_q, (torch.float32,))
        if out.shape[0] != rows:
            raise ValueError(f"out must have Q's shape {tuple(Q.shape)}, is {tuple(out.shape)}")
    if not 0 <= window <= _INT32_MAX or heads_q > _INT32_MAX:
        _int32(window=window, heads_q=heads_q)
    batch = _batch(cache, table, lens, starts, rows, max_new)
    lib = _lib()
    ws, ws_bytes = None, 0
    if workspace is None:
        ws_bytes = lib.sgemm_kv4_attend_workspace_size(cache._struct, batch, heads_q, window, cache._cus)
        if ws_bytes:
            workspace = torch.empty(ws_bytes, dtype=torch.uint8, device=cache._device)
            ws = workspace.data_ptr()
    elif not isinstance(workspace, torch.Tensor) or workspace.device != cache._device or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous tensor on Q's device")
    else:
        ws, ws_bytes = workspace.data_ptr() or None, workspace.numel() * workspace.element_size()
    _launch(cache._device.index, lib.sgemm_kv4_attend, cache._struct, batch, _types()[Q.dtype], heads_q, Q.data_ptr() or None,
            ldq, hsq, dim**-0.5 if scale is None else scale, 1 if causal else 0, window, out.data_ptr() or None, ldo, hso, ws,
            ws_bytes)
    return out


def rope_frequencies(rot, base=10000.0, stretch=1.0, original=None, device="cuda"):
    """(freqs, amplitude) for :func:`rope`: radians a position that each of the
    rot / 2 pairs turns by, ``base ** (-2 i / rot)``, as a float64 tensor.

    ``stretch`` > 1 is for contexts that many times as long as the model's
    own. Without ``original`` every frequency is divided by it. With
    ``original`` (the tokens of the model's own context) pairs that turn at
    least 32 times within it keep their frequency, those that turn at most once
    have it divided, those between are blended by their turns, and amplitude is
    0.1 log(stretch) + 1 instead of 1.
    """
    import torch

    rot = int(rot)
    if rot < 2 or rot % 2:
        raise ValueError(f"rot must be positive and even, is {rot}")
    if not base > 0 or not stretch >= 1:
        raise ValueError("base must be positive and stretch at least 1")
    f = float(base) ** (-torch.arange(rot // 2, dtype=torch.float64) / (rot // 2))
    if original is None:
        return (f / stretch).to(device), 1.0
    if not original > 0:
        raise ValueError(f"original must be positive, is {original}")
    keep = ((f * (original / (2 * math.pi)) - 1) / 31).clamp(0, 1)
    return (f * keep + f / stretch * (1 - keep)).to(device), 0.1 * math.log(stretch) + 1.0


def _rope_rows(X, Y, dtype, name):
    """(RopeRows, Y) of an operand X and its output Y (allocated when None)."""
    index = X.get_device()
    rows, heads, dim = X.shape
    x = _usual(X, index, heads, dim)
    if x is None:
        x = _heads(X, name)
    if Y is None:
        Y = _like(X, dtype)
        y = heads * dim or 1, dim
    else:
        y = _usual(Y, index, heads, dim)
        if y is None or Y.dtype is not dtype or Y.shape[0] != rows:
            _need(Y, f"{name}'s output", 3, (dtype,), X.device)
            if Y.shape != X.shape:
                raise ValueError(f"{name}'s output must be {tuple(X.shape)}, is {tuple(Y.shape)}")
            y = _heads(Y, f"{name}'s output")
    if heads > _INT32_MAX or y[0] > _INT32_MAX:
        _int32(heads=heads, row_stride=y[0])
    return RopeRows(X.data_ptr() or None, Y.data_ptr() or None, heads, *x, *y), Y


def _asks_gradient(x):
    """Whether x, a tensor or a pair of tensors, requires a gradient."""
    if isinstance(x, (tuple, list)):
        return any(_asks_gradient(t) for t in x)
    return getattr(x, "requires_grad", False)


_ROPE = None


def _rope_function():
    """rope as a node of automatic differentiation: the gradient is turned back."""
    global _ROPE
    if _ROPE is None:
        import torch

        class Rope(torch.autograd.Function):
            @staticmethod
            def forward(ctx, Q, K, positions, freqs, interleaved, amplitude, inverse, dtype):
                ctx.save_for_backward(positions, freqs)
                ctx.set_materialize_grads(False)
                ctx.turn = {"interleaved": interleaved, "amplitude": amplitude, "inverse": not inverse, "dtype": Q.dtype}
                out = rope(Q, K, positions, freqs, interleaved, amplitude, inverse, dtype)
                if K is not None:
                    ctx.mark_non_differentiable(*(y for y, needed in zip(out, ctx.needs_input_grad) if not needed))
                return out

            @staticmethod
            def backward(ctx, dQ, dK=None):
                # An expanded gradient is laid out; one without rows may be expanded and contiguous.
                g = [None if d is None or not needed else d if d.is_contiguous() and d.stride(-1) == 1 else d.clone(memory_format=torch.contiguous_format)
                     for d, needed in zip((dQ, dK), ctx.needs_input_grad)]
                if g[0] is not None and g[1] is not None:
                    g = rope(*g, *ctx.saved_tensors, **ctx.turn)
                else:
                    g = [None if d is None else rope(d, None, *ctx.saved_tensors, **ctx.turn) for d in g]
                return (*g, None, None, None, None, None, None)

        _ROPE = Rope
    return _ROPE


def rope(Q, K, positions, freqs, interleaved=False, amplitude=1.0, inverse=False, dtype=None, out=None):
    """Rotary positions: the pairs of components of each head of Q and K (rows
    x heads x dim: float32, bfloat16 or float16; K may be None) turned by
    ``positions[row] * freqs[pair]`` radians and multiplied by ``amplitude``.

    ``freqs`` (float64, on the GPU; :func:`rope_frequencies` makes it) has half
    as many elements as components are turned, the first ones of each head; the
    others are copied. Pairs are components i and i + len(freqs), or with
    ``interleaved`` 2 i and 2 i + 1. positions is an int32 tensor of the rows.
    ``inverse`` turns back, which is also the gradient's way: with dQ' the
    gradient of what comes out, rope(dQ', ..., inverse=True) is Q's. Where Q or
    K require a gradient, automatic differentiation makes that call.

    Returns (Q', K'), or Q' alone without K, in ``dtype`` (the operands' type
    by default) or into ``out`` (likewise a pair or a tensor), which may be the
    operands themselves. There is no gradient through ``out``, nor with respect
    to freqs: calls that ask for one are refused.
    """
    import torch

    types = _types()
    try:
        (rows, _, dim), index, (pairs,), code = Q.shape, Q.get_device(), freqs.shape, types[Q.dtype]
        usual = (index >= 0 and positions.dtype is torch.int32 and positions.get_device() == index and positions.shape == (rows,)
                 and positions.is_contiguous() and freqs.dtype is torch.float64 and freqs.get_device() == index and freqs.is_contiguous())
    except (AttributeError, KeyError, TypeError, ValueError):
        usual = False
    if not usual:
        _need(Q, "Q", 3, types)
        rows = Q.shape[0]
        _need(positions, "positions", 1, (torch.int32,), Q.device)
        _need(freqs, "freqs", 1, (torch.float64,), Q.device)
        raise ValueError(f"positions must be {rows} contiguous elements (has {positions.shape[0]}), freqs contiguous")
    if 2 * pairs > dim:
        raise ValueError(f"{pairs} pairs do not fit heads of {dim} components")
    if (Q.requires_grad or freqs.requires_grad or _asks_gradient(K) or _asks_gradient(out)) and torch.is_grad_enabled():
        if out is not None or freqs.requires_grad:
            raise ValueError("there is no gradient through out or with respect to freqs")
        return _rope_function().apply(Q, K, positions, freqs, interleaved, amplitude, inverse, dtype)
    if out is None:
        outs = (None, None)
    elif K is None:
        if not isinstance(out, torch.Tensor):
            raise TypeError("out must be a tensor")
        outs = (out, None)
    else:
        if not isinstance(out, (tuple, list)) or len(out) != 2 or not all(isinstance(t, torch.Tensor) for t in out):
            raise TypeError("out must be a pair of tensors")
        outs = out
    if dtype is None:
        dtype = Q.dtype if out is None else outs[0].dtype
    otype = code if dtype is Q.dtype else _type_code(dtype, "dtype")
    first, Y = _rope_rows(Q, outs[0], dtype, "Q")
    second = Z = None
    if K is not None:
        if not isinstance(K, torch.Tensor) or K.dim() != 3 or K.get_device() != index or K.dtype is not Q.dtype:
            _need(K, "K", 3, (Q.dtype,), Q.device)
        if K.shape[0] != rows or K.shape[2] != dim:
            raise ValueError(f"K must be {rows} x heads x {dim}, is {tuple(K.shape)}")
        second, Z = _rope_rows(K, outs[1], dtype, "K")
    if rows > _INT32_MAX:
        _int32(rows=rows)
    _launch(index, _lib().sgemm_rope, code, otype, rows, dim, 2 * pairs, 1 if interleaved else 0,
            1 if inverse else 0, amplitude, positions.data_ptr() or None, freqs.data_ptr() or None, first, second)
    return Y if K is None else (Y, Z)


def kv_tables(table, lens, new, pool, taken, block, rows, starts=None, positions=None, slots=None, taken_after=None):
    """The tables of a step, made on the GPU from the sequences' lengths.

    Sequence b holds ``lens[b]`` tokens, the last ``new[b]`` of them new. The
    columns of ``table`` (sequences x columns) that the new tokens reach first
    are filled with pages of ``pool``, from its entry ``taken[0]`` on, sequence
    after sequence (-1 where the pool is used up). Returns

    * starts (sequences + 1): where each sequence's rows begin, as the calls
      over a cache want them;
    * positions (int32) of the ``rows`` new rows, as :func:`rope` wants them;
    * slots (int64): page * block + place of each row, -1 without a page;
    * taken_after: ``taken`` and the pages so filled; more than the pool has
      says that pages were missing. It may be ``taken`` itself.

    All are int32 GPU tensors but slots, and each is allocated unless given.
    ``rows`` is the host's count of new rows; rows behind the last sequence stay
    as they are in given outputs.
    """
    import torch

    i32, rows = torch.int32, int(rows)
    try:
        (seqs, columns), index, (entries,) = table.shape, table.get_device(), pool.shape
        usual = (table.dtype is i32 and lens.dtype is i32 and new.dtype is i32 and pool.dtype is i32 and taken.dtype is i32 and index >= 0
                 and lens.get_device() == index and new.get_device() == index and pool.get_device() == index and taken.get_device() == index
                 and lens.shape == (seqs,) and new.shape == (seqs,) and taken.shape == (1,) and table.is_contiguous()
                 and lens.is_contiguous() and new.is_contiguous() and pool.is_contiguous() and taken.is_contiguous())
    except (AttributeError, TypeError, ValueError):
        usual = False
    if not usual:
        _need(table, "table", 2, (i32,))
        for name, t in (("lens", lens), ("new", new), ("pool", pool), ("taken", taken)):
            _need(t, name, 1, (i32,), table.device)
        if not all(t.is_contiguous() for t in (table, lens, new, pool, taken)):
            raise ValueError("table, lens, new, pool and taken must be contiguous")
        raise ValueError(f"a table of {table.shape[0]} rows needs as many lens and new and one taken, got {lens.shape[0]}, "
                         f"{new.shape[0]}, {taken.shape[0]}")
    if not 0 <= rows <= _INT32_MAX or not 0 <= block <= _INT32_MAX or seqs >= _INT32_MAX or columns > _INT32_MAX or entries > _INT32_MAX:
        _int32(rows=rows, block=block, seqs=seqs + 1, columns=columns, pool=entries)
    if starts is None and positions is None and slots is None and taken_after is None:
        # One allocation for the three of one type.
        starts, positions, taken_after = torch.empty(seqs + rows + 2, dtype=i32, device=table.device).split_with_sizes((seqs + 1, rows, 1))
        outs = starts, positions, torch.empty(rows, dtype=torch.int64, device=table.device), taken_after
    else:
        outs = []
        for name, t, size, kind in (("starts", starts, seqs + 1, i32), ("positions", positions, rows, i32),
                                    ("slots", slots, rows, torch.int64), ("taken_after", taken_after, 1, i32)):
            if t is None:
                t = torch.empty(size, dtype=kind, device=table.device)
            elif not isinstance(t, torch.Tensor) or t.dtype is not kind or t.get_device() != index or t.shape != (size,) or not t.is_contiguous():
                _need(t, name, 1, (kind,), table.device)
                raise ValueError(f"{name} must have {size} contiguous elements, has {t.shape[0]}")
            outs.append(t)
    step = KVStep(lens.data_ptr() or None, new.data_ptr() or None, pool.data_ptr() or None, taken.data_ptr(), table.data_ptr() or None,
                  outs[0].data_ptr(), outs[1].data_ptr() or None, outs[2].data_ptr() or None, outs[3].data_ptr(), seqs, columns, block,
                  entries, rows)
    _launch(index, _lib().sgemm_kv_tables, step)
    return tuple(outs)
