"""Binding of the products by groups of rows (include/mfl_grouped.h): the
places of a list of choices, one product per group with its gradients, the sum
of a token's results, and adapters beside a shared projection.

Checks of shapes and types, allocation of outputs and workspaces; every step
of the operators runs in the HIP kernels.
"""
from __future__ import annotations

import ctypes
from typing import Optional, Tuple

import torch

from ._attention import _DTYPES, BF16, _ptr, _Run

GROUPED_ALGOS = {"auto": 0, "few": 1, "tile128": 2, "tile256": 3}
_NAMES = {v: k for k, v in GROUPED_ALGOS.items()}
_F32, _I32, _I64 = 2, 4, 5
_TYPES = {torch.float16: 1, torch.float32: _F32, torch.bfloat16: BF16}

_i32, _i64, _vp = ctypes.c_int32, ctypes.c_int64, ctypes.c_void_p
_int32, _float32 = torch.int32, torch.float32
_raw_stream, _current = torch._C._cuda_getCurrentRawStream, torch._C._cuda_getDevice


class GroupRowsArgs(ctypes.Structure):
    """mfl_group_rows_t"""
    _fields_ = [("ids_type", _i32)] + [(n, _i64) for n in ("count", "top", "groups")]


class GroupedArgs(ctypes.Structure):
    """mfl_grouped_t"""
    _fields_ = [("dtype", _i32), ("out", _i32), ("algo", _i32)] + \
        [(n, _i64) for n in ("groups", "places", "a_rows", "n", "k", "lda", "ldb", "b_group",
                             "ldd")]


class GroupedGradArgs(ctypes.Structure):
    """mfl_grouped_grad_t"""
    _fields_ = [("f", GroupedArgs)] + [(n, _i64) for n in ("ldda", "lddb", "db_group")]


class CombineArgs(ctypes.Structure):
    """mfl_combine_t"""
    _fields_ = [("dtype", _i32), ("out", _i32)] + \
        [(n, _i64) for n in ("tokens", "top", "n", "x_rows", "ldx", "ldo")]


class AdaptersArgs(ctypes.Structure):
    """mfl_adapters_t"""
    _fields_ = [("dtype", _i32), ("out", _i32), ("algo", _i32)] + \
        [(n, _i64) for n in ("groups", "places", "x_rows", "n", "k", "rank", "ldx", "ldw", "lda",
                             "a_group", "ldb", "b_group", "ldd")]


def declare(lib: ctypes.CDLL) -> None:
    """Argument types of the library's functions."""
    P = ctypes.POINTER
    lib.group_rows.argtypes = [P(GroupRowsArgs)] + [_vp] * 5 + [_i64, _vp]
    lib.group_rows_plan.argtypes = [P(GroupRowsArgs)] + [_vp] * 4 + [P(_i64)]
    lib.gemm_tn_grouped.argtypes = [P(GroupedArgs)] + [_vp] * 6
    lib.gemm_tn_grouped_plan.argtypes = [P(GroupedArgs)] + [_vp] * 5 + [P(_i32)]
    lib.gemm_tn_grouped_backward.argtypes = [P(GroupedGradArgs)] + [_vp] * 8
    lib.gemm_tn_grouped_backward_plan.argtypes = [P(GroupedGradArgs)] + [_vp] * 7
    lib.combine_rows.argtypes = [P(CombineArgs)] + [_vp] * 5
    lib.combine_rows_backward.argtypes = [P(CombineArgs), _i64] + [_vp] * 8
    lib.gemm_tn_adapters.argtypes = [P(AdaptersArgs)] + [_vp] * 9 + [_i64, _vp]
    lib.gemm_tn_adapters_plan.argtypes = [P(AdaptersArgs)] + [_vp] * 8 + [P(_i32), P(_i64)]
    for n in ("group_rows", "group_rows_plan", "gemm_tn_grouped", "gemm_tn_grouped_plan",
              "gemm_tn_grouped_backward", "gemm_tn_grouped_backward_plan", "combine_rows",
              "combine_rows_backward", "gemm_tn_adapters", "gemm_tn_adapters_plan"):
        getattr(lib, n).restype = ctypes.c_int


_lib = None        # the loaded library and the caller's check of its codes
_check = None


def bind(lib: ctypes.CDLL, check) -> None:
    """Give the functions below their library."""
    global _lib, _check
    declare(lib)
    _lib, _check = lib, check


# ---------------------------------------------------------------- marshalling
class _Here(_Run):
    """_Run of the tensors given, None left out, with less to do where they are
    on one device and the stream is the current one."""

    __slots__ = ("index",)

    def __init__(self, stream, *tensors):
        i = tensors[0].get_device()
        for t in tensors:
            if t is not None and t.get_device() != i:
                i = -1
        if i < 0 or stream is not None:
            super().__init__([t for t in tensors if t is not None], stream)
            i = self.device.index
        else:
            self.device = tensors[0].device
            self.handle = _raw_stream(i)
            self.other = None
        self.index = i


def _call(run: _Here, fn, *args) -> None:
    """fn, which takes no workspace, on the tensors' device."""
    if _current() != run.index:
        with torch.cuda.device(run.device):
            rc = fn(*args, run.handle)
    else:
        rc = fn(*args, run.handle)
    if rc:
        _check(rc)


def _call_with(run: _Here, fn, need: int, *args) -> None:
    """The same for a function with a workspace of `need` bytes."""
    if need == 0:
        return _call(run, fn, *args, None, 0)
    ws = run.empty((need,), torch.uint8, result=False)
    _call(run, fn, *args, ws.data_ptr(), need)


def _new(run: _Here, like: torch.Tensor, shape, dtype: Optional[torch.dtype]) -> torch.Tensor:
    """A new tensor of `like`'s type, or of dtype."""
    if run.other is not None:
        return run.empty(shape, like.dtype if dtype is None else dtype)
    return like.new_empty(shape) if dtype is None else like.new_empty(shape, dtype=dtype)


def _matrix(t: torch.Tensor, name: str) -> int:
    """Row stride of a 2-D tensor with contiguous rows."""
    s = t.stride()
    if len(s) != 2:
        raise ValueError(f"{name} must be 2-D")
    r, c = t.shape
    if s[1] != 1 and c > 1:
        raise ValueError(f"{name}'s rows must be contiguous")
    return s[0] if r > 1 else c


def _matrices(t: torch.Tensor, name: str) -> Tuple[int, int]:
    """Row and matrix stride of a 3-D tensor with contiguous rows."""
    s = t.stride()
    if len(s) != 3:
        raise ValueError(f"{name} must be 3-D")
    g, r, c = t.shape
    if s[2] != 1 and c > 1:
        raise ValueError(f"{name}'s rows must be contiguous")
    return (s[1] if r > 1 else c), (s[0] if g > 1 else 0)


def _numbers(t: Optional[torch.Tensor], name: str, count: Optional[int] = None) -> None:
    if t is None:
        return
    if t.dtype is not _int32:
        raise TypeError(f"{name} must be int32")
    if t.dim() != 1 or not t.is_contiguous() or (count is not None and t.shape[0] != count):
        raise ValueError(f"{name} must be contiguous" +
                         ("" if count is None else f", of {count} entries"))


def _type(dtype, given: torch.dtype, name: str) -> int:
    """Code of an output's type: the operands' own or float32."""
    if dtype is None or dtype is given:
        return _TYPES.get(given, 0)       # (0: refused with the operands)
    if dtype is not _float32:
        raise TypeError(f"{name} must be of the operands' type or float32")
    return _F32


def _code(names: str, first: torch.Tensor, *others) -> int:
    """Code of the operands' one type."""
    dt = first.dtype
    code = _DTYPES.get(dt)
    if code is None:
        raise TypeError(f"{names} must be float16 or bfloat16")
    for t in others:
        if t.dtype is not dt:
            raise TypeError(f"{names} must have one dtype")
    return code


def _grouped_args(A, B, offsets, rows, out: int, algo: str, places: int, ldd: int):
    # (a call for few rows is as long as this takes: one look at what is usual,
    # the helpers for the rest)
    sa, sb, dt = A.stride(), B.stride(), A.dtype
    code = _DTYPES.get(dt)
    if code is None or B.dtype is not dt or len(sa) != 2 or len(sb) != 3 or sa[1] != 1 or \
            sb[2] != 1:
        code = _code("A and B", A, B)
        _matrix(A, "A")
        _matrices(B, "B")
    m, ka = A.shape
    groups, n, k = B.shape
    if ka != k:
        raise ValueError("A and B disagree on K")
    if offsets.dtype is not _int32 or offsets.numel() != groups + 1 or offsets.dim() != 1 or \
            not offsets.is_contiguous():
        _numbers(offsets, "offsets", groups + 1)
    if rows is not None and (rows.dtype is not _int32 or rows.dim() != 1 or
                             not rows.is_contiguous()):
        _numbers(rows, "rows")
    return GroupedArgs(code, out, GROUPED_ALGOS[algo], groups, places, m, n, k,
                       sa[0] if m > 1 else k, sb[1] if n > 1 else k, sb[0] if groups > 1 else 0,
                       ldd)


def _dense(t: torch.Tensor, run: _Here) -> torch.Tensor:
    """t, or where its rows do not follow each other whole (a sum's gradient,
    expanded) a contiguous copy, made on the stream that reads it."""
    if t.dim() != 2 or t.numel() == 0:
        return t
    s, (r, c) = t.stride(), t.shape
    if s[1] == 1 and (r < 2 or s[0] >= c):
        return t
    if run.other is None:
        return t.contiguous()
    with torch.cuda.stream(run.other):
        return t.contiguous()


# ------------------------------------------------------------------ functions
def group_rows(ids: torch.Tensor, groups: int, *, stream=None):
    """The rows of every group, from a list of choices, on the GPU.

    ids (tokens,) or (tokens, top), int32 or int64, contiguous: the groups that
    each token goes to, as a router's top-k or a batch's adapters; numbers
    outside 0 .. groups - 1 are of no group.  Sorted by group, a group's
    choices in their own order and those of no group behind, the choices take
    places 0, 1, ...  Returns (int32, on the device)

      rows     (tokens * top,)  the token of each place
      offsets  (groups + 1,)    the first place of each group
      slots    ids' shape       the place of each choice, -1 for no group

    as gemm_grouped, combine_rows and gemm_adapters take them.  At most 4096
    groups."""
    dtype = ids.dtype
    if dtype is not torch.int64 and dtype is not _int32:
        raise TypeError("ids must be int32 or int64")
    if ids.dim() not in (1, 2):
        raise ValueError("ids must be (tokens,) or (tokens, top)")
    if not ids.is_contiguous():
        raise ValueError("ids must be contiguous")
    top = ids.shape[1] if ids.dim() == 2 else 1
    a = GroupRowsArgs(_I32 if dtype is _int32 else _I64, ids.numel(), max(top, 1), groups)
    if groups < 1:
        raise ValueError("there must be a group")
    run = _Here(stream, ids)
    # (one allocation: each takes a third of the time of the kernel for a few
    # choices)
    n = ids.numel()
    rows, offsets, slots = torch.unsafe_split_with_sizes(
        _new(run, ids, (2 * n + groups + 1,), _int32), (n, groups + 1, n))
    if ids.dim() == 2:
        slots = slots.view(ids.shape)
    ptrs = _ptr(ids), _ptr(rows), _ptr(offsets), _ptr(slots)
    need = 0
    if n > 1024:                  # (up to as many one workgroup does without)
        b = _i64(0)
        _check(_lib.group_rows_plan(a, *ptrs, b))
        need = b.value
    _call_with(run, _lib.group_rows, need, a, *ptrs)
    return rows, offsets, slots


def gemm_grouped(A: torch.Tensor, B: torch.Tensor, offsets: torch.Tensor, *,
                 rows: Optional[torch.Tensor] = None, out_dtype: Optional[torch.dtype] = None,
                 D: Optional[torch.Tensor] = None, algo: str = "auto", stream=None):
    """D[i] = A[rows[i]] @ B[g].T for every place i of group g, on the GPU.

    A (M, K) and B (groups, N, K), float16 or bfloat16 with contiguous rows,
    16-byte aligned, N and K multiples of 8.  offsets (groups + 1, int32, on
    the device): group g owns the places offsets[g] .. offsets[g + 1] - 1.
    rows (int32): the row of A at each place, gathered by the kernel; without
    it place i is row i.  D (places, N) is of A's type, or float32 with
    out_dtype; it is allocated when not given, and its rows of no group are
    not written.  No autograd graph is recorded: gemm_grouped_backward gives
    the gradients.  algo chooses the kernel; by itself it follows the mean
    number of places per group."""
    places = A.shape[0] if rows is None else rows.shape[0]
    n = B.shape[1] if B.dim() == 3 else 0
    if D is not None:
        if D.shape != (places, n):
            raise ValueError(f"D must have shape {(places, n)}")
        if out_dtype is not None and out_dtype != D.dtype:
            raise TypeError("D is not of out_dtype")
        out_dtype = D.dtype
    out = _type(out_dtype, A.dtype, "D")
    a = _grouped_args(A, B, offsets, rows, out, algo, places, n if D is None else _matrix(D, "D"))
    run = _Here(stream, A, B, offsets, rows, D)
    if D is None:
        D = _new(run, A, (places, n), out_dtype)
    _call(run, _lib.gemm_tn_grouped, a, _ptr(A), _ptr(B), _ptr(offsets), _ptr(rows), _ptr(D))
    return D


def gemm_grouped_plan(A, B, offsets, *, rows=None, out_dtype=None, algo="auto") -> str:
    """The kernel gemm_grouped() takes for these tensors; their data is not
    read."""
    places = A.shape[0] if rows is None else rows.shape[0]
    a = _grouped_args(A, B, offsets, rows, _type(out_dtype, A.dtype, "D"), algo, places,
                      B.shape[1])
    al = _i32(0)
    _check(_lib.gemm_tn_grouped_plan(a, _ptr(A), _ptr(B), _ptr(offsets), _ptr(rows), 1 << 40, al))
    return _NAMES[al.value]


def gemm_grouped_backward(dD: torch.Tensor, A: torch.Tensor, B: torch.Tensor,
                          offsets: torch.Tensor, *, rows: Optional[torch.Tensor] = None,
                          dB_dtype: Optional[torch.dtype] = None, stream=None):
    """(dA, dB) of sum(D * dD) for gemm_grouped()'s arguments.

    dA (places, K) has a row per place, 0 for those of no group; where rows
    gathers, combine_rows(dA, slots) adds the rows of each token.  dB has B's
    shape and type, or float32 with dB_dtype; 0 for groups without places.
    An expanded or transposed dD is copied first.  The same arguments give the
    same bits."""
    places = A.shape[0] if rows is None else rows.shape[0]
    out = _type(dB_dtype, A.dtype, "dB")
    if dD.dtype != A.dtype:
        raise TypeError("dD must have A's dtype")
    if B.dim() != 3 or dD.shape != (places, B.shape[1]):
        raise ValueError("dD must be (places, N)")
    run = _Here(stream, dD, A, B, offsets, rows)
    dD = _dense(dD, run)
    f = _grouped_args(A, B, offsets, rows, out, "auto", places, _matrix(dD, "dD"))
    k, n = B.shape[2], B.shape[1]
    a = GroupedGradArgs(f, k, k, n * k)
    dA = _new(run, A, (places, k), None)
    dB = run.like(B) if dB_dtype is None else _new(run, B, B.shape, dB_dtype)
    _call(run, _lib.gemm_tn_grouped_backward, a, _ptr(dD), _ptr(A), _ptr(B), _ptr(offsets),
          _ptr(rows), _ptr(dA), _ptr(dB))
    return dA, dB


def _combine_args(X, slots, weights, out: int, ldo: int) -> CombineArgs:
    code = _code("X", X)
    if slots.dtype is not _int32:
        raise TypeError("slots must be int32")
    shape = slots.shape
    if len(shape) not in (1, 2) or not slots.is_contiguous():
        raise ValueError("slots must be (tokens,) or (tokens, top), contiguous")
    if weights is not None:
        if weights.dtype is not _float32:
            raise TypeError("weights must be float32")
        if weights.shape != shape or not weights.is_contiguous():
            raise ValueError("weights must have slots' shape, contiguous")
    ldx = _matrix(X, "X")
    rows, n = X.shape
    return CombineArgs(code, out, shape[0], shape[1] if len(shape) == 2 else 1, n, rows, ldx, ldo)


def combine_rows(X: torch.Tensor, slots: torch.Tensor, weights: Optional[torch.Tensor] = None, *,
                 out_dtype: Optional[torch.dtype] = None, out: Optional[torch.Tensor] = None,
                 stream=None):
    """out[t] = sum over j of weights[t, j] * X[slots[t, j]], on the GPU.

    X (places, N), float16 or bfloat16 with contiguous rows, N a multiple of
    8; slots (tokens,) or (tokens, top <= 64) int32, as group_rows gives them:
    one outside X's rows adds nothing.  weights: slots' shape, float32; 1
    without them.  out (tokens, N) is of X's type, or float32 with out_dtype.
    Sums are float32, in the order of j."""
    n = X.shape[1] if X.dim() == 2 else 0
    if out is not None:
        if out.shape != (slots.shape[0], n):
            raise ValueError(f"out must have shape {(slots.shape[0], n)}")
        if out_dtype is not None and out_dtype != out.dtype:
            raise TypeError("out is not of out_dtype")
        out_dtype = out.dtype
    a = _combine_args(X, slots, weights, _type(out_dtype, X.dtype, "out"),
                      n if out is None else _matrix(out, "out"))
    run = _Here(stream, X, slots, weights, out)
    if out is None:
        out = _new(run, X, (slots.shape[0], n), out_dtype)
    _call(run, _lib.combine_rows, a, _ptr(X), _ptr(slots), _ptr(weights), _ptr(out))
    return out


def combine_rows_backward(dout: torch.Tensor, X: torch.Tensor, slots: torch.Tensor,
                          weights: Optional[torch.Tensor] = None, *, rows: torch.Tensor,
                          stream=None):
    """(dX, dweights) of sum(out * dout) for combine_rows()'s arguments.

    rows (places,) int32: each place's token, as group_rows gives it with
    slots.  dX has X's shape; a place that no choice of its token leads to has
    gradient 0, and so has the weight of a choice without a place.  dweights is
    None without weights.  An expanded or transposed dout is copied first."""
    if dout.dtype != X.dtype:
        raise TypeError("dout must have X's dtype")
    if X.dim() != 2 or dout.shape != (slots.shape[0], X.shape[1]):
        raise ValueError("dout must be (tokens, N)")
    run = _Here(stream, dout, X, slots, weights, rows)
    dout = _dense(dout, run)
    a = _combine_args(X, slots, weights, _TYPES.get(X.dtype, 0), _matrix(dout, "dout"))
    _numbers(rows, "rows", X.shape[0])
    dX = run.like(X)
    dw = None if weights is None else run.like(weights)
    _call(run, _lib.combine_rows_backward, a, X.shape[1], _ptr(dout), _ptr(X), _ptr(slots),
          _ptr(rows), _ptr(weights), _ptr(dX), _ptr(dw))
    return dX, dw


def _adapters_args(x, W, A, B, offsets, rows, scale, out: int, algo: str, ldd: int):
    sx, sw, sa, sb, dt = x.stride(), W.stride(), A.stride(), B.stride(), x.dtype
    code = _DTYPES.get(dt)
    if code is None or not dt is W.dtype is A.dtype is B.dtype:
        code = _code("x, W, A and B", x, W, A, B)
    if len(sx) != 2 or len(sw) != 2 or len(sa) != 3 or len(sb) != 3 or \
            not sx[1] == sw[1] == sa[2] == sb[2] == 1:
        _matrix(x, "x")
        _matrix(W, "W")
        _matrices(A, "A")
        _matrices(B, "B")
    (m, k), (n, kw), (groups, rank, ka) = x.shape, W.shape, A.shape
    if kw != k or ka != k:
        raise ValueError("x, W and A disagree on K")
    if B.shape != (groups, n, rank):
        raise ValueError("W, A and B disagree on the adapters, N or the rank")
    if offsets.dtype is not _int32 or offsets.numel() != groups + 1 or offsets.dim() != 1 or \
            not offsets.is_contiguous():
        _numbers(offsets, "offsets", groups + 1)
    places = m
    if rows is not None:
        if rows.dtype is not _int32 or rows.dim() != 1 or not rows.is_contiguous():
            _numbers(rows, "rows")
        places = rows.shape[0]
        if places > m:
            raise ValueError("rows holds each row at most once")
    if scale is not None:
        if scale.dtype is not _float32:
            raise TypeError("scale must be float32")
        if scale.dim() != 1 or scale.numel() != groups or not scale.is_contiguous():
            raise ValueError("scale must hold one factor per adapter, contiguous")
    return AdaptersArgs(code, out, GROUPED_ALGOS[algo], groups, places, m, n, k, rank,
                        sx[0] if m > 1 else k, sw[0] if n > 1 else k, sa[1] if rank > 1 else k,
                        sa[0] if groups > 1 else 0, sb[1] if n > 1 else rank,
                        sb[0] if groups > 1 else 0, ldd)


def gemm_adapters(x: torch.Tensor, W: torch.Tensor, A: torch.Tensor, B: torch.Tensor,
                  offsets: torch.Tensor, *, rows: Optional[torch.Tensor] = None,
                  scale: Optional[torch.Tensor] = None,
                  out_dtype: Optional[torch.dtype] = None, D: Optional[torch.Tensor] = None,
                  algo: str = "auto", stream=None):
    """x @ W.T, plus scale[g] * (x @ A[g].T) @ B[g].T in the rows of adapter g,
    on the GPU: one step of a batch whose requests use different adapters.

    x (M, K), W (N, K), A (adapters, rank, K), B (adapters, N, rank), float16
    or bfloat16 with contiguous rows, 16-byte aligned, N, K and the rank
    multiples of 8.  offsets (adapters + 1, int32, on the device): adapter g
    owns the places offsets[g] .. offsets[g + 1] - 1; places behind the last
    have no adapter.  rows (int32): the row of x and of the result at each
    place, every row at most once, as group_rows(adapter of each row, adapters)
    gives them; without it places are rows.  scale: (adapters,) float32, 1
    without it.  D (M, N) is of x's type, or float32 with out_dtype; it is
    allocated when not given, and rows that no place leads to are not written.
    An adapter's values reach its own rows alone.  x @ A[g].T, scaled, is held
    in float32.  No autograd graph is recorded.  algo chooses the kernel."""
    m, n = x.shape[0], W.shape[0]
    if D is not None:
        if D.shape != (m, n):
            raise ValueError(f"D must have shape {(m, n)}")
        if out_dtype is not None and out_dtype != D.dtype:
            raise TypeError("D is not of out_dtype")
        out_dtype = D.dtype
    a = _adapters_args(x, W, A, B, offsets, rows, scale, _type(out_dtype, x.dtype, "D"), algo,
                       n if D is None else _matrix(D, "D"))
    run = _Here(stream, x, W, A, B, offsets, rows, scale, D)
    if D is None:
        D = _new(run, x, (m, n), out_dtype)
    ptrs = (_ptr(x), _ptr(W), _ptr(A), _ptr(B), _ptr(offsets), _ptr(rows), _ptr(scale), _ptr(D))
    b = _i64(0)
    rc = _lib.gemm_tn_adapters_plan(a, *ptrs, None, b)
    if rc:
        _check(rc)
    _call_with(run, _lib.gemm_tn_adapters, b.value, a, *ptrs)
    return D


def gemm_adapters_plan(x, W, A, B, offsets, *, rows=None, scale=None, out_dtype=None,
                       algo="auto") -> Tuple[str, int]:
    """(kernel, workspace bytes) gemm_adapters() takes for these tensors; their
    data is not read."""
    a = _adapters_args(x, W, A, B, offsets, rows, scale, _type(out_dtype, x.dtype, "D"), algo,
                       W.shape[0])
    al, b = _i32(0), _i64(0)
    _check(_lib.gemm_tn_adapters_plan(a, _ptr(x), _ptr(W), _ptr(A), _ptr(B), _ptr(offsets),
                                      _ptr(rows), _ptr(scale), 1 << 40, al, b))
    return _NAMES[al.value], b.value
