"""Binding of the attention functions (include/mfl_attention.h): packed
prompts, their gradients, and decoding behind a shared prefix.

Checks of shapes and types, allocation of outputs and workspaces; every step
of the operators runs in the HIP kernels.
"""
from __future__ import annotations

import ctypes
import math
from typing import Optional, Tuple

import torch

BF16 = 3
ATTENTION_ALGOS = {"auto": 0, "tall": 1, "flat": 2}
_NAMES = {v: k for k, v in ATTENTION_ALGOS.items()}
_DTYPES = {torch.float16: 1, torch.bfloat16: BF16}

_i32, _i64, _f32, _vp = ctypes.c_int32, ctypes.c_int64, ctypes.c_float, ctypes.c_void_p


class AttentionArgs(ctypes.Structure):
    """mfl_attention_t"""
    _fields_ = [("dtype", _i32), ("causal", _i32)] + \
        [(n, _i64) for n in ("batch", "total_q", "total_k", "heads_q", "heads_kv", "head_dim",
                             "q_token", "q_head", "k_token", "k_head", "v_token", "v_head",
                             "out_token", "out_head")] + \
        [("scale", _f32), ("algo", _i32), ("splits", _i32)]


class AttentionGradArgs(ctypes.Structure):
    """mfl_attention_grad_t"""
    _fields_ = [("f", AttentionArgs)] + \
        [(n, _i64) for n in ("dout_token", "dout_head", "dq_token", "dq_head", "dk_token",
                             "dk_head", "dv_token", "dv_head")]


class AttentionPrefixArgs(ctypes.Structure):
    """mfl_attention_prefix_t"""
    _fields_ = [("dtype", _i32), ("algo", _i32)] + \
        [(n, _i64) for n in ("batch", "q_tokens", "prefix", "capacity", "heads_q", "heads_kv",
                             "head_dim", "q_batch", "q_token", "q_head", "prefix_k_token",
                             "prefix_k_head", "prefix_v_token", "prefix_v_head", "k_batch",
                             "k_token", "k_head", "v_batch", "v_token", "v_head", "out_batch",
                             "out_token", "out_head")] + \
        [("scale", _f32), ("splits_prefix", _i32), ("splits_own", _i32)]


def declare(lib: ctypes.CDLL) -> None:
    """Argument types of the library's attention functions."""
    P = ctypes.POINTER
    lib.attention_packed.argtypes = [P(AttentionArgs)] + [_vp] * 8 + [_i64, _vp]
    lib.attention_packed_plan.argtypes = [P(AttentionArgs)] + [_vp] * 7 + \
        [P(_i32), P(_i32), P(_i64)]
    lib.attention_packed_backward.argtypes = [P(AttentionGradArgs)] + [_vp] * 12 + [_i64, _vp]
    lib.attention_packed_backward_plan.argtypes = [P(AttentionGradArgs)] + [_vp] * 11 + [P(_i64)]
    lib.attention_prefix.argtypes = [P(AttentionPrefixArgs)] + [_vp] * 9 + [_i64, _vp]
    lib.attention_prefix_plan.argtypes = [P(AttentionPrefixArgs)] + [_vp] * 8 + \
        [P(_i32), P(_i32), P(_i32), P(_i64)]
    for n in ("attention_packed", "attention_packed_backward", "attention_prefix"):
        getattr(lib, n).restype = ctypes.c_int
        getattr(lib, n + "_plan").restype = ctypes.c_int


# ---------------------------------------------------------------- marshalling
_lib = None        # the loaded library and the caller's check of its codes
_check = None
_E_WORKSPACE = -10


def bind(lib: ctypes.CDLL, check) -> None:
    """Give the functions below their library."""
    global _lib, _check
    declare(lib)
    _lib, _check = lib, check


class _Run:
    """Where a call runs: the tensors' device and the stream.  Outputs and
    workspaces are allocated for the stream that uses them; on a stream that
    is not the current one the caller's tensors are recorded there too."""

    __slots__ = ("device", "handle", "cur", "other")

    def __init__(self, tensors, stream):
        self.device = dev = tensors[0].device
        for t in tensors:
            if t.device != dev or not t.is_cuda:
                raise ValueError("all tensors must be device tensors (no CPU path)"
                                 if not t.is_cuda else "all tensors must be on one device")
        self.handle = torch._C._cuda_getCurrentRawStream(dev.index)
        self.other = None
        if stream is not None and int(stream) != self.handle:
            self.handle = int(stream)
            self.cur = torch.cuda.current_stream(dev)
            self.other = torch.cuda.ExternalStream(self.handle, device=dev)
            for t in tensors:
                t.record_stream(self.other)

    def like(self, t):
        """A new contiguous tensor of t's shape and type."""
        if self.other is None:
            return torch.empty_like(t, memory_format=torch.contiguous_format)
        return self.empty(t.shape, t.dtype)

    def empty(self, shape, dtype, result=True):
        if self.other is None:
            return torch.empty(shape, dtype=dtype, device=self.device)
        with torch.cuda.stream(self.other):
            t = torch.empty(shape, dtype=dtype, device=self.device)
        if result:
            t.record_stream(self.cur)
        return t

    def call(self, fn, args, ptrs, need):
        """fn on the tensors' device.  `need` gives the workspace's size, asked
        only when the call says that it wants one."""
        if torch.cuda.current_device() != self.device.index:
            with torch.cuda.device(self.device):
                return self._call(fn, args, ptrs, need)
        return self._call(fn, args, ptrs, need)

    def _call(self, fn, args, ptrs, need):
        rc = fn(args, *ptrs, None, 0, self.handle)
        if rc == _E_WORKSPACE:
            n = need()
            ws = self.empty((n,), torch.uint8, result=False)
            rc = fn(args, *ptrs, ws.data_ptr(), n, self.handle)
        if rc:
            _check(rc)


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else t.data_ptr()      # (no elements: NULL)


def _dtype(names, first, *others):
    dt = first.dtype
    code = _DTYPES.get(dt)
    if code is None:
        raise TypeError(f"{names} must be float16 or bfloat16")
    for t in others:
        if t.dtype != dt:
            raise TypeError(f"{names} must have one dtype")
    return code


def _strides3(t: torch.Tensor, name: str):
    """Token and head stride in elements; the last dimension is contiguous.  0
    for a dimension of one."""
    if t.dim() != 3:
        raise ValueError(f"{name} must be 3-D")
    n, h, d = t.shape
    x, y, z = t.stride()
    if z != 1 and d > 1:
        raise ValueError(f"{name}'s last dimension must be contiguous")
    return x if n > 1 else 0, y if h > 1 else 0


def _strides4(t: torch.Tensor, name: str):
    """Batch, token and head stride, as _strides3."""
    if t.dim() != 4:
        raise ValueError(f"{name} must be 4-D")
    b, n, h, d = t.shape
    w, x, y, z = t.stride()
    if z != 1 and d > 1:
        raise ValueError(f"{name}'s last dimension must be contiguous")
    return w if b > 1 else 0, x if n > 1 else 0, y if h > 1 else 0


def _strides_q(t: torch.Tensor, name: str):
    """_strides4 of (batch, tokens, heads, dim), or of (batch, heads, dim) as
    one token each."""
    if t.dim() == 4:
        return _strides4(t, name)
    w, y = _strides3(t, name)
    return w, 0, y


def _scale(scale, dim):
    scale = 1.0 / math.sqrt(dim or 1) if scale is None else float(scale)
    if not (scale > 0.0 and math.isfinite(scale)):
        raise ValueError("scale must be positive and finite")
    return scale


def _offsets(seq_q, seq_k):
    if seq_q is None:
        if seq_k is not None:
            raise ValueError("seq_k without seq_q")
        return 1
    for t, n in ((seq_q, "seq_q"),) if seq_k is seq_q else ((seq_q, "seq_q"), (seq_k, "seq_k")):
        if t.dtype != torch.int32:
            raise TypeError(f"{n} must be int32")
        if t.dim() != 1 or t.shape[0] < 2 or t.stride(0) != 1:
            raise ValueError(f"{n} must hold sequences + 1 offsets, contiguous")
    if seq_q.shape != seq_k.shape:
        raise ValueError("seq_q and seq_k disagree on the number of sequences")
    return seq_q.shape[0] - 1


def _heads(hq, hk):
    if hk == 0 or hq == 0 or hq % hk:
        raise ValueError("the query heads must be a multiple of the key heads")


def _packed_args(q, k, v, seq_q, seq_k, causal, scale, out, algo, splits):
    code = _dtype("q, k and v", q, k, v)
    q0, q1 = _strides3(q, "q")
    k0, k1 = _strides3(k, "k")
    v0, v1 = _strides3(v, "v")
    o0, o1 = _fresh(q.shape) if out is None else _strides3(out, "out")
    total_q, hq, d = q.shape
    total_k, hk, dk = k.shape
    if v.shape != k.shape:
        raise ValueError("k and v must have one shape")
    if dk != d:
        raise ValueError("q and k disagree on the head dimension")
    _heads(hq, hk)
    return AttentionArgs(code, 1 if causal else 0, _offsets(seq_q, seq_k), total_q, total_k, hq,
                         hk, d, q0, q1, k0, k1, v0, v1, o0, o1,
                         _scale(scale, d), ATTENTION_ALGOS[algo], splits)


def _like(t, ref, name):
    if t.dtype != ref.dtype:
        raise TypeError(f"{name} must have q's dtype")
    if t.shape != ref.shape:
        raise ValueError(f"{name} must have shape {tuple(ref.shape)}")


def _fresh(shape):
    """Strides of a new 3-D tensor, as _strides."""
    return [shape[1] * shape[2] if shape[0] > 1 else 0, shape[2] if shape[1] > 1 else 0]


def _rows(t, stream):
    """t, or where its elements do not follow each other or its tokens lie less
    than a row apart (a sum's gradient, expanded) a contiguous copy, made on
    the stream that reads it."""
    if t.dim() != 3 or t.numel() == 0 or \
            (t.stride(2) == 1 and (t.shape[0] < 2 or t.stride(0) >= t.shape[2])):
        return t
    if stream is None or not t.is_cuda:
        return t.contiguous()
    other = torch.cuda.ExternalStream(int(stream), device=t.device)
    t.record_stream(other)
    with torch.cuda.stream(other):
        return t.contiguous()


# ------------------------------------------------------------------ functions
def attention(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, *,
              seq_q: Optional[torch.Tensor] = None, seq_k: Optional[torch.Tensor] = None,
              causal: bool = True, scale: Optional[float] = None,
              out: Optional[torch.Tensor] = None, return_lse: bool = False,
              algo: str = "auto", splits: int = 0, stream=None):
    """softmax(scale q k^T) v over packed sequences on the GPU.

    q (tokens, heads, dim), k and v (tokens, kv heads, dim), float16 or
    bfloat16, any 16-byte aligned token and head strides; heads is a multiple
    of kv heads (grouped heads), dim a multiple of 8 up to 256.  seq_q, seq_k:
    sequences + 1 int32 offsets on the device (one sequence without them;
    seq_k defaults to seq_q).  causal: query token t of a sequence with lq
    queries and lk keys sees the keys up to t + lk - lq.  scale defaults to
    dim ** -0.5.  Returns out (tokens, heads, dim), with return_lse also the
    log-sum-exp (tokens, heads) float32; a query without visible keys has out
    0 and -inf.  Rows behind the last sequence are not written.  No autograd
    graph is recorded: attention_backward gives the gradients.  algo and
    splits choose the kernel and the parts its keys are split into; by
    themselves they follow the mean lengths, so for one long sequence among
    many short ones it pays to give them."""
    if seq_k is None:
        seq_k = seq_q
    if out is not None:
        _like(out, q, "out")
    a = _packed_args(q, k, v, seq_q, seq_k, causal, scale, out, algo, splits)
    run = _Run([t for t in (q, k, v, seq_q, seq_k, out) if t is not None], stream)
    if out is None:
        out = run.like(q)
    lse = run.empty(q.shape[:2], torch.float32) if return_lse else None
    ptrs = (_ptr(q), _ptr(k), _ptr(v), _ptr(seq_q), _ptr(seq_k), _ptr(out), _ptr(lse))

    def need():
        n = _i64(0)
        _check(_lib.attention_packed_plan(a, *ptrs, None, None, n))
        return n.value

    run.call(_lib.attention_packed, a, ptrs, need)
    return (out, lse) if return_lse else out


def attention_plan(q, k, v, *, seq_q=None, seq_k=None, causal=True, scale=None, algo="auto",
                   splits=0) -> Tuple[str, int, int]:
    """(kernel, key splits, workspace bytes) attention() takes for these
    tensors; their data is not read."""
    if seq_k is None:
        seq_k = seq_q
    a = _packed_args(q, k, v, seq_q, seq_k, causal, scale, None, algo, splits)
    al, sp, n = _i32(0), _i32(0), _i64(0)
    _check(_lib.attention_packed_plan(a, _ptr(q), _ptr(k), _ptr(v), _ptr(seq_q), _ptr(seq_k),
                                      1 << 40, None, al, sp, n))
    return _NAMES[al.value], sp.value, n.value


def attention_backward(dout: torch.Tensor, q: torch.Tensor, k: torch.Tensor, v: torch.Tensor,
                       out: torch.Tensor, lse: torch.Tensor, *,
                       seq_q: Optional[torch.Tensor] = None,
                       seq_k: Optional[torch.Tensor] = None, causal: bool = True,
                       scale: Optional[float] = None, stream=None):
    """(dq, dk, dv) of sum(out * dout) for attention()'s arguments and its out
    and lse.  The gradients of a group's shared kv head are summed over its
    query heads; tokens of no sequence have gradient 0.  Expanded or
    transposed q and dout are copied first.  The same arguments give
    the same bits."""
    if seq_k is None:
        seq_k = seq_q
    _like(dout, q, "dout")
    _like(out, q, "out")
    dout, q = _rows(dout, stream), _rows(q, stream)
    f = _packed_args(q, k, v, seq_q, seq_k, causal, scale, out, "auto", 0)
    if lse.dtype != torch.float32:
        raise TypeError("lse must be float32")
    if lse.shape != q.shape[:2] or not lse.is_contiguous():
        raise ValueError(f"lse must be contiguous, of shape {tuple(q.shape[:2])}")
    g = AttentionGradArgs(f, *_strides3(dout, "dout"), *_fresh(q.shape), *_fresh(k.shape),
                          *_fresh(v.shape))
    run = _Run([t for t in (dout, q, k, v, out, lse, seq_q, seq_k) if t is not None], stream)
    dq, dk, dv = run.like(q), run.like(k), run.like(v)
    ptrs = tuple(_ptr(t) for t in (dout, q, k, v, out, lse, seq_q, seq_k, dq, dk, dv))

    def need():
        n = _i64(0)
        _check(_lib.attention_packed_backward_plan(g, *ptrs, n))
        return n.value

    run.call(_lib.attention_packed_backward, g, ptrs, need)
    return dq, dk, dv


def attention_prefix(q: torch.Tensor, prefix_k: torch.Tensor, prefix_v: torch.Tensor,
                     k: torch.Tensor, v: torch.Tensor, lengths: torch.Tensor, *,
                     scale: Optional[float] = None, out: Optional[torch.Tensor] = None,
                     return_lse: bool = False, algo: str = "auto",
                     splits: Tuple[int, int] = (0, 0), stream=None):
    """Attention of a decoding batch whose sequences share a prefix.

    q (batch, heads, dim) or (batch, new tokens, heads, dim); prefix_k,
    prefix_v (prefix, kv heads, dim); k, v (batch, capacity, kv heads, dim):
    each sequence's own cache, of which lengths[b] (int32, on the device) keys
    are held, those of the new tokens last.  A new token sees the whole prefix
    and its own sequence's keys up to itself.  The prefix is read for the whole
    batch together, per tile of rows.  Returns out of q's shape, with return_lse also the
    log-sum-exp (float32, q's shape without dim).  algo and splits choose the
    prefix's kernel and the parts the prefix and the caches are split into."""
    code = _dtype("q, the prefix, k and v", q, prefix_k, prefix_v, k, v)
    if q.dim() not in (3, 4):
        raise ValueError("q must be (batch, heads, dim) or (batch, tokens, heads, dim)")
    if q.dim() == 4:
        batch, tokens, hq, d = q.shape
    else:
        (batch, hq, d), tokens = q.shape, 1
    qs = _strides_q(q, "q")
    pks, pvs = _strides3(prefix_k, "prefix_k"), _strides3(prefix_v, "prefix_v")
    ks, vs = _strides4(k, "k"), _strides4(v, "v")
    prefix, hk, dim = prefix_k.shape
    if prefix_v.shape != prefix_k.shape or v.shape != k.shape:
        raise ValueError("keys and values must have one shape")
    capacity = k.shape[1]
    if dim != d or k.shape != (batch, capacity, hk, d):
        raise ValueError("q, the prefix and the cache disagree on batch, heads or dim")
    if batch == 0:
        raise ValueError("the batch is empty")
    _heads(hq, hk)
    if lengths.dtype != torch.int32:
        raise TypeError("lengths must be int32")
    if lengths.shape != (batch,) or (batch > 1 and lengths.stride(0) != 1):
        raise ValueError("lengths must hold one length per sequence, contiguous")
    if out is not None:
        _like(out, q, "out")
    run = _Run([t for t in (q, prefix_k, prefix_v, k, v, lengths, out) if t is not None], stream)
    if out is None:
        out = run.like(q)
        os = (tokens * hq * d if batch > 1 else 0, hq * d if tokens > 1 else 0, d if hq > 1 else 0)
    else:
        os = _strides_q(out, "out")
    a = AttentionPrefixArgs(code, ATTENTION_ALGOS[algo], batch, tokens, prefix, capacity, hq, hk,
                            d, *qs, *pks, *pvs, *ks, *vs, *os, _scale(scale, d),
                            *splits)
    lse = run.empty(q.shape[:-1], torch.float32) if return_lse else None
    ptrs = (_ptr(q), _ptr(prefix_k), _ptr(prefix_v), _ptr(k), _ptr(v), _ptr(lengths), _ptr(out),
            _ptr(lse))

    def need():
        n = _i64(0)
        _check(_lib.attention_prefix_plan(a, *ptrs, None, None, None, n))
        return n.value

    run.call(_lib.attention_prefix, a, ptrs, need)
    return (out, lse) if return_lse else out
