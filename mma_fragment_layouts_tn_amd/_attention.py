"""Binding of the attention functions (include/mfl_attention.h): packed
prompts, their gradients, and decoding behind a shared prefix.

Checks of shapes and types, allocation of outputs and workspaces; every step
of the operators runs in the HIP kernels.
"""
from __future__ import annotations

import contextlib
import ctypes
import math
from typing import Optional, Tuple

import torch

BF16 = 3
ATTENTION_ALGOS = {"auto": 0, "tall": 1, "tall4": 2, "flat": 3}
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
class _Run:
    """Where a call runs: the tensors' device and the stream.  Outputs and
    workspaces are allocated for the stream that uses them; on a stream that
    is not the current one the caller's tensors are recorded there too."""

    def __init__(self, device, stream, tensors):
        self.device = device
        cur = torch.cuda.current_stream(device)
        self.handle = cur.cuda_stream if stream is None else int(stream)
        self.cur = self.other = None
        if self.handle != cur.cuda_stream:
            self.cur = cur
            self.other = torch.cuda.ExternalStream(self.handle, device=device)
            for t in tensors:
                if t is not None:
                    t.record_stream(self.other)

    def empty(self, shape, dtype, result=True):
        if self.other is None:
            return torch.empty(shape, dtype=dtype, device=self.device)
        with torch.cuda.stream(self.other):
            t = torch.empty(shape, dtype=dtype, device=self.device)
        if result:
            t.record_stream(self.cur)
        return t

    def workspace(self, nbytes):
        return self.empty((nbytes,), torch.uint8, result=False) if nbytes else None

    def on_device(self):
        if torch.cuda.current_device() == self.device.index:
            return contextlib.nullcontext()
        return torch.cuda.device(self.device)


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None or t.numel() == 0 else t.data_ptr()


def _check_type(tensors, names):
    dt = tensors[0].dtype
    if dt not in _DTYPES:
        raise TypeError(f"{names} must be float16 or bfloat16")
    for t in tensors:
        if t.dtype != dt:
            raise TypeError(f"{names} must have one dtype")
    return _DTYPES[dt]


def _check_device(tensors):
    dev = tensors[0].device
    for t in tensors:
        if not t.is_cuda:
            raise ValueError("all tensors must be device tensors (no CPU path)")
        if t.device != dev:
            raise ValueError("all tensors must be on one device")
    return dev


def _strides(t: torch.Tensor, name: str, dims: int):
    """Element strides of all but the last dimension, which is contiguous; 0
    for a dimension of one."""
    if t.dim() != dims:
        raise ValueError(f"{name} must be {dims}-D")
    if t.shape[-1] > 1 and t.stride(-1) != 1:
        raise ValueError(f"{name}'s last dimension must be contiguous")
    return [t.stride(i) if t.shape[i] > 1 else 0 for i in range(dims - 1)]


def _scale(scale, dim):
    scale = 1.0 / math.sqrt(dim) if scale is None else float(scale)
    if not (scale > 0.0 and math.isfinite(scale)):
        raise ValueError("scale must be positive and finite")
    return scale


def _offsets(seq_q, seq_k):
    if seq_q is None and seq_k is None:
        return 1
    if seq_q is None:
        raise ValueError("seq_k without seq_q")
    for t, n in ((seq_q, "seq_q"), (seq_k, "seq_k")):
        if t.dtype != torch.int32:
            raise TypeError(f"{n} must be int32")
        if t.dim() != 1 or t.shape[0] < 2 or (t.stride(0) != 1):
            raise ValueError(f"{n} must hold sequences + 1 offsets, contiguous")
    if seq_q.shape != seq_k.shape:
        raise ValueError("seq_q and seq_k disagree on the number of sequences")
    return seq_q.shape[0] - 1


def _packed_args(q, k, v, seq_q, seq_k, causal, scale, algo, splits):
    a = AttentionArgs()
    a.dtype = _check_type((q, k, v), "q, k and v")
    a.q_token, a.q_head = _strides(q, "q", 3)
    a.k_token, a.k_head = _strides(k, "k", 3)
    a.v_token, a.v_head = _strides(v, "v", 3)
    a.total_q, a.heads_q, a.head_dim = q.shape
    a.total_k, a.heads_kv, dk = k.shape
    if tuple(v.shape) != tuple(k.shape):
        raise ValueError("k and v must have one shape")
    if dk != a.head_dim:
        raise ValueError("q and k disagree on the head dimension")
    if a.heads_kv == 0 or a.heads_q == 0 or a.heads_q % a.heads_kv:
        raise ValueError("the query heads must be a multiple of the key heads")
    a.batch = _offsets(seq_q, seq_k)
    a.causal = 1 if causal else 0
    a.scale = _scale(scale, a.head_dim or 1)
    a.algo = ATTENTION_ALGOS[algo]
    a.splits = splits
    return a


def _like(t, ref, name):
    if t.dtype != ref.dtype:
        raise TypeError(f"{name} must have q's dtype")
    if tuple(t.shape) != tuple(ref.shape):
        raise ValueError(f"{name} must have shape {tuple(ref.shape)}")


def _check_lse(lse, shape):
    if lse.dtype != torch.float32:
        raise TypeError("lse must be float32")
    if tuple(lse.shape) != tuple(shape) or not lse.is_contiguous():
        raise ValueError(f"lse must be contiguous, of shape {tuple(shape)}")


def bind(lib, check):
    """The public functions over a loaded library."""

    def attention(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, *,
                  seq_q: Optional[torch.Tensor] = None, seq_k: Optional[torch.Tensor] = None,
                  causal: bool = True, scale: Optional[float] = None,
                  out: Optional[torch.Tensor] = None, return_lse: bool = False,
                  algo: str = "auto", splits: int = 0, stream=None):
        """softmax(scale q k^T) v over packed sequences on the GPU.

        q (tokens, heads, dim), k and v (tokens, kv heads, dim), float16 or
        bfloat16, any 16-byte aligned token and head strides; heads is a
        multiple of kv heads (grouped heads), dim a multiple of 8 up to 256.
        seq_q, seq_k: sequences + 1 int32 offsets on the device (one sequence
        without them; seq_k defaults to seq_q).  causal: query token t of a
        sequence with lq queries and lk keys sees the keys up to t + lk - lq.
        scale defaults to dim ** -0.5.  Returns out (tokens, heads, dim), with
        return_lse also the log-sum-exp (tokens, heads) float32; a query
        without visible keys has out 0 and -inf.  Rows behind the last
        sequence are not written.  No autograd graph is recorded:
        attention_backward gives the gradients."""
        if seq_q is not None and seq_k is None:
            seq_k = seq_q
        a = _packed_args(q, k, v, seq_q, seq_k, causal, scale, algo, splits)
        if out is not None:
            _like(out, q, "out")
            a.out_token, a.out_head = _strides(out, "out", 3)
        tensors = [t for t in (q, k, v, seq_q, seq_k, out) if t is not None]
        run = _Run(_check_device(tensors), stream, tensors)
        if out is None:
            out = run.empty(q.shape, q.dtype)
            a.out_token, a.out_head = _strides(out, "out", 3)
        lse = run.empty(q.shape[:2], torch.float32) if return_lse else None
        ptrs = [_ptr(t) for t in (q, k, v)] + \
            [None if t is None else t.data_ptr() for t in (seq_q, seq_k)] + [_ptr(out), _ptr(lse)]
        need = _i64(0)
        check(lib.attention_packed_plan(a, *ptrs, None, None, need))
        ws = run.workspace(need.value)
        with run.on_device():
            check(lib.attention_packed(a, *ptrs, _ptr(ws), need.value, run.handle))
        return (out, lse) if return_lse else out

    def attention_plan(q, k, v, *, seq_q=None, seq_k=None, causal=True, scale=None, algo="auto",
                       splits=0) -> Tuple[str, int, int]:
        """(kernel, key splits, workspace bytes) attention() takes for these
        tensors; their data is not read."""
        if seq_q is not None and seq_k is None:
            seq_k = seq_q
        a = _packed_args(q, k, v, seq_q, seq_k, causal, scale, algo, splits)
        a.out_token, a.out_head = a.heads_q * a.head_dim, a.head_dim
        al, sp, need = _i32(0), _i32(0), _i64(0)
        check(lib.attention_packed_plan(
            a, *[_ptr(t) for t in (q, k, v)],
            *[None if t is None else t.data_ptr() for t in (seq_q, seq_k)],
            1 << 40, None, al, sp, need))
        return _NAMES[al.value], sp.value, need.value

    def attention_backward(dout: torch.Tensor, q: torch.Tensor, k: torch.Tensor, v: torch.Tensor,
                           out: torch.Tensor, lse: torch.Tensor, *,
                           seq_q: Optional[torch.Tensor] = None,
                           seq_k: Optional[torch.Tensor] = None, causal: bool = True,
                           scale: Optional[float] = None, stream=None):
        """(dq, dk, dv) of sum(out * dout) for attention()'s arguments and
        its out and lse.  The gradients of a group's shared kv head are summed
        over its query heads; tokens of no sequence have gradient 0.  The same
        arguments give the same bits."""
        if seq_q is not None and seq_k is None:
            seq_k = seq_q
        g = AttentionGradArgs()
        g.f = _packed_args(q, k, v, seq_q, seq_k, causal, scale, "auto", 0)
        _like(dout, q, "dout")
        _like(out, q, "out")
        _check_lse(lse, q.shape[:2])
        g.f.out_token, g.f.out_head = _strides(out, "out", 3)
        g.dout_token, g.dout_head = _strides(dout, "dout", 3)
        tensors = [t for t in (dout, q, k, v, out, lse, seq_q, seq_k) if t is not None]
        run = _Run(_check_device(tensors), stream, tensors)
        dq, dk, dv = (run.empty(t.shape, t.dtype) for t in (q, k, v))
        g.dq_token, g.dq_head = _strides(dq, "dq", 3)
        g.dk_token, g.dk_head = _strides(dk, "dk", 3)
        g.dv_token, g.dv_head = _strides(dv, "dv", 3)
        ptrs = [_ptr(t) for t in (dout, q, k, v, out, lse)] + \
            [None if t is None else t.data_ptr() for t in (seq_q, seq_k)] + \
            [_ptr(t) for t in (dq, dk, dv)]
        need = _i64(0)
        check(lib.attention_packed_backward_plan(g, *ptrs, need))
        ws = run.workspace(need.value)
        with run.on_device():
            check(lib.attention_packed_backward(g, *ptrs, _ptr(ws), need.value, run.handle))
        return dq, dk, dv

    def attention_prefix(q: torch.Tensor, prefix_k: torch.Tensor, prefix_v: torch.Tensor,
                         k: torch.Tensor, v: torch.Tensor, lengths: torch.Tensor, *,
                         scale: Optional[float] = None, out: Optional[torch.Tensor] = None,
                         return_lse: bool = False, algo: str = "auto",
                         splits: Tuple[int, int] = (0, 0), stream=None):
        """Attention of a decoding batch whose sequences share a prefix.

        q (batch, heads, dim) or (batch, new tokens, heads, dim); prefix_k,
        prefix_v (prefix, kv heads, dim); k, v (batch, capacity, kv heads,
        dim): each sequence's own cache, of which lengths[b] (int32, on the
        device) keys are held, those of the new tokens last.  A new token sees
        the whole prefix and its own sequence's keys up to itself.  The prefix
        is read once for the whole batch.  Returns out of q's shape, with
        return_lse also the log-sum-exp (float32, q's shape without dim)."""
        a = AttentionPrefixArgs()
        a.dtype = _check_type((q, prefix_k, prefix_v, k, v), "q, the prefix, k and v")
        if q.dim() not in (3, 4):
            raise ValueError("q must be (batch, heads, dim) or (batch, tokens, heads, dim)")
        x = q if q.dim() == 4 else q.unsqueeze(1)
        a.q_batch, a.q_token, a.q_head = _strides(x, "q", 4)
        a.batch, a.q_tokens, a.heads_q, a.head_dim = x.shape
        a.prefix_k_token, a.prefix_k_head = _strides(prefix_k, "prefix_k", 3)
        a.prefix_v_token, a.prefix_v_head = _strides(prefix_v, "prefix_v", 3)
        a.k_batch, a.k_token, a.k_head = _strides(k, "k", 4)
        a.v_batch, a.v_token, a.v_head = _strides(v, "v", 4)
        a.prefix, a.heads_kv, dim = prefix_k.shape
        a.capacity = k.shape[1]
        if prefix_v.shape != prefix_k.shape or v.shape != k.shape:
            raise ValueError("keys and values must have one shape")
        if dim != a.head_dim or k.shape[3] != dim or k.shape[2] != a.heads_kv or \
                k.shape[0] != a.batch:
            raise ValueError("q, the prefix and the cache disagree on batch, heads or dim")
        if a.batch == 0:
            raise ValueError("the batch is empty")
        if a.heads_kv == 0 or a.heads_q == 0 or a.heads_q % a.heads_kv:
            raise ValueError("the query heads must be a multiple of the key heads")
        if lengths.dtype != torch.int32:
            raise TypeError("lengths must be int32")
        if tuple(lengths.shape) != (a.batch,) or (a.batch > 1 and lengths.stride(0) != 1):
            raise ValueError("lengths must hold one length per sequence, contiguous")
        a.scale = _scale(scale, a.head_dim or 1)
        a.algo = ATTENTION_ALGOS[algo]
        a.splits_prefix, a.splits_own = splits
        if out is not None:
            _like(out, q, "out")
        tensors = [t for t in (q, prefix_k, prefix_v, k, v, lengths, out) if t is not None]
        run = _Run(_check_device(tensors), stream, tensors)
        if out is None:
            out = run.empty(q.shape, q.dtype)
        y = out if q.dim() == 4 else out.unsqueeze(1)
        a.out_batch, a.out_token, a.out_head = _strides(y, "out", 4)
        lse = run.empty(q.shape[:-1], torch.float32) if return_lse else None
        ptrs = [_ptr(t) for t in (q, prefix_k, prefix_v, k, v)] + [lengths.data_ptr()] + \
            [_ptr(out), _ptr(lse)]
        need = _i64(0)
        check(lib.attention_prefix_plan(a, *ptrs, None, None, None, need))
        ws = run.workspace(need.value)
        with run.on_device():
            check(lib.attention_prefix(a, *ptrs, _ptr(ws), need.value, run.handle))
        return (out, lse) if return_lse else out

    return attention, attention_plan, attention_backward, attention_prefix
