"""The attention functions' refusals, without a GPU: the C ABI on addresses
that are never followed, the Python entry points on CPU tensors; and their
plans."""
import ctypes

import pytest
import torch

import mma_fragment_layouts_tn_amd as mfl
from mma_fragment_layouts_tn_amd import _attention as B

P = 0x100000         # fake, aligned device addresses (never followed)
(NEG, LD, NULL, ALIGN, ALIAS, UNSUP, LARGE, WS) = (-1, -2, -3, -7, -8, -4, -9, -10)


def packed(**kw):
    a = dict(dtype=B.BF16, causal=1, batch=2, total_q=40, total_k=50, heads_q=8, heads_kv=2,
             head_dim=128, q_token=1024, q_head=128, k_token=256, k_head=128, v_token=256,
             v_head=128, out_token=1024, out_head=128, scale=0.1, algo=0, splits=0)
    a.update(kw)
    return B.AttentionArgs(*[a[n] for n, _ in B.AttentionArgs._fields_])


PTRS = dict(q=P, k=2 * P, v=3 * P, seq_q=4 * P, seq_k=5 * P, out=6 * P, lse=7 * P)


def plan(a, **kw):
    p = dict(PTRS, **kw)
    al, sp, n = ctypes.c_int32(-1), ctypes.c_int32(-1), ctypes.c_int64(-1)
    rc = B._lib.attention_packed_plan(a, *p.values(), al, sp, n)
    # the call itself refuses alike, before anything is launched
    if rc:
        assert B._lib.attention_packed(a, *p.values(), None, 0, None) == rc
    return rc, al.value, sp.value, n.value


def test_codes_are_named():
    seen = {mfl.lib.gemm_strerror(c) for c in (NEG, LD, NULL, ALIGN, ALIAS, UNSUP, LARGE, WS)}
    assert len(seen) == 8


@pytest.mark.parametrize("kw,code", [
    (dict(total_q=-1), NEG), (dict(total_k=-1), NEG), (dict(batch=-1), NEG),
    (dict(heads_q=-8), NEG), (dict(head_dim=-8), NEG),
    (dict(dtype=2), UNSUP), (dict(dtype=0), UNSUP), (dict(batch=0), UNSUP),
    (dict(heads_kv=0), UNSUP), (dict(heads_q=0), UNSUP), (dict(heads_q=9), UNSUP),
    (dict(head_dim=0), UNSUP), (dict(head_dim=100), UNSUP), (dict(head_dim=264), UNSUP),
    (dict(scale=0.0), UNSUP), (dict(scale=-1.0), UNSUP), (dict(scale=float("inf")), UNSUP),
    (dict(scale=float("nan")), UNSUP), (dict(causal=2), UNSUP), (dict(algo=3), UNSUP),
    (dict(algo=-1), UNSUP), (dict(splits=-1), UNSUP), (dict(splits=1025), UNSUP),
    (dict(q_token=-8), LD), (dict(out_head=-128), LD),
    (dict(q_token=1025), ALIGN), (dict(k_head=4), ALIGN), (dict(v_token=257), ALIGN),
    (dict(k_token=(1 << 23) + 8), LARGE), (dict(q_token=(1 << 23) + 8), LARGE),
    (dict(v_head=1 << 41), LARGE), (dict(total_q=1 << 31), LARGE), (dict(total_k=1 << 31), LARGE),
    (dict(total_q=1 << 29, out_token=1024), LARGE), (dict(batch=(1 << 24) + 1), LARGE),
    (dict(heads_q=1 << 17), LARGE),
    (dict(out_token=1016), ALIAS), (dict(out_token=0), ALIAS), (dict(out_head=0), ALIAS),
    (dict(out_head=120), ALIAS),
])
def test_packed_refuses_sizes(kw, code):
    assert plan(packed(**kw))[0] == code


@pytest.mark.parametrize("kw,code", [
    (dict(q=0), NULL), (dict(k=0), NULL), (dict(v=0), NULL), (dict(out=0), NULL),
    (dict(seq_q=0), NULL), (dict(seq_k=0), NULL), (dict(seq_q=0, seq_k=0), NULL),
    (dict(q=P + 8), ALIGN), (dict(k=P + 2), ALIGN), (dict(out=6 * P + 8), ALIGN),
    (dict(lse=7 * P + 2), ALIGN), (dict(seq_q=4 * P + 1), ALIGN),
    (dict(out=P), ALIAS), (dict(out=3 * P), ALIAS),
])
def test_packed_refuses_pointers(kw, code):
    assert plan(packed(), **kw)[0] == code


def test_packed_allows():
    assert plan(packed())[0] == 0
    assert plan(packed(), lse=0)[0] == 0
    assert plan(packed(batch=1), seq_q=0, seq_k=0)[0] == 0
    assert plan(packed(total_q=0), q=0, out=0)[0] == 0
    assert plan(packed(total_k=0), k=0, v=0)[0] == 0
    assert plan(packed(k_head=0, v_head=0, k_token=0))[0] == 0          # shared inputs
    # heads outside tokens
    assert plan(packed(out_token=128, out_head=128 * 40, q_token=128, q_head=128 * 40))[0] == 0
    assert plan(packed(total_q=1, out_token=0, q_token=0))[0] == 0


def test_packed_plans():
    """What is written in include/mfl_attention.h and what the rules say."""
    def p(q, k, **kw):
        return plan(packed(batch=1, total_q=q, total_k=k, heads_q=32, heads_kv=8, q_token=4096,
                           out_token=4096, **kw), seq_q=0, seq_k=0)[1:]
    assert p(1, 1) == (2, 1, 0)
    assert p(8192, 8192) == (1, 1, 0)
    algo, splits, n = p(1, 100000)
    assert algo == 2 and splits > 1 and n == splits * 32 * (4 * 128 + 8)
    algo, splits, n = p(64, 8192)
    assert algo == 1 and splits > 1 and n == splits * 64 * 32 * (4 * 128 + 8)
    assert p(8192, 8192, algo=2, splits=3) == (2, 3, 3 * 8192 * 32 * (4 * 128 + 8))


def test_packed_asks_for_its_workspace():
    a = packed(splits=2)
    need = plan(a)[3]
    assert need > 0
    for ws, n in ((None, 0), (9 * P, need - 1), (9 * P + 8, need)):
        assert B._lib.attention_packed(a, *PTRS.values(), ws, n, None) == WS


GPTRS = dict(dout=8 * P, q=P, k=2 * P, v=3 * P, out=6 * P, lse=7 * P, seq_q=4 * P, seq_k=5 * P,
             dq=10 * P, dk=11 * P, dv=12 * P)


def grad_plan(f=None, ptr=None, **kw):
    g = dict(dout_token=1024, dout_head=128, dq_token=1024, dq_head=128, dk_token=256,
             dk_head=128, dv_token=256, dv_head=128)
    g.update(kw)
    a = B.AttentionGradArgs(packed(**(f or {})), *g.values())
    p = dict(GPTRS, **(ptr or {}))
    n = ctypes.c_int64(-1)
    rc = B._lib.attention_packed_backward_plan(a, *p.values(), n)
    got = B._lib.attention_packed_backward(a, *p.values(), None, 0, None) if rc or n.value else 0
    assert got == (rc or (WS if n.value else 0))
    return rc


@pytest.mark.parametrize("f,ptr,kw,code", [
    ({}, {}, {}, 0),
    (dict(algo=7, splits=99), {}, {}, 0),            # not read
    (dict(head_dim=12), {}, {}, UNSUP),
    (dict(total_q=-1), {}, {}, NEG),
    ({}, dict(dout=0), {}, NULL), ({}, dict(lse=0), {}, NULL), ({}, dict(dq=0), {}, NULL),
    ({}, dict(dk=0), {}, NULL), ({}, dict(dv=0), {}, NULL), ({}, dict(out=0), {}, NULL),
    ({}, dict(dout=8 * P + 8), {}, ALIGN), ({}, dict(dk=11 * P + 4), {}, ALIGN),
    ({}, dict(dq=P), {}, ALIAS), ({}, dict(dk=11 * P, dv=11 * P), {}, ALIAS),
    ({}, dict(dq=7 * P), {}, ALIAS), ({}, dict(dv=8 * P), {}, ALIAS),
    ({}, {}, dict(dout_token=-8), LD), ({}, {}, dict(dout_token=0), LD),
    (dict(q_token=0), {}, {}, LD), (dict(q_token=120), {}, {}, LD),
    ({}, {}, dict(dout_token=(1 << 23) + 8), LARGE), ({}, {}, dict(dk_head=4), ALIGN),
    ({}, {}, dict(dq_token=0), ALIAS), ({}, {}, dict(dk_token=248), ALIAS),
    ({}, {}, dict(dv_head=0), ALIAS),
    (dict(total_q=1, q_token=0), {}, dict(dout_token=0), 0),
    (dict(total_q=0), dict(dout=0, q=0, out=0, lse=0, dq=0), {}, 0),
])
def test_backward_refuses(f, ptr, kw, code):
    assert grad_plan(f, ptr, **kw) == code


def prefix(**kw):
    a = dict(dtype=B.BF16, algo=0, batch=3, q_tokens=2, prefix=100, capacity=64, heads_q=8,
             heads_kv=2, head_dim=128, q_batch=2048, q_token=1024, q_head=128,
             prefix_k_token=256, prefix_k_head=128, prefix_v_token=256, prefix_v_head=128,
             k_batch=64 * 256, k_token=256, k_head=128, v_batch=64 * 256, v_token=256,
             v_head=128, out_batch=2048, out_token=1024, out_head=128, scale=0.1,
             splits_prefix=0, splits_own=0)
    a.update(kw)
    return B.AttentionPrefixArgs(*[a[n] for n, _ in B.AttentionPrefixArgs._fields_])


PPTRS = dict(q=P, prefix_k=2 * P, prefix_v=3 * P, k=4 * P, v=5 * P, lengths=6 * P, out=7 * P,
             lse=8 * P)


def prefix_plan(a, **kw):
    p = dict(PPTRS, **kw)
    out = [ctypes.c_int32(-1) for _ in range(3)] + [ctypes.c_int64(-1)]
    rc = B._lib.attention_prefix_plan(a, *p.values(), *out)
    if rc:
        assert B._lib.attention_prefix(a, *p.values(), None, 0, None) == rc
    return (rc, *[x.value for x in out])


@pytest.mark.parametrize("kw,ptr,code", [
    ({}, {}, 0),
    (dict(batch=-1), {}, NEG), (dict(q_tokens=-1), {}, NEG), (dict(prefix=-1), {}, NEG),
    (dict(capacity=-1), {}, NEG),
    (dict(batch=0), {}, UNSUP), (dict(dtype=5), {}, UNSUP), (dict(heads_q=3), {}, UNSUP),
    (dict(head_dim=20), {}, UNSUP), (dict(scale=0.0), {}, UNSUP), (dict(algo=3), {}, UNSUP),
    (dict(splits_own=-1), {}, UNSUP), (dict(splits_prefix=2000), {}, UNSUP),
    (dict(prefix=1 << 31), {}, LARGE), (dict(capacity=1 << 31), {}, LARGE),
    (dict(batch=1 << 20, q_tokens=1 << 10, out_batch=1 << 20), {}, LARGE),
    (dict(k_token=(1 << 23) + 8), {}, LARGE), (dict(prefix_v_token=1 << 24), {}, LARGE),
    (dict(k_batch=-8), {}, LD), (dict(k_batch=12), {}, ALIGN), (dict(prefix_k_head=2), {}, ALIGN),
    (dict(out_batch=1024), {}, ALIAS), (dict(out_token=0), {}, ALIAS),
    ({}, dict(q=0), NULL), ({}, dict(out=0), NULL), ({}, dict(prefix_k=0), NULL),
    ({}, dict(prefix_v=0), NULL), ({}, dict(k=0), NULL), ({}, dict(v=0), NULL),
    ({}, dict(lengths=0), NULL),
    ({}, dict(k=4 * P + 2), ALIGN), ({}, dict(lengths=6 * P + 2), ALIGN),
    ({}, dict(out=P), ALIAS), ({}, dict(out=5 * P), ALIAS),
    (dict(prefix=0), dict(prefix_k=0, prefix_v=0), 0),
    (dict(capacity=0), dict(k=0, v=0, lengths=0), 0),
    (dict(q_tokens=0), dict(q=0, out=0, k=0, v=0, prefix_k=0, prefix_v=0, lengths=0), 0),
    (dict(k_batch=0, v_batch=0), {}, 0),             # one cache for all
])
def test_prefix_refuses(kw, ptr, code):
    assert prefix_plan(prefix(**kw), **ptr)[0] == code


def test_prefix_asks_for_its_workspace():
    """Two parts at least are joined, unless one of the two has no keys."""
    rc, algo, x, y, need = prefix_plan(prefix())
    assert rc == 0 and algo == 2 and x >= 1 and y >= 1 and need == (x + y) * 48 * (4 * 128 + 8)
    assert prefix_plan(prefix(prefix=0, splits_own=1))[2:] == (0, 1, 0)
    assert prefix_plan(prefix(capacity=0, splits_prefix=1))[2:] == (1, 0, 0)
    for ws, n in ((None, 0), (9 * P, need - 1), (9 * P + 4, need)):
        assert B._lib.attention_prefix(prefix(), *PPTRS.values(), ws, n, None) == WS


# ------------------------------------------------------------ Python checks
def tensors(tq=6, tk=7, h=4, g=2, d=16, dtype=torch.float16):
    return (torch.zeros(tq, h, d, dtype=dtype), torch.zeros(tk, g, d, dtype=dtype),
            torch.zeros(tk, g, d, dtype=dtype))


def off(*x):
    return torch.tensor(x, dtype=torch.int32)


@pytest.mark.parametrize("change,error", [
    (dict(), ValueError),                                     # CPU tensors
    (dict(q=torch.zeros(6, 4, 16)), TypeError),
    (dict(k=torch.zeros(7, 2, 16, dtype=torch.bfloat16)), TypeError),
    (dict(q=torch.zeros(6, 64, dtype=torch.float16)), ValueError),
    (dict(q=torch.zeros(6, 3, 16, dtype=torch.float16)), ValueError),
    (dict(q=torch.zeros(6, 4, 24, dtype=torch.float16)), ValueError),
    (dict(v=torch.zeros(8, 2, 16, dtype=torch.float16)), ValueError),
    (dict(q=torch.zeros(6, 16, 4, dtype=torch.float16).transpose(1, 2)), ValueError),
    (dict(seq_k=off(0, 7)), ValueError),
    (dict(seq_q=off(0, 6), seq_k=off(0, 3, 7)), ValueError),
    (dict(seq_q=torch.tensor([0, 6])), TypeError),
    (dict(seq_q=off(0)), ValueError),
    (dict(seq_q=off(0, 1, 6, 7)[::2], seq_k=off(0, 7)), ValueError),
    (dict(scale=0.0), ValueError), (dict(scale=float("nan")), ValueError),
    (dict(algo="other"), KeyError),
    (dict(out=torch.zeros(6, 4, 16)), TypeError),
    (dict(out=torch.zeros(5, 4, 16, dtype=torch.float16)), ValueError),
])
def test_attention_refuses(change, error):
    q, k, v = tensors()
    kw = dict(q=q, k=k, v=v)
    kw.update(change)
    with pytest.raises(error):
        mfl.attention(kw.pop("q"), kw.pop("k"), kw.pop("v"), **kw)


@pytest.mark.parametrize("change,error", [
    (dict(), ValueError),
    (dict(dout=torch.zeros(6, 4, 16)), TypeError),
    (dict(out=torch.zeros(6, 4, 8, dtype=torch.float16)), ValueError),
    (dict(lse=torch.zeros(6, 4, dtype=torch.float64)), TypeError),
    (dict(lse=torch.zeros(4, 6)), ValueError),
    (dict(lse=torch.zeros(4, 6).t()), ValueError),
])
def test_backward_refuses_tensors(change, error):
    q, k, v = tensors()
    kw = dict(dout=torch.zeros_like(q), q=q, k=k, v=v, out=torch.zeros_like(q),
              lse=torch.zeros(6, 4))
    kw.update(change)
    with pytest.raises(error):
        mfl.attention_backward(*kw.values())


@pytest.mark.parametrize("change,error", [
    (dict(), ValueError),
    (dict(q=torch.zeros(2, 64, dtype=torch.float16)), ValueError),
    (dict(q=torch.zeros(3, 4, 16, dtype=torch.float16)), ValueError),
    (dict(pk=torch.zeros(5, 2, 16)), TypeError),
    (dict(pv=torch.zeros(4, 2, 16, dtype=torch.float16)), ValueError),
    (dict(k=torch.zeros(2, 9, 1, 16, dtype=torch.float16)), ValueError),
    (dict(lengths=torch.zeros(2, dtype=torch.int64)), TypeError),
    (dict(lengths=off(1, 2, 3)), ValueError),
    (dict(lengths=off(1, 2, 3, 4)[::2]), ValueError),
    (dict(q=torch.zeros(0, 4, 16, dtype=torch.float16)), ValueError),
])
def test_prefix_refuses_tensors(change, error):
    f = torch.float16
    kw = dict(q=torch.zeros(2, 4, 16, dtype=f), pk=torch.zeros(5, 2, 16, dtype=f),
              pv=torch.zeros(5, 2, 16, dtype=f), k=torch.zeros(2, 9, 2, 16, dtype=f),
              v=torch.zeros(2, 9, 2, 16, dtype=f), lengths=off(9, 9))
    kw.update(change)
    with pytest.raises(error):
        mfl.attention_prefix(*kw.values())


def test_plan_on_cpu_tensors():
    """attention_plan reads no data: (kernel, splits, workspace bytes)."""
    q, k, v = tensors(1, 4096, 4, 2, 64)
    kind, splits, n = mfl.attention_plan(q, k, v)
    assert kind == "flat" and splits > 1 and n == splits * 4 * (4 * 64 + 8)
    assert mfl.attention_plan(*tensors(2000, 2000, 32, 8, 64))[0] == "tall"
