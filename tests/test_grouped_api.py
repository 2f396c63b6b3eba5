"""Refusals of the products by groups of rows, without a GPU: the C ABI on
addresses that are never followed, the Python entry points on CPU tensors; and
their plans."""
import ctypes

import pytest
import torch

import mma_fragment_layouts_tn_amd as mfl
from mma_fragment_layouts_tn_amd import _grouped as B

P = 0x100000         # fake, aligned device addresses (never followed)
(NEG, LD, NULL, UNSUP, CASE, ALIGN, ALIAS, LARGE, WS) = (-1, -2, -3, -4, -6, -7, -8, -9, -10)
BF16, F16, F32, I32 = mfl.BF16, mfl.F16, mfl.F32, 4


# ---------------------------------------------------------------- the C ABI
def grouped(**kw):
    a = dict(dtype=BF16, out=BF16, algo=0, groups=4, places=100, a_rows=100, n=64, k=128, lda=128,
             ldb=128, b_group=64 * 128, ldd=64)
    a.update(kw)
    return B.GroupedArgs(*[a[n] for n, _ in B.GroupedArgs._fields_])


GPTRS = dict(A=P, B=2 * P, offsets=3 * P, rows=4 * P, D=5 * P)


def plan(a, **kw):
    p = dict(GPTRS, **kw)
    al = ctypes.c_int32(-1)
    rc = B._lib.gemm_tn_grouped_plan(a, *p.values(), al)
    if rc:      # the call itself refuses alike, before anything is launched
        assert B._lib.gemm_tn_grouped(a, *p.values(), None) == rc
    return rc, al.value


SIZES = [
    (dict(groups=-1), NEG), (dict(places=-1), NEG), (dict(a_rows=-1), NEG), (dict(n=-8), NEG),
    (dict(k=-8), NEG),
    (dict(groups=0), UNSUP), (dict(n=0), UNSUP), (dict(k=0), UNSUP), (dict(dtype=F32), UNSUP),
    (dict(dtype=0), UNSUP), (dict(out=F16), UNSUP), (dict(out=0), UNSUP), (dict(algo=-1), UNSUP),
    (dict(algo=4), UNSUP),
    (dict(groups=4097), LARGE), (dict(places=1 << 31), LARGE), (dict(n=(1 << 21) + 8), LARGE),
    (dict(k=(1 << 21) + 8), LARGE), (dict(lda=(1 << 21) + 8), LARGE),
    (dict(ldb=(1 << 21) + 8), LARGE), (dict(b_group=1 << 43), LARGE),
    (dict(a_rows=1 << 23), LARGE),          # gathered rows over 2 GiB of A
    (dict(n=60), ALIGN), (dict(k=124, lda=128, ldb=128), ALIGN), (dict(lda=132), ALIGN),
    (dict(ldb=130), ALIGN), (dict(ldd=66), ALIGN), (dict(b_group=8193), ALIGN),
    (dict(lda=120), LD), (dict(ldb=120), LD), (dict(ldd=56), LD), (dict(b_group=-8), LD),
]


@pytest.mark.parametrize("kw,code", SIZES)
def test_grouped_refuses_sizes(kw, code):
    assert plan(grouped(**kw))[0] == code


@pytest.mark.parametrize("kw,code", [
    (dict(A=0), NULL), (dict(B=0), NULL), (dict(offsets=0), NULL), (dict(D=0), NULL),
    (dict(A=P + 8), ALIGN), (dict(B=P + 2), ALIGN), (dict(D=P + 8), ALIGN),
    (dict(offsets=P + 2), ALIGN), (dict(rows=P + 1), ALIGN),
    (dict(D=P), ALIAS), (dict(D=2 * P), ALIAS), (dict(D=4 * P), ALIAS),
])
def test_grouped_refuses_pointers(kw, code):
    assert plan(grouped(), **kw)[0] == code


def test_grouped_accepts():
    assert plan(grouped())[0] == 0
    assert plan(grouped(out=F32, ldd=128))[0] == 0
    assert plan(grouped(places=0), A=0, D=0)[0] == 0
    assert plan(grouped(b_group=0))[0] == 0                       # one matrix for all
    assert plan(grouped(a_rows=1 << 23, places=1 << 23), rows=0)[0] == 0    # not gathered
    assert plan(grouped(a_rows=99), rows=0)[0] == UNSUP           # fewer rows than places
    assert plan(grouped(a_rows=3))[0] == 0                        # gathered: any number
    assert plan(None)[0] == NULL


def test_grouped_chooses():
    """Few rows, and tiles by the mean; a given kernel is taken."""
    assert plan(grouped(groups=8, places=2, n=2048, k=4096, lda=4096, ldb=4096, ldd=2048))[1] == 1
    big = dict(groups=8, places=16384, n=2048, k=4096, lda=4096, ldb=4096, ldd=2048)
    assert plan(grouped(**big), rows=0)[0] == UNSUP
    assert plan(grouped(a_rows=8192, **big))[1] == 3
    for algo in (1, 2, 3):
        assert plan(grouped(algo=algo))[1] == algo


def test_grouped_refuses_too_many_workgroups():
    a = grouped(groups=1, places=1 << 30, a_rows=1 << 30, n=1 << 21, ldd=1 << 21, k=8, lda=8, ldb=8,
                b_group=1 << 24)
    assert plan(a, rows=0)[0] == LARGE


def backward(a, grad=(), **kw):
    p = dict(dD=6 * P, A=P, B=2 * P, offsets=3 * P, rows=4 * P, dA=7 * P, dB=8 * P)
    p.update(kw)
    g = dict(ldda=a.k, lddb=a.k, db_group=a.n * a.k)
    g.update(grad)
    g = B.GroupedGradArgs(a, *g.values())
    rc = B._lib.gemm_tn_grouped_backward_plan(g, *p.values())
    if rc:
        assert B._lib.gemm_tn_grouped_backward(g, *p.values(), None) == rc
    return rc


@pytest.mark.parametrize("kw,code", SIZES)
def test_backward_refuses_sizes(kw, code):
    assert backward(grouped(**kw)) == code


def test_backward_refuses():
    a = grouped()
    assert backward(a) == 0
    assert backward(a, dA=0) == 0 and backward(a, dB=0) == 0
    assert backward(a, dD=P) == 0                      # inputs may share memory
    assert backward(grouped(algo=2)) == CASE
    for kw, code in [(dict(dD=0), NULL), (dict(dA=P), ALIAS), (dict(dB=2 * P), ALIAS),
                     (dict(dA=8 * P), ALIAS), (dict(dB=6 * P), ALIAS), (dict(dA=7 * P + 8), ALIGN),
                     (dict(dB=8 * P + 4), ALIGN)]:
        assert backward(a, **kw) == code
    for grad, code in [(dict(ldda=120), LD), (dict(lddb=132), ALIGN),
                       (dict(db_group=64 * 128 - 8), ALIAS), (dict(db_group=0), ALIAS),
                       (dict(ldda=1 << 22), LARGE)]:
        assert backward(a, grad) == code
    assert B._lib.gemm_tn_grouped_backward_plan(None, *[P] * 7) == NULL


def sort(**kw):
    a = dict(ids_type=I32, count=100, top=2, groups=8)
    a.update({k: kw.pop(k) for k in list(kw) if k in a})
    p = dict(ids=P, rows=2 * P, offsets=3 * P, slots=4 * P)
    p.update(kw)
    g, n = B.GroupRowsArgs(*a.values()), ctypes.c_int64(-1)
    rc = B._lib.group_rows_plan(g, *p.values(), n)
    if rc:
        assert B._lib.group_rows(g, *p.values(), None, 0, None) == rc
    elif n.value:
        for ws, size in ((None, 1 << 40), (9 * P, n.value - 1), (9 * P + 8, n.value)):
            assert B._lib.group_rows(g, *p.values(), ws, size, None) == WS
    return rc, n.value


def test_group_rows_refuses():
    assert sort() == (0, 0)
    for kw, code in [(dict(count=-2), NEG), (dict(top=-1), NEG), (dict(groups=-1), NEG),
                     (dict(groups=0), UNSUP), (dict(top=0), UNSUP), (dict(top=3), UNSUP),
                     (dict(ids_type=BF16), UNSUP), (dict(groups=4097), LARGE),
                     (dict(count=1 << 31), LARGE), (dict(ids=0), NULL), (dict(rows=0), NULL),
                     (dict(offsets=0), NULL), (dict(slots=0), NULL), (dict(ids=P + 2), ALIGN),
                     (dict(ids_type=5, ids=P + 4), ALIGN), (dict(slots=P + 1), ALIGN),
                     (dict(rows=P), ALIAS), (dict(slots=2 * P), ALIAS), (dict(offsets=P), ALIAS)]:
        assert sort(**kw)[0] == code, kw
    assert sort(count=0, ids=0, rows=0, slots=0) == (0, 0)


def test_group_rows_workspace_is_as_documented():
    """None up to one workgroup's choices, 4 (groups + 1) bytes per chunk begun,
    256 chunks at most."""
    for groups, alone, chunks in ((8, 8192, 3), (256, 8192, 3), (257, 1024, 2), (4096, 1024, 2)):
        assert sort(count=alone, top=1, groups=groups)[1] == 0
        assert sort(count=alone + 1, top=1, groups=groups)[1] == chunks * 4 * (groups + 1)
        for count in (1 << 20, (1 << 20) + 1, 1 << 24, (1 << 31) - (1 << 16) - 1):
            assert 0 < sort(count=count, top=1, groups=groups)[1] <= 256 * 4 * (groups + 1)


def combine(**kw):
    a = dict(dtype=BF16, out=BF16, tokens=50, top=2, n=64, x_rows=100, ldx=64, ldo=64)
    a.update({k: kw.pop(k) for k in list(kw) if k in a})
    p = dict(X=P, slots=2 * P, weights=3 * P, out=4 * P)
    p.update(kw.pop("ptrs", {}))
    c = B.CombineArgs(*a.values())
    return c, p


@pytest.mark.parametrize("kw,code", [
    (dict(tokens=-1), NEG), (dict(top=-1), NEG), (dict(n=-8), NEG), (dict(x_rows=-1), NEG),
    (dict(dtype=F32), UNSUP), (dict(out=F16), UNSUP), (dict(n=0), UNSUP), (dict(top=65), UNSUP),
    (dict(tokens=1 << 31), LARGE), (dict(tokens=1 << 30, top=4), LARGE),
    (dict(tokens=1 << 30, n=1024, ldx=1024, ldo=1024, top=1), LARGE),
    (dict(n=60), ALIGN), (dict(ldx=68), ALIGN), (dict(ldx=56), LD), (dict(ldo=56), LD),
    (dict(ptrs=dict(X=0)), NULL), (dict(ptrs=dict(slots=0)), NULL), (dict(ptrs=dict(out=0)), NULL),
    (dict(ptrs=dict(X=P + 8)), ALIGN), (dict(ptrs=dict(weights=P + 2)), ALIGN),
    (dict(ptrs=dict(out=P)), ALIAS), (dict(ptrs=dict(out=3 * P)), ALIAS),
])
def test_combine_refuses(kw, code):
    c, p = combine(**kw)
    assert B._lib.combine_rows(c, *p.values(), None) == code


@pytest.mark.parametrize("kw,code", [
    (dict(out=F32), UNSUP), (dict(lddx=56), LD), (dict(lddx=68), ALIGN), (dict(rows=0), NULL),
    (dict(dX=0), NULL), (dict(weights=0), UNSUP), (dict(dX=P), ALIAS), (dict(dX=4 * P), ALIAS),
    (dict(dw=3 * P), ALIAS), (dict(dX=7 * P + 8), ALIGN), (dict(tokens=1 << 28, top=8), LARGE),
])
def test_combine_backward_refuses(kw, code):
    p = dict(lddx=64, dout=4 * P, X=P, slots=2 * P, rows=5 * P, weights=3 * P, dX=7 * P, dw=8 * P)
    p.update({k: v for k, v in kw.items() if k in p})
    c, _ = combine(**{k: v for k, v in kw.items() if k not in p})
    assert B._lib.combine_rows_backward(c, *p.values(), None) == code


def adapters(ptrs=None, **kw):
    a = dict(dtype=BF16, out=BF16, algo=0, groups=4, places=100, x_rows=100, n=64, k=128, rank=16,
             ldx=128, ldw=128, lda=128, a_group=16 * 128, ldb=16, b_group=64 * 16, ldd=64)
    a.update(kw)
    p = dict(x=P, W=2 * P, A=3 * P, B=4 * P, offsets=5 * P, rows=6 * P, scale=7 * P, D=8 * P)
    p.update(ptrs or {})
    c, al, n = B.AdaptersArgs(*a.values()), ctypes.c_int32(-1), ctypes.c_int64(-1)
    rc = B._lib.gemm_tn_adapters_plan(c, *p.values(), al, n)
    if rc:
        assert B._lib.gemm_tn_adapters(c, *p.values(), 9 * P, 1 << 40, None) == rc
    elif a["places"] and n.value:
        for ws, size in ((None, 1 << 40), (9 * P, n.value - 1), (9 * P + 8, n.value)):
            assert B._lib.gemm_tn_adapters(c, *p.values(), ws, size, None) == WS
    return rc, al.value, n.value


@pytest.mark.parametrize("kw,code", [
    (dict(groups=-1), NEG), (dict(places=-1), NEG), (dict(x_rows=-1), NEG), (dict(rank=-8), NEG),
    (dict(groups=0), UNSUP), (dict(rank=0), UNSUP), (dict(n=0), UNSUP), (dict(dtype=F32), UNSUP),
    (dict(out=F16), UNSUP), (dict(algo=4), UNSUP),
    (dict(groups=4097), LARGE), (dict(rank=(1 << 21) + 8), LARGE), (dict(x_rows=1 << 23), LARGE),
    (dict(rank=12), ALIGN), (dict(n=68), ALIGN), (dict(ldx=132), ALIGN), (dict(ldb=20), ALIGN),
    (dict(a_group=2049), ALIGN), (dict(b_group=1), ALIGN),
    (dict(ldx=120), LD), (dict(ldw=120), LD), (dict(lda=120), LD), (dict(ldb=8), LD),
    (dict(ldd=56), LD), (dict(a_group=-8), LD),
] + [(dict(ptrs={x: 0}), NULL) for x in ("x", "W", "A", "B", "offsets", "D")] + [
    (dict(ptrs=dict(W=P + 8)), ALIGN), (dict(ptrs=dict(scale=P + 2)), ALIGN),
    (dict(ptrs=dict(D=P)), ALIAS), (dict(ptrs=dict(D=4 * P)), ALIAS),
])
def test_adapters_refuses(kw, code):
    assert adapters(**kw)[0] == code


def test_adapters_plans():
    """The workspace is as documented."""
    for places in (1, 48, 191, 193, 1000, 8192):
        for rank in (8, 16, 64):
            for out in (BF16, F32):
                for algo in (0, 1, 2, 3):
                    rc, al, n = adapters(places=places, x_rows=places, rank=rank, ldb=rank, out=out,
                                         algo=algo, k=4608, ldx=4608, ldw=4608, lda=4608, n=512,
                                         ldd=512)
                    assert rc == 0 and al == (algo or al) and al in (1, 2, 3)
                    least = 4 * places + places * rank * (6 if al > 1 and out == F32 else 4)
                    part = 4 * places * 512
                    if al > 1:
                        assert least <= n <= least + 32
                    else:
                        parts = (n - least) // part
                        assert 1 <= parts <= 18 and n - least - parts * part <= 32
    assert adapters(places=0, ptrs=dict(x=0, D=0))[0] == 0
    # small problems need none, unless their rank is large or tiles are asked for
    assert adapters()[1:] == (1, 0) and adapters(algo=1)[1:] == (1, 0)
    assert adapters(rank=72, ldb=72)[2] > 0 and adapters(algo=2)[2] > 0


# ------------------------------------------------------- the Python functions
def half(*shape):
    return torch.zeros(*shape, dtype=torch.bfloat16)


OFF = torch.tensor([0, 3, 6], dtype=torch.int32)


@pytest.mark.parametrize("kw,err", [
    (dict(A=torch.zeros(6, 16)), TypeError), (dict(B=half(2, 8, 16).half()), TypeError),
    (dict(A=half(6)), ValueError), (dict(B=half(8, 16)), ValueError),
    (dict(A=half(6, 24)), ValueError), (dict(A=half(16, 6).t()), ValueError),
    (dict(B=half(2, 16, 8).transpose(1, 2)), ValueError),
    (dict(offsets=OFF.long()), TypeError), (dict(offsets=OFF[:2]), ValueError),
    (dict(offsets=torch.zeros(6, dtype=torch.int32)[::2]), ValueError),
    (dict(rows=torch.arange(6)), TypeError),
    (dict(rows=torch.zeros(2, 3, dtype=torch.int32)), ValueError),
    (dict(out_dtype=torch.float16), TypeError), (dict(D=half(5, 8)), ValueError),
    (dict(D=half(6, 8), out_dtype=torch.float32), TypeError), (dict(algo="none"), KeyError),
    (dict(), ValueError),      # CPU tensors
])
def test_python_grouped_refuses(kw, err):
    a = dict(A=half(6, 16), B=half(2, 8, 16), offsets=OFF)
    a.update(kw)
    with pytest.raises(err):
        mfl.gemm_grouped(a.pop("A"), a.pop("B"), a.pop("offsets"), **a)


def test_python_other_functions_refuse_cpu_tensors_and_shapes():
    A, Bm, i32 = half(6, 16), half(2, 8, 16), torch.int32
    slots = torch.zeros(3, 2, dtype=i32)
    for f, err in [
            (lambda: mfl.group_rows(torch.zeros(4), 2), TypeError),
            (lambda: mfl.group_rows(torch.zeros(2, 2, 2, dtype=i32), 2), ValueError),
            (lambda: mfl.group_rows(torch.zeros(4, 2, dtype=i32).t(), 2), ValueError),
            (lambda: mfl.group_rows(torch.zeros(4, dtype=i32), 0), ValueError),
            (lambda: mfl.group_rows(torch.zeros(4, dtype=i32), 2), ValueError),
            (lambda: mfl.gemm_grouped_backward(half(6, 8).half(), A, Bm, OFF), TypeError),
            (lambda: mfl.gemm_grouped_backward(half(5, 8), A, Bm, OFF), ValueError),
            (lambda: mfl.gemm_grouped_backward(half(6, 8), A, Bm, OFF, dB_dtype=torch.float16),
             TypeError),
            (lambda: mfl.gemm_grouped_backward(half(6, 8), A, Bm, OFF), ValueError),
            (lambda: mfl.combine_rows(torch.zeros(6, 8), slots), TypeError),
            (lambda: mfl.combine_rows(half(6, 8), slots.long()), TypeError),
            (lambda: mfl.combine_rows(half(6, 8), slots, torch.zeros(3, 3)), ValueError),
            (lambda: mfl.combine_rows(half(6, 8), slots, half(3, 2)), TypeError),
            (lambda: mfl.combine_rows(half(6, 8), slots.t()), ValueError),
            (lambda: mfl.combine_rows(half(6, 8), slots, out=half(2, 8)), ValueError),
            (lambda: mfl.combine_rows(half(6, 8), slots), ValueError),
            (lambda: mfl.combine_rows_backward(half(3, 9), half(6, 8), slots,
                                               rows=torch.zeros(6, dtype=i32)), ValueError),
            (lambda: mfl.combine_rows_backward(half(3, 8).half(), half(6, 8), slots,
                                               rows=torch.zeros(6, dtype=i32)), TypeError)]:
        with pytest.raises(err):
            f()


@pytest.mark.parametrize("kw,err", [
    (dict(x=torch.zeros(6, 16)), TypeError), (dict(W=half(8, 16).half()), TypeError),
    (dict(W=half(8, 24)), ValueError), (dict(A=half(2, 8, 24)), ValueError),
    (dict(B=half(2, 8, 16)), ValueError), (dict(x=half(16, 6).t()), ValueError),
    (dict(scale=torch.ones(3)), ValueError), (dict(scale=half(2)), TypeError),
    (dict(rows=torch.zeros(7, dtype=torch.int32)), ValueError),
    (dict(rows=torch.zeros(6)), TypeError), (dict(offsets=OFF[:1]), ValueError),
    (dict(D=half(5, 8)), ValueError), (dict(out_dtype=torch.float16), TypeError),
    (dict(), ValueError),
])
def test_python_adapters_refuses(kw, err):
    a = dict(x=half(6, 16), W=half(8, 16), A=half(2, 8, 16), B=half(2, 8, 8), offsets=OFF)
    a.update(kw)
    with pytest.raises(err):
        mfl.gemm_adapters(*[a.pop(n) for n in ("x", "W", "A", "B", "offsets")], **a)


def test_plans_need_no_gpu():
    assert mfl.gemm_grouped_plan(half(6, 16), half(2, 8, 16), OFF) == "few"
    for rank in (8, 72):
        algo, need = mfl.gemm_adapters_plan(half(6, 16), half(8, 16), half(2, rank, 16),
                                            half(2, 8, rank), OFF)
        assert algo == "few" and (need > 0) == (rank > 64)
