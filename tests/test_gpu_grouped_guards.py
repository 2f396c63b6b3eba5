"""Products by groups of rows through the C ABI, on buffers with canaries before
and behind every operand, output and workspace: for offsets out of range and
out of order, rows, slots and ids from outside, and odd sizes, nothing beside
the outputs is written and no operand is, and the gaps between padded rows keep
what they held.  Offsets that grow once they are held inside the places give the
results of what they say, and rows of no group stay as they were; of others
(groups that overlap have more tiles than a launch of that many places) only
the bounds are kept.  A workspace's contents change no result."""
import ctypes

import numpy as np
import pytest
import torch

import mma_fragment_layouts_tn_amd as mfl
from gpu_helpers import say
from mma_fragment_layouts_tn_amd import _grouped as B
from oracle import grouped as G
from test_gpu_grouped import ALGOS, DT, f64, values, within

pytestmark = pytest.mark.gpu

GUARD = 4096              # bytes before and behind
CODE = {"f16": mfl.F16, "bf16": mfl.BF16, "f32": mfl.F32}
CANARY = 0x5a             # (as 16 or 32 bits a finite number)


class Held:
    """A tensor in the middle of a buffer of canaries; an output without data
    holds canaries too."""

    def __init__(self, data=None, *, shape=None, dtype=None, ld=None, fill=CANARY):
        shape, dtype = (data.shape, data.dtype) if data is not None else (shape, dtype)
        self.shape, size = shape, torch.empty(0, dtype=dtype).element_size()
        width = shape[-1] if shape else 1
        self.ld = width if ld is None else ld
        lines = int(np.prod(shape[:-1])) if len(shape) else 1
        self.bytes = lines * self.ld * size
        self.buf = torch.full((self.bytes + 2 * GUARD,), CANARY, dtype=torch.uint8, device="cuda")
        self.buf[GUARD:GUARD + self.bytes] = fill
        self.lines = self.buf[GUARD:GUARD + self.bytes].view(dtype).view(lines, self.ld)
        self.t = self.lines[:, :width]
        if data is not None:
            self.t.copy_(data.reshape(lines, width))
        self.before = self.buf.clone()

    @property
    def ptr(self):
        return self.buf.data_ptr() + GUARD

    def get(self):
        return self.t.reshape(self.shape)

    def intact(self):
        """The canaries around, and between the rows."""
        edge = torch.cat([self.buf[:GUARD], self.buf[GUARD + self.bytes:]])
        gaps = self.lines[:, self.t.shape[1]:].reshape(-1).view(torch.uint8)
        return bool((edge == CANARY).all()) and bool((gaps == CANARY).all())

    def unchanged(self):
        return torch.equal(self.buf, self.before)

    def canary_rows(self):
        """Which rows still hold canaries alone."""
        return (self.t.contiguous().view(torch.uint8).view(self.t.shape[0], -1) == CANARY) \
            .all(1).cpu().numpy()


def stream():
    return torch.cuda.current_stream().cuda_stream


def ints(x):
    return Held(torch.as_tensor(x).to(torch.int32))


def finish(name, rc, inputs, outputs):
    torch.cuda.synchronize()
    assert rc == 0, (name, mfl.strerror(rc))
    for i, t in enumerate(inputs):
        assert t.unchanged(), f"{name}: operand {i} written"
    for i, t in enumerate(outputs):
        assert t.intact(), f"{name}: beside output {i}"


def growing(offsets, places):
    return bool((np.diff(np.clip(offsets, 0, places)) >= 0).all())


def membership(offsets, places):
    """How many groups hold each place, the one behind the last among them."""
    count = np.zeros(places, int)
    for a, b in G._spans(np.concatenate([np.asarray(offsets, np.int64), [places]]), places):
        count[a:b] += 1
    return count


BAD = [[0, 30, 70, 90], [-5, 30, 1 << 30, 90], [0, 80, 20, 90], [0, 0, 0, -1], [90, 90, 90, 90],
       [2 ** 31 - 1, -2 ** 31, 50, 3], [40, 45, 50, 60], [0, 80, 20, 50]]


class Product:
    def __init__(self, kind, places, offsets, n, k, *, gather, pad, seed=0):
        gen = torch.Generator().manual_seed(seed + n + k + places)
        self.kind, self.n, self.k, self.offsets = kind, n, k, np.asarray(offsets)
        self.places, self.groups = places, len(offsets) - 1
        self.m = max(1, places // 2) if gather else places
        self.pad = pad
        self.hA = values(gen, (self.m, k), kind)
        self.hB = values(gen, (self.groups, n, k), kind, k ** -0.5)
        self.hd = values(gen, (places, n), kind)
        self.hr = torch.randint(-2, self.m + 2, (places,), generator=gen) if gather else None
        self.A, self.B = Held(self.hA, ld=k + pad), Held(self.hB, ld=k + pad)
        self.dD, self.o = Held(self.hd, ld=n + pad), ints(offsets)
        self.rows = ints(self.hr) if gather else None
        self.operands = [self.A, self.B, self.o] + ([self.rows] if gather else [])

    def args(self, out, algo, ldd):
        p = self.pad
        return B.GroupedArgs(CODE[self.kind], CODE[out], B.GROUPED_ALGOS[algo], self.groups,
                             self.places, self.m, self.n, self.k, self.k + p, self.k + p,
                             self.n * (self.k + p), ldd)

    def ref(self):
        return None if self.hr is None else self.hr.numpy()

    def forward(self, out, algo):
        D = Held(shape=(self.places, self.n), dtype=DT[out], ld=self.n + 2 * self.pad)
        rc = B._lib.gemm_tn_grouped(self.args(out, algo, D.ld), self.A.ptr, self.B.ptr, self.o.ptr,
                                    self.rows and self.rows.ptr, D.ptr, stream())
        finish(f"forward {algo}", rc, self.operands, [D])
        if not growing(self.offsets, self.places):
            return
        want, tol = G.product(f64(self.hA), f64(self.hB), self.offsets, self.ref(), out)
        count = membership(self.offsets, self.places)
        once = (count == 1) & ~np.isnan(want[:, 0])
        want[~once] = np.nan
        within(f"D {algo}", D.get(), want, tol)
        held = D.canary_rows()
        assert held[count == 0].all()
        behind = (count == 1) & ~once            # of no group
        assert held[behind].all()

    def backward(self, out):
        dA = Held(shape=(self.places, self.k), dtype=DT[self.kind], ld=self.k + self.pad)
        dB = Held(shape=(self.groups, self.n, self.k), dtype=DT[out], ld=self.k + self.pad)
        f = self.args(out, "auto", self.n + self.pad)
        a = B.GroupedGradArgs(f, dA.ld, dB.ld, self.n * dB.ld)
        rc = B._lib.gemm_tn_grouped_backward(a, self.dD.ptr, self.A.ptr, self.B.ptr, self.o.ptr,
                                             self.rows and self.rows.ptr, dA.ptr, dB.ptr, stream())
        finish("backward", rc, self.operands + [self.dD], [dA, dB])
        if not growing(self.offsets, self.places):
            return
        want, tol = G.gradients(f64(self.hd), f64(self.hA), f64(self.hB), self.offsets, self.ref(),
                                self.kind, out)
        count = membership(self.offsets, self.places)
        want[0][count != 1] = np.nan
        within("dA", dA.get(), want[0], tol[0])
        within("dB", dB.get(), want[1], tol[1])
        assert dA.canary_rows()[count == 0].all()


@pytest.mark.parametrize("offsets", BAD)
@pytest.mark.parametrize("gather", [False, True])
def test_product_offsets(offsets, gather):
    say(f"[gpu] offsets {offsets}, gather={gather}")
    c = Product("f16", 90, offsets, 72, 104, gather=gather, pad=8)
    for algo in ALGOS:
        c.forward("f16", algo)
    c.forward("f32", "tile256")
    c.backward("f16")


@pytest.mark.parametrize("lens", [[1], [17, 0, 33], [0, 257, 1], [130, 5, 64, 0]])
@pytest.mark.parametrize("n,k,pad", [(8, 8, 0), (72, 136, 24), (264, 72, 8)])
def test_product_sizes(lens, n, k, pad):
    say(f"[gpu] lens {lens}, n={n} k={k} pad={pad}")
    offsets = [0] + np.cumsum(lens).tolist()
    for tail in (0, 19):
        c = Product("bf16", offsets[-1] + tail, offsets, n, k, gather=tail > 0, pad=pad)
        for algo in ALGOS:
            c.forward("bf16" if n > 8 else "f32", algo)
        c.backward("f32" if pad else "bf16")


def test_many_groups_out_of_order():
    """Groups beyond those that are numbered without gaps."""
    gen = torch.Generator().manual_seed(3)
    offsets = torch.randint(-50, 700, (301,), generator=gen).tolist()
    for o in (offsets, sorted(offsets)):
        c = Product("f16", 600, o, 40, 64, gather=True, pad=8)
        for algo in ("few", "tile128"):
            c.forward("f16", algo)
        c.backward("f16")


# ---------------------------------------------------------------- adapters
class Adapters:
    def __init__(self, kind, places, offsets, rank, n, k, *, pad, rows=False, seed=0):
        gen = torch.Generator().manual_seed(seed + places + rank + n + k)
        a = len(offsets) - 1
        self.kind, self.places, self.rank, self.n, self.k = kind, places, rank, n, k
        self.offsets, self.groups, self.pad = np.asarray(offsets), a, pad
        self.x, self.W = values(gen, (places, k), kind), values(gen, (n, k), kind, k ** -0.5)
        self.a = values(gen, (a, rank, k), kind, k ** -0.5)
        self.b = values(gen, (a, n, rank), kind, rank ** -0.5)
        self.scale = torch.rand(a, generator=gen) + 0.5
        # rows: two of them from outside
        self.r = None
        if rows:
            self.r = torch.randperm(places, generator=gen)
            self.r[0], self.r[-1] = -1, places
        self.held = [Held(self.x, ld=k + pad), Held(self.W, ld=k + pad), Held(self.a, ld=k + pad),
                     Held(self.b, ld=rank + pad), ints(offsets)] + \
            ([ints(self.r)] if rows else []) + [Held(self.scale)]

    def run(self, out, algo, fill):
        p, n, k, rank = self.pad, self.n, self.k, self.rank
        D = Held(shape=(self.places, n), dtype=DT[out], ld=n + p)
        c = B.AdaptersArgs(CODE[self.kind], CODE[out], B.GROUPED_ALGOS[algo], self.groups,
                           self.places, self.places, n, k, rank, k + p, k + p, k + p,
                           rank * (k + p), rank + p, n * (rank + p), n + p)
        ptrs = [t.ptr for t in self.held]
        if self.r is None:
            ptrs.insert(5, None)
        need = ctypes.c_int64(-1)
        rc = B._lib.gemm_tn_adapters_plan(c, *ptrs, D.ptr, None, need)
        assert rc == 0
        # (the workspace to the byte; canaries follow it)
        ws = Held(shape=(need.value,), dtype=torch.uint8, fill=fill) if need.value else None
        rc = B._lib.gemm_tn_adapters(c, *ptrs, D.ptr, ws and ws.ptr, need.value, stream())
        finish(f"adapters {algo}", rc, self.held, [D] + ([ws] if ws else []))
        return D

    def check(self, out, algo):
        # owners that the workspace held before: numbers of groups, or NaN for what follows
        first, second = (self.run(out, algo, fill) for fill in (0, 0xff))
        if not growing(self.offsets, self.places):
            return
        rows = np.arange(self.places) if self.r is None else self.r.numpy()
        want, tol = G.adapters(f64(self.x), f64(self.W), f64(self.a), f64(self.b), self.offsets,
                               rows, f64(self.scale), out)
        count = membership(self.offsets, self.places)
        listed = np.isin(np.arange(self.places), rows)
        ask = np.zeros(self.places, bool)
        for i, r in enumerate(rows):
            if 0 <= r < self.places and count[i] == 1:
                ask[r] = True
        want[~ask] = np.nan
        within(f"D {algo}", first.get(), want, tol)
        assert first.canary_rows()[~listed].all()
        keep = torch.from_numpy(ask)
        assert torch.equal(first.get()[keep], second.get()[keep])


@pytest.mark.parametrize("offsets", BAD)
@pytest.mark.parametrize("algo", ALGOS)
@pytest.mark.parametrize("rank", [8, 72])
def test_adapters_offsets(offsets, algo, rank):
    """Rank 8 by one launch, 72 by two, where FEW."""
    say(f"[gpu] adapters {algo} rank={rank} offsets {offsets}")
    c = Adapters("f16", 90, offsets, rank, 72, 104, pad=8)
    c.check("f16", algo)


@pytest.mark.parametrize("algo", ALGOS)
@pytest.mark.parametrize("places,rank,n,k,pad", [(1, 8, 8, 8, 0), (33, 72, 72, 136, 24),
                                                 (257, 40, 264, 72, 8), (130, 136, 520, 1032, 0)])
def test_adapters_sizes(places, rank, n, k, pad, algo):
    say(f"[gpu] adapters {algo} places={places} rank={rank} n={n} k={k} pad={pad}")
    offsets = [0, places // 3, places // 3, places - places // 4]
    for out in ("bf16", "f32"):
        Adapters("bf16", places, offsets, rank, n, k, pad=pad, rows=places > 1).check(out, algo)


# --------------------------------------------------------------- the sort
@pytest.mark.parametrize("count,top,groups,kind", [
    (1, 1, 1, "i32"), (1000, 4, 5, "i64"), (8192, 8, 256, "i32"), (8200, 8, 256, "i64"),
    (1030, 2, 300, "i32"), (20000, 5, 4096, "i64")])
def test_group_rows(count, top, groups, kind):
    say(f"[gpu] group_rows {count} to {groups}, {kind}")
    gen = torch.Generator().manual_seed(count)
    host = torch.randint(-3, groups + 3, (count,), generator=gen)
    host[::7] = -2 ** 31
    ids = Held(host.to(torch.int32 if kind == "i32" else torch.int64))
    a = B.GroupRowsArgs(4 if kind == "i32" else 5, count, top, groups)
    outs = [Held(shape=(n,), dtype=torch.int32) for n in (count, groups + 1, count)]
    ptrs = [ids.ptr] + [t.ptr for t in outs]
    need = ctypes.c_int64(-1)
    assert B._lib.group_rows_plan(a, *ptrs, need) == 0
    ws = Held(shape=(need.value,), dtype=torch.uint8, fill=0xff) if need.value else None
    rc = B._lib.group_rows(a, *ptrs, ws and ws.ptr, need.value, stream())
    finish("group_rows", rc, [ids], outs + ([ws] if ws else []))
    for t, want in zip(outs, G.group_rows(host.numpy().reshape(-1, top), groups)):
        assert np.array_equal(t.get().cpu().numpy(), want.reshape(-1))


# ----------------------------------------------------------- the rows' sum
@pytest.mark.parametrize("tokens,top,x_rows,n,pad", [(1, 1, 1, 8, 0), (37, 3, 100, 72, 8),
                                                     (50, 64, 7, 520, 0), (9, 2, 40, 264, 24)])
def test_combine(tokens, top, x_rows, n, pad):
    """Slots and rows from outside and twice."""
    say(f"[gpu] combine {tokens} x {top} of {x_rows} rows of {n}")
    gen = torch.Generator().manual_seed(tokens)
    X, dout = values(gen, (x_rows, n), "f16"), values(gen, (tokens, n), "f16")
    slots = torch.randint(-2, x_rows + 2, (tokens, top), generator=gen)
    rows = torch.randint(-2, tokens + 2, (x_rows,), generator=gen)
    w = torch.rand(tokens, top, generator=gen)
    hX, hd, hs, hr, hw = Held(X, ld=n + pad), Held(dout, ld=n + pad), ints(slots), ints(rows), Held(w)
    out = Held(shape=(tokens, n), dtype=torch.float32, ld=n + pad)
    c = B.CombineArgs(mfl.F16, mfl.F32, tokens, top, n, x_rows, n + pad, n + pad)
    rc = B._lib.combine_rows(c, hX.ptr, hs.ptr, hw.ptr, out.ptr, stream())
    finish("combine", rc, [hX, hs, hw], [out])
    within("out", out.get(), *G.combine(f64(X), slots.numpy(), f64(w), "f32"))
    dX, dw = Held(shape=(x_rows, n), dtype=torch.float16, ld=n + 2 * pad), \
        Held(shape=(tokens, top), dtype=torch.float32)
    c = B.CombineArgs(mfl.F16, mfl.F16, tokens, top, n, x_rows, n + pad, n + pad)
    rc = B._lib.combine_rows_backward(c, dX.ld, hd.ptr, hX.ptr, hs.ptr, hr.ptr, hw.ptr, dX.ptr,
                                      dw.ptr, stream())
    finish("combine backward", rc, [hX, hd, hs, hr, hw], [dX, dw])
    want, tol = G.combine_gradients(f64(dout), f64(X), slots.numpy(), rows.numpy(), f64(w), "f16")
    within("dX", dX.get(), want[0], tol[0])
    within("dw", dw.get(), want[1], tol[1])
