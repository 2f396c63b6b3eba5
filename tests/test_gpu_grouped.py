"""Products by groups of rows on the GPU against their float64 definitions
(oracle/grouped.py): places of a list of choices (exact), the product of every
group and its gradients, the sum of a token's results, and adapters beside a
projection, every element within the bound that fp32 sums and one rounding of the result give.

Sizes sit where the kernels change: empty groups, one row, the 16 rows of an
atom, tiles of 16, 32, 64, 128 and 256 rows, contractions that end inside a
step of 64 or a sub-step of 32, widths between the tiles', rows gathered
twice or from outside, padded and shared strides, values of other groups and
behind the last one that must not be read.
"""
import numpy as np
import pytest
import torch

import mma_fragment_layouts_tn_amd as mfl
from gpu_helpers import say
from oracle import grouped as G

pytestmark = pytest.mark.gpu

DT = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}


def f64(t):
    return t.detach().cpu().double().numpy()


def values(gen, shape, kind, gain=1.0):
    return (torch.randn(*shape, generator=gen) * gain).to(DT[kind])


def within(name, got, want, tol):
    got = f64(got)
    assert got.shape == want.shape, (name, got.shape, want.shape)
    ask = ~np.isnan(want)
    err = np.abs(np.where(ask, got, 0) - np.where(ask, want, 0))
    bad = ~(err <= tol) & ask
    if bad.any():
        i = np.unravel_index(np.argmax(np.where(bad, np.nan_to_num(err, nan=np.inf), 0)), got.shape)
        raise AssertionError(f"{name}: {bad.sum()} of {bad.size} outside, worst at {i}: "
                             f"{got[i]} for {want[i]} +- {tol[i]}")
    say(f"[gpu]   {name}: worst {np.max(err / np.where(tol > 0, tol, 1), initial=0):.3f} "
        "of the bound")


# ------------------------------------------------------------- group_rows
@pytest.mark.parametrize("tokens,top,groups", [
    (1, 1, 1), (1, 2, 8), (63, 1, 3), (64, 8, 64), (65, 3, 5), (512, 8, 256), (1000, 4, 257),
    (4096, 1, 7), (4097, 1, 7), (2500, 8, 64), (30000, 5, 300), (70001, 8, 256), (5000, 2, 4096)])
@pytest.mark.parametrize("kind", [torch.int32, torch.int64])
def test_group_rows(tokens, top, groups, kind):
    say(f"[gpu] group_rows {tokens} x {top} of {groups} {kind}")
    gen = torch.Generator().manual_seed(tokens + groups)
    ids = torch.randint(-1, groups + 1, (tokens, top), generator=gen).to(kind)
    got = mfl.group_rows(ids.cuda(), groups)
    torch.cuda.synchronize()
    for name, x, want in zip(("rows", "offsets", "slots"), got, G.group_rows(ids.numpy(), groups)):
        assert x.dtype == torch.int32
        assert np.array_equal(x.cpu().numpy(), want), name


def test_group_rows_edges():
    for ids in (torch.zeros(0, 2, dtype=torch.int32), torch.full((300,), -7, dtype=torch.int64),
                torch.full((9000,), 2, dtype=torch.int32),
                torch.tensor([1 << 40, -(1 << 40), 1, 0, (1 << 32) + 1], dtype=torch.int64)):
        say(f"[gpu] group_rows {tuple(ids.shape)} {ids.dtype}")
        got = mfl.group_rows(ids.cuda(), 3)
        torch.cuda.synchronize()
        for x, want in zip(got, G.group_rows(ids.numpy(), 3)):
            assert np.array_equal(x.cpu().numpy(), want)


# ----------------------------------------------------------- gemm_grouped
class Case:
    def __init__(self, kind, lens, n, k, *, gather=False, tail=0, seed=0, pad=0):
        gen = torch.Generator().manual_seed(seed + n + k + len(lens))
        self.kind, self.lens, self.n, self.k = kind, lens, n, k
        self.offsets = torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32)
        self.used = int(self.offsets[-1])
        places = self.used + tail
        m = max(1, places // 2) if gather else places
        self.A = values(gen, (m, k + pad), kind)[:, :k]
        self.B = values(gen, (len(lens), n, k + pad), kind, k ** -0.5)[:, :, :k]
        self.dD = values(gen, (places, n + pad), kind)[:, :n]
        self.rows = torch.randint(0, m, (places,), generator=gen).int() if gather else None
        if tail:           # places of no group hold what must not be read
            self.dD[self.used:] = float("nan")
            if not gather:
                self.A[self.used:] = float("inf")
        say(f"[gpu] grouped {kind} lens={lens} n={n} k={k} gather={gather} tail={tail} pad={pad}")

    def cuda(self, t):
        """On the device with the strides it has here."""
        if t is None:
            return None
        c = torch.empty_strided(t.shape, t.stride(), dtype=t.dtype, device="cuda")
        c.copy_(t)
        return c

    def ref_rows(self):
        return None if self.rows is None else self.rows.numpy()

    def forward(self, out="", **kw):
        D = mfl.gemm_grouped(self.cuda(self.A), self.cuda(self.B), self.offsets.cuda(),
                             rows=self.cuda(self.rows), out_dtype=DT[out or self.kind], **kw)
        torch.cuda.synchronize()
        return D

    def check_forward(self, out="", **kw):
        D = self.forward(out, **kw)
        want, tol = G.product(f64(self.A), f64(self.B), self.offsets.numpy(), self.ref_rows(),
                              out or self.kind)
        within("D", D, want, tol)
        return D

    def check_backward(self, db="", **kw):
        dA, dB = mfl.gemm_grouped_backward(self.cuda(self.dD), self.cuda(self.A),
                                           self.cuda(self.B), self.offsets.cuda(),
                                           rows=self.cuda(self.rows),
                                           dB_dtype=DT[db or self.kind], **kw)
        torch.cuda.synchronize()
        want, tol = G.gradients(f64(self.dD), f64(self.A), f64(self.B), self.offsets.numpy(),
                                self.ref_rows(), self.kind, db or self.kind)
        within("dA", dA, want[0], tol[0])
        within("dB", dB, want[1], tol[1])


LENS = [[1], [0, 1, 0], [16, 17, 1], [0, 0, 33, 64, 65, 0], [127, 128, 129, 2], [300, 5, 257]]


@pytest.mark.parametrize("algo", ["few", "tile128", "tile256"])
@pytest.mark.parametrize("gather", [False, True])
@pytest.mark.parametrize("lens", LENS, ids=str)
def test_product_lengths(lens, gather, algo):
    Case("bf16", lens, 136, 200, gather=gather).check_forward(algo=algo)


@pytest.mark.parametrize("algo", ["few", "tile128", "tile256"])
@pytest.mark.parametrize("n,k", [(8, 8), (16, 64), (264, 128), (248, 72), (512, 1000), (40, 2056)])
@pytest.mark.parametrize("kind,out", [("f16", "f16"), ("f16", "f32"), ("bf16", "bf16"),
                                      ("bf16", "f32")])
def test_product_sizes(kind, out, n, k, algo):
    Case(kind, [40, 3, 70], n, k, gather=True).check_forward(out, algo=algo)


@pytest.mark.parametrize("rows", [1, 11, 40, 200])
def test_few_shapes(rows):
    """The mean decides between 16, 32 and 64 places per workgroup, the width
    between 16 and 32 columns."""
    for n in (24, 1048):
        Case("f16", [rows, 2 * rows, 0], n, 520, gather=True).check_forward(algo="few")


@pytest.mark.parametrize("gather", [False, True])
@pytest.mark.parametrize("lens", LENS, ids=str)
def test_gradient_lengths(lens, gather):
    Case("bf16", lens, 136, 200, gather=gather).check_backward()


@pytest.mark.parametrize("n,k", [(8, 8), (16, 64), (264, 128), (248, 72), (512, 1000)])
@pytest.mark.parametrize("kind,db", [("f16", "f16"), ("f16", "f32"), ("bf16", "bf16"),
                                     ("bf16", "f32")])
@pytest.mark.parametrize("gather", [False, True])
def test_gradient_sizes(kind, db, n, k, gather):
    Case(kind, [40, 3, 70, 0, 130], n, k, gather=gather).check_backward(db)


@pytest.mark.parametrize("gather", [False, True])
def test_strides(gather):
    c = Case("f16", [40, 0, 150], 104, 88, gather=gather, pad=24)
    for algo in ("few", "tile128", "tile256"):
        c.check_forward(algo=algo)
    c.check_backward()


@pytest.mark.parametrize("algo", ["few", "tile128", "tile256"])
def test_places_of_no_group(algo):
    """Their rows of D stay as they were, their gradient is 0, and what they
    hold is not read."""
    c = Case("bf16", [20, 0, 33], 64, 96, tail=150)
    D = torch.full((203, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    got = mfl.gemm_grouped(c.cuda(c.A), c.cuda(c.B), c.offsets.cuda(), D=D, algo=algo)
    torch.cuda.synchronize()
    assert got is D and bool((D[c.used:] == 7).all())
    want, tol = G.product(f64(c.A), f64(c.B), c.offsets.numpy(), None, "bf16")
    within("D", D[:c.used], want[:c.used], tol[:c.used])
    if algo == "few":
        c.check_backward()


@pytest.mark.parametrize("algo", ["few", "tile128", "tile256"])
def test_rows_from_outside_are_zeros(algo):
    c = Case("f16", [30, 40], 64, 96, gather=True)
    c.rows[::3] = torch.tensor([-1, c.A.shape[0], 2 ** 31 - 1, -2 ** 31]).repeat(20)[:24].int()
    c.check_forward(algo=algo)
    if algo == "few":
        c.check_backward()


@pytest.mark.parametrize("algo", ["few", "tile128", "tile256"])
def test_groups_are_apart(algo):
    """A group whose matrix and rows hold infinities and NaN leaves the others
    as they are."""
    c = Case("bf16", [17, 30, 70], 72, 136, seed=3)
    clean = c.forward(algo=algo)
    c.B[1], c.A[17:47] = float("nan"), float("inf")
    D = c.forward(algo=algo)
    keep = torch.cat([torch.arange(17), torch.arange(47, 117)])
    assert torch.equal(D[keep], clean[keep])
    if algo == "few":
        c.dD[17:47] = float("inf")
        dA, dB = mfl.gemm_grouped_backward(c.dD.cuda(), c.A.cuda(), c.B.cuda(), c.offsets.cuda())
        assert bool(torch.isfinite(dA[keep]).all())
        assert bool(torch.isfinite(dB[0]).all()) and bool(torch.isfinite(dB[2]).all())


def test_offsets_out_of_range():
    """Held inside the places whatever they are: nothing is read or written
    beside the tensors."""
    c = Case("f16", [30, 40, 20], 64, 96)
    for bad in ([-5, 30, 1 << 30, 90], [0, 80, 20, 90], [0, 0, 0, -1], [90, 90, 90, 90],
                [2 ** 31 - 1, -2 ** 31, 50, 3]):
        say(f"[gpu] offsets {bad}")
        o = torch.tensor(bad, dtype=torch.int32).cuda()
        for algo in ("few", "tile128", "tile256"):
            mfl.gemm_grouped(c.A.cuda(), c.B.cuda(), o, algo=algo)
        mfl.gemm_grouped_backward(c.dD.cuda(), c.A.cuda(), c.B.cuda(), o)
        torch.cuda.synchronize()


def test_shared_matrices():
    """Groups that share one matrix (a group stride of 0)."""
    c = Case("bf16", [9, 21], 64, 96)
    c.B = c.B[:1].expand(2, 64, 96)
    D = mfl.gemm_grouped(c.A.cuda(), c.B[:1].cuda().expand(2, 64, 96), c.offsets.cuda())
    torch.cuda.synchronize()
    want, tol = G.product(f64(c.A), f64(c.B), c.offsets.numpy(), None, "bf16")
    within("D", D, want, tol)


def test_many_groups():
    gen = torch.Generator().manual_seed(1)
    lens = torch.randint(0, 4, (700,), generator=gen).tolist()
    c = Case("f16", lens, 40, 64, gather=True)
    for algo in ("few", "tile128"):
        c.check_forward(algo=algo)
    c.check_backward()


def test_gradients_against_differences():
    """Directional derivatives of sum(D * dD) by central differences of the
    kernel's own forward pass in fp32 results."""
    c = Case("bf16", [33, 0, 70], 64, 128, gather=True, seed=5)
    dA, dB = mfl.gemm_grouped_backward(c.dD.cuda(), c.A.cuda(), c.B.cuda(), c.offsets.cuda(),
                                       rows=c.rows.cuda(), dB_dtype=torch.float32)
    gen = torch.Generator().manual_seed(9)

    def loss(A, B):
        D = mfl.gemm_grouped(A.cuda(), B.cuda(), c.offsets.cuda(), rows=c.rows.cuda(),
                             out_dtype=torch.float32)
        return float((D.double() * c.dD.cuda().double()).sum())

    # a step of a whole power of two keeps the shifted operands near bf16
    # values; the product is bilinear, so central differences are exact but for
    # roundings: take the step as it comes out after rounding
    for which in ("A", "B"):
        x = c.A if which == "A" else c.B
        step = torch.randn(x.shape, generator=gen) * 0.25
        up, down = (x.float() + step).to(x.dtype), (x.float() - step).to(x.dtype)
        d = up.double() - down.double()
        if which == "A":
            got = loss(up, c.B) - loss(down, c.B)
            g = torch.zeros(c.A.shape, dtype=torch.float64)
            g.index_add_(0, c.rows.long(), dA.cpu().double())
            mag = torch.zeros_like(g).index_add_(0, c.rows.long(), dA.cpu().double().abs())
        else:
            got = loss(c.A, up) - loss(c.A, down)
            g, mag = dB.cpu().double(), dB.cpu().double().abs()
        want = float((g * d).sum())
        # dA's rounding to bf16, and both forward passes' fp32 sums
        tol = float((mag * d.abs()).sum()) * 2 ** -8 + 1e-4 * abs(want) + 0.05
        say(f"[gpu] d{which}: {got} for {want} +- {tol}")
        assert abs(got - want) <= tol


# ----------------------------------------------------------- combine_rows
@pytest.mark.parametrize("kind,out", [("f16", "f16"), ("bf16", "bf16"), ("bf16", "f32")])
@pytest.mark.parametrize("tokens,top,n", [(1, 1, 8), (5, 2, 64), (33, 8, 520), (100, 3, 2048),
                                          (7, 64, 24)])
@pytest.mark.parametrize("weighted", [True, False])
def test_combine(kind, out, tokens, top, n, weighted):
    say(f"[gpu] combine {kind} {tokens} x {top} x {n} weighted={weighted}")
    gen = torch.Generator().manual_seed(tokens * top + n)
    ids = torch.randint(-1, 4, (tokens, top), generator=gen).int()
    rows, offsets, slots = mfl.group_rows(ids.cuda(), 4)
    X, dout = values(gen, (tokens * top, n), kind), values(gen, (tokens, n), kind)
    X[int(offsets[-1]):] = float("nan")          # places of no group
    w = torch.randn(tokens, top, generator=gen) if weighted else None
    got = mfl.combine_rows(X.cuda(), slots, None if w is None else w.cuda(), out_dtype=DT[out])
    dX, dw = mfl.combine_rows_backward(dout.cuda(), X.cuda(), slots,
                                       None if w is None else w.cuda(), rows=rows)
    torch.cuda.synchronize()
    w64 = np.ones((tokens, top)) if w is None else f64(w)
    s, r = slots.cpu().numpy(), rows.cpu().numpy()
    want, tol = G.combine(f64(X), s, w64, out)
    within("out", got, want, tol)
    want, tol = G.combine_gradients(f64(dout), f64(X), s, r, w64, kind)
    within("dX", dX, want[0], tol[0])
    if w is None:
        assert dw is None
    else:
        within("dw", dw, want[1], tol[1])


def test_combine_slots_from_outside_and_twice():
    X = torch.randn(6, 16).half()
    slots = torch.tensor([[0, 0, 6], [-1, 2, 3], [2 ** 31 - 1, -2 ** 31, 5]], dtype=torch.int32)
    rows = torch.tensor([0, 0, 1, 1, -1, 2], dtype=torch.int32)
    w, dout = torch.randn(3, 3), torch.randn(3, 16).half()
    got = mfl.combine_rows(X.cuda(), slots.cuda(), w.cuda())
    dX, dw = mfl.combine_rows_backward(dout.cuda(), X.cuda(), slots.cuda(), w.cuda(),
                                       rows=rows.cuda())
    want, tol = G.combine(f64(X), slots.numpy(), f64(w), "f16")
    within("out", got, want, tol)
    want, tol = G.combine_gradients(f64(dout), f64(X), slots.numpy(), rows.numpy(), f64(w), "f16")
    within("dX", dX, want[0], tol[0])
    within("dw", dw, want[1], tol[1])


def test_combine_strides():
    X, out = torch.randn(12, 48).bfloat16(), torch.zeros(4, 64, dtype=torch.bfloat16).cuda()
    slots = torch.arange(12, dtype=torch.int32).flip(0).view(4, 3)
    got = mfl.combine_rows(X.cuda()[:, :40], slots.cuda(), out=out[:, :40])
    want, tol = G.combine(f64(X[:, :40]), slots.numpy(), np.ones((4, 3)), "bf16")
    within("out", got, want, tol)
    assert bool((out[:, 40:] == 0).all())


# ---------------------------------------------------------- gemm_adapters
class Adapted:
    def __init__(self, kind, m, adapters, rank, n, k, *, mode="mixed", seed=0, pad=0):
        gen = torch.Generator().manual_seed(seed + m + rank + n + k)
        self.kind = kind
        ids = torch.randint(-1, adapters, (m,), generator=gen)
        if mode == "runs":
            ids = ids.sort().values
        if mode == "none":
            ids[:] = -1
        if mode == "one":
            ids[:] = adapters - 1
        self.ids = ids
        self.x = values(gen, (m, k + pad), kind)[:, :k]
        self.W = values(gen, (n, k + pad), kind, k ** -0.5)[:, :k]
        self.A = values(gen, (adapters, rank, k + pad), kind, k ** -0.5)[:, :, :k]
        self.B = values(gen, (adapters, n, rank + pad), kind, rank ** -0.5)[:, :, :rank]
        self.scale = torch.rand(adapters, generator=gen) * 2 - 0.5
        self.adapters = adapters
        say(f"[gpu] adapters {kind} m={m} adapters={adapters} rank={rank} n={n} k={k} {mode}")

    def run(self, out="", scale=True, **kw):
        rows, offsets, _ = mfl.group_rows(self.ids.cuda(), self.adapters)
        self.rows, self.offsets = rows.cpu(), offsets.cpu()

        def put(t):
            c = torch.empty_strided(t.shape, t.stride(), dtype=t.dtype, device="cuda")
            return c.copy_(t)

        D = mfl.gemm_adapters(put(self.x), put(self.W), put(self.A), put(self.B), offsets,
                              rows=rows, scale=self.scale.cuda() if scale else None,
                              out_dtype=DT[out or self.kind], **kw)
        torch.cuda.synchronize()
        return D

    def check(self, out="", scale=True, **kw):
        D = self.run(out, scale, **kw)
        s = f64(self.scale) if scale else np.ones(self.adapters)
        want, tol = G.adapters(f64(self.x), f64(self.W), f64(self.A), f64(self.B),
                               self.offsets.numpy(), self.rows.numpy(), s, out or self.kind)
        within("D", D, want, tol)
        return D


ALGOS = ["few", "tile128", "tile256"]


@pytest.mark.parametrize("algo", ALGOS)
@pytest.mark.parametrize("m", [1, 16, 33, 64, 130, 300])
@pytest.mark.parametrize("mode", ["mixed", "runs", "none", "one"])
def test_adapters_rows(m, mode, algo):
    Adapted("bf16", m, 5, 16, 136, 200, mode=mode).check(algo=algo)


@pytest.mark.parametrize("algo", ALGOS)
@pytest.mark.parametrize("rank", [8, 24, 32, 40, 64, 136])
@pytest.mark.parametrize("kind,out", [("f16", "f16"), ("f16", "f32"), ("bf16", "bf16"),
                                      ("bf16", "f32")])
def test_adapters_ranks(kind, out, rank, algo):
    Adapted(kind, 70, 3, rank, 72, 264).check(out, scale=rank != 24, algo=algo)


@pytest.mark.parametrize("algo", ALGOS)
@pytest.mark.parametrize("n,k", [(8, 8), (264, 128), (512, 1000)])
def test_adapters_sizes(n, k, algo):
    Adapted("f16", 90, 40, 8, n, k, pad=16).check(algo=algo)


def test_adapters_auto_and_many():
    Adapted("bf16", 400, 100, 16, 1032, 64).check()
    Adapted("f16", 1200, 7, 32, 1024, 72, mode="runs").check()


@pytest.mark.parametrize("algo", ALGOS)
def test_adapters_without_rows(algo):
    """Places are rows; those behind the last adapter have the shared term
    alone."""
    c = Adapted("bf16", 100, 4, 16, 72, 136)
    offsets = torch.tensor([0, 30, 30, 47, 80], dtype=torch.int32)
    D = mfl.gemm_adapters(c.x.cuda(), c.W.cuda(), c.A.cuda(), c.B.cuda(), offsets.cuda(),
                          algo=algo)
    want, tol = G.adapters(f64(c.x), f64(c.W), f64(c.A), f64(c.B), offsets.numpy(), None,
                           np.ones(4), "bf16")
    within("D", D, want, tol)


@pytest.mark.parametrize("algo", ALGOS)
def test_adapters_are_apart(algo):
    """An adapter of infinities and NaN changes no other request's row."""
    c = Adapted("f16", 150, 5, 16, 72, 136, seed=2)
    clean = c.run(algo=algo)
    c.B[2, 5:9], c.A[3] = float("nan"), float("inf")
    c.B[2, 20, 3] = float("inf")
    D = c.run(algo=algo)
    others = (c.ids != 2) & (c.ids != 3)
    assert torch.equal(D[others], clean[others])
    mine = (c.ids == 2).nonzero().flatten()
    rest = [n for n in range(72) if not 5 <= n < 9 and n != 20]
    assert bool(D[mine][:, 5:9].isnan().all()) and bool((~D[mine][:, 20].isfinite()).all())
    assert torch.equal(D[mine][:, rest], clean[mine][:, rest])
    assert bool((~D[c.ids == 3].isfinite()).all())


@pytest.mark.parametrize("algo", ALGOS)
def test_adapters_rows_listed_in_part(algo):
    """Rows that no place leads to stay as they were; numbers outside are
    skipped."""
    c = Adapted("bf16", 90, 3, 8, 64, 72, seed=4)
    rows = torch.arange(0, 90, 2, dtype=torch.int32)
    rows[3], rows[7] = -1, 90
    offsets = torch.tensor([0, 10, 25, 40], dtype=torch.int32)
    D = torch.full((90, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    mfl.gemm_adapters(c.x.cuda(), c.W.cuda(), c.A.cuda(), c.B.cuda(), offsets.cuda(),
                      rows=rows.cuda(), D=D, algo=algo)
    want, tol = G.adapters(f64(c.x), f64(c.W), f64(c.A), f64(c.B), offsets.numpy(), rows.numpy(),
                           np.ones(3), "bf16")
    kept = torch.from_numpy(np.isnan(want[:, 0]))
    assert int(kept.sum()) == 47 and bool((D[kept] == 7).all())
    within("D", D, want, tol)


@pytest.mark.parametrize("algo", ALGOS)
def test_adapters_offsets_out_of_range(algo):
    c = Adapted("f16", 90, 3, 8, 64, 72)
    for bad in ([-5, 30, 1 << 30, 90], [0, 80, 20, 90], [90, 90, 90, 90],
                [2 ** 31 - 1, -2 ** 31, 50, 3]):
        say(f"[gpu] offsets {bad}")
        mfl.gemm_adapters(c.x.cuda(), c.W.cuda(), c.A.cuda(), c.B.cuda(),
                          torch.tensor(bad, dtype=torch.int32).cuda(), algo=algo)
    torch.cuda.synchronize()
