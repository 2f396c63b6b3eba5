"""gemm_adapters holds the low-rank term's own factor s_g h as fp32 does, by
every kernel: numbers beyond fp16's range and far below its smallest step, and
numbers of 20 bits that a shared term takes away again.  The same request has
the same result whatever batch it is in."""
import numpy as np
import pytest
import torch

import mma_fragment_layouts_tn_amd as mfl
from gpu_helpers import say
from oracle import grouped as G
from test_gpu_grouped import ALGOS, DT, f64, values, within

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("algo", ALGOS)
@pytest.mark.parametrize("rank", [16, 72])
@pytest.mark.parametrize("kind,out", [("f16", "f16"), ("f16", "f32"), ("bf16", "bf16"),
                                      ("bf16", "f32")])
def test_whole_numbers_are_exact(kind, out, rank, algo):
    """Every product and every sum is a whole number below 2^24 (times a power
    of two), so fp32 is exact in any order.  h has up to 20 bits; the shared
    term takes away all but some 13."""
    say(f"[gpu] whole numbers, {kind} to {out}, rank {rank}, {algo}")
    gen = torch.Generator().manual_seed(rank)
    m, n, k, adapters = 150, 72, 64, 4
    ids = torch.randint(-1, adapters, (m,), generator=gen)
    x = torch.randint(0, 128, (m, k), generator=gen).double()
    A0 = torch.randint(0, 128, (rank, k), generator=gen).double()
    of = torch.randint(0, rank, (n,), generator=gen)
    B0 = torch.zeros(n, rank).double()
    B0[torch.arange(n), of] = torch.randint(0, 2, (n,), generator=gen).double() * 2 - 1
    W = torch.randint(-1, 2, (n, k), generator=gen) - B0 @ A0
    A, B, scale = [], [], 2.0 ** -torch.tensor([0, 3, -4, 10])
    for s in scale:
        order = torch.randperm(rank, generator=gen)
        A.append(A0[order])
        B.append(B0[:, order] / s)
    A, B = torch.stack(A), torch.stack(B)
    want = x @ W.t()
    for g in range(adapters):
        low = x @ A[g].t() * scale[g] @ B[g].t()
        assert float((x @ A[g].t()).max()) > 2 ** 16
        want = torch.where((ids == g)[:, None], want + low, want)
    assert bool((want == want.round()).all())
    rows, offsets, _ = mfl.group_rows(ids.cuda(), adapters)
    ops = [t.to(DT[kind]) for t in (x, W, A, B)]
    assert all(torch.equal(a.double(), b.double()) for a, b in zip(ops, (x, W, A, B)))
    D = mfl.gemm_adapters(*[t.cuda() for t in ops], offsets, rows=rows, scale=scale.cuda(),
                          out_dtype=DT[out], algo=algo)
    assert torch.equal(D.cpu(), want.to(DT[out]))


class Scaled:
    """Adapters of scales far apart, each with a B that brings its term back."""

    def __init__(self, kind, m, n, k, rank, scales, shared, seed=0):
        gen = torch.Generator().manual_seed(seed + m + rank)
        self.ids = torch.randint(-1, len(scales), (m,), generator=gen)
        self.x = values(gen, (m, k), kind)
        self.W = values(gen, (n, k), kind, shared * k ** -0.5)
        self.A = values(gen, (len(scales), rank, k), kind, k ** -0.5)
        self.B = torch.stack([values(gen, (n, rank), kind, min(1 / abs(s), 1e4)) for s in scales])
        self.scale = torch.tensor(scales)

    def tensors(self):
        return [t.cuda() for t in (self.x, self.W, self.A, self.B)]

    def check(self, out, algo):
        rows, offsets, _ = mfl.group_rows(self.ids.cuda(), len(self.scale))
        D = mfl.gemm_adapters(*self.tensors(), offsets, rows=rows, scale=self.scale.cuda(),
                              out_dtype=DT[out], algo=algo)
        torch.cuda.synchronize()
        assert bool(D.isfinite().all())
        want, tol = G.adapters(f64(self.x), f64(self.W), f64(self.A), f64(self.B),
                               offsets.cpu().numpy(), rows.cpu().numpy(), f64(self.scale), out)
        within("D", D, want, tol)
        return D


@pytest.mark.parametrize("algo", ALGOS)
@pytest.mark.parametrize("rank", [8, 40, 72])
@pytest.mark.parametrize("kind,out", [("f16", "f16"), ("f16", "f32"), ("bf16", "bf16"),
                                      ("bf16", "f32")])
def test_scales_far_apart(kind, out, rank, algo):
    say(f"[gpu] scales far apart, {kind} to {out}, rank {rank}, {algo}")
    Scaled(kind, 150, 72, 136, rank, [1e5, -3e4, 1.0, 1e-3, 1e-5, 2.0 ** -30], 1.0).check(out, algo)


@pytest.mark.parametrize("algo", ALGOS)
@pytest.mark.parametrize("kind", ["f16", "bf16"])
def test_terms_alone(kind, algo):
    """Nothing beside the low-rank terms, which keep their relative accuracy."""
    say(f"[gpu] low-rank terms alone, {kind}, {algo}")
    Scaled(kind, 150, 72, 136, 40, [1e20, 1e7, -1.0, 1e-4, 1e-9, 1e-20], 0.0).check("f32", algo)


def test_the_size_of_the_batch_does_not_matter():
    """500 rows go by one kernel and 1000 by another."""
    plans = []
    for m in (500, 1000):
        c = Scaled("f16", m, 1024, 1024, 16, [1e5, -1e5, 1e6, 1.0], 1.0, seed=3)
        plans.append(mfl.gemm_adapters_plan(*c.tensors(), torch.zeros(5).int().cuda())[0])
        say(f"[gpu] {m} rows by {plans[-1]}")
        c.check("f16", "auto")
    assert plans[0] == "few" and plans[1].startswith("tile")
