"""gemm_adapters for few rows: one launch for small problems, two that share
the contraction for others, at sizes on both sides and at the edges of the
tiles; the same inputs by every path."""
import numpy as np
import pytest
import torch

import mma_fragment_layouts_tn_amd as mfl
from gpu_helpers import say
from oracle import grouped as G
from test_gpu_grouped import DT, Adapted, f64, values, within

pytestmark = pytest.mark.gpu


def launches(c, out="", algo="few"):
    _, need = mfl.gemm_adapters_plan(c.x, c.W, c.A, c.B, torch.zeros(c.adapters + 1).int(),
                                     out_dtype=DT[out or c.kind], algo=algo)
    return 1 if need == 0 else 2


@pytest.mark.parametrize("m", [1, 15, 16, 17, 100])
@pytest.mark.parametrize("rank", [8, 16, 24, 32, 40, 56, 64])
def test_one_launch_ranks(m, rank):
    c = Adapted("bf16" if rank % 16 else "f16", m, 4, rank, 72, 520)
    assert launches(c) == 1
    c.check("f32" if m == 17 else "", algo="few")


@pytest.mark.parametrize("n,k", [(8, 8), (24, 2048), (32, 40), (40, 504), (1032, 256)])
@pytest.mark.parametrize("kind", ["f16", "bf16"])
def test_one_launch_sizes(n, k, kind):
    c = Adapted(kind, 37, 9, 16, n, k, pad=24)
    assert launches(c) == 1
    c.check(algo="few")
    c.check("f32", scale=False, algo="few")


@pytest.mark.parametrize("m,adapters,rank,n,k", [(1, 1, 16, 520, 4096), (1, 9, 8, 4096, 4096),
                                                 (37, 3, 16, 40, 4000), (16, 1, 32, 72, 2056),
                                                 (3, 2, 24, 8, 2560), (150, 1, 16, 200, 2736)])
@pytest.mark.parametrize("kind,out", [("f16", "f32"), ("bf16", "bf16")])
def test_one_launch_long(m, adapters, rank, n, k, kind, out):
    """Sixteen columns a workgroup."""
    c = Adapted(kind, m, adapters, rank, n, k)
    assert launches(c, out) == 1
    c.check(out, algo="few")


def test_one_launch_many_adapters():
    """More groups than are numbered without gaps; most without a row."""
    c = Adapted("f16", 200, 300, 8, 32, 64)
    assert launches(c) == 1
    c.check(algo="few")


@pytest.mark.parametrize("m", [1, 16, 31, 64, 65, 190])
@pytest.mark.parametrize("mode", ["mixed", "runs", "none", "one"])
def test_two_launches_rows(m, mode):
    c = Adapted("bf16", m, 5, 16, 136, 4168, mode=mode)
    assert launches(c) == 2
    c.check(algo="few")


@pytest.mark.parametrize("rank,n,k", [(72, 8, 8), (136, 264, 200), (64, 520, 2056), (8, 2056, 2056),
                                      (16, 40, 8200)])
@pytest.mark.parametrize("kind,out", [("f16", "f16"), ("bf16", "f32")])
def test_two_launches_sizes(rank, n, k, kind, out):
    c = Adapted(kind, 70, 3, rank, n, k)
    assert launches(c, out) == 2
    c.check(out, scale=rank != 64, algo="few")


@pytest.mark.parametrize("k", [264, 4168])
def test_are_apart(k):
    """An adapter of infinities and NaN changes no other request's row, by one
    launch and by two."""
    c = Adapted("f16", 150, 5, 16, 72, k, seed=2)
    assert launches(c) == (1 if k == 264 else 2)
    clean = c.run(algo="few")
    c.B[2], c.A[3] = float("nan"), float("inf")
    D = c.run(algo="few")
    others = (c.ids != 2) & (c.ids != 3)
    assert torch.equal(D[others], clean[others])
    assert bool((~D[c.ids == 3].isfinite()).all()) and bool(D[c.ids == 2].isnan().all())


@pytest.mark.parametrize("k", [264, 4168])
def test_rows_of_infinities(k):
    """A request's own infinities stay in its row."""
    c = Adapted("bf16", 40, 3, 16, 72, k, seed=3)
    clean = c.run(algo="few")
    c.x[7] = float("inf")
    D = c.run(algo="few")
    rest = torch.arange(40) != 7
    assert torch.equal(D[rest], clean[rest]) and bool((~D[7].isfinite()).all())


@pytest.mark.parametrize("k", [72, 4168])
def test_listed_in_part_and_out_of_range(k):
    c = Adapted("bf16", 90, 3, 8, 64, k, seed=4)
    rows = torch.arange(0, 90, 2, dtype=torch.int32)
    rows[3], rows[7] = -1, 90
    offsets = torch.tensor([0, 10, 25, 40], dtype=torch.int32)
    D = torch.full((90, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    dev = [t.cuda() for t in (c.x, c.W, c.A, c.B)]
    mfl.gemm_adapters(*dev, offsets.cuda(), rows=rows.cuda(), D=D, algo="few")
    want, tol = G.adapters(f64(c.x), f64(c.W), f64(c.A), f64(c.B), offsets.numpy(), rows.numpy(),
                           np.ones(3), "bf16")
    kept = torch.from_numpy(np.isnan(want[:, 0]))
    assert int(kept.sum()) == 47 and bool((D[kept] == 7).all())
    within("D", D, want, tol)
    for bad in ([-5, 30, 1 << 30, 90], [0, 80, 20, 90], [90] * 4, [2 ** 31 - 1, -2 ** 31, 50, 3]):
        say(f"[gpu] offsets {bad}")
        mfl.gemm_adapters(*dev, torch.tensor(bad, dtype=torch.int32).cuda(), algo="few")
    torch.cuda.synchronize()


def test_paths_agree():
    """Results of every path, in float32, within twice the bound of each other."""
    gen = torch.Generator().manual_seed(0)
    x, W = values(gen, (60, 1024), "f16"), values(gen, (256, 1024), "f16", 1 / 32)
    A, B = values(gen, (4, 16, 1024), "f16", 1 / 32), values(gen, (4, 256, 16), "f16", 0.25)
    ids = torch.randint(-1, 4, (60,), generator=gen)
    rows, offsets, _ = mfl.group_rows(ids.cuda(), 4)
    got = [mfl.gemm_adapters(x.cuda(), W.cuda(), A.cuda(), B.cuda(), offsets, rows=rows,
                             out_dtype=torch.float32, algo=a) for a in ("few", "tile128", "tile256")]
    _, tol = G.adapters(f64(x), f64(W), f64(A), f64(B), offsets.cpu().numpy(), rows.cpu().numpy(),
                        np.ones(4), "f32")
    for D in got[1:]:
        assert (np.abs(f64(D) - f64(got[0])) <= 2 * tol).all()
