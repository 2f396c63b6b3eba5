"""Every tile that a launch's last round may be cut into: a round that is
nearly full keeps its tiles of 256 columns whole, emptier ones are cut in two,
four and eight, along rows and columns, and a tile of few rows is the smaller
one.  Groups of each height against widths that give each number of parts; more
groups than the kernels count; more choices than a walk of a wave."""
import numpy as np
import pytest
import torch

import mma_fragment_layouts_tn_amd as mfl
from oracle import grouped as G
from test_gpu_grouped import DT, Adapted, Case, f64, within

pytestmark = pytest.mark.gpu

# heights: whole, under a half, under a quarter of a tile; none; one row; over a half
LENS = [256, 100, 60, 0, 1, 129]
# columns of 5 tiles of rows: 8, 4, 2 parts, none; a round and 4 parts; each ragged
WIDTHS = [256 * 6 - 8, 256 * 9 + 64, 256 * 20 + 136, 256 * 30, 256 * 60 + 72]


@pytest.mark.parametrize("n", WIDTHS)
@pytest.mark.parametrize("kind,out", [("bf16", "bf16"), ("f16", "f32")])
def test_product(n, kind, out):
    Case(kind, LENS, n, 200, gather=True).check_forward(out, algo="tile256")


@pytest.mark.parametrize("n", WIDTHS)
@pytest.mark.parametrize("gather", [False, True])
def test_gradients(n, gather):
    """dA over n columns, dB over as many tiles of each group."""
    c = Case("bf16", LENS, 72, n, gather=gather, tail=70)
    c.check_backward("f32" if gather else "")


@pytest.mark.parametrize("n,k", [(264, 520), (1000, 2304), (2048, 4096)])
def test_weights(n, k):
    """dB whole, halved and in corners, groups of few places and of none."""
    Case("f16", [70, 0, 33, 1], n, k).check_backward()


# rows of adapters: a tile and a part of one of each height
@pytest.mark.parametrize("tail", [10, 100, 200])
@pytest.mark.parametrize("tiles", [6, 20, 40, 75, 150])
@pytest.mark.parametrize("kind,out", [("f16", "f16"), ("bf16", "f32")])
def test_adapters(tail, tiles, kind, out):
    n = 256 * (tiles // 2) - 56
    Adapted(kind, 256 + tail, 3, 40, n, 136, mode="runs").check(out, algo="tile256")


@pytest.mark.parametrize("n", [256 * 5, 256 * 40])
def test_adapters_are_apart(n):
    c = Adapted("f16", 300, 5, 16, n, 136, seed=2)
    clean = c.run(algo="tile256")
    c.B[2, 5:9], c.A[3] = float("nan"), float("inf")
    c.B[2, n - 3, 3] = float("inf")
    D = c.run(algo="tile256")
    others = (c.ids != 2) & (c.ids != 3)
    assert torch.equal(D[others], clean[others])
    mine = c.ids == 2
    assert bool(D[mine][:, 5:9].isnan().all()) and bool((~D[mine][:, n - 3].isfinite()).all())
    assert torch.equal(D[mine][:, 9:n - 3], clean[mine][:, 9:n - 3])


@pytest.mark.parametrize("algo", ["few", "tile128", "tile256"])
def test_more_groups_than_are_counted(algo):
    """300 groups, most of them empty, places of none behind: product,
    gradients, adapters."""
    gen = torch.Generator().manual_seed(1)
    lens = torch.zeros(300, dtype=torch.int64)
    lens[torch.randperm(300, generator=gen)[:40]] = torch.randint(1, 90, (40,), generator=gen)
    c = Case("bf16", lens.tolist(), 40, 72, tail=300)
    D = torch.full((c.used + 300, 40), 7.0, dtype=torch.bfloat16, device="cuda")
    mfl.gemm_grouped(c.cuda(c.A), c.cuda(c.B), c.offsets.cuda(), D=D, algo=algo)
    want, tol = G.product(f64(c.A), f64(c.B), c.offsets.numpy(), None, "bf16")
    within("D", D[:c.used], want[:c.used], tol[:c.used])
    assert bool((D[c.used:] == 7).all())
    if algo == "few":
        c.check_backward()
    Adapted("f16", 700, 300, 8, 264, 72).check(algo=algo)


def test_alignment_of_parts_with_strides():
    for n in (256 * 9 + 64, 256 * 30):
        c = Case("f16", LENS, n, 88, gather=True, pad=24)
        c.check_forward(algo="tile256")
        D = torch.full((c.used, n + 40), 3.0, dtype=torch.float16, device="cuda")
        mfl.gemm_grouped(c.cuda(c.A), c.cuda(c.B), c.offsets.cuda(), rows=c.cuda(c.rows),
                         D=D[:, :n], algo="tile256")
        assert bool((D[:, n:] == 3).all()) and torch.equal(D[:, :n], c.forward(algo="tile256"))


@pytest.mark.parametrize("tokens,top,groups", [(4093, 2, 64), (8192, 1, 256), (8193, 1, 3),
                                               (300001, 8, 64), (60001, 8, 1000), (1100000, 1, 256),
                                               (131073, 2, 4096)])
def test_more_choices_than_a_chunk_each(tokens, top, groups):
    """Chunks grow beyond one walk of a wave: against a stable sort."""
    gen = torch.Generator().manual_seed(tokens)
    ids = torch.randint(-1, groups + 1, (tokens, top), generator=gen)
    rows, offsets, slots = mfl.group_rows(ids.cuda(), groups)
    torch.cuda.synchronize()
    key = torch.where((ids < 0) | (ids >= groups), groups, ids).flatten()
    order = torch.sort(key, stable=True).indices
    place = torch.empty_like(order)
    place[order] = torch.arange(len(order))
    counts = torch.bincount(key, minlength=groups + 1)
    assert torch.equal(rows.cpu().long(), order // top)
    assert int(offsets[0]) == 0 and torch.equal(offsets[1:].cpu().long(), counts[:-1].cumsum(0))
    assert torch.equal(slots.cpu().long().flatten(), torch.where(key < groups, place, -1))
