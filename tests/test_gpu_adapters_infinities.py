"""Infinities and NaN in an adapter's matrices: its own rows hold what IEEE
arithmetic gives for the sum (an infinity of one sign stays one, also against a
finite part that the result's type cannot hold), by every kernel."""
import numpy as np
import pytest
import torch

import mma_fragment_layouts_tn_amd as mfl
from gpu_helpers import say
from test_gpu_grouped import ALGOS, DT, f64, values

pytestmark = pytest.mark.gpu

INF = float("inf")


def kinds(t):
    """0 finite, 1 +inf, 2 -inf, 3 NaN."""
    return np.select([np.isnan(t), t == INF, t == -INF], [3, 1, 2], 0)


class Case:
    """Rows of positive numbers, so that an infinity's sign is A's and B's."""

    def __init__(self, kind, rank, n=72, k=136, m=150):
        gen = torch.Generator().manual_seed(rank)
        self.ids = torch.randint(-1, 3, (m,), generator=gen)
        self.x = values(gen, (m, k), kind).abs() + 0.125
        self.W = values(gen, (n, k), kind, k ** -0.5)
        self.A = values(gen, (3, rank, k), kind, k ** -0.5)
        self.B = values(gen, (3, n, rank), kind).abs() + 0.125

    def check(self, out, algo):
        rows, offsets, _ = mfl.group_rows(self.ids.cuda(), 3)
        D = f64(mfl.gemm_adapters(self.x.cuda(), self.W.cuda(), self.A.cuda(), self.B.cuda(),
                                  offsets, rows=rows, out_dtype=DT[out], algo=algo))
        with np.errstate(all="ignore"):
            x, W = f64(self.x), f64(self.W)
            want = (x[:, None] * W[None]).sum(-1)
            for g in range(3):
                h = (x[:, None] * f64(self.A[g])[None]).sum(-1)
                low = (h[:, None] * f64(self.B[g])[None]).sum(-1)
                want = np.where((self.ids.numpy() == g)[:, None], want + low, want)
            held = f64(torch.from_numpy(want).to(DT[out]))
        wrong = kinds(D) != kinds(held)
        assert not wrong.any(), (np.argwhere(wrong)[:5], D[wrong][:5], held[wrong][:5])
        return kinds(held)


CASES = [(kind, rank, algo) for kind in ("f16", "bf16") for rank in (16, 72) for algo in ALGOS]


@pytest.mark.parametrize("kind,rank,algo", CASES)
def test_infinities_in_both_matrices(kind, rank, algo):
    say(f"[gpu] infinities in A and B, {kind}, rank {rank}, {algo}")
    c = Case(kind, rank)
    c.A[1, 3, 5] = INF                 # h of column 3: +inf
    c.B[1, 10, 3] = INF                # inf inf
    c.B[1, 11, 3] = -INF
    c.B[1, 12, 2] = INF                # beside it: an infinity of either sign
    c.B[1, 13, 3] = 0                  # inf 0
    c.B[1, 14, 7] = float("nan")
    c.A[2, 0, 9] = -INF
    c.B[2, 20, 1] = 6.0
    seen = c.check("f32", algo)
    c.check(kind, algo)
    mine = seen[c.ids.numpy() == 1]
    assert (mine[:, 10] == 1).all() and (mine[:, 11] == 2).all() and (mine[:, 0] == 1).all()
    assert (mine[:, 13] == 3).all() and (mine[:, 14] == 3).all()


@pytest.mark.parametrize("rank", [16, 72])
@pytest.mark.parametrize("algo", ALGOS)
def test_infinity_against_an_overflow(rank, algo):
    """Finite parts beyond fp16's largest number, with either sign, beside an
    infinity of the other."""
    say(f"[gpu] infinities against overflows, rank {rank}, {algo}")
    c = Case("f16", rank)
    c.x[:, 0], c.W[:, 0] = 400.0, 400.0
    c.W[::2, 0] = -400.0
    c.A[:, :, 0] = c.A[:, :, 0].abs()  # (h positive: 400 |A| is most of it)
    c.A[:, :, 0] += 1.0
    c.B[0, 8:24, 1] = -INF
    c.B[0, 30:40, 4] = INF
    seen = c.check("f16", algo)
    mine = seen[c.ids.numpy() == 0]
    assert (mine[:, 8:24] == 2).all() and (mine[:, 30:40] == 1).all()
