"""The float64 oracle of the products by groups of rows, pinned: a sort by
hand, its properties, the products and gradients against torch's in float64,
and planted mistakes."""
import numpy as np
import pytest
import torch

from oracle import grouped as G


def test_group_rows_by_hand():
    ids = [[2, 0], [1, 2], [-1, 0], [2, 3]]
    rows, offsets, slots = G.group_rows(ids, 3)
    # group 0: choices 1, 5; 1: 2; 2: 0, 3, 6; none: 4, 7
    assert rows.tolist() == [0, 2, 1, 0, 1, 3, 2, 3]
    assert offsets.tolist() == [0, 2, 3, 6]
    assert slots.tolist() == [[3, 0], [2, 4], [-1, 1], [5, -1]]


@pytest.mark.parametrize("tokens,top,groups", [(1, 1, 1), (7, 3, 4), (50, 2, 9)])
def test_group_rows_properties(tokens, top, groups):
    rng = np.random.default_rng(tokens)
    ids = rng.integers(-1, groups + 1, (tokens, top))
    rows, offsets, slots = G.group_rows(ids, groups)
    kept = slots >= 0
    assert (kept == ((ids >= 0) & (ids < groups))).all()
    assert sorted(slots[kept].tolist()) == list(range(offsets[-1]))
    for t in range(tokens):
        for j in range(top):
            if kept[t, j]:
                g = ids[t, j]
                assert offsets[g] <= slots[t, j] < offsets[g + 1] and rows[slots[t, j]] == t
    for g in range(groups):     # a group's choices in their own order
        assert (np.diff(slots.reshape(-1)[ids.reshape(-1) == g]) == 1).all()


def setup(seed=0, gather=True):
    rng = np.random.default_rng(seed)
    lens = [3, 0, 5, 1]
    offsets = np.concatenate([[0], np.cumsum(lens)])
    A, B = rng.normal(size=(6, 7)), rng.normal(size=(4, 5, 7))
    rows = rng.integers(0, 6, 9) if gather else None
    if not gather:
        A = rng.normal(size=(9, 7))
    return A, B, offsets, rows, rng.normal(size=(9, 5)), lens


def by_torch(A, B, rows, dD, lens):
    a, b = (torch.tensor(x, requires_grad=True) for x in (A, B))
    which = torch.repeat_interleave(torch.arange(len(lens)), torch.tensor(lens))
    x = a if rows is None else a[torch.tensor(rows)]
    x.retain_grad()
    D = torch.einsum("ik,ink->in", x, b[which])
    (D * torch.tensor(dD)).sum().backward()
    return D.detach().numpy(), x.grad.numpy(), b.grad.numpy()


@pytest.mark.parametrize("gather", [True, False])
def test_products_and_gradients(gather):
    A, B, offsets, rows, dD, lens = setup(gather=gather)
    D, dA, dB = by_torch(A, B, rows, dD, lens)
    got, tol = G.product(A, B, offsets, rows, "f32")
    assert np.allclose(got, D, rtol=1e-13) and (tol > 0).all()
    grads, tols = G.gradients(dD, A, B, offsets, rows, "bf16", "f32")
    assert np.allclose(grads[0], dA, rtol=1e-12) and np.allclose(grads[1], dB, rtol=1e-12)
    assert (grads[1][1] == 0).all()       # the empty group


def test_rows_of_no_group_and_from_outside():
    A, B, offsets, rows, dD, _ = setup()
    rows = np.concatenate([rows, [0, 1]])
    rows[0] = 99
    D, _ = G.product(A, B, offsets, rows, "f32")
    assert np.isnan(D[9:]).all() and (D[0] == 0).all()


@pytest.mark.parametrize("plant", ["transposed", "group", "row"])
def test_planted_mistakes_show(plant):
    A, B, offsets, rows, dD, lens = setup()
    D, _, _ = by_torch(A, B, rows, dD, lens)
    wrong_b = np.roll(B, 1, axis=1) if plant == "transposed" else \
        B[::-1] if plant == "group" else B
    wrong_rows = (rows + 1) % 6 if plant == "row" else rows
    got, tol = G.product(A, wrong_b, offsets, wrong_rows, "bf16")
    assert (np.abs(got - D) > tol).any()


def test_combine_and_its_gradients():
    rng = np.random.default_rng(5)
    ids = rng.integers(-1, 3, (6, 2))
    rows, _, slots = G.group_rows(ids, 3)
    X, w, dout = rng.normal(size=(12, 4)), rng.normal(size=(6, 2)), rng.normal(size=(6, 4))
    x, v = torch.tensor(X, requires_grad=True), torch.tensor(w, requires_grad=True)
    kept = torch.tensor(slots >= 0)
    each = x[torch.tensor(np.maximum(slots, 0))] * (v * kept)[..., None]
    out = each.sum(1)
    (out * torch.tensor(dout)).sum().backward()
    got, _ = G.combine(X, slots, w, "f32")
    assert np.allclose(got, out.detach().numpy(), rtol=1e-13)
    (dX, dw), _ = G.combine_gradients(dout, X, slots, rows, w, "f32")
    assert np.allclose(dX, x.grad.numpy()) and np.allclose(dw, v.grad.numpy())


def test_adapters():
    rng = np.random.default_rng(7)
    x, W = rng.normal(size=(5, 6)), rng.normal(size=(3, 6))
    A, B, s = rng.normal(size=(2, 4, 6)), rng.normal(size=(2, 3, 4)), np.array([0.5, -2.0])
    rows, offsets = np.array([4, 0, 2, 1, 3]), np.array([0, 2, 3])
    D, tol = G.adapters(x, W, A, B, offsets, rows, s, "f16")
    for r, g in ((4, 0), (0, 0), (2, 1), (1, -1), (3, -1)):
        want = W @ x[r] + (0 if g < 0 else s[g] * B[g] @ (A[g] @ x[r]))
        assert np.allclose(D[r], want, rtol=1e-13)
        assert (tol[r] >= 2.0 ** -11 * np.abs(want)).all()


def test_bound_covers_fp32_and_is_not_loose():
    """The product formed in fp32 and rounded once lies within the bound, and
    one further bf16 rounding of an operand does not."""
    rng = np.random.default_rng(3)
    A = torch.tensor(rng.normal(size=(64, 512))).bfloat16()
    B = torch.tensor(rng.normal(size=(1, 32, 512))).bfloat16()
    want, tol = G.product(A.double().numpy(), B.double().numpy(), np.array([0, 64]), None, "f32")
    got = (A.float() @ B[0].float().t()).double().numpy()
    assert (np.abs(got - want) <= tol).all()
    off = (A.float() * 1.004).bfloat16().float() @ B[0].float().t()
    assert (np.abs(off.double().numpy() - want) > tol).any()
