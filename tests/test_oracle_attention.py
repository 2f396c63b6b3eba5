"""The float64 definition of attention (oracle/attention.py) against closed
forms, against differences, and its forms against each other."""
import numpy as np
import pytest

from oracle import attention as A


def data(rng, lq, lk, h, g, d):
    return (rng.standard_normal((lq, h, d)), rng.standard_normal((lk, g, d)),
            rng.standard_normal((lk, g, d)))


def forward(q, k, v, sq, sk, causal, scale=0.3):
    out, lse, _, _ = A.attention(q, k, v, sq, sk, causal, scale, "f16")
    return out, lse


def test_one_key_is_its_value():
    q, k, v = data(np.random.default_rng(0), 3, 1, 4, 2, 8)
    out, lse = forward(q, k, v, [0, 3], [0, 1], False)
    assert np.allclose(out, v[0][[0, 0, 1, 1]][None].repeat(3, 0), rtol=1e-14)
    s = 0.3 * np.einsum("thd,hd->th", q, k[0][[0, 0, 1, 1]])
    assert np.allclose(lse, s, rtol=1e-13)


def test_equal_scores_give_the_mean():
    _, k, v = data(np.random.default_rng(1), 1, 7, 1, 1, 8)
    out, lse = forward(np.zeros((1, 1, 8)), k, v, [0, 1], [0, 7], True)
    assert np.allclose(out[0, 0], v[:, 0].mean(axis=0), rtol=1e-13)
    assert np.isclose(lse[0, 0], np.log(7.0), rtol=1e-14)


def test_rows_without_keys():
    """Five queries, three keys, the last of both aligned: two rows see nothing."""
    q, k, v = data(np.random.default_rng(2), 5, 3, 2, 1, 8)
    out, lse = forward(q, k, v, [0, 5], [0, 3], True)
    assert not out[:2].any() and np.isneginf(lse[:2]).all()
    assert np.allclose(out[2], v[0], rtol=1e-14) and np.isfinite(lse[2:]).all()
    (dq, dk, dv), _ = A.gradients(np.ones_like(q), q, k, v, out, lse, [0, 5], [0, 3], True, 0.3,
                                  "f16")
    assert not dq[:2].any() and np.isfinite(dk).all() and np.isfinite(dv).all()


def test_packing_is_sequence_by_sequence():
    rng = np.random.default_rng(3)
    q, k, v = data(rng, 9, 11, 4, 2, 8)
    out, lse = forward(q, k, v, [0, 4, 4, 9], [0, 6, 7, 11], True)
    for a, b, x, y in ((0, 4, 0, 6), (4, 9, 7, 11)):
        o, l = forward(q[a:b], k[x:y], v[x:y], [0, b - a], [0, y - x], True)
        assert np.array_equal(out[a:b], o) and np.array_equal(lse[a:b], l)


@pytest.mark.parametrize("causal", [True, False])
def test_gradients_against_differences(causal):
    """Central differences of sum(out * dout): step 1e-5, error of the order
    of 1e-10, of the differences' rounding 1e-11."""
    rng = np.random.default_rng(4)
    q, k, v = data(rng, 6, 8, 4, 2, 4)
    dout = rng.standard_normal(q.shape)
    sq, sk = [0, 2, 2, 6], [0, 3, 4, 8]
    out, lse = forward(q, k, v, sq, sk, causal)
    grads, _ = A.gradients(dout, q, k, v, out, lse, sq, sk, causal, 0.3, "f16")
    for which in range(3):
        for _ in range(6):
            u = rng.standard_normal((q, k, v)[which].shape)
            x, y = [q, k, v], [q, k, v]
            x[which], y[which] = x[which] + 1e-5 * u, y[which] - 1e-5 * u
            slope = ((forward(*x, sq, sk, causal)[0] - forward(*y, sq, sk, causal)[0]) *
                     dout).sum() / 2e-5
            assert abs(slope - (grads[which] * u).sum()) < 1e-8


def test_prefix_is_the_longer_sequence():
    rng = np.random.default_rng(5)
    b, t, n0, cap, h, g, d = 3, 2, 5, 7, 4, 2, 8
    q = rng.standard_normal((b, t, h, d))
    pk, pv = rng.standard_normal((2, n0, g, d))
    k, v = rng.standard_normal((2, b, cap, g, d))
    lengths = [7, 2, 4]
    out, lse, _, _ = A.prefix_attention(q, pk, pv, k, v, lengths, 0.3, "f16")
    for i, n in enumerate(lengths):
        kk, vv = np.concatenate([pk, k[i, :n]]), np.concatenate([pv, v[i, :n]])
        o, l = forward(q[i], kk, vv, [0, t], [0, n0 + n], True)
        assert np.allclose(out[i], o, rtol=1e-13) and np.allclose(lse[i], l, rtol=1e-13)
