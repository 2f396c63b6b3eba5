"""Workspaces that attention's functions ask for stay within the bounds that
include/mfl_attention.h states, whatever the batch is made of."""
import ctypes

import pytest

from mma_fragment_layouts_tn_amd import _attention as B
from test_attention_api import GPTRS, packed, plan


def columns(dim):
    return 64 if dim <= 64 else 128 if dim <= 128 else 256


def layout(h, hk, d):
    return dict(heads_q=h, heads_kv=hk, head_dim=d, q_token=h * d, q_head=d, k_token=hk * d,
                k_head=d, v_token=hk * d, v_head=d, out_token=h * d, out_head=d)


@pytest.mark.parametrize("dim", [64, 80, 256])
@pytest.mark.parametrize("heads", [(32, 8), (16, 16), (8, 1), (40, 5)], ids=str)
def test_forward(heads, dim):
    """Batches of chunks against keys far longer: every plane of partial sums
    holds all rows, so the number of parts is what counts."""
    dc = columns(dim)
    most = 1 << 28
    split = 0
    for batch in (1, 2, 7, 16, 32, 64, 200):
        for q in (1, 5, 32, 64, 300):
            for keys in (300, 2000, 8192, 100000):
                rc, algo, splits, need = plan(packed(batch=batch, total_q=batch * q,
                                                     total_k=batch * keys,
                                                     **layout(*heads, dim)))
                assert rc == 0 and 1 <= splits <= 64
                assert need == (splits > 1) * splits * batch * q * heads[0] * (4 * dc + 8)
                assert need <= most, (batch, q, keys)
                split += splits > 1
    assert split > 10


def test_forward_few_rows_keep_their_parts():
    """Few rows and one sequence far longer than the others: its keys still go
    to many workgroups."""
    rc, algo, splits, need = plan(packed(batch=8, total_q=8, total_k=8 * 8300,
                                         **layout(32, 8, 128)))
    assert (rc, algo) == (0, 2) and splits >= 32 and need < 10e6


def test_no_rows():
    for keys in (0, 1, 100000):
        assert plan(packed(total_q=0, total_k=keys), q=0, out=0)[0] == 0


# ---------------------------------------------------------------- gradients
def grad_bytes(batch, tokens, heads, dim, causal):
    h, hk = heads
    f = packed(batch=batch, total_q=tokens, total_k=tokens, causal=causal, **layout(h, hk, dim))
    n = ctypes.c_int64(-1)
    a = B.AttentionGradArgs(f, h * dim, dim, h * dim, dim, hk * dim, dim, hk * dim, dim)
    assert B._lib.attention_packed_backward_plan(a, *GPTRS.values(), n) == 0
    return n.value


@pytest.mark.parametrize("causal", [0, 1])
@pytest.mark.parametrize("dim", [64, 128, 256])
def test_gradients(dim, causal):
    """Beside 8 bytes per row of q: a place of fp32 sums for every workgroup
    and every tile of keys, and never more than two per workgroup.  Up to 256
    key heads there are at most 256 workgroups, or where these would leave
    more than a sixteenth of the CUs idle, 1024."""
    dc = columns(dim)
    keys = 256 if dc == 128 else 128
    place = 8 * keys * dc
    for hk in list(range(1, 41)) + [48, 64, 85, 100, 128, 129, 200, 256]:
        whole = hk * (256 // hk) >= 240
        shares = (256 if whole else 1024) // hk
        for batch, tokens in ((1, 1), (1, 64), (3, 1045), (4, 2048), (4, 8192), (100, 5000)):
            tiles = tokens // keys + batch
            most = min(2 * shares, shares + tiles - 1) * hk * place
            n = grad_bytes(batch, tokens, (2 * hk, hk), dim, causal)
            assert 8 * 2 * hk * tokens <= n <= 8 * 2 * hk * tokens + most + 16 * shares + 16


def test_gradients_named():
    """16/4, 12/3 and 40/20 heads of 128."""
    assert grad_bytes(3, 1045, (16, 4), 128, 1) < 75e6
    assert grad_bytes(3, 1045, (12, 3), 128, 1) < 75e6
    assert grad_bytes(4, 2048, (40, 20), 128, 1) < 130e6
    assert grad_bytes(4, 8192, (32, 8), 128, 1) < 137e6
