"""Workspaces that attention's functions ask for stay within the bounds that
include/mfl_attention.h states, whatever the batch is made of."""
import pytest

from test_attention_api import packed, plan


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
