"""Sizes whose launches would have more workgroups than the GPU takes are
refused by the plan and by the call, before anything is launched; the sizes
just below are planned."""
import ctypes

import pytest

from mma_fragment_layouts_tn_amd import _attention as B
from test_attention_api import GPTRS, LARGE, UNSUP, packed, plan, prefix, prefix_plan

FLAT, TALL = 2, 1


def one_head(**kw):
    """Heads of 8 elements, one query and one key head."""
    return packed(**dict(dict(heads_q=1, heads_kv=1, head_dim=8, q_token=8, q_head=8, k_token=8,
                              k_head=8, v_token=8, v_head=8, out_token=8, out_head=8), **kw))


@pytest.mark.parametrize("kw,fits", [
    # one workgroup per 16 rows
    (dict(batch=1, total_q=(1 << 28) - 16, total_k=8, algo=FLAT), True),
    (dict(batch=1, total_q=1 << 28, total_k=8, algo=FLAT), False),
    (dict(batch=1, total_q=1 << 28, total_k=8, algo=TALL), True),
    # one per sequence, kv head and split
    (dict(batch=1 << 20, total_q=1 << 20, total_k=1 << 20, heads_q=15, heads_kv=15, q_token=120,
          out_token=120, k_token=120, v_token=120), True),
    (dict(batch=1 << 20, total_q=1 << 20, total_k=1 << 20, heads_q=16, heads_kv=16, q_token=128,
          out_token=128, k_token=128, v_token=128), False),
    (dict(batch=1 << 20, total_q=1 << 20, total_k=1 << 20, algo=FLAT, splits=16), False),
    # TALL in two splits: joining takes one per 8 rows
    (dict(batch=1, total_q=1 << 26, total_k=8, algo=TALL, splits=2), True),
    (dict(batch=1, total_q=1 << 27, total_k=8, algo=TALL, splits=2), False),
], ids=str)
def test_forward(kw, fits):
    p = dict(seq_q=0, seq_k=0) if kw["batch"] == 1 else {}
    assert plan(one_head(**kw), **p)[0] == (0 if fits else LARGE)


@pytest.mark.parametrize("heads,fits", [(15, True), (16, False)])
def test_backward(heads, fits):
    """One workgroup at least per sequence and kv head."""
    t = 8 * heads
    f = one_head(batch=1 << 20, total_q=1 << 20, total_k=1 << 20, heads_q=heads, heads_kv=heads,
                 q_token=t, k_token=t, v_token=t, out_token=t)
    a = B.AttentionGradArgs(f, *[t, 8] * 4)
    n = ctypes.c_int64(-1)
    want = 0 if fits else LARGE
    assert B._lib.attention_packed_backward_plan(a, *GPTRS.values(), n) == want
    if not fits:
        assert B._lib.attention_packed_backward(a, *GPTRS.values(), None, 0, None) == want


@pytest.mark.parametrize("kw,fits", [
    (dict(batch=1 << 20, heads_q=8, heads_kv=8), True),        # own keys: one each
    (dict(batch=1 << 21, heads_q=8, heads_kv=8), False),
    (dict(batch=1 << 20, heads_q=32, heads_kv=1), True),       # the join: 4 rows each
    (dict(batch=1 << 20, heads_q=64, heads_kv=1), False),
    (dict(batch=1 << 20, heads_q=64, heads_kv=1, prefix=0, splits_own=1), True),   # no join
], ids=str)
def test_prefix(kw, fits):
    h, hk = kw["heads_q"], kw["heads_kv"]
    a = dict(q_tokens=1, head_dim=8, q_batch=8 * h, q_token=0, q_head=8, out_batch=8 * h,
             out_token=0, out_head=8, prefix_k_token=8 * hk, prefix_k_head=8,
             prefix_v_token=8 * hk, prefix_v_head=8, k_token=8 * hk, k_head=8, v_token=8 * hk,
             v_head=8, k_batch=0, v_batch=0)
    assert prefix_plan(prefix(**dict(a, **kw)))[0] == (0 if fits else LARGE)


@pytest.mark.parametrize("scale,code", [(2.3e38, 0), (2.4e38, UNSUP), (3.4e38, UNSUP)])
def test_scale(scale, code):
    """The kernels work in powers of two: scale * log2(e) has to be a number."""
    assert plan(packed(scale=scale))[0] == code
    assert prefix_plan(prefix(scale=scale))[0] == code
