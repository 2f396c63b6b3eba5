"""Rows behind the last sequence where the keys are split: nothing of theirs is
written, whatever the workspace held before the call."""
import ctypes

import pytest
import torch

from mma_fragment_layouts_tn_amd import _attention as B
from gpu_helpers import say
from oracle import attention as A
from test_gpu_attention import DT, Packed, f64, within
from test_gpu_use_attention import same

pytestmark = pytest.mark.gpu


def call(p, algo, splits, fill):
    """The C entry with a workspace, out and lse that held `fill`, 7 and 5."""
    q, k, v = (t.cuda() for t in (p.q, p.k, p.v))
    sq, sk = p.sq.cuda(), p.sk.cuda()
    out = torch.full(q.shape, 7.0, dtype=DT[p.kind]).cuda()
    lse = torch.full(q.shape[:2], 5.0).cuda()
    a = B.AttentionArgs(B._DTYPES[q.dtype], int(p.causal), sq.numel() - 1, q.shape[0], k.shape[0],
                        q.shape[1], k.shape[1], q.shape[2], *q.stride()[:2], *k.stride()[:2],
                        *v.stride()[:2], *out.stride()[:2], p.scale, B.ATTENTION_ALGOS[algo],
                        splits)
    ptrs = [t.data_ptr() for t in (q, k, v, sq, sk, out, lse)]
    n, parts = ctypes.c_int64(0), ctypes.c_int32(0)
    assert B._lib.attention_packed_plan(a, *ptrs, None, parts, n) == 0
    ws = torch.full((max(n.value, 16) // 4,), fill).cuda()
    torch.cuda.synchronize()
    stream = torch.cuda.current_stream().cuda_stream
    assert B._lib.attention_packed(a, *ptrs, ws.data_ptr(), n.value, stream) == 0
    torch.cuda.synchronize()
    say(f"[gpu]   {algo} splits={splits}: {parts.value} parts")
    return out, lse, parts.value


@pytest.mark.parametrize("splits", [0, 1, 2, 7])
@pytest.mark.parametrize("algo", ["tall", "flat"])
@pytest.mark.parametrize("ql,kl,tail", [
    ([33, 0, 100], [33, 5, 100], 1),
    ([33, 100], [500, 700], 40),
    ([2], [9000], 300),            # few rows, many keys: parts by themselves
], ids=str)
def test_tail_rows_of_split_keys(ql, kl, tail, algo, splits):
    p = Packed("bf16", ql, kl, 4, 2, 64, True, tail=tail)
    n = sum(ql)
    first = None
    for fill in (1.0, float("nan")):
        out, lse, parts = call(p, algo, splits, fill)
        assert (out[n:] == 7).all() and (lse[n:] == 5).all()
        if first is not None:
            assert same(out, first[0]) and same(lse, first[1])
        first = out, lse
    assert splits == 0 or parts == splits
    p.check_forward(algo=algo, splits=splits)


@pytest.mark.parametrize("algo", ["tall", "flat"])
def test_rows_before_the_first_sequence(algo):
    """Offsets that do not begin at 0: the rows before them are no rows either."""
    p = Packed("f16", [45], [45], 4, 2, 64, True, tail=5)
    p.sq, p.sk = (torch.tensor([8, 30, 45], dtype=torch.int32) for _ in range(2))
    want, wl, tol, tl = A.attention(f64(p.q), f64(p.k), f64(p.v), [8, 30, 45], [8, 30, 45], True,
                                    p.scale, p.kind)
    for splits in (1, 3):
        out, lse, _ = call(p, algo, splits, 1.0)
        for x, y in ((out, 7), (lse, 5)):
            assert (x[:8] == y).all() and (x[45:] == y).all()
        within("out", out[8:45], want[8:45], tol[8:45])
        within("lse", lse[8:45], wl[8:45], tl[8:45])
