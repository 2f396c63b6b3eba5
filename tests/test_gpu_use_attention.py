"""The attention functions as they are used: strided, shared and expanded
operands, rows of no sequence, other streams, captured graphs, caches beyond
32-bit offsets, the same bits every time, gradients against differences, and
the three together (a prompt, then decoding behind it, then training on it).

The file's name sorts behind test_gpu_probe.py: once a process has used several
streams, the die that a launch on the default one starts on is no longer the
first (the dies still take turns, which is what the kernels need), and a test
there asks for the first.
"""
import numpy as np
import pytest
import torch

import mma_fragment_layouts_tn_amd as mfl
from gpu_helpers import say
from oracle import attention as A
from test_gpu_attention import DT, Packed, Prefix, f64, offsets, values, within

pytestmark = pytest.mark.gpu


def same(a, b):
    return torch.equal(a.contiguous().view(torch.uint8), b.contiguous().view(torch.uint8))


@pytest.mark.parametrize("algo", ["tall", "flat"])
@pytest.mark.parametrize("tail", [1, 40, 400])
def test_tail_rows(tail, algo):
    """Rows behind the last sequence are not read (NaN, inf), out and lse of
    theirs stay, their gradients are 0."""
    p = Packed("bf16", [33, 100], [33, 100], 4, 2, 64, True, tail=tail)
    out, lse = p.check_forward(algo=algo)
    n = 133
    mark = torch.full_like(out, 7.0)
    got = mfl.attention(p.q.cuda(), p.k.cuda(), p.v.cuda(), out=mark, algo=algo, **p.how())
    assert got is mark and same(mark[:n], out[:n]) and (mark[n:] == 7).all()
    out[n:], lse[n:] = float("nan"), float("nan")
    dq, dk, dv = p.check_backward(out, lse)
    for x in (dq, dk, dv):
        assert not x[n:].any()


def test_sequences_at_the_end_only():
    """Every token behind the sequences: nothing to attend to."""
    p = Packed("f16", [0, 0], [0, 0], 4, 2, 64, True, tail=300)
    mark = torch.full(p.q.shape, 3.0, dtype=torch.float16).cuda()
    out, lse = mfl.attention(p.q.cuda(), p.k.cuda(), p.v.cuda(), out=mark, return_lse=True,
                             **p.how())
    assert (out == 3).all()
    for x in mfl.attention_backward(p.dout.cuda(), p.q.cuda(), p.k.cuda(), p.v.cuda(), out, lse,
                                    **p.how()):
        assert not x.any()


@pytest.mark.parametrize("tq,tk", [(0, 5), (5, 0), (0, 0)])
@pytest.mark.parametrize("packed", [True, False])
def test_no_tokens(tq, tk, packed):
    q = torch.ones(tq, 4, 64, dtype=torch.bfloat16).cuda()
    k = torch.ones(tk, 2, 64, dtype=torch.bfloat16).cuda()
    how = dict(seq_q=offsets([tq]).cuda(), seq_k=offsets([tk]).cuda()) if packed else {}
    out, lse = mfl.attention(q, k, k, return_lse=True, **how)
    assert out.shape == q.shape and not out.any() and torch.isneginf(lse).all()
    dq, dk, dv = mfl.attention_backward(q, q, k, k, out, lse, **how)
    assert not dq.any() and not dk.any() and not dv.any() and dk.shape == k.shape


@pytest.mark.parametrize("seq_q,seq_k", [
    ([0, -5, 40, 1 << 30], [0, 20, 20, 1 << 30]),
    ([0, 30, 10, 50], [0, 50, 10, 50]),
    ([5, 30, 40, 50], [10, 30, 40, 45]),
    ([-(1 << 31), (1 << 31) - 1, 0, 0], [(1 << 31) - 1, 0, -1, 0]),
])
def test_offsets_out_of_order(seq_q, seq_k):
    """Offsets that are wrong give wrong rows, never an access outside."""
    gen = torch.Generator().manual_seed(0)
    q, k = values(gen, (50, 4, 64), "bf16").cuda(), values(gen, (50, 2, 64), "bf16").cuda()
    how = dict(seq_q=torch.tensor(seq_q, dtype=torch.int32).cuda(),
               seq_k=torch.tensor(seq_k, dtype=torch.int32).cuda())
    for algo in ("tall", "flat"):
        for splits in (0, 3):
            say(f"[gpu] offsets {seq_q} {seq_k} {algo} {splits}")
            out, lse = mfl.attention(q, k, k, return_lse=True, algo=algo, splits=splits, **how)
            torch.cuda.synchronize()
    mfl.attention_backward(q, q, k, k, torch.zeros_like(q), torch.zeros_like(lse), **how)
    torch.cuda.synchronize()


def test_strided_operands():
    """q, k and v as slices of one projection, out as a slice; heads outside
    tokens; equal to the same values laid out plainly."""
    gen = torch.Generator().manual_seed(1)
    t, h, g, d = 150, 4, 2, 72
    qkv = values(gen, (t, h + 2 * g, d + 8), "bf16").cuda()[:, :, :d]
    q, k, v = qkv[:, :h], qkv[:, h:h + g], qkv[:, h + g:]
    how = dict(seq_q=offsets([90, 60]).cuda())
    plain, lse = mfl.attention(q.contiguous(), k.contiguous(), v.contiguous(), return_lse=True,
                               **how)
    big = torch.full((t, h, 2 * d), 5.0, dtype=torch.bfloat16).cuda()
    out, l2 = mfl.attention(q, k, v, out=big[:, :, :d], return_lse=True, **how)
    assert same(out, plain) and same(lse, l2) and (big[:, :, d:] == 5).all()
    hq, hk, hv = (x.transpose(0, 1).contiguous().transpose(0, 1) for x in (q, k, v))
    ho = torch.empty(h, t, d, dtype=torch.bfloat16).cuda().transpose(0, 1)
    assert same(mfl.attention(hq, hk, hv, out=ho, **how), plain)
    dout = values(gen, (t, h, d), "bf16").cuda()
    want = mfl.attention_backward(dout, q.contiguous(), k.contiguous(), v.contiguous(), plain, lse,
                                  **how)
    for args in ((dout, q, k, v, out, lse), (dout, hq, hk, hv, ho, lse)):
        for x, y in zip(mfl.attention_backward(*args, **how), want):
            assert same(x, y)


def test_expanded_operands():
    """One value for all tokens or heads (stride 0), as a sum's gradient is."""
    gen = torch.Generator().manual_seed(2)
    q, k = values(gen, (70, 4, 64), "f16").cuda(), values(gen, (70, 1, 64), "f16").cuda()
    ek = k.expand(70, 2, 64)
    dout = torch.ones(1, 1, 64, dtype=torch.float16).cuda().expand(70, 4, 64)
    out, lse = mfl.attention(q, ek, ek, return_lse=True)
    ck = ek.contiguous()
    o2, l2 = mfl.attention(q, ck, ck, return_lse=True)
    assert same(out, o2) and same(lse, l2)
    want = mfl.attention_backward(dout.contiguous(), q, ck, ck, out, lse)
    for x, y in zip(mfl.attention_backward(dout, q, ek, ek, out, lse), want):
        assert same(x, y)
    one = q[:1].expand(70, 4, 64)                       # every query the same
    a, l1 = mfl.attention(one, ck, ck, return_lse=True)
    b, _ = mfl.attention(one.contiguous(), ck, ck, return_lse=True)
    assert same(a, b)
    want = mfl.attention_backward(dout.contiguous(), one.contiguous(), ck, ck, a, l1)
    for x, y in zip(mfl.attention_backward(dout, one, ck, ck, a, l1), want):
        assert same(x, y)


def test_same_bits():
    """Gradients of shared heads and split keys: no order left to chance."""
    p = Packed("bf16", [700, 1, 350], [700, 1, 350], 8, 2, 128, True)
    dev = [x.cuda() for x in (p.dout, p.q, p.k, p.v)]
    out, lse = p.forward(splits=5)
    want = mfl.attention_backward(*dev, out, lse, **p.how())
    for _ in range(4):
        o, l = p.forward(splits=5)
        assert same(o, out) and same(l, lse)
        for x, y in zip(mfl.attention_backward(*dev, out, lse, **p.how()), want):
            assert same(x, y)


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("heads", [(8, 4, 64), (8, 2, 128), (4, 2, 256)], ids=str)
def test_backward_shares(heads, causal):
    """Tiles cut between workgroups in many ways: many sequences, long beside
    short, keys without queries."""
    p = Packed("bf16", [1500, 0, 3, 128, 257, 64], [1500, 300, 40, 100, 257, 1], *heads, causal)
    p.check_backward(*p.check_forward())


def test_backward_a_tile_each():
    """More sequences than shares are made for."""
    n = [(7 * i) % 5 for i in range(300)]
    p = Packed("f16", n, [x + i % 3 for i, x in enumerate(n)], 4, 2, 64, True)
    p.check_backward(*p.check_forward())


@pytest.mark.parametrize("gain", [1.0, 30.0])
def test_large_scores(gain):
    """Scores to a thousand and beyond: the running maximum moves by more than
    its slack, weights leave fp32's range below."""
    p = Packed("bf16", [200], [333], 4, 2, 128, True, gain=gain, scale=1.0)
    p.check_backward(*p.check_forward(algo="tall"))
    p.check_forward(algo="flat")


def test_other_stream():
    p = Packed("bf16", [300, 77], [300, 77], 8, 2, 128, True)
    want_o, want_l = p.forward()
    dev = [x.cuda() for x in (p.q, p.k, p.v, p.dout)]
    how = p.how()
    want = mfl.attention_backward(dev[3], *dev[:3], want_o, want_l, **how)
    ones = torch.ones(1, 1, 128, dtype=torch.bfloat16).cuda().expand(377, 8, 128)
    want1 = mfl.attention_backward(ones, *dev[:3], want_o, want_l, **how)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    for _ in range(3):
        out, lse = mfl.attention(*dev[:3], return_lse=True, splits=3, stream=s.cuda_stream, **how)
        out, lse = mfl.attention(*dev[:3], return_lse=True, stream=s.cuda_stream, **how)
        got = mfl.attention_backward(dev[3], *dev[:3], out, lse, stream=s.cuda_stream, **how)
        got1 = mfl.attention_backward(ones, *dev[:3], out, lse, stream=s.cuda_stream, **how)
        s.synchronize()
        assert same(out, want_o) and same(lse, want_l)
        assert all(same(x, y) for x, y in zip(got, want))
        assert all(same(x, y) for x, y in zip(got1, want1))
    with torch.cuda.stream(s):                          # the current stream, without the argument
        out = mfl.attention(*dev[:3], **how)
    s.synchronize()
    assert same(out, want_o)


def test_graphs():
    """Captured, replayed with other inputs, with eager calls between; two
    graphs, each with workspaces of its own."""
    p = Packed("bf16", [250, 700], [250, 700], 8, 2, 128, True)
    x = Prefix("bf16", 6, 1, 900, 64, [64, 0, 1, 33, 20, 64], 8, 2, 128)
    x.k, x.v = torch.nan_to_num(x.k), torch.nan_to_num(x.v, posinf=1.0)
    dev = [t.cuda() for t in (p.q, p.k, p.v, p.dout)]
    pre = [t.cuda() for t in (x.q, x.pk, x.pv, x.k, x.v, x.lengths)]
    how = p.how()

    def train():
        out, lse = mfl.attention(*dev[:3], return_lse=True, splits=2, **how)
        return (out, lse, *mfl.attention_backward(dev[3], *dev[:3], out, lse, **how))

    def decode():
        return mfl.attention_prefix(*pre, return_lse=True)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        train(), decode()
    torch.cuda.current_stream().wait_stream(side)
    graphs = []
    for f in (train, decode):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            got = f()
        graphs.append((g, got, f))
    gen = torch.Generator().manual_seed(9)
    for i in range(4):
        for t in dev + pre[:5]:
            t.copy_(values(gen, t.shape, "bf16"))
        pre[5].copy_(torch.tensor([i, 64, 0, 5 * i, 64 - i, 7], dtype=torch.int32))
        for g, got, f in graphs if i % 2 else graphs[::-1]:
            g.replay()
        eager = [f() for _, _, f in graphs]
        torch.cuda.synchronize()
        for (_, got, _), want in zip(graphs, eager):
            assert all(same(a, b) for a, b in zip(got, want)), i


def test_long_offsets():
    """Elements beyond 2^32 of the first: a cache by its batch, head and token
    strides, k and v of packed sequences by theirs."""
    big = torch.empty((1 << 32) + (1 << 26), dtype=torch.bfloat16, device="cuda")
    gen = torch.Generator().manual_seed(3)

    def view(shape, strides, at=0):
        t = big.as_strided(shape, strides, at)
        t.copy_(values(gen, shape, "bf16"))
        return t
    q = values(gen, (2, 1, 4, 64), "bf16").cuda()
    pk, pv = (values(gen, (70, 2, 64), "bf16").cuda() for _ in range(2))
    n = torch.tensor([90, 41], dtype=torch.int32).cuda()
    for strides in (((1 << 32), 128, 64), (128 * 90, 128, 1 << 32)):
        shape = (2, 90, 2, 64)
        strides = (*strides, 1)
        k, v = view(shape, strides), view(shape, strides, 1 << 20)
        assert same(mfl.attention_prefix(q, pk, pv, k, v, n),
                    mfl.attention_prefix(q, pk, pv, k.contiguous(), v.contiguous(), n))
    q = values(gen, (513, 2, 64), "bf16").cuda()
    how = dict(seq_q=offsets([200, 313]).cuda())
    k, v = view((513, 1, 64), (1 << 23, 64, 1)), view((513, 1, 64), (1 << 23, 64, 1), 1 << 20)
    for algo in ("tall", "flat"):
        out, lse = mfl.attention(q, k, v, return_lse=True, algo=algo, **how)
        assert same(out, mfl.attention(q, k.contiguous(), v.contiguous(), algo=algo, **how))
    want = mfl.attention_backward(q, q, k.contiguous(), v.contiguous(), out, lse, **how)
    for x, y in zip(mfl.attention_backward(q, q, k, v, out, lse, **how), want):
        assert same(x, y)
    fq = view((513, 2, 64), (1 << 23, 64, 1), 1 << 21)          # q, dout and out too
    o = view((513, 2, 64), (1 << 23, 64, 1), 1 << 22)
    out, lse = mfl.attention(fq, k, v, return_lse=True, out=o, **how)
    c = [t.contiguous() for t in (fq, k, v, o)]
    assert same(o, mfl.attention(*c[:3], **how))
    want = mfl.attention_backward(c[0], *c, lse, **how)
    for x, y in zip(mfl.attention_backward(fq, fq, k, v, o, lse, **how), want):
        assert same(x, y)
    say("[gpu] long offsets done")


@pytest.mark.parametrize("kind", ["f16", "bf16"])
def test_gradients_against_differences(kind):
    """Along random directions u: the differences of the float64 definition,
    at a step whose own error is below 1e-6 of the bound, against the
    kernels' gradients.  Beside their bound for the out and lse they are
    given, those two's own errors count: a row's delta is off by at most
    sum(|dout| tol_out), its weights by a factor 1 + tol_lse."""
    p = Packed(kind, [37], [37], 4, 2, 64, True, gain=1.0)
    q, k, v, dout = (f64(t) for t in (p.q, p.k, p.v, p.dout))
    seq = [0, 37]
    how = (seq, seq, True, p.scale, kind)
    exact, el, tol_o, tol_l = A.attention(q, k, v, *how)
    out, lse = p.forward()
    got = mfl.attention_backward(*(t.cuda() for t in (p.dout, p.q, p.k, p.v)), out, lse, **p.how())
    torch.cuda.synchronize()
    (wq, wk, wv), tols = A.gradients(dout, q, k, v, exact, el, *how)
    more = [np.zeros_like(x) for x in (q, k, v)]
    for i in range(4):
        j = i // 2
        r = A.one_head(q[:, i], k[:, j], v[:, j], p.scale, A.visible(37, 37, True))
        dd = (np.abs(dout[:, i]) * tol_o[:, i]).sum(axis=1)[:, None]
        ds = np.abs(r.p * (dout[:, i] @ v[:, j].T - (dout[:, i] * r.out).sum(axis=1)[:, None]))
        off = r.p * dd + 1.1 * tol_l[:, i][:, None] * (ds + r.p * dd)
        more[0][:, i] = p.scale * off @ np.abs(k[:, j])
        more[1][:, j] += p.scale * off.T @ np.abs(q[:, i])
        more[2][:, j] += (1.1 * tol_l[:, i][:, None] * r.p).T @ np.abs(dout[:, i])
    rng = np.random.default_rng(0)
    for which, name in enumerate("qkv"):
        for _ in range(5):
            u = rng.standard_normal((q, k, v)[which].shape)
            x, y = [q, k, v], [q, k, v]
            x[which], y[which] = x[which] + 1e-5 * u, y[which] - 1e-5 * u
            slope = ((A.attention(*x, *how)[0] - A.attention(*y, *how)[0]) * dout).sum() / 2e-5
            bound = ((1.1 * tols[which] + 1.1 * more[which]) * np.abs(u)).sum()
            off = abs((f64(got[which]) * u).sum() - slope)
            say(f"[gpu]   d{name}: off {off:.2e}, bound {bound:.2e}")
            assert off <= bound


def test_prompt_then_decoding_then_training():
    """As they are used together: a prompt is attended to, its keys are the
    prefix of a batch that decodes token by token, each step equal to packed
    attention over the whole sequence so far; the finished sequences are
    trained on."""
    gen = torch.Generator().manual_seed(5)
    h, g, d, n0, steps, b = 8, 2, 64, 150, 4, 5
    kind, scale = "bf16", 64 ** -0.5
    pq, pk, pv = (values(gen, (n0, x, d), kind) for x in (h, g, g))
    out, lse = mfl.attention(pq.cuda(), pk.cuda(), pv.cuda(), return_lse=True)
    want, wl, tol, tl = A.attention(f64(pq), f64(pk), f64(pv), [0, n0], [0, n0], True, scale, kind)
    within("prompt", out, want, tol)
    within("prompt lse", lse, wl, tl)
    kc, vc = (torch.full((b, steps, g, d), float("nan"), dtype=DT[kind]).cuda() for _ in range(2))
    qs, ks, vs = (values(gen, (b, steps, x, d), kind) for x in (h, g, g))
    outs = []
    for t in range(steps):
        kc[:, t], vc[:, t] = ks[:, t].cuda(), vs[:, t].cuda()
        n = torch.full((b,), t + 1, dtype=torch.int32).cuda()
        outs.append(mfl.attention_prefix(qs[:, t].cuda(), pk.cuda(), pv.cuda(), kc, vc, n))
    got = torch.stack(outs, 1)
    # the same sequences, whole
    q = torch.cat([torch.cat([pq, qs[i]]) for i in range(b)])
    k = torch.cat([torch.cat([pk, ks[i]]) for i in range(b)])
    v = torch.cat([torch.cat([pv, vs[i]]) for i in range(b)])
    seq = [i * (n0 + steps) for i in range(b + 1)]
    want, wl, tol, tl = A.attention(f64(q), f64(k), f64(v), seq, seq, True, scale, kind)
    rows = np.concatenate([np.arange(s + n0, s + n0 + steps) for s in seq[:-1]])
    within("decoded", got.reshape(b * steps, h, d), want[rows], tol[rows])
    p = Packed(kind, [n0 + steps] * b, [n0 + steps] * b, h, g, d, True)
    p.q, p.k, p.v = q, k, v
    p.check_backward(*p.check_forward())


@pytest.mark.parametrize("dim", [8, 24, 136, 248])
def test_head_dims(dim):
    p = Packed("bf16", [70, 1, 140], [95, 1, 140], 4, 2, dim, True)
    p.check_backward(*p.check_forward(algo="tall"))
    p.check_forward(algo="flat")
    Prefix("bf16", 3, 2, 100, 40, [0, 2, 40], 4, 2, dim).check()


def test_many_sequences():
    """Thousands of sequences of up to three tokens, many empty."""
    n = [(11 * i) % 7 % 4 for i in range(5000)]
    p = Packed("bf16", n, n, 2, 1, 64, True)
    for algo in ("flat", "tall"):
        out, lse = p.check_forward(algo=algo)
    p.check_backward(out, lse)


def test_neighbours_do_not_leak():
    """A sequence full of NaN between two others: theirs stay the same bits."""
    lens = [37, 50, 90]
    p = Packed("bf16", lens, lens, 4, 2, 64, True)
    dev = [x.cuda() for x in (p.q, p.k, p.v, p.dout)]
    how = p.how()

    def run():
        res = []
        for algo in ("tall", "flat"):
            for splits in (1, 3):
                res += mfl.attention(*dev[:3], return_lse=True, algo=algo, splits=splits, **how)
        out, lse = mfl.attention(*dev[:3], return_lse=True, **how)
        return [*res, *mfl.attention_backward(dev[3], *dev[:3], out, lse, **how)]
    clean = run()
    for x in dev:
        x[37:87] = float("nan")
    for a, b in zip(run(), clean):
        assert same(a[:37], b[:37]) and same(a[87:], b[87:])


def test_prefix_lengths_are_held():
    """Lengths below 0 and beyond the capacity count as 0 and the capacity;
    one cache for the whole batch."""
    x = Prefix("bf16", 4, 2, 70, 33, [0, 33, 33, 0], 4, 2, 64)
    dev = [t.cuda() for t in (x.q, x.pk, x.pv, x.k, x.v)]
    want = mfl.attention_prefix(*dev, x.lengths.cuda())
    wrong = torch.tensor([-7, 34, (1 << 31) - 1, -(1 << 31)], dtype=torch.int32).cuda()
    assert same(mfl.attention_prefix(*dev, wrong), want)
    k, v = (t[1:2].expand(4, 33, 2, 64) for t in dev[3:])
    n = torch.tensor([33, 5, 1, 20], dtype=torch.int32).cuda()
    assert same(mfl.attention_prefix(*dev[:3], k, v, n),
                mfl.attention_prefix(*dev[:3], k.contiguous(), v.contiguous(), n))


def test_one_token_sum():
    """The gradient of a sum at one token: every stride 0."""
    gen = torch.Generator().manual_seed(4)
    q, k = values(gen, (1, 4, 64), "f16").cuda(), values(gen, (9, 2, 64), "f16").cuda()
    out, lse = mfl.attention(q, k, k, return_lse=True)
    ones = torch.ones((), dtype=torch.float16).cuda().expand(1, 4, 64)
    want = mfl.attention_backward(ones.contiguous(), q, k, k, out, lse)
    for a, b in zip(mfl.attention_backward(ones, q, k, k, out, lse), want):
        assert same(a, b)


def test_two_streams_at_once():
    """Calls with workspaces in flight on two streams together."""
    p = Packed("bf16", [600, 300], [600, 300], 8, 2, 128, True)
    x = Prefix("bf16", 32, 1, 2000, 100, [3 * i for i in range(32)], 8, 2, 128)
    dev = [t.cuda() for t in (p.q, p.k, p.v, p.dout)]
    pre = [t.cuda() for t in (x.q, x.pk, x.pv, x.k, x.v, x.lengths)]
    how = p.how()
    out, lse = mfl.attention(*dev[:3], return_lse=True, splits=4, **how)
    grads = mfl.attention_backward(dev[3], *dev[:3], out, lse, **how)
    dec = mfl.attention_prefix(*pre)
    torch.cuda.synchronize()
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    got = []
    for _ in range(5):
        with torch.cuda.stream(a):
            o, l = mfl.attention(*dev[:3], return_lse=True, splits=4, **how)
            got.append((o, out))
            got += zip(mfl.attention_backward(dev[3], *dev[:3], o, l, **how), grads)
        with torch.cuda.stream(b):
            for _ in range(4):
                got.append((mfl.attention_prefix(*pre), dec))
    torch.cuda.synchronize()
    assert all(same(x, y) for x, y in got)


@pytest.mark.parametrize("heads", [(300, 300, 64), (1100, 1100, 8), (64, 1, 64), (34, 2, 128)],
                         ids=str)
def test_many_heads(heads):
    """More key heads than workgroups for shares of the keys; groups wider
    than a tile's 16 rows, and not a power of two."""
    p = Packed("bf16", [33, 2], [40, 2], *heads, True)
    p.check_backward(*p.check_forward(algo="flat"))
    p.check_forward(algo="tall")
    Prefix("bf16", 2, 1, 40, 9, [9, 3], *heads).check()
