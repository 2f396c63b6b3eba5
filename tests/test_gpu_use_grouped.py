"""Products by groups of rows as they are used: an experts' layer with its
gradients, a batch of requests with adapters, captured and replayed, on other
streams, beside each other, with tensors that pass 4 GiB; and the same bits
every time."""
import numpy as np
import pytest
import torch

import mma_fragment_layouts_tn_amd as mfl
from gpu_helpers import say
from oracle import grouped as G
from test_gpu_grouped import DT, f64, values, within

pytestmark = pytest.mark.gpu
U = 2.0 ** -8            # half a step of bf16


class Layer:
    """Experts of two products with a SiLU between them, a token's two best
    added by the router's weights; some tokens are padding."""

    def __init__(self, tokens=200, dim=128, inner=192, experts=6, top=2, seed=0):
        gen = torch.Generator().manual_seed(seed)
        self.x = values(gen, (tokens, dim), "bf16").cuda()
        self.W1 = values(gen, (experts, inner, dim), "bf16", dim ** -0.5).cuda()
        self.W2 = values(gen, (experts, dim, inner), "bf16", inner ** -0.5).cuda()
        self.dout = values(gen, (tokens, dim), "bf16").cuda()
        score = torch.randn(tokens, experts, generator=gen)
        best = score.softmax(1).topk(top)
        self.ids = best.indices
        self.ids[::17] = -1
        self.ids, self.w = self.ids.cuda(), best.values.contiguous().cuda()
        self.experts = experts

    def forward(self):
        s = self
        s.rows, s.offsets, s.slots = mfl.group_rows(s.ids, s.experts)
        s.h = mfl.gemm_grouped(s.x, s.W1, s.offsets, rows=s.rows)
        s.a = torch.nn.functional.silu(s.h)
        s.y = mfl.gemm_grouped(s.a, s.W2, s.offsets)
        s.out = mfl.combine_rows(s.y, s.slots, s.w)
        return s.out

    def backward(self):
        s = self
        s.dy, s.dw = mfl.combine_rows_backward(s.dout, s.y, s.slots, s.w, rows=s.rows)
        s.da, s.dW2 = mfl.gemm_grouped_backward(s.dy, s.a, s.W2, s.offsets)
        sig = torch.sigmoid(s.h.float())
        s.dh = (s.da.float() * sig * (1 + s.h.float() * (1 - sig))).bfloat16()
        s.dxs, s.dW1 = mfl.gemm_grouped_backward(s.dh, s.x, s.W1, s.offsets, rows=s.rows)
        s.dx = mfl.combine_rows(s.dxs, s.slots)
        return s.dx, s.dW1, s.dW2, s.dw


def test_experts_layer_step_by_step():
    """Each step within the oracle's bound of its own inputs."""
    s = Layer()
    s.forward()
    s.backward()
    torch.cuda.synchronize()
    ids = s.ids.cpu().numpy()
    rows, offsets, slots = G.group_rows(ids, s.experts)
    n = offsets[-1]
    assert np.array_equal(s.rows.cpu().numpy(), rows) and \
        np.array_equal(s.offsets.cpu().numpy(), offsets) and \
        np.array_equal(s.slots.cpu().numpy(), slots)
    x, W1, W2, w, dout = (f64(t) for t in (s.x, s.W1, s.W2, s.w, s.dout))
    want, tol = G.product(x, W1, offsets, rows, "bf16")
    within("h", s.h, want, tol)
    a = np.nan_to_num(f64(s.a)[:n])
    a = np.concatenate([a, np.zeros((len(rows) - n, a.shape[1]))])
    want, tol = G.product(a, W2, offsets, None, "bf16")
    within("y", s.y, want, tol)
    y = np.concatenate([f64(s.y)[:n], np.zeros((len(rows) - n, x.shape[1]))])
    want, tol = G.combine(y, slots, w, "bf16")
    within("out", s.out, want, tol)
    want, tol = G.combine_gradients(dout, y, slots, rows, w, "bf16")
    within("dy", s.dy, want[0], tol[0])
    within("dw", s.dw, want[1], tol[1])
    want, tol = G.gradients(f64(s.dy), a, W2, offsets, None, "bf16", "bf16")
    within("da", s.da, want[0], tol[0])
    within("dW2", s.dW2, want[1], tol[1])
    dh = np.concatenate([f64(s.dh)[:n], np.zeros((len(rows) - n, a.shape[1]))])
    want, tol = G.gradients(dh, x, W1, offsets, rows, "bf16", "bf16")
    within("dxs", s.dxs, want[0], tol[0])
    within("dW1", s.dW1, want[1], tol[1])
    want, tol = G.combine(f64(s.dxs), slots, np.ones(slots.shape), "bf16")
    within("dx", s.dx, want, tol)


def test_experts_layer_end_to_end():
    """Out and gradients against autograd in float64.  The bound: a rounding of
    half a step per stored intermediate, carried through the products' absolute
    values (SiLU and its derivative change by at most 1.1 and 0.5 times an
    error), a thousandth more for fp32 sums and what is of second order."""
    s = Layer(seed=3)
    s.forward()
    got = s.backward()
    x, W1, W2, w = (t.double().cpu().requires_grad_() for t in (s.x, s.W1, s.W2, s.w))
    dout = s.dout.double().cpu()
    ids = s.ids.cpu()
    out = torch.zeros_like(x)
    e_out, e_dx = torch.zeros(x.shape).double(), torch.zeros(x.shape).double()
    e_W1, e_W2 = torch.zeros(W1.shape).double(), torch.zeros(W2.shape).double()
    e_w = torch.zeros(w.shape).double()
    parts = []
    for j in range(ids.shape[1]):
        for g in range(s.experts):
            t = torch.nonzero(ids[:, j] == g).flatten()
            h = x[t] @ W1[g].t()
            a = torch.nn.functional.silu(h)
            y = a @ W2[g].t()
            parts.append((t, w[t, j, None] * y))
            with torch.no_grad():
                e_h = U * h.abs()
                e_a = 1.1 * e_h + U * a.abs()
                e_y = e_a @ W2[g].abs().t() + U * y.abs()
                e_out[t] += w[t, j, None] * e_y
                e_w[t, j] += (dout[t].abs() * e_y).sum(1)
                dy = w[t, j, None] * dout[t]
                e_dy = U * dy.abs()
                da = dy @ W2[g]
                e_da = e_dy @ W2[g].abs() + U * da.abs()
                e_W2[g] += e_dy.t() @ a.abs() + dy.abs().t() @ e_a
                sig = torch.sigmoid(h)
                d = sig * (1 + h * (1 - sig))
                dh = da * d
                e_dh = e_da * d.abs() + 0.5 * e_h * da.abs() + U * dh.abs()
                dxs = dh @ W1[g]
                e_dx[t] += e_dh @ W1[g].abs() + U * dxs.abs()
                e_W1[g] += e_dh.t() @ x[t].abs()
    for t, p in parts:
        out = out.index_add(0, t, p)
    (out * dout).sum().backward()
    for name, g, want, e in (("out", s.out, out, e_out), ("dx", got[0], x.grad, e_dx),
                             ("dW1", got[1], W1.grad, e_W1), ("dW2", got[2], W2.grad, e_W2),
                             ("dw", got[3], w.grad, e_w)):
        want = want.detach().numpy()
        within(name, g, want, 1.05 * e.numpy() + 1e-3 * np.abs(want) + U * np.abs(want) + 1e-4)


def eager(fs):
    r = [f() for f in fs]
    torch.cuda.synchronize()
    return [[t.clone() for t in (x if isinstance(x, (tuple, list)) else [x])] for x in r]


def same(a, b):
    return all(torch.equal(x, y) for p, q in zip(a, b) for x, y in zip(p, q))


def calls(seed=0):
    """Calls of every function on inputs of their own, results whole."""
    s = Layer(seed=seed, tokens=301)
    gen = torch.Generator().manual_seed(seed)
    ad = torch.randint(-1, 5, (40,), generator=gen)
    x, W = values(gen, (40, 256), "f16").cuda(), values(gen, (512, 256), "f16", 0.06).cuda()
    A, B = values(gen, (5, 16, 256), "f16", 0.06).cuda(), values(gen, (5, 512, 16), "f16").cuda()
    ids = torch.randint(0, 7, (9000,), generator=gen).cuda()
    rows, offsets, _ = mfl.group_rows(ad.cuda(), 5)

    def layer():
        s.forward()
        n = int(301 - len(range(0, 301, 17))) * 2        # the kept places
        return (s.out, s.h[:n], s.y[:n])

    return s, [layer, lambda: s.backward(),
               lambda: mfl.group_rows(ids, 7),
               lambda: mfl.gemm_adapters(x, W, A, B, offsets, rows=rows),
               lambda: mfl.gemm_adapters(x, W, A, B, offsets, rows=rows, algo="tile128")]


def test_same_bits():
    _, fs = calls(1)
    first = eager(fs)
    for _ in range(3):
        assert same(first, eager(fs))


def test_captured_and_replayed():
    """A graph of every function, replayed on changed inputs between eager
    calls, gives the eager results' bits."""
    s, fs = calls(2)
    eager(fs)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for f in fs:
            f()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = [f() for f in fs]
    for k in range(4):
        say(f"[gpu] replay {k}")
        gen = torch.Generator().manual_seed(100 + k)
        s.x.copy_(values(gen, tuple(s.x.shape), "bf16"))
        ids = torch.rand(301, s.experts, generator=gen).topk(2).indices
        ids[::17] = -1
        s.ids.copy_(ids)
        graph.replay()
        torch.cuda.synchronize()
        got = [[t.clone() for t in (x if isinstance(x, (tuple, list)) else [x])] for x in held]
        assert same(got, eager(fs))
        torch.randn(1 << 20, device="cuda").sum().item()      # the program's own work between


def test_two_graphs_replayed_in_turn():
    """Their workspaces are their own."""
    graphs, helds, wants = [], [], []
    sets = [calls(seed)[1] for seed in (5, 6)]      # hold the graphs' inputs
    for fs in sets:
        wants.append(eager(fs))
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            helds.append([f() for f in fs])
        graphs.append(g)
    for _ in range(3):
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        for held, want in zip(helds, wants):
            got = [x if isinstance(x, (tuple, list)) else [x] for x in held]
            assert same(got, want)


def test_other_streams():
    """On a stream given, while it is not the current one; results used on the
    current one after waiting."""
    s, _ = calls(7)
    want = eager([lambda: mfl.group_rows(s.ids, s.experts)])[0]
    rows, offsets, slots = want
    D = mfl.gemm_grouped(s.x, s.W1, offsets, rows=rows)
    n = int(offsets[-1])
    grads = mfl.gemm_grouped_backward(torch.ones_like(D), s.x, s.W1, offsets, rows=rows)
    side = torch.cuda.Stream()
    for _ in range(3):
        side.wait_stream(torch.cuda.current_stream())
        h = side.cuda_stream
        r2, o2, s2 = mfl.group_rows(s.ids, s.experts, stream=h)
        D2 = mfl.gemm_grouped(s.x, s.W1, o2, rows=r2, stream=h)
        # (an expanded gradient is copied on the stream that reads it)
        one = torch.ones(1, 1, dtype=torch.bfloat16, device="cuda").expand(D.shape)
        side.wait_stream(torch.cuda.current_stream())
        g2 = mfl.gemm_grouped_backward(one, s.x, s.W1, o2, rows=r2, stream=h)
        c2 = mfl.combine_rows(D2, s2, s.w, stream=h)
        torch.cuda.current_stream().wait_stream(side)
        assert torch.equal(r2, rows) and torch.equal(o2, offsets) and torch.equal(s2, slots)
        assert torch.equal(D2[:n], D[:n])
        assert torch.equal(g2[0], grads[0]) and torch.equal(g2[1], grads[1])
        assert torch.equal(c2, mfl.combine_rows(D, slots, s.w))


def test_two_streams_at_once():
    """Calls beside each other do not meet."""
    streams = [torch.cuda.Stream() for _ in range(2)]
    sets = [calls(seed)[1] for seed in (8, 9)]
    wants = [eager(fs) for fs in sets]
    for _ in range(3):
        got = []
        for st, fs in zip(streams, sets):
            st.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(st):
                got.append([f() for f in fs])
        torch.cuda.synchronize()
        for r, want in zip(got, wants):
            assert same([x if isinstance(x, (tuple, list)) else [x] for x in r], want)


def test_requests_with_adapters_step_by_step():
    """Decoding steps of a batch whose requests come and go: the assignment
    changes between steps, the weights stay."""
    gen = torch.Generator().manual_seed(4)
    E, R, N, K = 6, 16, 264, 520
    W, A = values(gen, (N, K), "bf16", K ** -0.5), values(gen, (E, R, K), "bf16", K ** -0.5)
    B, scale = values(gen, (E, N, R), "bf16", R ** -0.5), torch.rand(E, generator=gen)
    dev = [t.cuda() for t in (W, A, B)]
    for batch in (1, 7, 64, 65, 200, 331):
        x = values(gen, (batch, K), "bf16")
        ids = torch.randint(-1, E, (batch,), generator=gen)
        rows, offsets, _ = mfl.group_rows(ids.cuda(), E)
        D = mfl.gemm_adapters(x.cuda(), *dev, offsets, rows=rows, scale=scale.cuda())
        want, tol = G.adapters(f64(x), f64(W), f64(A), f64(B), offsets.cpu().numpy(),
                               rows.cpu().numpy(), f64(scale), "bf16")
        within(f"D of {batch}", D, want, tol)


def test_rows_past_4_gib():
    """A, D and dA of more than 4 GiB each, and the place numbers that go with
    them: the last rows against float64."""
    places, k, n = 300_000, 8192, 8
    gen = torch.Generator(device="cuda").manual_seed(0)
    A = torch.empty(places, k, dtype=torch.bfloat16, device="cuda").normal_(generator=gen)
    B = torch.randn(2, n, k, device="cuda", generator=gen).bfloat16()
    offsets = torch.tensor([0, 299_700, places], dtype=torch.int32, device="cuda")
    for algo in ("few", "tile128", "tile256"):
        say(f"[gpu] {places} rows of {k}, {algo}")
        D = mfl.gemm_grouped(A, B, offsets, algo=algo)
        tail = slice(places - 400, places)
        a = f64(A[tail])
        want, tol = G.product(a, f64(B), np.array([0, 100, 400]), None, "bf16")
        within("D", D[tail], want, tol)
    dD = torch.randn(places, n, device="cuda", generator=gen).bfloat16()
    dA, dB = mfl.gemm_grouped_backward(dD, A, B, offsets, dB_dtype=torch.float32)
    want, tol = G.gradients(f64(dD[tail]), a, f64(B), np.array([0, 100, 400]), None, "bf16", "f32")
    within("dA", dA[tail], want[0], tol[0])
    within("dB", dB[1], want[1][1], tol[1][1])
    slots = torch.arange(places - 8, places, dtype=torch.int32, device="cuda").view(4, 2)
    out = mfl.combine_rows(dA, slots)
    want, tol = G.combine(f64(dA[-8:]), np.arange(8).reshape(4, 2), np.ones((4, 2)), "bf16")
    within("combined", out, want, tol)


def test_matrices_past_4_gib():
    """B of 5 GiB: the last group's product and gradients."""
    E, n, k = 40, 8192, 8192
    B = torch.zeros(E, n, k, dtype=torch.float16, device="cuda")
    gen = torch.Generator(device="cuda").manual_seed(1)
    B[-1].normal_(generator=gen)
    A = torch.randn(E + 30, k, device="cuda", generator=gen).half()
    offsets = torch.cat([torch.arange(E), torch.tensor([E + 30])]).int().cuda()
    cols = slice(n - 64, n)
    for algo in ("few", "tile128", "tile256"):
        say(f"[gpu] {E} matrices of {n} x {k}, {algo}")
        D = mfl.gemm_grouped(A, B, offsets, algo=algo, out_dtype=torch.float32)
        want, tol = G.product(f64(A[E - 1:]), f64(B[-1:, cols]), np.array([0, 31]), None, "f32")
        within("D", D[E - 1:, cols], want, tol)
        assert bool((D[:E - 1] == 0).all())
    dD = torch.randn(E + 30, n, device="cuda", generator=gen).half()
    dA, dB = mfl.gemm_grouped_backward(dD, A, B, offsets)
    want, tol = G.gradients(f64(dD[E - 1:, cols]), f64(A[E - 1:]), f64(B[-1:, cols]),
                            np.array([0, 31]), None, "f16", "f16")
    within("dB", dB[-1, cols], want[1][0], tol[1][0])
    want = f64(dD[E - 1:]) @ f64(B[-1])
    mag = np.abs(f64(dD[E - 1:])) @ np.abs(f64(B[-1]))
    within("dA", dA[E - 1:], want, G._bound(mag, n, want, "f16"))
