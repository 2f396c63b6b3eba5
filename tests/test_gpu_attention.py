"""Attention on the GPU against its float64 definition (oracle/attention.py):
packed sequences, gradients, and decoding behind a shared prefix, every
element within the bound that fp32 sums and one rounding of weights, score
gradients and results give.

Sizes sit where the kernels change: one row, the 32 rows of a wave, the 32
and 64 keys of a chunk, tiles of 128 and 256 rows, empty sequences, rows
without keys, head dimensions between the accumulators' classes, strided and
shared operands, values behind the sequences that must not be read.
"""
import numpy as np
import pytest
import torch

import mma_fragment_layouts_tn_amd as mfl
from gpu_helpers import say
from oracle import attention as A

pytestmark = pytest.mark.gpu

DT = {"f16": torch.float16, "bf16": torch.bfloat16}


def values(gen, shape, kind, gain=1.0):
    return (torch.randn(*shape, generator=gen) * gain).to(DT[kind])


def f64(t):
    return t.detach().cpu().double().numpy()


def offsets(lens):
    return torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32)


def within(name, got, want, tol):
    got = f64(got)
    bad = ~(np.abs(got - want) <= tol) & ~((got == want) | (np.isnan(want)))
    if bad.any():
        i = np.unravel_index(np.argmax(np.where(bad, np.abs(got - want), 0)), got.shape)
        raise AssertionError(f"{name}: {bad.sum()} of {bad.size} outside, worst at {i}: "
                             f"{got[i]} for {want[i]} +- {tol[i]}")
    fin = np.isfinite(want) & (tol > 0)
    say(f"[gpu]   {name}: worst {np.max(np.abs(got - want)[fin] / tol[fin], initial=0):.3f} of the bound")


class Packed:
    def __init__(self, kind, ql, kl, heads, kv, dim, causal, seed=0, scale=None, tail=0, gain=1.5):
        gen = torch.Generator().manual_seed(seed + 1000 * dim + heads)
        self.kind, self.causal = kind, causal
        self.scale = dim ** -0.5 if scale is None else scale
        self.ql, self.kl = ql, kl
        self.q = values(gen, (sum(ql) + tail, heads, dim), kind, gain)
        self.k = values(gen, (sum(kl) + tail, kv, dim), kind)
        self.v = values(gen, (sum(kl) + tail, kv, dim), kind)
        self.dout = values(gen, (sum(ql) + tail, heads, dim), kind)
        if tail:    # rows of no sequence hold what must not be read
            for x in (self.q, self.dout):
                x[sum(ql):] = float("nan")
            self.k[sum(kl):] = float("inf")
            self.v[sum(kl):] = float("nan")
        self.sq, self.sk = offsets(ql), offsets(kl)
        say(f"[gpu] attention {kind} q={ql} k={kl} heads={heads}/{kv} dim={dim} causal={causal}")

    def how(self):
        return dict(seq_q=self.sq.cuda(), seq_k=self.sk.cuda(), causal=self.causal,
                    scale=self.scale)

    def forward(self, **kw):
        out, lse = mfl.attention(self.q.cuda(), self.k.cuda(), self.v.cuda(), return_lse=True,
                                 **self.how(), **kw)
        torch.cuda.synchronize()
        return out, lse

    def check_forward(self, **kw):
        out, lse = self.forward(**kw)
        want, wl, tol, tl = A.attention(f64(self.q), f64(self.k), f64(self.v), self.sq.tolist(),
                                        self.sk.tolist(), self.causal, self.scale, self.kind)
        n = sum(self.ql)
        within("out", out[:n], want[:n], tol[:n])
        within("lse", lse[:n], wl[:n], tl[:n])
        return out, lse

    def check_backward(self, out, lse):
        dq, dk, dv = mfl.attention_backward(self.dout.cuda(), self.q.cuda(), self.k.cuda(),
                                            self.v.cuda(), out, lse, **self.how())
        torch.cuda.synchronize()
        want, tol = A.gradients(f64(self.dout), f64(self.q), f64(self.k), f64(self.v), f64(out),
                                f64(lse), self.sq.tolist(), self.sk.tolist(), self.causal,
                                self.scale, self.kind)
        for name, x, w, t in zip(("dq", "dk", "dv"), (dq, dk, dv), want, tol):
            within(name, x, w, t)
        return dq, dk, dv


LENGTHS = [
    ([1], [1]),
    ([33], [33]),
    ([64, 1, 65], [64, 1, 65]),
    ([5, 0, 31, 32], [70, 3, 0, 33]),
    ([130, 257], [130, 257]),
    ([40, 10], [17, 10]),              # causal: the first 23 rows see nothing
    ([300], [411]),
]
HEADS = [(1, 1, 64), (4, 1, 128), (6, 2, 64), (3, 3, 128), (2, 1, 256), (5, 5, 32), (8, 2, 80),
         (2, 2, 200)]


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("lens", LENGTHS, ids=str)
@pytest.mark.parametrize("algo", ["tall", "flat", "auto"])
def test_forward_lengths(algo, lens, causal):
    p = Packed("bf16", *lens, 4, 2, 128, causal)
    p.check_forward(algo=algo)


@pytest.mark.parametrize("kind", ["f16", "bf16"])
@pytest.mark.parametrize("heads", HEADS, ids=str)
@pytest.mark.parametrize("algo", ["tall", "flat"])
def test_forward_heads(algo, heads, kind):
    p = Packed(kind, [70, 1, 130], [95, 1, 130], *heads, True)
    p.check_forward(algo=algo)


@pytest.mark.parametrize("algo", ["tall", "flat"])
@pytest.mark.parametrize("splits", [2, 3, 7])
def test_forward_splits(algo, splits):
    """Key ranges computed apart and joined; some have no visible key."""
    p = Packed("f16", [33, 1, 100], [500, 700, 90], 4, 1, 64, True)
    p.check_forward(algo=algo, splits=splits)


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("lens", LENGTHS, ids=str)
def test_backward_lengths(lens, causal):
    p = Packed("bf16", *lens, 4, 2, 128, causal)
    p.check_backward(*p.check_forward())


@pytest.mark.parametrize("kind", ["f16", "bf16"])
@pytest.mark.parametrize("heads", HEADS, ids=str)
def test_backward_heads(heads, kind):
    p = Packed(kind, [70, 1, 140], [95, 1, 140], *heads, True)
    p.check_backward(*p.check_forward())


# ------------------------------------------------------------ shared prefix
class Prefix:
    def __init__(self, kind, batch, tokens, prefix, capacity, lengths, heads, kv, dim, seed=0):
        gen = torch.Generator().manual_seed(seed + 77 * dim + batch)
        self.kind, self.scale = kind, dim ** -0.5
        self.q = values(gen, (batch, tokens, heads, dim), kind, 1.5)
        self.pk, self.pv = (values(gen, (prefix, kv, dim), kind) for _ in range(2))
        self.k, self.v = (values(gen, (batch, capacity, kv, dim), kind) for _ in range(2))
        self.lengths = torch.tensor(lengths, dtype=torch.int32)
        for b, n in enumerate(lengths):      # places of the cache that hold no key
            self.k[b, max(n, 0):] = float("nan")
            self.v[b, max(n, 0):] = float("inf")
        say(f"[gpu] prefix {kind} batch={batch} tokens={tokens} prefix={prefix} own={lengths} "
            f"of {capacity} heads={heads}/{kv} dim={dim}")

    def check(self, **kw):
        out, lse = mfl.attention_prefix(self.q.cuda(), self.pk.cuda(), self.pv.cuda(),
                                        self.k.cuda(), self.v.cuda(), self.lengths.cuda(),
                                        return_lse=True, **kw)
        torch.cuda.synchronize()
        want, wl, tol, tl = A.prefix_attention(
            f64(self.q), f64(self.pk), f64(self.pv), f64(self.k), f64(self.v),
            self.lengths.tolist(), self.scale, self.kind)
        within("out", out, want, tol)
        within("lse", lse, wl, tl)
        return out, lse


@pytest.mark.parametrize("kind", ["f16", "bf16"])
@pytest.mark.parametrize("heads", [(8, 2, 128), (4, 4, 64), (3, 1, 256), (16, 1, 80)], ids=str)
@pytest.mark.parametrize("shape", [
    (1, 1, 1, 1, [1]),
    (3, 1, 100, 40, [0, 1, 40]),
    (5, 3, 65, 70, [3, 70, 2, 0, 33]),       # fewer keys than new tokens: only the prefix
    (2, 1, 0, 300, [300, 0]),                # no prefix; a sequence without any key
    (2, 2, 700, 0, [0, 0]),                  # no cache
], ids=str)
def test_prefix(shape, heads, kind):
    b, t, p, cap, lengths = shape
    Prefix(kind, b, t, p, cap, lengths, *heads).check()


@pytest.mark.parametrize("algo", ["tall", "flat"])
@pytest.mark.parametrize("splits", [(1, 1), (4, 1), (3, 5), (70, 2)])
def test_prefix_kernels(algo, splits):
    Prefix("bf16", 40, 2, 333, 200, [(7 * i) % 201 for i in range(40)], 8, 2, 64).check(
        algo=algo, splits=splits)
