"""Gradients whose key tiles are cut between workgroups: both numberings of the
places that the cut tiles' sums take in the workspace, in one sequence and in
many, with tiles cut once and several times."""
import pytest
import torch

import mma_fragment_layouts_tn_amd as mfl
from test_gpu_attention import Packed
from test_gpu_use_attention import same

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("heads,lens", [
    ((2, 1, 64), [1500]),                          # 256 shares of one sequence's 12 tiles
    ((6, 3, 128), [700, 0, 0, 300, 45]),           # as many shares as fill one round
    ((16, 8, 64), [(37 * i) % 200 for i in range(60)]),    # more tiles than shares
    ((8, 8, 128), [(53 * i) % 300 for i in range(40)]),
    ((3, 3, 256), [129, 1, 400]),
], ids=str)
def test_places(heads, lens, causal):
    p = Packed("bf16", lens, lens, *heads, causal)
    p.check_backward(*p.check_forward())


def test_offsets_out_of_order():
    """The numbers stay inside the workspace whatever the offsets are, and
    good offsets give the same bits afterwards."""
    p = Packed("bf16", [900, 300], [900, 300], 4, 1, 64, True)
    dev = [t.cuda() for t in (p.dout, p.q, p.k, p.v)]
    out, lse = p.forward()
    want = mfl.attention_backward(*dev, out, lse, **p.how())
    for seq in ([0, 1 << 30, 5, 1 << 30, 0, 1200], [1200, 0, 1200, 0], [700, 100, 1200, 1100]):
        s = torch.tensor(seq, dtype=torch.int32).cuda()
        mfl.attention_backward(*dev, out, lse, seq_q=s)
        torch.cuda.synchronize()
        for a, b in zip(mfl.attention_backward(*dev, out, lse, **p.how()), want):
            assert same(a, b)
