"""Runs of rows of one adapter, as the kernels that multiply them together find
them among a wave's 64 rows: every run begins once, at its first row, whatever
the numbers are."""
import pytest
import torch

import mma_fragment_layouts_tn_amd as mfl
from gpu_helpers import say

pytestmark = pytest.mark.gpu


def cases():
    gen = torch.Generator().manual_seed(1)
    yield "one", torch.full((64,), 3)
    yield "zeros", torch.zeros(64)
    yield "none", torch.full((64,), -1)
    yield "second row", torch.cat([torch.tensor([5]), torch.zeros(63)])
    yield "falling", torch.arange(64, 0, -1)
    yield "two", torch.arange(64) // 32 + 1
    for n in (2, 3, 9):
        yield f"any of {n}", torch.randint(-1, n, (64,), generator=gen)
        yield f"sorted of {n}", torch.randint(-1, n, (64,), generator=gen).sort().values


@pytest.mark.parametrize("name,own", list(cases()), ids=[n for n, _ in cases()])
def test_every_run_begins_once(name, own):
    say(f"[gpu] run starts, {name}")
    own = own.int()
    want = sum(1 << i for i in range(64) if i == 0 or own[i] != own[i - 1])
    assert mfl.probe_run_starts(own.cuda()) == want
