"""The build's check of kernels that tie other matrix instructions by hand
than the 16x16x32 one (`prefix`): every access to an accumulator between them
is rejected, wherever it stands, until the drain."""
import pytest

from test_build_check import B, DRAIN, T32, _kernel

TIED = dict(tied=True, prefix="v_mfma_")
BF16 = "v_mfma_f32_32x32x16_bf16 a[0:15], v[0:3], v[4:7], a[0:15]"


def test_accepts_after_the_drain():
    for t in (T32, BF16):
        k = _kernel("v_accvgpr_write_b32 a0, 0", "s_nop 4", t, t, *DRAIN,
                    "v_accvgpr_read_b32 v2, a0")
        assert B.check_mfma_fences(k, "good", **TIED) == 1


@pytest.mark.parametrize("body", [
    ("s_nop 4", BF16, "v_accvgpr_read_b32 v2, a0", *DRAIN),
    ("s_nop 4", T32, "v_accvgpr_mov_b32 a16, a0", T32, *DRAIN),
    ("s_nop 4", ".LBB0_1:", BF16, "s_cbranch_scc1 .LBB0_1", "v_accvgpr_read_b32 v2, a0", *DRAIN),
])
def test_rejects_before_it(body):
    with pytest.raises(RuntimeError, match="in flight"):
        B.check_mfma_fences(_kernel(*body), "bad", **TIED)


def test_the_sources_meant_are_checked_so():
    assert B.TIED_SOURCES == {"attention_dkv.hip"} and B.TIED_SOURCES <= set(B.SOURCES)
