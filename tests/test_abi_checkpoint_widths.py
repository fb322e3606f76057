"""The widest rows that the checkpoint calls address: a pass forward whose
gradient would be refused, or whose weight rows lie further apart than its 32-bit
offsets reach, is refused itself."""
import pytest

import expert_grouped_gemm_amd as moe
from test_abi_int8 import L, UNSUPPORTED, WS_BYTES, _at, _call  # noqa: F401  (the fixture)


@pytest.mark.parametrize("fn", ["moe_expert_forward_checkpoint", "moe_expert_backward_checkpoint"])
@pytest.mark.parametrize("d,f", [((1 << 24) + 128, 128), ((1 << 20) + 128, 128), (128, (1 << 20) + 128)])
def test_wider_rows_are_refused(L, fn, d, f):  # noqa: F811
    assert _call(L, fn, _at(fn), p=moe.make_problem(2, d, f, 1, 1)) == UNSUPPORTED


@pytest.mark.parametrize("fn", ["moe_expert_forward_checkpoint", "moe_expert_backward_checkpoint"])
@pytest.mark.parametrize("d,f", [(1 << 20, 128), (128, 1 << 20)])
def test_the_widest(L, fn, d, f):  # noqa: F811
    """Only the workspace is too small for these."""
    assert _call(L, fn, _at(fn), p=moe.make_problem(64, d, f, 1, 1), ws_bytes=256) == 3
