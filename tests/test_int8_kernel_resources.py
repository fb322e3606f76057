"""The kernels of the 8-bit integer products and checkpoints keep their
accumulators and fragments in registers: none spills."""
import pytest

from test_kernel_resources import _one, kernels  # noqa: F401  (the fixture)


@pytest.mark.parametrize("kernel", [r"15moe_gemm_kernelILi4E", r"15moe_gemm_kernelILi5E", r"16int8_rows_kernelILb0E",
                                    r"16int8_rows_kernelILb1E", r"22expert_backward_kernelILi3E",
                                    r"22expert_backward_kernelILi4E", r"22expert_backward_kernelILi5E"])
def test_products_spill_nothing(kernels, kernel):  # noqa: F811
    assert _one(kernels, kernel) == dict(vgpr_spill_count=0, private_segment_fixed_size=0)


def test_codecs_spill_nothing(kernels):  # noqa: F811
    names = [n for n in kernels if "int8_quantize_kernel" in n or "int8_dequantize_kernel" in n]
    assert len(names) == 8 + 2 + 2 + 2
    for n in names:
        assert kernels[n] == dict(vgpr_spill_count=0, private_segment_fixed_size=0), n
