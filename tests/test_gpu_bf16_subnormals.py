"""Values below bf16's smallest normal number (2^-126) pass the roundings to
bf16 whole: nothing is flushed to zero."""
import numpy as np
import pytest
import torch

import expert_grouped_gemm_amd as moe
import oracle

pytestmark = pytest.mark.gpu


def test_dequantize_to_bf16_subnormals():
    """Every code under the scale bytes 0 .. 8; the values (2^-128 and up) are all bf16 values."""
    codes = torch.tensor([[(2 * i) % 16 | ((2 * i + 1) % 16) << 4 for i in range(16)]] * 9, dtype=torch.uint8)
    scales = torch.arange(9, dtype=torch.uint8)[:, None]
    ref = oracle.decode_mxfp4(codes.numpy(), scales.numpy())
    for dt in (torch.bfloat16, torch.float32):
        out = torch.empty(9, 32, dtype=dt, device="cuda")
        moe.mxfp4_dequantize(codes.cuda(), scales.cuda(), out)
        np.testing.assert_array_equal(out.double().cpu().numpy(), ref)


@pytest.mark.parametrize("d", [128, 1152])
def test_permutations_of_subnormal_gradients(d):
    """Gate weight 1 and one slot per token: both gradients are copies, bit for bit (signed zeros too)."""
    T, E = 9, 4
    bits = torch.randint(0, 0x80, (T, d), generator=torch.Generator().manual_seed(d)).to(torch.int32)
    bits |= torch.randint(0, 2, (T, d), generator=torch.Generator().manual_seed(d + 1)).to(torch.int32) << 15
    dY = bits.to(torch.int16).view(torch.bfloat16).cuda()
    p = moe.make_problem(T, d, 128, E, 1)
    idx = torch.arange(T, dtype=torch.int32, device="cuda") % E
    off = torch.arange(T + 1, dtype=torch.int32, device="cuda")
    d_buf = torch.empty(T, d, dtype=torch.bfloat16, device="cuda")
    moe.combine_backward(p, dY, torch.ones(T, d, device="cuda"), off, idx, torch.ones(T, 1, device="cuda"), d_buf,
                         torch.empty(T, 1, device="cuda"))
    assert torch.equal(d_buf.view(torch.int16), dY.view(torch.int16))
    dX = torch.empty_like(dY)
    moe.dispatch_backward(p, dY, off, dX)
    # a sum that starts at +0 loses the sign of a zero, nothing else
    assert torch.equal(dX.float(), dY.float())
    assert torch.equal(dX.view(torch.int16)[dY != 0], dY.view(torch.int16)[dY != 0])
