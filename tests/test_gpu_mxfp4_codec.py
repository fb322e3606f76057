"""MXFP4 quantiser and its inverse: bit-exact against the fp64 codec (the
nearest code is found by comparing distances), at ties, block maxima next to
powers of two, subnormals, non-finite elements, one row and many."""
import numpy as np
import pytest
import torch

import expert_grouped_gemm_amd as moe
import moe_synth
import oracle
from oracle import backward

pytestmark = pytest.mark.gpu


def _quantize(x):
    codes = torch.full((*x.shape[:-1], x.shape[-1] // 2), 0xAB, dtype=torch.uint8, device="cuda")
    scales = torch.full((*x.shape[:-1], x.shape[-1] // 32), 0xAB, dtype=torch.uint8, device="cuda")
    moe.mxfp4_quantize(x.cuda(), codes, scales)
    return codes, scales


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,cols", [(1, 32), (1, 7168), (3, 96), (257, 384), (4099, 160)])
def test_codes_and_scales(rows, cols, dtype):
    print(f"[mxfp4] {rows}x{cols} {dtype}", flush=True)
    g = torch.Generator().manual_seed(rows + cols)
    x = torch.randn(rows, cols, generator=g) * torch.exp2(torch.randint(-60, 60, (rows, cols // 32), generator=g)
                                                          .float()).repeat_interleave(32, 1)
    x = x.to(dtype)
    codes, scales = _quantize(x)
    c, s = backward.quantize_mxfp4(x.double().numpy())
    np.testing.assert_array_equal(scales.cpu().numpy(), s)
    np.testing.assert_array_equal(codes.cpu().numpy(), c)
    for out_dtype in (torch.bfloat16, torch.float32):
        out = torch.empty(rows, cols, dtype=out_dtype, device="cuda")
        moe.mxfp4_dequantize(codes, scales, out)
        np.testing.assert_array_equal(out.double().cpu().numpy(), oracle.decode_mxfp4(c, s))


def test_every_tie_border_and_exponent():
    rows = []
    ties = [0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0, 7.0, 7.96875]
    for e in range(-149, 128):                       # every fp32 binade, subnormals included
        base = 2.0 ** e
        row = [base, -base] + [s * v * base / 4 for v in ties for s in (1, -1)]
        rows.append(row + [0.0] * (32 - len(row)))
    x64 = np.clip(np.array(rows), -3.3e38, 3.3e38)
    x = torch.tensor(x64.astype(np.float32))
    codes, scales = _quantize(x)
    c, s = backward.quantize_mxfp4(x.double().numpy())
    np.testing.assert_array_equal(scales.cpu().numpy(), s)
    np.testing.assert_array_equal(codes.cpu().numpy(), c)
    out = torch.empty(x.shape, dtype=torch.float32, device="cuda")
    moe.mxfp4_dequantize(codes, scales, out)
    np.testing.assert_array_equal(out.double().cpu().numpy(), oracle.decode_mxfp4(c, s))
    border = torch.tensor([[float(np.float32(v))] + [0.0] * 31 for e in (-20, 0, 19)
                           for v in (np.nextafter(np.float32(2.0 ** e), np.float32(0)), 2.0 ** e,
                                     np.nextafter(np.float32(2.0 ** e), np.float32(9e9)))])
    codes, scales = _quantize(border)
    c, s = backward.quantize_mxfp4(border.double().numpy())
    np.testing.assert_array_equal(scales.cpu().numpy(), s)
    np.testing.assert_array_equal(codes.cpu().numpy(), c)


def test_poisoned_and_zero_blocks():
    x = torch.ones(4, 96)
    x[0, 40] = float("nan")
    x[1, 95] = float("-inf")
    x[2, 32:64] = 0.0
    x[3, 0:32] = -0.0
    for dt in (torch.float32, torch.bfloat16):
        codes, scales = _quantize(x.to(dt))
        c, s = backward.quantize_mxfp4(x.numpy())
        np.testing.assert_array_equal(scales.cpu().numpy(), s)
        np.testing.assert_array_equal(codes.cpu().numpy(), c)
        out = torch.empty(4, 96, dtype=dt, device="cuda")
        moe.mxfp4_dequantize(codes, scales, out)
        nan = torch.isnan(out).cpu()
        assert nan[0, 32:64].all() and nan[1, 64:].all() and int(nan.sum()) == 64


def test_weights_as_the_generator_draws_them():
    cfg = moe_synth.make_config("tiny", T=128, dtype="w4a8_mxfp4")
    inp = moe_synth.generate(cfg)
    g = torch.Generator().manual_seed(cfg.seed)
    torch.randn(cfg.T, cfg.d, generator=g), torch.randn(cfg.T, cfg.E_global, generator=g)
    w1 = torch.stack([torch.randn(2 * cfg.f, cfg.d, generator=g).mul_(0.02) for _ in range(cfg.E_local)])
    codes, scales = _quantize(w1)
    assert torch.equal(codes.cpu(), inp["W1"]) and torch.equal(scales.cpu(), inp["W1_scale"])


def test_past_2_31_elements():
    """2^31 + 64 elements: offsets past 32 bits, checked in the first and last blocks."""
    n = (1 << 31) + 64
    x = torch.ones(n // 32, 32, dtype=torch.bfloat16, device="cuda")
    x[-1] = 3.0
    codes = torch.empty(n // 32, 16, dtype=torch.uint8, device="cuda")
    scales = torch.empty(n // 32, 1, dtype=torch.uint8, device="cuda")
    moe.mxfp4_quantize(x, codes, scales)
    assert (codes[:-1] == 0x66).all() and (scales[:-1] == 125).all()     # 1 = 4 * 2^-2
    assert (codes[-1] == 0x77).all() and int(scales[-1]) == 126          # 3 = 6 * 2^-1
    out = torch.empty_like(x)
    moe.mxfp4_dequantize(codes, scales, out)
    assert torch.equal(out, x)


def test_empty_and_refused():
    e = torch.empty(0, 64, device="cuda")
    moe.mxfp4_quantize(e, torch.empty(0, 32, dtype=torch.uint8, device="cuda"),
                       torch.empty(0, 2, dtype=torch.uint8, device="cuda"))
    x = torch.ones(2, 64, device="cuda")
    c, s = torch.empty(2, 32, dtype=torch.uint8, device="cuda"), torch.empty(2, 2, dtype=torch.uint8, device="cuda")
    for bad in ((x[:, :48].contiguous(), c, s), (x.half(), c, s), (x, c[:1], s), (x, c, s[:1]), (x, c.char(), s),
                (x.cpu(), c, s), (x.t(), c, s)):
        with pytest.raises(ValueError):
            moe.mxfp4_quantize(*bad)
        with pytest.raises(ValueError):
            moe.mxfp4_dequantize(bad[1], bad[2], bad[0])
