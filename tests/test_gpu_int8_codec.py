"""The 8-bit integer codecs: bit-exact against the fp64 codecs, at ties,
borders, subnormals, non-finite elements, one row and many."""
import numpy as np
import pytest
import torch

import expert_grouped_gemm_amd as moe
from oracle import int8

pytestmark = pytest.mark.gpu

SHAPES = [(1, 32), (1, 7168), (3, 96), (257, 384), (4099, 160), (2, 16384), (3, 20000), (5, 40992)]


def _rows(x):
    codes = torch.full(x.shape, 0x55, dtype=torch.int8, device="cuda")
    scales = torch.full(x.shape[:-1], 7.0, device="cuda")
    moe.int8_quantize(x.cuda(), codes, scales)
    return codes, scales


def _blocks(x):
    codes = torch.full(x.shape, 0x55, dtype=torch.int8, device="cuda")
    scales = torch.full((*x.shape[:-1], x.shape[-1] // 32), 0x55, dtype=torch.uint8, device="cuda")
    moe.mxint8_quantize(x.cuda(), codes, scales)
    return codes, scales


def _check_rows(x):
    codes, scales = _rows(x)
    c, s = int8.quantize_int8(x.double().numpy())
    np.testing.assert_array_equal(scales.cpu().numpy(), s)
    np.testing.assert_array_equal(codes.cpu().numpy(), c)
    out = torch.empty(x.shape, device="cuda")
    moe.int8_dequantize(codes, scales, out)
    v = c.astype(np.float32) * s[:, None]              # one fp32 product
    np.testing.assert_array_equal(out.cpu().numpy(), v)
    out = torch.empty(x.shape, dtype=torch.bfloat16, device="cuda")
    moe.int8_dequantize(codes, scales, out)
    want = torch.tensor(v).to(torch.bfloat16)
    assert torch.equal(torch.isnan(out.cpu()), torch.isnan(want))
    assert torch.equal(out.cpu().nan_to_num(), want.nan_to_num())


def _check_blocks(x):
    codes, scales = _blocks(x)
    c, s = int8.quantize_mxint8(x.double().numpy())
    np.testing.assert_array_equal(scales.cpu().numpy(), s)
    np.testing.assert_array_equal(codes.cpu().numpy(), c)
    for dt in (torch.float32, torch.bfloat16):
        out = torch.empty(x.shape, dtype=dt, device="cuda")
        moe.mxint8_dequantize(codes, scales, out)
        np.testing.assert_array_equal(out.double().cpu().numpy(), int8.decode_mxint8(c, s))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,cols", SHAPES + [(1, 16), (7, 48)])
def test_rows(rows, cols, dtype):
    print(f"[int8] {rows}x{cols} {dtype}", flush=True)
    g = torch.Generator().manual_seed(rows + cols)
    x = torch.randn(rows, cols, generator=g) * torch.exp2(torch.randint(-60, 60, (rows, 1), generator=g).float())
    _check_rows(x.to(dtype))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_rows_of_ties(dtype):
    """Ratios of small whole numbers: many quotients lie halfway between two codes, and next to it in fp32."""
    g = torch.Generator().manual_seed(4)
    x = torch.randint(-255, 256, (4096, 64), generator=g).float()
    x[:, 0] = torch.randint(1, 256, (4096,), generator=g).float()
    x[2048:] *= torch.exp2(torch.randint(-9, 1, (2048, 64), generator=g).float())
    _check_rows(x.to(dtype))
    if dtype is torch.float32:
        _check_rows(torch.nextafter(x, torch.tensor(0.0)))
        _check_rows(torch.nextafter(x, torch.tensor(1e30)))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_rows_of_every_exponent(dtype):
    g = torch.Generator().manual_seed(5)
    e = torch.arange(-149, 128)
    x = torch.ldexp(torch.rand(e.numel(), 32, generator=g, dtype=torch.float64) * 1.9 - 0.95, e[:, None]).clamp(
        -3.38e38, 3.38e38)
    x[:, 0] = torch.ldexp(torch.tensor(1.0, dtype=torch.float64), e)
    _check_rows(x.float().to(dtype))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("cols", [96, 7168, 20000])
def test_poisoned_and_zero_rows(dtype, cols):
    x = torch.ones(6, cols)
    x[0, cols - 1] = float("nan")
    x[1, 0] = float("-inf")
    x[2] = 0.0
    x[3] = -0.0
    x[4, 5] = torch.finfo(dtype).min
    x[5] = torch.finfo(dtype).max
    _check_rows(x.to(dtype))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,cols", [s for s in SHAPES if s[1] % 32 == 0])
def test_blocks(rows, cols, dtype):
    print(f"[mxint8] {rows}x{cols} {dtype}", flush=True)
    g = torch.Generator().manual_seed(rows + cols)
    x = torch.randn(rows, cols, generator=g) * torch.exp2(torch.randint(-60, 60, (rows, cols // 32), generator=g)
                                                          .float()).repeat_interleave(32, 1)
    _check_blocks(x.to(dtype))


def test_blocks_of_ties_borders_and_every_exponent():
    rows = []
    for e in range(-149, 128):                         # every fp32 binade, subnormals included
        base = 2.0 ** e
        row = [base * 1.5, -base] + [s * (n + 0.5) * base / 64 for n in (0, 1, 2, 62, 63, 126, 127) for s in (1, -1)]
        rows.append(row + [0.0] * (32 - len(row)))
    _check_blocks(torch.tensor(np.clip(np.array(rows), -3.3e38, 3.3e38).astype(np.float32)))
    _check_blocks(torch.tensor([[float(v)] + [0.0] * 31 for e in (-126, -121, -120, -20, 0, 19, 127)
                                for v in (np.nextafter(np.float32(2.0 ** e), np.float32(0)), np.float32(2.0 ** e),
                                          np.nextafter(np.float32(2.0 ** e), np.float32(3e38)))]))


def test_poisoned_and_zero_blocks():
    x = torch.ones(4, 96)
    x[0, 40] = float("nan")
    x[1, 95] = float("-inf")
    x[2, 32:64] = 0.0
    x[3, 0:32] = -0.0
    for dt in (torch.float32, torch.bfloat16):
        _check_blocks(x.to(dt))


def test_every_code_and_scale_byte_read_back():
    codes = torch.arange(-128, 128, dtype=torch.int8).repeat(256, 1)
    scales = torch.arange(256, dtype=torch.uint8)[:, None].repeat(1, 8)
    want = int8.decode_mxint8(codes.numpy(), scales.numpy())
    want[254, codes[254].numpy() == -128] = -np.inf    # -2^128
    for dt in (torch.float32, torch.bfloat16):
        out = torch.empty(256, 256, dtype=dt, device="cuda")
        moe.mxint8_dequantize(codes.cuda(), scales.cuda(), out)
        np.testing.assert_array_equal(out.double().cpu().numpy(), want)


def test_past_2_31_elements():
    """Offsets past 32 bits, checked in the first and last rows."""
    n = (1 << 31) + 4096
    x = torch.ones(n // 4096, 4096, dtype=torch.bfloat16, device="cuda")
    x[-1, 1:] = 0.5
    codes = torch.empty(x.shape, dtype=torch.int8, device="cuda")
    scales = torch.empty(n // 4096, device="cuda")
    moe.int8_quantize(x, codes, scales)
    assert (codes[:-1] == 127).all() and int(codes[-1, 0]) == 127 and (codes[-1, 1:] == 64).all()
    out = torch.empty_like(x)
    moe.int8_dequantize(codes, scales, out)
    assert (out[:-1] == 1).all() and (out[-1, 1:] == float(torch.tensor(64 / 127).to(torch.bfloat16))).all()
    bytes_ = torch.empty(n // 4096, 128, dtype=torch.uint8, device="cuda")
    moe.mxint8_quantize(x, codes, bytes_)
    assert (codes[-1, 32:] == 64).all() and (bytes_[-1, 1:] == 126).all() and (bytes_[:-1] == 127).all()
    out.zero_()
    moe.mxint8_dequantize(codes, bytes_, out)
    assert torch.equal(out, x)


def test_empty_and_refused():
    z = dict(device="cuda")
    i8, u8 = torch.int8, torch.uint8
    moe.int8_quantize(torch.empty(0, 64, **z), torch.empty(0, 64, dtype=i8, **z), torch.empty(0, **z))
    moe.mxint8_quantize(torch.empty(0, 64, **z), torch.empty(0, 64, dtype=i8, **z), torch.empty(0, 2, dtype=u8, **z))
    x, c = torch.ones(2, 64, **z), torch.empty(2, 64, dtype=i8, **z)
    s, b = torch.empty(2, **z), torch.empty(2, 2, dtype=u8, **z)
    for quantize, dequantize, sc, cut in ((moe.int8_quantize, moe.int8_dequantize, s, 40),
                                          (moe.mxint8_quantize, moe.mxint8_dequantize, b, 48)):
        for bad in ((x[:, :cut].contiguous(), c, sc), (x.half(), c, sc), (x, c[:1], sc), (x, c, sc[:1]),
                    (x, c.view(u8), sc), (x, c, sc.double()), (x.cpu(), c, sc), (x.t(), c, sc)):
            with pytest.raises(ValueError):
                quantize(*bad)
            with pytest.raises(ValueError):
                dequantize(bad[1], bad[2], bad[0])


def test_replayed_graph_and_another_stream():
    x = torch.randn(37, 4096, device="cuda").to(torch.bfloat16)
    c, s, o = torch.empty_like(x, dtype=torch.int8), torch.empty(37, device="cuda"), torch.empty_like(x)
    c2, b2, o2 = torch.empty_like(c), torch.empty(37, 128, dtype=torch.uint8, device="cuda"), torch.empty_like(x)

    def run(stream=None):
        moe.int8_quantize(x, c, s, stream=stream)
        moe.int8_dequantize(c, s, o, stream=stream)
        moe.mxint8_quantize(x, c2, b2, stream=stream)
        moe.mxint8_dequantize(c2, b2, o2, stream=stream)

    run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run()
    side = torch.cuda.Stream()
    for i in range(3):
        x.normal_()
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in (c, s, o, c2, b2, o2)]
        for t in (c, s, o, c2, b2, o2):
            t.zero_()
        torch.cuda.synchronize()
        run(side if i == 1 else None)
        torch.cuda.synchronize()
        for a, b in zip(got, (c, s, o, c2, b2, o2)):
            assert torch.equal(a, b)
