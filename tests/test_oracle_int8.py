"""Pins of the oracle's 8-bit integer codecs: against exact rational
arithmetic, hand-worked rows, and the OCP definition of MXINT8."""
from fractions import Fraction

import numpy as np
import pytest
import torch

from oracle import backward, int8


def _exact_row(row):
    """Codes of a row by rational arithmetic."""
    v = [Fraction(float(t)) for t in row]
    amax = max(abs(t) for t in v)
    least = Fraction(127) / 2 ** 126
    return [round(127 * t / max(amax, least)) for t in v] if amax else [0] * len(v)  # Python rounds half to even


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("scale", [1.0, 1e-38, 3e-36, 1e30])
def test_rows_against_rational_arithmetic(dtype, scale):
    g = torch.Generator().manual_seed(3)
    x = (torch.randn(40, 48, generator=g) * scale).to(dtype)
    x[::3] = torch.randint(-40, 41, x[::3].shape, generator=g).to(dtype) * scale  # ratios of small numbers: ties
    codes, scales = int8.quantize_int8(x.double().numpy())
    for r in range(x.shape[0]):
        assert codes[r].tolist() == _exact_row(x[r].double().numpy())
        amax = float(x[r].double().abs().max())
        want = np.float32(max(np.float32(amax / 127), np.float32(2.0 ** -126))) if amax else np.float32(1)
        assert scales[r] == want


def test_worked_row():
    # amax 254: codes are x / 2; 3, 5 and 7 are ties, which go to the even code
    codes, scales = int8.quantize_int8([[254.0, -254.0, 3.0, 5.0, 7.0, -3.0, 1.0, 0.0]])
    assert codes.tolist() == [[127, -127, 2, 2, 4, -2, 0, 0]] and scales.tolist() == [2.0]


def test_largest_row_reads_back_finite():
    top = float(np.finfo(np.float32).max)
    codes, scales = int8.quantize_int8([[top, -top / 2]])
    assert codes.tolist() == [[127, -64]] and np.isfinite(np.float32(127) * scales[0])
    assert abs(127 * float(scales[0]) - top) < 2e-7 * top


def test_bad_and_zero_rows():
    codes, scales = int8.quantize_int8([[0.0, -0.0], [1.0, np.inf], [np.nan, 5.0], [2.0, -1.0]])
    assert codes.tolist() == [[0, 0], [0, 0], [0, 0], [127, -64]]      # 63.5 is a tie
    assert scales[0] == 1 and np.isnan(scales[1:3]).all() and scales[3] == np.float32(2 / 127)


def test_mxint8_from_the_format_definition():
    # elements are code / 64 times the scale: the largest is 1 + 63/64 of it
    codes = np.zeros((1, 64), np.int8)
    codes[0, :4], codes[0, 32] = [1, 64, 127, -127], -64
    got = int8.decode_mxint8(codes, np.array([[127, 130]], np.uint8))
    np.testing.assert_array_equal(got[0, :4], [1 / 64, 1.0, 1 + 63 / 64, -(1 + 63 / 64)])
    assert got[0, 32] == -8.0 and np.count_nonzero(got) == 5
    assert np.isnan(int8.decode_mxint8(codes, np.array([[255, 127]], np.uint8))[0, :32]).all()


def test_mxint8_worked_block():
    x = np.zeros((1, 32))
    x[0, :6] = [1.5, -1.0, 1.999, 1 / 128, 3 / 128, -5 / 128]          # scale 1, step 1/64
    codes, scales = int8.quantize_mxint8(x)
    assert scales.tolist() == [[127]] and codes[0, :6].tolist() == [96, -64, 127, 0, 2, -2]


def test_mxint8_values_are_exact_in_bf16_and_near():
    rng = np.random.default_rng(1)
    x = rng.normal(size=(64, 256)) * np.exp2(rng.integers(-100, 100, size=(64, 8))).repeat(32, 1)
    codes, scales = int8.quantize_mxint8(x)
    v = int8.decode_mxint8(codes, scales)
    np.testing.assert_array_equal(torch.tensor(v).to(torch.bfloat16).double().numpy(), v)
    step = np.exp2(scales.astype(np.float64) - 133).repeat(32, 1)
    big = np.abs(x) > 127.5 * step                                      # saturated
    assert np.all(np.abs(v - x)[~big] <= step[~big] / 2) and np.all(np.abs(v - x)[big] < step[big])
    # coding values that lie on a block's grid gives them back
    again = int8.quantize_mxint8(v)
    np.testing.assert_array_equal(int8.decode_mxint8(*again), v)


def test_backward_formulas_against_differences():
    """dg, du and with them dx, dW1, dW2 of the formulas that the gradient from a checkpoint uses, against central
    differences of <do, W2 (silu(g) u)> in g, u and W2."""
    rng = np.random.default_rng(2)
    d, f, A = 3, 4, 5
    x, do = rng.normal(size=(A, d)), rng.normal(size=(A, d))
    w1, w2 = rng.normal(size=(2 * f, d)), rng.normal(size=(d, f))
    gu = x @ w1.T

    def loss(gu, w2):
        g, u = np.split(gu, 2, axis=1)
        return float(np.sum(do * ((g / (1 + np.exp(-g)) * u) @ w2.T)))

    def numeric(fn, at, h=1e-5):
        out = np.zeros_like(at)
        for i in np.ndindex(at.shape):
            up, lo = at.copy(), at.copy()
            up[i] += h
            lo[i] -= h
            out[i] = (fn(up) - fn(lo)) / (2 * h)
        return out

    dh = numeric(lambda v: loss(v, w2), gu)
    dx, dW1, dW2 = backward.expert_backward(x, do, [0, A], w1[None], w2[None])
    np.testing.assert_allclose(dx, dh @ w1, atol=1e-8)
    np.testing.assert_allclose(dW1[0], dh.T @ x, atol=1e-8)
    np.testing.assert_allclose(dW2[0], numeric(lambda v: loss(gu, v), w2), atol=1e-8)
