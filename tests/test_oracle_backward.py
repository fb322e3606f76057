"""The fp64 gradients of oracle.backward against central differences of the
forward formulas, and the MXFP4 quantiser against the input generator's codec.

Central differences with step h of a function with third derivative of order
one err by h^2 plus rounding eps / h; at h = 1e-5 both are below 1e-9 here.
"""
import numpy as np
import pytest
import torch

import moe_synth
import oracle
from oracle import backward


def _num_grad(fn, x, h=1e-5):
    g = np.zeros_like(x)
    it = np.nditer(x, flags=["multi_index"])
    for _ in it:
        i = it.multi_index
        old = x[i]
        x[i] = old + h
        up = fn()
        x[i] = old - h
        dn = fn()
        x[i] = old
        g[i] = (up - dn) / (2 * h)
    return g


@pytest.mark.parametrize("S", [1, 2])
def test_whole_chain_against_differences(S):
    """loss = <R, Y> of the share; the chain combine -> experts -> dispatch, and the router."""
    rng = np.random.default_rng(3 + S)
    T, d, f, E, k, eb, ee = 4, 3, 2, 5, 3, 1, 4
    X, logits = rng.normal(size=(T, d)), rng.normal(size=(T, E))
    W1, W2 = rng.normal(size=(ee - eb, 2 * f, d)), rng.normal(size=(ee - eb, d, f))
    R = rng.normal(size=(T, d))
    idx, _, _ = oracle.route_topk(logits, k)
    disp = oracle.dispatch(idx, np.ones((T, k)) / k, eb, ee, S)
    rs, rd, off = disp["row_src"], disp["row_dst"], disp["offsets"]

    def gates():
        sel = np.take_along_axis(logits, idx, 1)
        ex = np.exp(sel - sel.max(1, keepdims=True))
        return ex / ex.sum(1, keepdims=True)

    def slots():
        O = np.zeros((disp["A"], d))
        for e in range(ee - eb):
            r = slice(off[e], off[e + 1])
            g, u = np.split(X[rs[r] // k] @ W1[e].T, 2, axis=1)
            O[rd[r]] = (g / (1 + np.exp(-g)) * u) @ W2[e].T
        return O

    def loss():
        w, O = gates(), slots()
        Y = np.zeros((T, d))
        for r in range(disp["A"]):
            t, j = rs[r] // k, rs[r] % k
            Y[oracle.y_row_of_token(t, T, S)] += w[t, j] * O[rd[r]]
        return float((R * Y).sum())

    d_buf, d_w, d_logits = backward.combine_backward(R, slots(), disp["tok_off"], idx, gates(), eb, ee, E, S)
    dx, dW1, dW2 = backward.expert_backward(X[rs // k], d_buf[rd], off, W1, W2)
    d_slots = np.zeros_like(dx)
    d_slots[rd] = dx
    dX = backward.dispatch_backward(d_slots, disp["tok_off"], T, S)
    for got, x in ((d_logits, logits), (dX, X), (dW1, W1), (dW2, W2)):
        np.testing.assert_allclose(got, _num_grad(loss, x), rtol=1e-7, atol=1e-8)


def test_quantiser_matches_the_generators_codec():
    g = torch.Generator().manual_seed(5)
    x = torch.randn(64, 256, generator=g) * torch.exp2(torch.randint(-30, 30, (64, 1), generator=g).float())
    x[3, 32:64] = 0
    codes, scales = moe_synth._quant_mxfp4_rows(x)
    c, s = backward.quantize_mxfp4(x.numpy())
    np.testing.assert_array_equal(c, codes.numpy())
    np.testing.assert_array_equal(s, scales.numpy())


def test_quantiser_ties_borders_and_poison():
    x = np.zeros((1, 64))
    x[0, :16] = [4.0, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, -0.25, -5.0, 6.0, 7.99, -7.0, 0.2, -0.0, 1e-300]
    x[0, 40] = np.inf
    c, s = backward.quantize_mxfp4(x)
    nib = np.stack([c & 15, c >> 4], -1).reshape(-1)
    vals = oracle.e2m1_to_f64(nib[:16])
    np.testing.assert_array_equal(vals, [4, 0, 1, 1, 2, 2, 4, 4, 0, -4, 6, 6, -6, 0, 0, 0])
    assert s[0, 0] == 127 and s[0, 1] == 255 and not nib[32:].any()
    for amax, byte in ((1.0, 125), (np.nextafter(2.0, 0), 125), (2.0, 126), (2.0 ** -126, 0), (2.0 ** -140, 0)):
        row = np.zeros((1, 32))
        row[0, 7] = amax
        assert backward.quantize_mxfp4(row)[1][0, 0] == byte, amax
