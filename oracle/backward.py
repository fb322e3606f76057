"""fp64 gradients of the layer's steps, written from their formulas (one token,
one expert at a time), and the MXFP4 quantiser of whole rows.

With O[p] the expert outputs in token-order slots, q(t) the output row of
token t and s = sigmoid(g):
  combine   dO[p] = w[t,j] dY[q(t)],  dw[t,j] = <dY[q(t)], O[p]>
  router    dl[t,e] = sum_{j: idx[t,j] = e} w_j (dw_j - sum_i w_i dw_i)
  experts   [g u] = W1 x, a = g s u, o = W2 a; da = W2^T do,
            dg = da u (s + g s (1 - s)), du = da g s,
            dx = W1^T [dg du], dW1 = sum_r [dg du] x^T, dW2 = sum_r do a^T
  dispatch  dX[t] = sum of the slots of t
"""
from __future__ import annotations

import numpy as np

from .moe_oracle import f64_to_bf16_bits, y_row_of_token  # noqa: F401

__all__ = ["combine_backward", "dispatch_backward", "expert_backward", "quantize_mxfp4"]


def _slots_of(t, tok_off, local_t, T, S):
    q = int(y_row_of_token(t, T, S))
    return q, int(tok_off[q]) + np.arange(int(local_t.sum()))


def combine_backward(dY, buf, tok_off, idx, w, e_begin, e_end, E_global, num_segments=1):
    """(d_buf [A, d], d_w [T, k], d_logits [T, E])"""
    dY, buf, w = (np.asarray(x, dtype=np.float64) for x in (dY, buf, w))
    idx = np.asarray(idx)
    T, k = idx.shape
    A = int(tok_off[-1])
    d_buf = np.zeros((A, dY.shape[1]))
    d_w = np.zeros((T, k))
    d_logits = np.zeros((T, E_global))
    for t in range(T):
        local = (idx[t] >= e_begin) & (idx[t] < e_end)
        q, slots = _slots_of(t, tok_off, local, T, num_segments)
        for j, p in zip(np.flatnonzero(local), slots):
            d_buf[p] = w[t, j] * dY[q]
            d_w[t, j] = float(dY[q] @ buf[p])
        mean = float(w[t] @ d_w[t])
        for j in range(k):
            if 0 <= idx[t, j] < E_global:
                d_logits[t, idx[t, j]] += w[t, j] * (d_w[t, j] - mean)
    return d_buf, d_w, d_logits


def dispatch_backward(d_slots, tok_off, T, num_segments=1):
    d_slots = np.asarray(d_slots, dtype=np.float64)
    dX = np.zeros((T, d_slots.shape[1]))
    for t in range(T):
        q = int(y_row_of_token(t, T, num_segments))
        dX[t] = d_slots[int(tok_off[q]):int(tok_off[q + 1])].sum(axis=0)
    return dX


def expert_backward(X_rows, dO_rows, offsets, W1, W2):
    """X_rows, dO_rows [A, d] in expert order, W1 [E_l, 2f, d], W2 [E_l, d, f]:
    (dx_rows [A, d], dW1, dW2)."""
    X_rows, dO_rows = np.asarray(X_rows, dtype=np.float64), np.asarray(dO_rows, dtype=np.float64)
    El, f2, d = W1.shape
    f = f2 // 2
    dx = np.zeros_like(X_rows)
    dW1, dW2 = np.zeros((El, f2, d)), np.zeros((El, d, f))
    for e in range(El):
        r = slice(int(offsets[e]), int(offsets[e + 1]))
        w1, w2 = np.asarray(W1[e], dtype=np.float64), np.asarray(W2[e], dtype=np.float64)
        g, u = np.split(X_rows[r] @ w1.T, 2, axis=1)
        s = 1.0 / (1.0 + np.exp(-g))
        da = dO_rows[r] @ w2
        dh = np.concatenate([da * u * (s + g * s * (1.0 - s)), da * g * s], axis=1)
        dx[r] = dh @ w1
        dW1[e] = dh.T @ X_rows[r]
        dW2[e] = dO_rows[r].T @ (g * s * u)
    return dx, dW1, dW2


_E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def quantize_mxfp4(x):
    """x [rows, K] -> (packed codes uint8 [rows, K/2], E8M0 bytes [rows, K/32]):
    the nearest E2M1 value of x / 2^e, ties to the even code, e = floor(log2
    amax) - 2 >= -127; a block with an infinite or NaN element is byte 255 and
    codes 0."""
    x = np.asarray(x, dtype=np.float64)
    R, K = x.shape
    b = x.reshape(R, K // 32, 32)
    finite = np.isfinite(b).all(axis=2)
    v = np.where(finite[..., None], b, 0.0)
    amax = np.abs(v).max(axis=2)
    e = np.where(amax > 0, np.maximum(np.frexp(amax)[1] - 3, -127), 0)
    y = np.abs(v) / np.exp2(e.astype(np.float64))[..., None]
    dist = np.abs(y[..., None] - _E2M1)
    best = dist.min(axis=-1, keepdims=True)
    near = dist == best                              # one code, or two at a tie
    code = np.where((near & (np.arange(8) % 2 == 0)).any(axis=-1),
                    np.argmax(near & (np.arange(8) % 2 == 0), axis=-1), np.argmax(near, axis=-1))
    code = np.where(y > 6.0, 7, code)
    code = (code | (np.signbit(v).astype(np.int64) << 3)).astype(np.uint8)
    code = np.where(finite[..., None], code, 0).reshape(R, K).astype(np.uint8)
    byte = np.where(finite, e + 127, 255).astype(np.uint8)
    return code[:, 0::2] | (code[:, 1::2] << 4), byte
