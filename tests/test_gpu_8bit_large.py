"""The 8-bit Linears and the checkpoint calls at the largest row counts that a
problem may have (row capacity x width just below 2^31 elements, byte offsets up
to 2^32), and on a padded layout with a row capacity of its own. Rows picked
from all over have the bits that a small problem of those rows alone gives."""
import numpy as np
import pytest
import torch

import expert_grouped_gemm_amd as moe
from oracle import int8
from test_gpu_checkpoint import _check, _reference

pytestmark = pytest.mark.gpu


def _picked(A, width, seed=1):
    """Rows at the ends, around a band's border and around 2^30, 2^31 and 2^32 bytes of rows of 2 x width bytes."""
    rows = {0, 1, 255, 256, A - 257, A - 2, A - 1}
    for b in (30, 31, 32):
        r = (1 << b) // (2 * width)
        rows |= {r - 1, r, r + 1}
    rows |= set(np.random.default_rng(seed).integers(0, A, 20).tolist())
    return sorted(r for r in rows if 0 <= r < A)


def _normal(g, *shape, std=1.0):
    return torch.empty(shape, dtype=torch.bfloat16, device="cuda").normal_(std=std, generator=g)


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _perm(g, n):
    return torch.randperm(n, generator=g, device="cuda").to(torch.int32)


def _checkpoint(p, X, Xs, src, off, dst, W1, W2, dO):
    cap, d, f = moe.row_capacity(p), p.d, p.f
    z = dict(device="cuda")
    gu, gus = torch.zeros(cap, 2 * f, dtype=torch.int8, **z), torch.zeros(cap, f // 16, dtype=torch.uint8, **z)
    C, ws = torch.zeros(cap, d, **z), moe.alloc_checkpoint_workspace(p)
    moe.expert_forward_checkpoint(p, X, src, off, dst, W1, W2, gu, gus, C, ws)
    z["dtype"] = torch.bfloat16
    out = torch.zeros(cap, d, **z), torch.zeros(W1.shape, **z), torch.zeros(W2.shape, **z)
    if Xs is not None:
        X, Xs = Xs
    moe.expert_backward_checkpoint(p, X, Xs, src, off, dst, gu, gus, W1, W2, dO, *out, ws)
    moe.check_workspace(p, ws)
    return C, gu, gus, *out


@pytest.mark.parametrize("x8", [False, True])
@pytest.mark.parametrize("E_global", [1, 1024])  # the weight gradients of many and of few rows
@pytest.mark.parametrize("T,d,f", [(262016, 128, 8064), (131968, 16256, 128)])
def test_checkpoint_of_the_most_rows(T, d, f, E_global, x8):
    print(f"[large] {T} {d} {f} {E_global} x8={x8}", flush=True)
    g = torch.Generator(device="cuda").manual_seed(d)
    p = moe.make_problem(T, d, f, E_global, 1, 0, 1, sched="auto")
    X, W1, W2 = _normal(g, T, d), _normal(g, 1, 2 * f, d, std=d ** -0.5), _normal(g, 1, d, f, std=f ** -0.5)
    Xs = None
    if x8:
        Xs = torch.empty(T, d, dtype=torch.int8, device="cuda"), torch.empty(T, d // 32, dtype=torch.uint8, device="cuda")
        moe.mxint8_quantize(X, *Xs)
    src, dst = _perm(g, T), _perm(g, T)
    rows = _picked(T, max(d, f))
    n, at = len(rows), torch.tensor(rows, device="cuda")
    tok, slot = src[at].long(), dst[at].long()
    dO = torch.zeros(T, d, dtype=torch.bfloat16, device="cuda")  # every other row's gradient is zero
    dO[slot] = _normal(g, n, d)
    big = _checkpoint(p, X, Xs, src, _i32([0, T]), dst, W1, W2, dO)
    few = moe.make_problem(n, d, f, 1, 1, sched="auto")
    some = _checkpoint(few, X[tok], None if Xs is None else (Xs[0][tok], Xs[1][tok]), None, _i32([0, n]),
                       _i32(list(range(n))), W1, W2, dO[slot])
    for i, where in ((0, slot), (1, at), (2, at), (3, slot)):
        assert torch.equal(big[i][where], some[i]), i
    others = torch.ones(T, dtype=torch.bool, device="cuda")
    others[slot] = False
    assert not big[3][others].any() and bool(big[0][others].any(1).all())
    x = int8.decode_mxint8(*(t[tok].cpu().numpy() for t in Xs)) if x8 else X[tok].double().cpu().numpy()
    gu = int8.decode_mxint8(some[1].cpu().numpy(), some[2].cpu().numpy())
    ref = _reference(x, dO[slot].double().cpu().numpy(), [0, n], gu, W1.double().cpu().numpy(), W2.double().cpu().numpy())
    _check((big[3][slot].double().cpu().numpy(), big[4].double().cpu().numpy(), big[5].double().cpu().numpy()), ref, d)


def _codes(g, *shape):
    return (torch.empty(shape, dtype=torch.int8, device="cuda").random_(-128, 128, generator=g),
            torch.rand(shape[:-1], generator=g, device="cuda") * 2e-3 + 1e-4)


def test_int8_linears_of_the_most_rows():
    g = torch.Generator(device="cuda").manual_seed(6)
    T, d, f = 131968, 16256, 128
    (x, xs), (w, ws_) = _codes(g, T, d), _codes(g, 1, 2 * f, d)
    src, rows = _perm(g, T), torch.tensor(_picked(T, d // 2), device="cuda")
    tok, n = src[rows].long(), rows.numel()
    outs = []
    for p, a, b, s in ((moe.make_problem(T, d, f, 1, 1), x, xs, src), (moe.make_problem(n, d, f, 1, 1), x[tok], xs[tok], None)):
        H, ws = torch.zeros(p.T, f, dtype=torch.bfloat16, device="cuda"), moe.alloc_workspace(p)
        moe.int8_linear1(p, a, b, s, _i32([0, p.T]), w, ws_, H, ws)
        moe.check_workspace(p, ws)
        outs.append(H)
    assert torch.equal(outs[0][rows], outs[1]) and bool(outs[0].any(1).all())
    del x, xs, w, outs
    T, d, f = 262016, 128, 8064
    (h, hs), (w, ws_) = _codes(g, T, f), _codes(g, 1, d, f)
    dst, rows = _perm(g, T), torch.tensor(_picked(T, f // 2), device="cuda")
    n = rows.numel()
    outs = []
    for p, a, b, s in ((moe.make_problem(T, d, f, 1, 1), h, hs, dst),
                       (moe.make_problem(n, d, f, 1, 1), h[rows], hs[rows], _i32(list(range(n))))):
        C, ws = torch.zeros(p.T, d, device="cuda"), moe.alloc_workspace(p)
        moe.int8_linear2(p, a, b, _i32([0, p.T]), s, w, ws_, C, ws)
        moe.check_workspace(p, ws)
        outs.append(C)
    assert torch.equal(outs[0][dst[rows].long()], outs[1]) and bool(outs[0].any(1).all())


@pytest.mark.parametrize("x8", [False, True])
@pytest.mark.parametrize("counts", [[0, 300, 0, 400], [1, 0, 699, 0], [128, 129, 256, 1]])
def test_checkpoint_on_a_padded_layout(counts, x8):
    """Four tokens, whose problem has room for 700 rows: the bits that a problem of 700 tokens gives for them."""
    cap, E, d, f = 700, 4, 384, 256
    g = torch.Generator(device="cuda").manual_seed(counts[0])
    X, dO = _normal(g, cap, d), _normal(g, cap, d)
    W1, W2, dst = _normal(g, E, 2 * f, d, std=0.05), _normal(g, E, d, f, std=0.05), _perm(g, cap)
    off = _i32(np.concatenate([[0], np.cumsum(counts)]).tolist())
    Xs = None
    if x8:
        Xs = torch.empty(cap, d, dtype=torch.int8, device="cuda"), torch.empty(cap, d // 32, dtype=torch.uint8, device="cuda")
        moe.mxint8_quantize(X, *Xs)
    padded = moe.make_problem(4, d, f, E, 2, sched="auto", row_capacity=cap)
    plain = moe.make_problem(cap, d, f, E, 1, sched="auto")
    assert moe.row_capacity(padded) == moe.row_capacity(plain) == cap
    for a, b in zip(*(_checkpoint(p, X, Xs, None, off, dst, W1, W2, dO) for p in (padded, plain))):
        assert torch.equal(a, b)
