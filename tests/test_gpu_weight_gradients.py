"""The two kernels of the experts' weight gradients: for few rows per expert and
for many (chosen by the router's mean, T k / E_global > 256), on row counts
around their stages and tiles, experts without rows among long ones, widths
that end inside a tile. The same rows give the same bits from either: every
element is summed over an expert's rows in one order."""
import numpy as np
import pytest
import torch

import expert_grouped_gemm_amd as moe
from oracle import backward

pytestmark = pytest.mark.gpu

U, B = 2.0 ** -24, 2.0 ** -8


def _i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


def _operands(counts, d, f, seed=3):
    A, E = sum(counts), len(counts)
    g = torch.Generator().manual_seed(seed + A)
    X, dO = (torch.randn(A, d, generator=g).to(torch.bfloat16) for _ in range(2))
    W1, W2 = (torch.randn(*s, generator=g).mul_(0.05).to(torch.bfloat16) for s in ((E, 2 * f, d), (E, d, f)))
    gu = torch.randint(-127, 128, (A, 2 * f), generator=g, dtype=torch.int8)
    gus = torch.randint(125, 129, (A, f // 16), generator=g, dtype=torch.uint8)
    off = np.concatenate([[0], np.cumsum(counts)])
    return off, np.random.default_rng(A).permutation(A), *(t.cuda() for t in (X, dO, W1, W2, gu, gus))


def _run(E_global, ops, checkpoint, grid=0):
    off, dst, X, dO, W1, W2, gu, gus = ops
    (A, d), E, f = X.shape, W1.shape[0], W2.shape[2]
    p = moe.make_problem(A, d, f, E_global, 1, 0, E, sched="auto", grid=grid)
    z = dict(dtype=torch.bfloat16, device="cuda")
    out = torch.full((A, d), 3.0, **z), torch.full((E, 2 * f, d), 3.0, **z), torch.full((E, d, f), 3.0, **z)
    if checkpoint:
        ws = moe.alloc_checkpoint_workspace(p).fill_(255)
        moe.expert_backward_checkpoint(p, X, None, None, _i32(off), _i32(dst), gu, gus, W1, W2, dO, *out, ws)
    else:
        ws = moe.alloc_backward_workspace(p).fill_(255)
        moe.expert_backward(p, X, None, _i32(off), _i32(dst), W1, W2, dO, *out, ws)
    moe.check_workspace(p, ws)
    return out


COUNTS = [[0, 0, 1100, 0], [1025, 1, 0, 31], [33, 700, 0, 500], [256, 257, 511, 640], [32, 64, 1500, 96], [2000, 0, 0, 0]]


@pytest.mark.parametrize("checkpoint", [False, True])
@pytest.mark.parametrize("d,f", [(128, 384), (384, 128), (640, 256)])
@pytest.mark.parametrize("counts", COUNTS)
def test_both_kernels_give_the_same_bits(counts, d, f, checkpoint):
    print(f"[weights] {counts} {d} {f} {checkpoint}", flush=True)
    ops = _operands(counts, d, f)
    many, few = _run(4, ops, checkpoint), _run(1024, ops, checkpoint)  # the mean above 256, and 2
    for a, b in zip(many, few):
        assert torch.equal(a, b)
    for grid in (1, 3, 200):
        for a, b in zip(many, _run(4, ops, checkpoint, grid)):
            assert torch.equal(a, b)
    for e in range(4):
        if counts[e] == 0:
            assert not many[1][e].any() and not many[2][e].any()


@pytest.mark.parametrize("counts", COUNTS[:4])
def test_many_rows_against_the_formulas(counts):
    """dW against fp64, the sums' and the roundings' errors as a bound on the norm: a and dh are rounded to bf16, half a
    step each, and so is the result; sums of fp32 are off by 2000 u at most, far below a tenth of that."""
    ops = _operands(counts, 384, 256)
    off, dst, X, dO, W1, W2, _, _ = ops
    _, dW1, dW2 = _run(4, ops, False)
    _, r1, r2 = backward.expert_backward(X.cpu().double().numpy(), dO.cpu().double().numpy()[dst], off,
                                         W1.cpu().double().numpy(), W2.cpu().double().numpy())
    for got, ref in ((dW1, r1), (dW2, r2)):
        err = np.linalg.norm(got.double().cpu().numpy() - ref)
        assert err <= 2.2 * B * np.linalg.norm(ref)


def test_infinities_stay_in_their_expert_and_row():
    """The rows behind an expert's last belong to the next one: theirs are not seen, infinite or not."""
    counts = [300, 301, 500, 600]
    off, dst, X, dO, W1, W2, gu, gus = _operands(counts, 128, 128)
    dO[dst[300], 7] = float("inf")           # the first row of expert 1, right behind expert 0's last
    X[600, 5] = float("nan")                 # its last row, right before expert 2's first
    out = _run(4, (off, dst, X, dO, W1, W2, gu, gus), True)
    for e in (0, 2, 3):
        assert torch.isfinite(out[1][e]).all() and torch.isfinite(out[2][e]).all()
    assert not torch.isfinite(out[2][1][7]).any() and torch.isnan(out[1][1][:, 5]).all()
