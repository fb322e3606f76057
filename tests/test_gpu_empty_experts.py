"""Weight gradients of a share on which few experts have rows. An expert without
rows costs its zeros and no more: the kernel for many rows looks ahead for the
next tile that has any, and would spend a time that grows with the square of the
tiles if it looked again from every one of them."""
import numpy as np
import pytest
import torch

import expert_grouped_gemm_amd as moe

pytestmark = pytest.mark.gpu

El, D, F, K, T = 64, 512, 512, 1, 64 * 600


def _call(E_global, rows, at, o, grid):
    """A call of expert_backward, with every row on expert `at`: for many rows where the router's mean is 600 (E_global
    64), for few where it is 37 (1024)."""
    p = moe.make_problem(T, D, F, E_global, K, 0, El, sched="auto", grid=grid)
    off = torch.tensor([0] * (at + 1) + [rows] * (El - at), dtype=torch.int32, device="cuda")
    ws = moe.alloc_backward_workspace(p)
    return lambda: moe.expert_backward(p, o["X"], None, off, o["dst"], o["W1"], o["W2"], o["dO"], o["dx"], o["dW1"],
                                       o["dW2"], ws)


@pytest.fixture(scope="module")
def operands():
    g = torch.Generator(device="cuda").manual_seed(2)

    def rand(*s, std=1.0):
        return torch.randn(s, generator=g, device="cuda").mul_(std).to(torch.bfloat16)

    z = dict(dtype=torch.bfloat16, device="cuda")
    return dict(X=rand(T, D), dO=rand(T, D), W1=rand(El, 2 * F, D, std=0.05), W2=rand(El, D, F, std=0.05),
                dst=torch.arange(T, dtype=torch.int32, device="cuda"), dx=torch.empty(T, D, **z),
                dW1=torch.empty(El, 2 * F, D, **z), dW2=torch.empty(El, D, F, **z))


@pytest.mark.parametrize("at", [0, 1, 40, El - 1])
@pytest.mark.parametrize("rows", [0, 1, 33, 700])
def test_rows_on_one_expert(rows, at, operands):
    """Both kernels, the same bits, and zeros for every other expert."""
    o, outs = operands, []
    for E_global, grid in ((El, 0), (El, 2), (El, 6), (1024, 0)):
        o["dW1"].fill_(3.0)
        o["dW2"].fill_(3.0)
        _call(E_global, rows, at, o, grid)()
        outs.append((o["dW1"].clone(), o["dW2"].clone()))
    for a, b in outs[1:]:
        assert torch.equal(a, outs[0][0]) and torch.equal(b, outs[0][1])
    for w in outs[0]:
        others = [e for e in range(El) if e != at or rows == 0]
        assert not w[others].any() and (rows == 0 or bool(w[at].any()))


def test_experts_without_rows_are_walked_once(operands):
    """On a grid of two workgroups each has 128 and 256 tiles, all but a few without rows. The kernel for few rows, which
    looks for nothing, is the measure: it has twice the workgroups, which store the zeros in half the time (0.75 ms; the
other 1.5, and 6.0 when it looked from every tile)."""
    times = {}
    for E_global in (El, 1024):
        call = _call(E_global, 64, 0, operands, 2)
        call()
        torch.cuda.synchronize()
        best = []
        for _ in range(5):
            e = [torch.cuda.Event(enable_timing=True) for _ in range(2)]
            e[0].record()
            call()
            e[1].record()
            torch.cuda.synchronize()
            best.append(e[0].elapsed_time(e[1]))
        times[E_global] = min(best)
    print(f"[empty experts] many rows {times[El]:.3f} ms, few rows {times[1024]:.3f} ms", flush=True)
    assert times[El] <= 4 * times[1024], times
