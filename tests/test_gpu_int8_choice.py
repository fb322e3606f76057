"""Which kernel the Linears on 8-bit integers take. The kernel for few rows walks
an expert's rows in passes of 32 and reads the weights again for each, so it is
for calls in which no expert can have many: the router's mean says nothing about
the rows of one expert on a share that holds the favoured ones. The persistent
GEMM plans its row bands in the workspace, the other kernel does not: a workspace
that held something else before tells them apart."""
import numpy as np
import pytest
import torch

import expert_grouped_gemm_amd as moe

pytestmark = pytest.mark.gpu


def _i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


def _operands(T, k, El, d, f, counts, seed=5):
    cap, A = T * min(k, El), sum(counts)
    g = torch.Generator(device="cuda").manual_seed(seed)

    def codes(*s):
        return torch.randint(-128, 128, s, generator=g, dtype=torch.int8, device="cuda")

    def scales(*s):
        return torch.rand(s, generator=g, device="cuda") * 2e-3 + 1e-4

    src = torch.zeros(cap, dtype=torch.int32, device="cuda")
    src[:A] = torch.randint(0, T * k, (A,), generator=g, device="cuda").to(torch.int32)
    dst = torch.randperm(cap, generator=g, device="cuda").to(torch.int32)
    return dict(X=codes(T, d), Xs=scales(T), src=src, off=_i32(np.concatenate([[0], np.cumsum(counts)])), dst=dst,
                W1=codes(El, 2 * f, d), W1s=scales(El, 2 * f), H=codes(cap, f), Hs=scales(cap),
                W2=codes(El, d, f), W2s=scales(El, d))


def _run(first, o, T, k, E, El, d, f, row_capacity=0):
    """The output, and whether the call left row bands in its workspace."""
    p = moe.make_problem(T, d, f, E, k, 0, El, sched="auto", row_capacity=row_capacity)
    cap = moe.row_capacity(p)
    ws = moe.alloc_workspace(p).fill_(0xA5)
    ops = {n: t for n, t in o.items()}
    if cap > o["H"].shape[0]:
        for n in ("src", "dst", "H", "Hs"):
            ops[n] = torch.cat([o[n], o[n].new_zeros((cap - o[n].shape[0],) + o[n].shape[1:])])
    if first:
        out = torch.zeros(cap, f, dtype=torch.bfloat16, device="cuda")
        moe.int8_linear1(p, ops["X"], ops["Xs"], ops["src"], ops["off"], ops["W1"], ops["W1s"], out, ws)
    else:
        out = torch.zeros(cap, d, device="cuda")
        moe.int8_linear2(p, ops["H"], ops["Hs"], ops["off"], ops["dst"], ops["W2"], ops["W2s"], out, ws)
    moe.check_workspace(p, ws)
    L = moe.workspace_layout(p)
    return out[:T * min(k, El)], bool((ws[L.meta + 256:L.topk_idx] != 0xA5).any())


# T, k, experts, local experts, d, f
HOT = [(2048, 8, 256, 1, 1024, 256), (1395, 6, 160, 20, 1024, 256), (1542, 2, 64, 8, 384, 256), (256, 8, 256, 32, 512, 384),
       (320, 1, 64, 8, 2304, 1408)]


@pytest.mark.parametrize("first", [True, False])
@pytest.mark.parametrize("shape", HOT)
def test_an_expert_that_every_token_reaches_goes_to_the_persistent_kernel(shape, first):
    print(f"[int8 choice] {shape} first={first}", flush=True)
    T, k, E, El, d, f = shape
    counts = [T] + [3] * (El - 1) if k > 1 else [T] + [0] * (El - 1)
    o = _operands(T, k, El, d, f, counts)
    out, bands = _run(first, o, *shape)
    assert bands
    padded, _ = _run(first, o, *shape, row_capacity=T * min(k, El) + 1)
    assert torch.equal(out, padded)


# ... and the two sides of the bounds, Linear-1 and Linear-2 (None: either): few tokens, and tiles that leave most of 256
# CUs idle or not
BOUNDS = [((1, 2, 8, 8, 512, 1408), False, False), ((64, 8, 256, 32, 1152, 2048), False, False),
          ((65, 8, 256, 32, 2176, 2048), True, True), ((128, 8, 256, 1, 2304, 1408), False, False),
          ((129, 8, 256, 1, 2304, 1408), True, True), ((128, 1, 1, 1, 640, 512), True, True),
          ((64, 1, 1, 1, 640, 512), False, False), ((64, 2, 8, 8, 2304, 2176), False, False),  # 16 rows in the mean
          ((64, 2, 4, 4, 4224, 2176), True, True)]  # 32


@pytest.mark.parametrize("shape,one,two", BOUNDS)
def test_both_sides_of_the_bounds(shape, one, two):
    """Every token's first choice is one expert: as many rows as it can have. Either kernel gives the same bits."""
    T, k, E, El, d, f = shape
    counts = [0] * El
    counts[El // 2] = T
    o = _operands(T, k, El, d, f, counts)
    for first, want in ((True, one), (False, two)):
        out, bands = _run(first, o, *shape)
        assert bands == want, first
        padded, there = _run(first, o, *shape, row_capacity=T * min(k, El) + 1)
        assert there and torch.equal(out, padded)
        if first:
            x, w, s = o["X"][o["src"][:T].long() // k].double(), o["W1"][El // 2].double(), o["W1s"][El // 2].double()
            g, u = ((x @ w.t()) * o["Xs"][o["src"][:T].long() // k].double()[:, None] * s).chunk(2, 1)
            ref, got = g / (1 + torch.exp(-g)) * u, out[:T].double()
            u24 = 2.0 ** -24  # the bound of tests/test_gpu_int8_linear.py
            tol = 4 * u24 * (1.1 * (u * g).abs() + ref.abs()) + 16 * u24 * (1 + g.abs()) * ref.abs()
            tol = tol + 2.0 ** -8 * (ref.abs() + tol) + 1e-30
        else:
            ref = (o["H"][:T].double() @ o["W2"][El // 2].double().t()) * o["Hs"][:T].double()[:, None]
            ref = ref * o["W2s"][El // 2].double()
            got, tol = out[o["dst"][:T].long()].double(), 4 * 2.0 ** -24 * ref.abs() + 1e-30
        assert ((got - ref).abs() <= tol).all(), first
