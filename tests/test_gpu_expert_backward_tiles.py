"""Every form of tile the experts' gradient picks by its rule, against the fp64
formulas: products of 256 and of 128 columns, each with 2, 4, 5, 6 and 8 row
blocks, of experts with one row band (weights read past the caches) and with
several. A small grid makes whole rounds of wide tiles out of few of them; the
grids here leave a last round with and without a cut along the rows. Bounds and
references are those of test_gpu_expert_backward.

And rows, tokens and slots whose byte offsets pass 2^31."""
import numpy as np
import pytest
import torch

import expert_grouped_gemm_amd as moe
from oracle import backward
from test_gpu_expert_backward import _bounds, _check, _i32, _rounded_reference

pytestmark = pytest.mark.gpu

SINGLE, SEVERAL = (40, 100, 150, 180, 250, 256), (296, 356, 406, 442, 600, 512)
BF = dict(dtype=torch.bfloat16, device="cuda")


def _weights(g, E, d, f):
    return (torch.randn(E, 2 * f, d, generator=g).mul_(0.05).to(torch.bfloat16),
            torch.randn(E, d, f, generator=g).mul_(0.05).to(torch.bfloat16))


@pytest.mark.parametrize("counts,d,f,grids", [
    (SINGLE, 384, 640, (2,)), (SEVERAL, 384, 640, (2,)), (SINGLE, 640, 384, (22,)), (SEVERAL, 640, 384, (22, 34)),
    (SEVERAL, 640, 640, (16, 28)),
    ((700, 513, 1100, 900), 640, 384, (2, 8)),     # weight gradients of long experts, several tiles a workgroup
    ((0, 1600, 1, 1200, 0), 384, 640, (2, 0)),     # ... and of none and one row among them
    ((1, 0, 2) * 341 + (130,), 128, 128, (0, 6)),  # as many experts as there may be
])
def test_every_tile_form(counts, d, f, grids):
    A, E = sum(counts), len(counts)
    off = np.concatenate([[0], np.cumsum(counts)])
    rng, g = np.random.default_rng(A + d), torch.Generator().manual_seed(A + d)
    X, dO = (torch.randn(A, d, generator=g).to(torch.bfloat16) for _ in range(2))
    W1, W2 = _weights(g, E, d, f)
    src, dst = rng.permutation(A), rng.permutation(A)
    ops = (X.double().numpy()[src], dO.double().numpy()[dst], off, W1.double().numpy(), W2.double().numpy())
    want, rounded, bounds = backward.expert_backward(*ops), _rounded_reference(*ops), _bounds(*ops)
    args = (X.cuda(), _i32(src), _i32(off), _i32(dst), W1.cuda(), W2.cuda(), dO.cuda())
    for grid in grids:
        print(f"[expert_backward tiles] {counts} d={d} f={f} grid={grid}", flush=True)
        p = moe.make_problem(A, d, f, E, 1, sched="auto", grid=grid)
        out = torch.empty(A, d, **BF), torch.empty(E, 2 * f, d, **BF), torch.empty(E, d, f, **BF)
        ws = moe.alloc_backward_workspace(p)
        moe.expert_backward(p, *args, *out, ws)
        torch.cuda.synchronize()
        moe.check_workspace(p, ws)
        dxs, dW1, dW2 = (t.double().cpu().numpy() for t in out)
        _check((dxs[dst], dW1, dW2), want, rounded, bounds, (counts, grid))


@pytest.mark.parametrize("gather", [True, False])
@pytest.mark.parametrize("E_global", [4, 512])    # long experts' and short experts' weight gradients
def test_byte_offsets_past_2_31(E_global, gather):
    """160000 rows of 8192 bf16 values, 2.6 GB: the rows in use stand at the far end of every array."""
    T, d, f, El, counts = 160000, 8192, 128, 4, (70, 300, 1, 213)
    n = sum(counts)
    first = T - n
    off = first + np.concatenate([[0], np.cumsum(counts)])
    rng, g = np.random.default_rng(E_global), torch.Generator().manual_seed(E_global)
    tok = np.concatenate([[T - 1, 0, 131071, 131072], first + rng.permutation(n - 4)])  # 2^31 bytes start at row 131072
    slot = np.concatenate([[T - 1, 131072, 0, 131071], first - 1 - rng.permutation(n - 4)])
    x, do = (torch.randn(n, d, generator=g).to(torch.bfloat16) for _ in range(2))
    W1, W2 = _weights(g, El, d, f)
    X, dO = torch.full((T, d), float("nan"), **BF), torch.full((T, d), float("nan"), **BF)
    src = np.zeros(T, np.int64)
    if gather:
        X[torch.tensor(tok, device="cuda")] = x.cuda()
        src[first:] = tok
    else:
        X[first:] = x.cuda()
    dO[torch.tensor(slot, device="cuda")] = do.cuda()
    dst = np.zeros(T, np.int64)
    dst[first:] = slot
    p = moe.make_problem(T, d, f, E_global, 1, 0, El, sched="auto")
    out = torch.full((T, d), 3.0, **BF), torch.empty(El, 2 * f, d, **BF), torch.empty(El, d, f, **BF)
    ws = moe.alloc_backward_workspace(p)
    print(f"[expert_backward 2^31] E_global={E_global} gather={gather} {ws.numel()} bytes", flush=True)
    moe.expert_backward(p, X, _i32(src) if gather else None, _i32(off), _i32(dst), W1.cuda(), W2.cuda(), dO, *out, ws)
    torch.cuda.synchronize()
    moe.check_workspace(p, ws)
    at = torch.tensor(slot, device="cuda")
    dx, dW1, dW2 = (t.double().cpu().numpy() for t in (out[0][at], out[1], out[2]))
    out[0][at] = 3.0
    assert torch.all(out[0] == 3.0)                # no other slot was written
    ops = x.double().numpy(), do.double().numpy(), off - first, W1.double().numpy(), W2.double().numpy()
    _check((dx, dW1, dW2), backward.expert_backward(*ops), _rounded_reference(*ops), _bounds(*ops), "far rows")
