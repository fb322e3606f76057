"""The two kernels of the experts' weight gradients on both sides of the row
counts between which the library chooses: the same bits from either."""
import pytest
import torch

import expert_grouped_gemm_amd as moe
from test_gpu_weight_gradients import _i32, _operands, _run

pytestmark = pytest.mark.gpu

# little weights: the mean above 512 of 4 experts, and 2 to 3 of 1024
COUNTS = [[0, 0, 2100, 0], [2049, 1, 0, 31], [33, 1400, 0, 900], [513, 1000, 511, 640], [64, 32, 3000, 96], [4100, 0, 0, 0],
          [1, 2, 3, 2100]]


@pytest.mark.parametrize("checkpoint", [False, True])
@pytest.mark.parametrize("d,f", [(128, 384), (384, 128), (640, 256)])
@pytest.mark.parametrize("counts", COUNTS)
def test_little_weights(counts, d, f, checkpoint):
    print(f"[weight kernels] {counts} {d} {f} {checkpoint}", flush=True)
    ops = _operands(counts, d, f)
    size = moe.checkpoint_workspace_size if checkpoint else moe.backward_workspace_size
    A = sum(counts)
    assert size(moe.make_problem(A, d, f, 4, 1)) > size(moe.make_problem(A, d, f, 1024, 1, 0, 4))  # copies, and none
    many, few = _run(4, ops, checkpoint), _run(1024, ops, checkpoint)
    for grid in (0, 1, 3, 200):
        for a, b in zip(few, many if grid == 0 else _run(4, ops, checkpoint, grid)):
            assert torch.equal(a, b)


@pytest.mark.parametrize("mxint8", [False, True])
def test_more_weights_from_257_rows(mxint8):
    """48 experts of 1024 x 1024, 257 rows in the mean, most of them of 0 to 540: the kernel for many rows. A router over
    1024 experts gives the other one."""
    E, d, f = 48, 1024, 1024
    counts = [(7 * e * e + 13 * e) % 540 for e in range(E)]
    counts[5] = 0
    counts[-1] += 257 * E - sum(counts)
    assert counts[-1] > 0 and sum(counts) == 257 * E
    A = sum(counts)
    g = torch.Generator(device="cuda").manual_seed(4)

    def rand(*s, std=1.0):
        return torch.randn(*s, generator=g, device="cuda").mul_(std).to(torch.bfloat16)

    X, dO, W1, W2 = rand(A, d), rand(A, d), rand(E, 2 * f, d, std=0.03), rand(E, d, f, std=0.03)
    gu = torch.randint(-127, 128, (A, 2 * f), generator=g, device="cuda", dtype=torch.int8)
    gus = torch.randint(125, 129, (A, f // 16), generator=g, device="cuda", dtype=torch.uint8)
    off = _i32([0] + torch.tensor(counts).cumsum(0).tolist())
    dst = torch.randperm(A, generator=g, device="cuda").to(torch.int32)
    Xs = None
    if mxint8:
        Xs = torch.empty(A, d // 32, dtype=torch.uint8, device="cuda")
        codes = torch.empty(A, d, dtype=torch.int8, device="cuda")
        moe.mxint8_quantize(X, codes, Xs)
        X = codes
    outs = []
    for E_global in (E, 1024):
        p = moe.make_problem(A, d, f, E_global, 1, 0, E, sched="auto")
        ws = moe.alloc_checkpoint_workspace(p).fill_(255)
        out = [torch.full(s, 3.0, dtype=torch.bfloat16, device="cuda") for s in ((A, d), (E, 2 * f, d), (E, d, f))]
        moe.expert_backward_checkpoint(p, X, Xs, None, off, dst, gu, gus, W1, W2, dO, *out, ws)
        moe.check_workspace(p, ws)
        outs.append(out)
    for a, b in zip(*outs):
        assert torch.equal(a, b)
    assert not outs[0][1][5].any() and not outs[0][2][5].any()
