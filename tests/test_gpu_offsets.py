"""Offsets whose differences 32 bits do not hold: 0, 2^31 - 1, -2^31, -1, 0 differ by
2^31 - 1 or by 1 if they are subtracted in 32 bits, and decrease all the same."""
import pytest
import torch

import expert_grouped_gemm_amd as moe

pytestmark = pytest.mark.gpu

FAR = [0, 2 ** 31 - 1, -2 ** 31, -1, 0]


def _problem(sched, T=96):
    p = moe.make_problem(T, 256, 128, 4, 2, sched=sched)
    g = torch.Generator().manual_seed(2)
    X, W1, W2 = (torch.randn(*s, generator=g).to(torch.bfloat16).cuda() for s in
                 ((2 * T, 256), (4, 256, 256), (4, 256, 128)))
    i = dict(dtype=torch.int32, device="cuda")
    return p, X, W1, W2, torch.randperm(2 * T, generator=g).to(torch.int32).cuda(), torch.tensor(FAR, **i), torch.tensor(
        [0, 40, 40, 150, 2 * T], **i)


def _rejected(p, ws):
    with pytest.raises(moe.MoEError) as ei:
        moe.check_workspace(p, ws)
    assert ei.value.status == 1


@pytest.mark.parametrize("sched", ["separate", "expert_wave", "interleaved"])
def test_expert_forward(sched):
    p, X, W1, W2, dst, far, good = _problem(sched)
    C, ws = torch.full((192, 256), 5.0, device="cuda"), moe.alloc_workspace(p)
    moe.expert_forward(p, X, None, far, dst, W1, None, W2, None, C, ws)
    _rejected(p, ws)
    assert torch.all(C == 5.0)
    moe.expert_forward(p, X, None, good, dst, W1, None, W2, None, C, ws)
    moe.check_workspace(p, ws)
    assert torch.isfinite(C).all() and not (C == 5.0).all(1).any()


def test_checkpoint_calls():
    p, X, W1, W2, dst, far, good = _problem("auto")
    C, ws = torch.full((192, 256), 5.0, device="cuda"), moe.alloc_checkpoint_workspace(p)
    gu = torch.full((192, 256), 7, dtype=torch.int8, device="cuda")
    gus = torch.full((192, 8), 9, dtype=torch.uint8, device="cuda")
    moe.expert_forward_checkpoint(p, X, None, far, dst, W1, W2, gu, gus, C, ws)
    _rejected(p, ws)
    assert torch.all(C == 5.0) and torch.all(gu == 7) and torch.all(gus == 9)
    moe.expert_forward_checkpoint(p, X, None, good, dst, W1, W2, gu, gus, C, ws)
    dO = C.to(torch.bfloat16)
    z = dict(dtype=torch.bfloat16, device="cuda")
    out = torch.full((192, 256), 3.0, **z), torch.full((4, 256, 256), 3.0, **z), torch.full((4, 256, 128), 3.0, **z)
    moe.expert_backward_checkpoint(p, X, None, None, far, dst, gu, gus, W1, W2, dO, *out, ws)
    _rejected(p, ws)
    for t in out:
        assert torch.all(t == 3.0)
    moe.expert_backward_checkpoint(p, X, None, None, good, dst, gu, gus, W1, W2, dO, *out, ws)
    moe.check_workspace(p, ws)
    for t in out:
        assert torch.isfinite(t.float()).all()
