"""The device-side error report of a workspace across a run of calls: a
rejection, or a wait that timed out, is still there after a later call of the
same layer that went well, until moe_check_workspace reads it; and what a
workspace's memory held before its first call is no report."""
import numpy as np
import pytest
import torch

import expert_grouped_gemm_amd as moe
import moe_synth
import oracle
from moe_cases import problem_of, run_layer, to_gpu

pytestmark = pytest.mark.gpu


def _i32(x, cap=None):
    x = np.asarray(x)
    if cap is not None:
        x = np.concatenate([x, np.zeros(cap - x.size, x.dtype)])
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _expect(status, p, ws):
    with pytest.raises(moe.MoEError) as ei:
        moe.check_workspace(p, ws)
    assert ei.value.status == status
    moe.check_workspace(p, ws)  # the report clears the words


class _W4A4:
    """A small share on MXFP4 operands; first and second are the two Linears."""

    def __init__(self):
        cfg = moe_synth.make_config("tiny", T=70, d=384, f=128, E_global=8, k=2, e_begin=1, e_end=6)
        idx, w, _ = oracle.route_topk(np.random.default_rng(4).normal(size=(cfg.T, 8)).astype(np.float32), cfg.k)
        disp = oracle.dispatch(idx, w, cfg.e_begin, cfg.e_end)
        g = torch.Generator().manual_seed(4)

        def mx(*shape):
            return (torch.randint(0, 256, (*shape[:-1], shape[-1] // 2), generator=g, dtype=torch.uint8).cuda(),
                    torch.randint(118, 128, (*shape[:-1], shape[-1] // 32), generator=g, dtype=torch.uint8).cuda())

        self.cfg, self.p = cfg, problem_of(cfg, sched="auto")
        self.x, self.w1 = mx(cfg.T, cfg.d), mx(cfg.E_local, 2 * cfg.f, cfg.d)
        self.h, self.w2 = mx(cfg.cap, cfg.f), mx(cfg.E_local, cfg.d, cfg.f)
        self.src, self.dst = _i32(disp["row_src"], cfg.cap), _i32(disp["row_dst"], cfg.cap)
        self.off = _i32(disp["offsets"])
        self.H = torch.zeros(cfg.cap, cfg.f, dtype=torch.bfloat16, device="cuda")
        self.C = torch.zeros(cfg.cap, cfg.d, device="cuda")

    def first(self, ws, src=None, off=None):
        moe.mxfp4_linear1(self.p, *self.x, self.src if src is None else src, self.off if off is None else off,
                          *self.w1, self.H, ws)

    def second(self, ws):
        moe.mxfp4_linear2(self.p, *self.h, self.off, self.dst, *self.w2, self.C, ws)


@pytest.mark.parametrize("bad", ["row_src", "offsets"])
def test_linear2_keeps_what_linear1_reported(bad):
    s = _W4A4()
    ws = moe.alloc_workspace(s.p)
    if bad == "row_src":
        src = s.src.clone()
        src[5] = s.cfg.T * s.cfg.k
        s.first(ws, src=src)
    else:
        off = s.off.clone()
        off[-1] = s.cfg.cap + 1
        s.first(ws, off=off)
    s.second(ws)
    _expect(1, s.p, ws)
    s.first(ws)                      # nothing of it is left for the next layer
    s.second(ws)
    moe.check_workspace(s.p, ws)


def test_the_next_layers_linear1_starts_a_new_report():
    s = _W4A4()
    ws = moe.alloc_workspace(s.p)
    src = s.src.clone()
    src[5] = -1
    s.first(ws, src=src)
    s.second(ws)
    s.first(ws)
    s.second(ws)
    moe.check_workspace(s.p, ws)


def test_the_linears_keep_a_dispatch_past_capacity():
    """topk_idx lists the one local expert twice for every token: 2 T assignments against a capacity of T."""
    s = _W4A4()
    cfg, p = s.cfg, moe.make_problem(s.cfg.T, s.cfg.d, s.cfg.f, 8, 2, 0, 1, sched="auto")
    ws = moe.alloc_workspace(p)
    v = moe.workspace_views(p, ws)
    idx = torch.zeros(cfg.T, 2, dtype=torch.int32, device="cuda")
    moe.dispatch(p, torch.ones(cfg.T, cfg.d, dtype=torch.bfloat16, device="cuda"), None, idx,
                 torch.full((cfg.T, 2), 0.5, device="cuda"), v["counts"], v["offsets"], v["row_src"], v["row_dst"],
                 v["tok_off"], v["comb_w"], v["x_perm"], None, ws)
    rows = _i32(np.arange(cfg.T))
    off = _i32([0, cfg.T])
    moe.mxfp4_linear1(p, *s.x, 2 * rows, off, *s.w1, s.H, ws)
    moe.mxfp4_linear2(p, *s.h, off, rows, *s.w2, s.C, ws)
    assert s.H[:cfg.T].any() and s.C[:cfg.T].any()   # they ran: their own rows are good
    _expect(1, p, ws)


@pytest.mark.parametrize("sched", ["interleaved", "expert_wave"])
def test_backward_keeps_a_timed_out_forward(sched):
    """The forward's bounded wait is forced to give up; the gradients that follow on its combine buffer go well."""
    cfg = moe_synth.make_config("tiny", T=512, d=128, f=256, E_global=4, k=2, seed=51)
    g = to_gpu(moe_synth.generate(cfg))
    bad, p = problem_of(cfg, sched=sched), problem_of(cfg, sched=sched)
    bad.flags |= moe.FLAG_TEST_WAIT_TIMEOUT
    ws = moe.alloc_backward_workspace(p)
    run_layer(bad, g, ws=ws, want_fp32=False)
    v = moe.workspace_views(p, ws)
    bf = dict(dtype=torch.bfloat16, device="cuda")
    dO, dxs = torch.ones(cfg.cap, cfg.d, **bf), torch.empty(cfg.cap, cfg.d, **bf)
    args = (p, g["X"], v["row_src"], v["offsets"], v["row_dst"], g["W1"], g["W2"], dO, dxs,
            torch.empty_like(g["W1"]), torch.empty_like(g["W2"]), ws)
    moe.expert_backward(*args)
    torch.cuda.synchronize()
    assert torch.isfinite(dxs).all()
    _expect(5, p, ws)
    run_layer(p, g, ws=ws)
    moe.expert_backward(*args)
    moe.check_workspace(p, ws)


@pytest.mark.parametrize("byte", [0x00, 0x01, 0x55, 0xFF])
def test_a_fresh_workspace_reports_nothing(byte):
    s = _W4A4()
    for call in (s.first, s.second):
        ws = torch.full((moe.workspace_size(s.p),), byte, dtype=torch.uint8, device="cuda")
        call(ws)
        moe.check_workspace(s.p, ws)
    cfg = s.cfg
    bf = dict(dtype=torch.bfloat16, device="cuda")
    ws = torch.full((moe.backward_workspace_size(s.p),), byte, dtype=torch.uint8, device="cuda")
    dW1 = torch.full((cfg.E_local, 2 * cfg.f, cfg.d), 3.0, **bf)
    moe.expert_backward(s.p, torch.ones(cfg.T, cfg.d, **bf), s.src, s.off, s.dst, torch.ones_like(dW1),
                        torch.ones(cfg.E_local, cfg.d, cfg.f, **bf), torch.ones(cfg.cap, cfg.d, **bf),
                        torch.empty(cfg.cap, cfg.d, **bf), dW1, torch.empty(cfg.E_local, cfg.d, cfg.f, **bf), ws)
    moe.check_workspace(s.p, ws)
    assert not torch.all(dW1 == 3.0)
