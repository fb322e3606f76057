"""Gradients of the combine (with the router's softmax) and of the dispatch
against the fp64 formulas, and the calls they refuse.

Tolerances, per element, from the roundings a result passes through (u = 2^-24
per fp32 operation, 2^-8 for a rounding to bf16):
  d_combine_buf  one product, one rounding to bf16: (2^-8 + 2 u) |ref|
  d_topk_w       a sum of d products in fp32, in whatever order: at most d
                 roundings, each at most u of the sum of magnitudes
  d_logits       the products of d_topk_w and its errors, k + 4 more roundings
  dX             a sum of at most k values, one rounding to bf16
"""
import numpy as np
import pytest
import torch

import expert_grouped_gemm_amd as moe
import moe_synth
import oracle
from moe_cases import problem_of
from oracle import backward

pytestmark = pytest.mark.gpu

U, B = 2.0 ** -24, 2.0 ** -8

CASES = {
    "one_token": dict(T=1, d=128, E_global=4, k=1),
    "odd_tokens": dict(T=77, d=384, E_global=16, k=4, e_begin=3, e_end=11),
    "k16": dict(T=50, d=256, E_global=24, k=16, e_begin=4, e_end=20),
    "segments": dict(T=96, d=640, E_global=8, k=3, e_begin=0, e_end=5, num_segments=4),
    "wide_rows": dict(T=33, d=7168, E_global=256, k=8, e_begin=0, e_end=32),
    "none_local": dict(T=5, d=128, E_global=512, k=2, e_begin=511, e_end=512),
    "rows_of_1024": dict(T=37, d=1024, E_global=12, k=5),
    "rows_past_1024": dict(T=19, d=1152, E_global=12, k=5, e_begin=2, e_end=9),
    "rows_of_256": dict(T=43, d=256, E_global=16, k=7, e_begin=0, e_end=9),
    "many_experts": dict(T=20, d=128, E_global=1024, k=8),
}


def _setup(case, seed=7):
    cfg = moe_synth.make_config("tiny", **{**dict(f=128, e_begin=0, e_end=case["E_global"]), **case})
    rng = np.random.default_rng(seed)
    idx, w, _ = oracle.route_topk(rng.normal(size=(cfg.T, cfg.E_global)).astype(np.float32), cfg.k)
    disp = oracle.dispatch(idx, w, cfg.e_begin, cfg.e_end, cfg.num_segments)
    g = torch.Generator().manual_seed(seed)
    dY = torch.randn(cfg.T, cfg.d, generator=g).to(torch.bfloat16)
    buf = torch.randn(cfg.cap, cfg.d, generator=g)
    return cfg, idx, torch.tensor(w, dtype=torch.float32), disp, dY, buf


def _i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("bf16_buf", [False, True])
@pytest.mark.parametrize("name", list(CASES))
def test_combine_backward(name, bf16_buf):
    print(f"[combine_backward] {name} bf16_buf={bf16_buf}", flush=True)
    cfg, idx, w, disp, dY, buf = _setup(CASES[name])
    if bf16_buf:
        buf = buf.to(torch.bfloat16)
    p = problem_of(cfg, sched="auto", bf16_combine_buf=bf16_buf)
    A = disp["A"]
    d_buf = torch.full((cfg.cap, cfg.d), 3.0, dtype=torch.bfloat16, device="cuda")
    d_w = torch.full((cfg.T, cfg.k), 9.0, device="cuda")
    d_l = torch.full((cfg.T, cfg.E_global), 9.0, device="cuda")
    moe.combine_backward(p, dY.cuda(), buf.cuda(), _i32(disp["tok_off"]), _i32(idx), w.cuda(), d_buf, d_w, d_l)
    torch.cuda.synchronize()
    buf64, dY64, w64 = buf.double().numpy(), dY.double().numpy(), w.double().numpy()
    r_buf, r_w, r_l = backward.combine_backward(dY64, buf64, disp["tok_off"], idx, w64, cfg.e_begin, cfg.e_end,
                                                cfg.E_global, cfg.num_segments)
    got = d_buf.double().cpu().numpy()
    assert np.all(np.abs(got[:A] - r_buf) <= (B + 2 * U) * np.abs(r_buf))
    assert np.all(got[A:] == 3.0)
    mag = backward.combine_backward(np.abs(dY64), np.abs(buf64), disp["tok_off"], idx, w64, cfg.e_begin, cfg.e_end,
                                    cfg.E_global, cfg.num_segments)[1]
    tol_w = cfg.d * U * mag
    assert np.all(np.abs(d_w.double().cpu().numpy() - r_w) <= tol_w)
    mean = (w64 * np.abs(r_w)).sum(1, keepdims=True)
    tol = w64 * (tol_w + (w64 * tol_w).sum(1, keepdims=True) + (cfg.k + 4) * U * (np.abs(r_w) + mean))
    tol_l = np.zeros_like(r_l)
    np.put_along_axis(tol_l, idx.astype(np.int64), tol, axis=1)
    assert np.all(np.abs(d_l.double().cpu().numpy() - r_l) <= tol_l)
    d_w2 = torch.empty_like(d_w)                 # without the logits' gradient
    moe.combine_backward(p, dY.cuda(), buf.cuda(), _i32(disp["tok_off"]), _i32(idx), w.cuda(), d_buf, d_w2)
    assert torch.equal(d_w, d_w2)


@pytest.mark.parametrize("name", list(CASES))
def test_dispatch_backward(name):
    print(f"[dispatch_backward] {name}", flush=True)
    cfg, idx, w, disp, dY, buf = _setup(CASES[name])
    p = problem_of(cfg, sched="auto")
    dxs = buf.to(torch.bfloat16)
    dxs[disp["A"]:] = float("nan")              # rows past the last slot are never read
    dX = torch.empty(cfg.T, cfg.d, dtype=torch.bfloat16, device="cuda")
    dX32 = torch.empty(cfg.T, cfg.d, device="cuda")
    moe.dispatch_backward(p, dxs.cuda(), _i32(disp["tok_off"]), dX, dX32)
    torch.cuda.synchronize()
    v = dxs[:disp["A"]].double().numpy()
    ref = backward.dispatch_backward(v, disp["tok_off"], cfg.T, cfg.num_segments)
    tol = cfg.k * U * backward.dispatch_backward(np.abs(v), disp["tok_off"], cfg.T, cfg.num_segments)
    assert np.all(np.abs(dX32.double().cpu().numpy() - ref) <= tol)
    assert np.all(np.abs(dX.double().cpu().numpy() - ref) <= tol + (B + B * U) * (np.abs(ref) + tol))
    dX2 = torch.empty_like(dX)
    moe.dispatch_backward(p, dxs.cuda(), _i32(disp["tok_off"]), dX2)
    assert torch.equal(dX2, dX)


def test_same_expert_twice_in_a_row_of_topk():
    """A caller's topk_idx may repeat an expert: both gates have a slot, and its logit takes both gradients."""
    T, d, E = 3, 128, 6
    idx = np.array([[2, 2], [2, 5], [5, 5]], dtype=np.int32)
    w = np.array([[0.25, 0.75], [0.5, 0.5], [0.125, 0.875]], dtype=np.float32)
    disp = oracle.dispatch(idx, w, 0, 4)
    g = torch.Generator().manual_seed(1)
    dY = torch.randn(T, d, generator=g).to(torch.bfloat16)
    p = moe.make_problem(T, d, 128, E, 2, 0, 4)
    buf = torch.randn(moe.row_capacity(p), d, generator=g)
    d_buf = torch.zeros(moe.row_capacity(p), d, dtype=torch.bfloat16, device="cuda")
    d_w, d_l = torch.empty(T, 2, device="cuda"), torch.empty(T, E, device="cuda")
    moe.combine_backward(p, dY.cuda(), buf.cuda(), _i32(disp["tok_off"]), _i32(idx), torch.tensor(w).cuda(), d_buf,
                         d_w, d_l)
    r_buf, r_w, r_l = backward.combine_backward(dY.double().numpy(), buf.double().numpy(), disp["tok_off"], idx, w, 0, 4,
                                                E)
    mag = np.abs(dY.double().numpy()) @ np.abs(buf.double().numpy()).T
    assert np.all(np.abs(d_w.double().cpu().numpy() - r_w) <= d * U * mag.max())
    assert np.all(np.abs(d_l.double().cpu().numpy() - r_l) <= 4 * d * U * mag.max())
    assert np.all(np.abs(d_buf.double().cpu().numpy()[:disp["A"]] - r_buf) <= (B + 2 * U) * np.abs(r_buf))


def test_slot_ranges_that_do_not_fit():
    """Ranges outside the buffer, reversed, or of another length than the token's local experts."""
    cfg, idx, w, disp, dY, buf = _setup(CASES["odd_tokens"])
    p = problem_of(cfg, sched="auto")
    t = next(t for t in range(cfg.T) if disp["tok_off"][t + 1] > disp["tok_off"][t])
    for lo, hi in ((-2, -1), (cfg.cap, cfg.cap + 1), (5, 4), (0, cfg.cap + 7)):
        off = np.asarray(disp["tok_off"]).copy()
        off[t], off[t + 1] = lo, hi
        touched = {x for x in (t - 1, t, t + 1) if 0 <= x < cfg.T}
        d_buf = torch.full((cfg.cap, cfg.d), 3.0, dtype=torch.bfloat16, device="cuda")
        d_w, d_l = torch.zeros(cfg.T, cfg.k, device="cuda"), torch.zeros(cfg.T, cfg.E_global, device="cuda")
        moe.combine_backward(p, dY.cuda(), buf.cuda(), _i32(off), _i32(idx), w.cuda(), d_buf, d_w, d_l)
        dX = torch.zeros(cfg.T, cfg.d, dtype=torch.bfloat16, device="cuda")
        moe.dispatch_backward(p, buf.to(torch.bfloat16).cuda(), _i32(off), dX)
        assert torch.isnan(d_w[t]).all() and torch.isnan(d_l[t]).all(), (lo, hi)
        others = [x for x in range(cfg.T) if x not in touched]
        assert torch.isfinite(d_w[others]).all() and torch.isfinite(d_l[others]).all()
        if not (0 <= lo <= hi <= cfg.cap):
            assert torch.isnan(dX[t]).all(), (lo, hi)
        assert torch.isfinite(dX[others]).all()


def test_non_finite_gradients_stay_with_their_token():
    cfg, idx, w, disp, dY, buf = _setup(CASES["odd_tokens"])
    p = problem_of(cfg, sched="auto")
    dY[4, 3] = float("inf")
    dY[9, 0] = float("nan")
    d_buf = torch.zeros(cfg.cap, cfg.d, dtype=torch.bfloat16, device="cuda")
    d_w, d_l = torch.empty(cfg.T, cfg.k, device="cuda"), torch.empty(cfg.T, cfg.E_global, device="cuda")
    moe.combine_backward(p, dY.cuda(), buf.cuda(), _i32(disp["tok_off"]), _i32(idx), w.cuda(), d_buf, d_w, d_l)
    keep = [t for t in range(cfg.T) if t not in (4, 9)]
    assert torch.isfinite(d_w[keep]).all() and torch.isfinite(d_l[keep]).all()
    bad = torch.zeros(cfg.cap, dtype=torch.bool)
    for t in (4, 9):
        bad[disp["tok_off"][t]:disp["tok_off"][t + 1]] = True
    assert torch.isfinite(d_buf[~bad.cuda()]).all()


def test_replayed_graph_and_another_stream():
    cfg, idx, w, disp, dY, buf = _setup(CASES["segments"])
    p = problem_of(cfg, sched="auto")
    dYg, bufg, off, ix, wg = dY.cuda(), buf.cuda(), _i32(disp["tok_off"]), _i32(idx), w.cuda()
    d_buf = torch.zeros(cfg.cap, cfg.d, dtype=torch.bfloat16, device="cuda")
    d_w, d_l = torch.empty(cfg.T, cfg.k, device="cuda"), torch.empty(cfg.T, cfg.E_global, device="cuda")
    dX = torch.empty(cfg.T, cfg.d, dtype=torch.bfloat16, device="cuda")

    def step():
        moe.combine_backward(p, dYg, bufg, off, ix, wg, d_buf, d_w, d_l)
        moe.dispatch_backward(p, d_buf, off, dX)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for i in range(3):
        dYg.copy_((dY * (i + 1)).to(torch.bfloat16))
        for out in (d_w, d_l, dX):
            out.fill_(7.0)
        graph.replay()
        torch.cuda.synchronize()
        replayed = [x.clone() for x in (d_buf, d_w, d_l, dX)]
        step()
        torch.cuda.synchronize()
        for a, b in zip(replayed, (d_buf, d_w, d_l, dX)):
            assert torch.equal(a, b)


@pytest.mark.parametrize("change", ["dtype", "small", "cpu", "strided", "missing"])
def test_refused_tensors(change):
    cfg, idx, w, disp, dY, buf = _setup(CASES["odd_tokens"])
    p = problem_of(cfg, sched="auto")
    d_buf = torch.full((cfg.cap, cfg.d), 3.0, dtype=torch.bfloat16, device="cuda")
    d_w = torch.empty(cfg.T, cfg.k, device="cuda")
    bad = {"dtype": dY.float().cuda(), "small": dY[:-1].cuda(), "cpu": dY, "missing": None,
           "strided": torch.empty(cfg.T, 2 * cfg.d, dtype=torch.bfloat16, device="cuda")[:, ::2]}[change]
    with pytest.raises(ValueError):
        moe.combine_backward(p, bad, buf.cuda(), _i32(disp["tok_off"]), _i32(idx), w.cuda(), d_buf, d_w)
    with pytest.raises(ValueError):
        moe.dispatch_backward(p, d_buf, _i32(disp["tok_off"]), bad)
    torch.cuda.synchronize()
    assert torch.all(d_buf == 3.0)
