"""The experts' gradient against the fp64 formulas, alone and in the whole
backward pass of a layer.

Two references. The exact one (oracle.backward) with a bound per element, from
the roundings on the way (u = 2^-24 per fp32 operation, b = 2^-8 per rounding
to bf16; |silu'| <= 1.1, |silu''| <= 0.5; the hardware's exp2 and reciprocal
and the products around them within 16 u (1 + |g|) of silu and 32 u (1 + |g|)
of its derivative):
  g, u, da   sums of d products: d u (sum of magnitudes)
  a          1.1 |u| eg + |silu| eu + (16 u (1 + |g|) + b) |a|
  dg         |u D| eda + |da D| eu + |da u| (0.5 eg + 32 u (1 + |g|)) + b |dg|
  du         |silu| eda + |da| (1.1 eg + 16 u (1 + |g|) |silu|) + b |du|
  dx, dW     the sum over the products of those errors, n u (sum of
             magnitudes) for n products, one more b
And one with a, dg and du rounded to bf16 where the kernel rounds them: what is
left is the outputs' one rounding, at most 2^-8 of every element and so of the
norm; sums of fp32 and a rounding that falls the other way for it are far
below a tenth of that.
"""
import numpy as np
import pytest
import torch

import expert_grouped_gemm_amd as moe
import moe_synth
import oracle
from moe_cases import problem_of, to_gpu
from oracle import backward

pytestmark = pytest.mark.gpu

U, B = 2.0 ** -24, 2.0 ** -8

CASES = {
    "one_token": dict(T=1, d=128, f=128, E_global=4, k=2),
    "odd_tokens": dict(T=77, d=384, f=128, E_global=8, k=2, e_begin=1, e_end=6),
    "odd_widths": dict(T=150, d=640, f=384, E_global=8, k=3),
    "bands": dict(T=700, d=256, f=256, E_global=2, k=1),
    "segments": dict(T=256, d=512, f=256, E_global=16, k=4, e_begin=4, e_end=12, num_segments=4),
    "empty_experts": dict(T=3, d=256, f=128, E_global=64, k=2),
    "none_local": dict(T=2, d=128, f=128, E_global=512, k=1, e_begin=511, e_end=512),
    "long_experts": dict(T=1500, d=384, f=640, E_global=2, k=1),
    "long_many_tiles": dict(T=1111, d=2304, f=1152, E_global=4, k=2),
    "one_expert": dict(T=274, d=896, f=384, E_global=1, k=1),
    "many_tiles": dict(T=900, d=1536, f=2048, E_global=3, k=1),
}


def _i32(x, cap=None):
    x = np.asarray(x)
    if cap is not None:
        x = np.concatenate([x, np.zeros(cap - x.size, x.dtype)])
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _setup(case, seed=5):
    cfg = moe_synth.make_config("tiny", **{**dict(e_begin=0, e_end=case["E_global"], seed=seed), **case})
    inp = moe_synth.generate(cfg)
    idx, w, _ = oracle.route_topk(inp["logits"].numpy(), cfg.k)
    disp = oracle.dispatch(idx, w, cfg.e_begin, cfg.e_end, cfg.num_segments)
    g = torch.Generator().manual_seed(seed)
    dO = torch.randn(cfg.cap, cfg.d, generator=g).to(torch.bfloat16)
    return cfg, inp, disp, dO


def _outputs(cfg):
    z = dict(dtype=torch.bfloat16, device="cuda")
    return (torch.full((cfg.cap, cfg.d), 3.0, **z), torch.full((cfg.E_local, 2 * cfg.f, cfg.d), 3.0, **z),
            torch.full((cfg.E_local, cfg.d, cfg.f), 3.0, **z))


def _rounded_reference(X, dO, off, W1, W2):
    dx, dW1, dW2 = np.zeros_like(X), np.zeros(W1.shape), np.zeros(W2.shape)
    for e in range(W1.shape[0]):
        r = slice(off[e], off[e + 1])
        g, u = np.split(X[r] @ W1[e].T, 2, axis=1)
        s = 1 / (1 + np.exp(-g))
        da = dO[r] @ W2[e]
        a = oracle.round_to_bf16(g * s * u)
        dh = oracle.round_to_bf16(np.concatenate([da * u * (s + g * s * (1 - s)), da * g * s], axis=1))
        dx[r], dW1[e], dW2[e] = dh @ W1[e], dh.T @ X[r], dO[r].T @ a
    return dx, dW1, dW2


def _bounds(X, dO, off, W1, W2):
    tx, t1, t2 = np.zeros_like(X), np.zeros(W1.shape), np.zeros(W2.shape)
    d, f = X.shape[1], W2.shape[2]
    for e in range(W1.shape[0]):
        r = slice(off[e], off[e + 1])
        n = off[e + 1] - off[e]
        x, do, w1, w2 = X[r], dO[r], W1[e], W2[e]
        g, u = np.split(x @ w1.T, 2, axis=1)
        eg, eu = np.split(d * U * (np.abs(x) @ np.abs(w1).T), 2, axis=1)
        s = 1 / (1 + np.exp(-g))
        silu, D = g * s, s + g * s * (1 - s)
        da = do @ w2
        eda = d * U * (np.abs(do) @ np.abs(w2))
        G = U * (1 + np.abs(g))
        ea = 1.1 * np.abs(u) * eg + np.abs(silu) * eu + (16 * G + B) * np.abs(silu * u)
        edg = (np.abs(u * D) * eda + np.abs(da * D) * eu + np.abs(da * u) * (0.5 * eg + 32 * G)
               + B * np.abs(da * u * D))
        edu = np.abs(silu) * eda + np.abs(da) * (1.1 * eg + 16 * G * np.abs(silu)) + B * np.abs(da * silu)
        dh, edh = np.concatenate([da * u * D, da * silu], 1), np.concatenate([edg, edu], 1)
        m = np.abs(dh) + edh
        tx[r] = edh @ np.abs(w1) + 2 * f * U * (m @ np.abs(w1))
        t1[e] = edh.T @ np.abs(x) + n * U * (m.T @ np.abs(x))
        t2[e] = np.abs(do).T @ ea + n * U * (np.abs(do).T @ (np.abs(silu * u) + ea))
    return tx, t1, t2


def _check(got, exact, rounded, bounds, label):
    for name, g, ref, rr, tol in zip(("dx", "dW1", "dW2"), got, exact, rounded, bounds):
        err = np.abs(g - ref)
        assert np.all(err <= tol + B * (np.abs(ref) + tol)), (label, name, float((err - tol).max()))
        norm = np.linalg.norm(rr)
        if norm:
            rel = np.linalg.norm(g - rr) / norm
            assert rel <= 1.1 * B, (label, name, rel)


@pytest.mark.parametrize("gather", [True, False])
@pytest.mark.parametrize("name", list(CASES))
def test_expert_backward(name, gather):
    print(f"[expert_backward] {name} gather={gather}", flush=True)
    cfg, inp, disp, dO = _setup(CASES[name])
    A, cap, off = disp["A"], cfg.cap, disp["offsets"]
    dO[A:] = float("nan")                        # slots of no row are never read
    p = problem_of(cfg, sched="auto")
    tok = disp["row_src"] // cfg.k
    X, src = inp["X"], _i32(disp["row_src"], cap)
    if not gather:
        X = torch.full((cap, cfg.d), float("nan"), dtype=torch.bfloat16)
        X[:A] = inp["X"][torch.tensor(tok)]
        src = None
    out = _outputs(cfg)
    ws = moe.alloc_backward_workspace(p)
    moe.expert_backward(p, X.cuda(), src, _i32(off), _i32(disp["row_dst"], cap), inp["W1"].cuda(), inp["W2"].cuda(),
                        dO.cuda(), *out, ws)
    torch.cuda.synchronize()
    moe.check_workspace(p, ws)
    dxs, dW1, dW2 = (t.double().cpu().numpy() for t in out)
    ops = (inp["X"].double().numpy()[tok], dO.double().numpy()[disp["row_dst"]], off, inp["W1"].double().numpy(),
           inp["W2"].double().numpy())
    _check((dxs[disp["row_dst"]], dW1, dW2), backward.expert_backward(*ops), _rounded_reference(*ops), _bounds(*ops),
           name)
    assert np.all(dxs[A:] == 3.0)
    again = _outputs(cfg)
    moe.expert_backward(p, X.cuda(), src, _i32(off), _i32(disp["row_dst"], cap), inp["W1"].cuda(), inp["W2"].cuda(),
                        dO.cuda(), *again, ws)
    for a, b in zip(out, again):
        assert torch.equal(a, b)                 # the same bits on every call


@pytest.mark.parametrize("counts", [[1, 63, 64, 65], [0, 0, 257, 0], [127, 128, 129, 2], [256, 0, 31, 33]])
def test_rows_per_expert_around_the_tile_borders(counts):
    print(f"[expert_backward] counts {counts}", flush=True)
    A, d, f = sum(counts), 256, 128
    off = np.concatenate([[0], np.cumsum(counts)])
    rng = np.random.default_rng(A)
    g = torch.Generator().manual_seed(A)
    p = moe.make_problem(A, d, f, 4, 1, sched="auto")
    X, dO = (torch.randn(A, d, generator=g).to(torch.bfloat16) for _ in range(2))
    W1, W2 = (torch.randn(*s, generator=g).mul_(0.05).to(torch.bfloat16) for s in ((4, 2 * f, d), (4, d, f)))
    dst = rng.permutation(A)
    z = dict(dtype=torch.bfloat16, device="cuda")
    out = torch.empty(A, d, **z), torch.empty(4, 2 * f, d, **z), torch.empty(4, d, f, **z)
    ws = moe.alloc_backward_workspace(p)
    moe.expert_backward(p, X.cuda(), None, _i32(off), _i32(dst), W1.cuda(), W2.cuda(), dO.cuda(), *out, ws)
    torch.cuda.synchronize()
    moe.check_workspace(p, ws)
    dxs, dW1, dW2 = (t.double().cpu().numpy() for t in out)
    ops = X.double().numpy(), dO.double().numpy()[dst], off, W1.double().numpy(), W2.double().numpy()
    _check((dxs[dst], dW1, dW2), backward.expert_backward(*ops), _rounded_reference(*ops), _bounds(*ops), counts)


def test_rows_that_do_not_start_at_zero():
    """offsets[0] > 0: the rows before it belong to no expert."""
    A, d, f, first = 90, 128, 128, 7
    off = np.array([first, 40, 40, A])
    g = torch.Generator().manual_seed(8)
    p = moe.make_problem(A, d, f, 3, 1, sched="auto")
    X, dO = (torch.randn(A, d, generator=g).to(torch.bfloat16) for _ in range(2))
    W1, W2 = (torch.randn(*s, generator=g).mul_(0.05).to(torch.bfloat16) for s in ((3, 2 * f, d), (3, d, f)))
    X[:first] = float("nan")
    z = dict(dtype=torch.bfloat16, device="cuda")
    out = torch.full((A, d), 3.0, **z), torch.empty(3, 2 * f, d, **z), torch.empty(3, d, f, **z)
    ws = moe.alloc_backward_workspace(p)
    moe.expert_backward(p, X.cuda(), None, _i32(off), _i32(np.arange(A)), W1.cuda(), W2.cuda(), dO.cuda(), *out, ws)
    torch.cuda.synchronize()
    moe.check_workspace(p, ws)
    dxs, dW1, dW2 = (t.double().cpu().numpy() for t in out)
    assert np.all(dxs[:first] == 3.0)
    ops = (X.double().numpy()[first:], dO.double().numpy()[first:], off - first, W1.double().numpy(),
           W2.double().numpy())
    _check((dxs[first:], dW1, dW2), backward.expert_backward(*ops), _rounded_reference(*ops), _bounds(*ops), "first")


@pytest.mark.parametrize("T", [300, 1300])
def test_on_another_stream(T):
    """Both weight-gradient forms on a stream of the caller's, against the default stream."""
    cfg, inp, disp, dO = _setup(dict(T=T, d=256, f=128, E_global=2, k=1))
    p = problem_of(cfg, sched="auto")
    args = (inp["X"].cuda(), _i32(disp["row_src"], cfg.cap), _i32(disp["offsets"]), _i32(disp["row_dst"], cfg.cap),
            inp["W1"].cuda(), inp["W2"].cuda(), dO.cuda())
    a, b = _outputs(cfg), _outputs(cfg)
    ws, ws2 = moe.alloc_backward_workspace(p), moe.alloc_backward_workspace(p)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    moe.expert_backward(p, *args, *a, ws, stream=side)
    moe.expert_backward(p, *args, *b, ws2)
    torch.cuda.synchronize()
    for x, y in zip(a, b):
        assert torch.equal(x, y)


def test_grid_changes_no_bit():
    cfg, inp, disp, dO = _setup(CASES["odd_widths"])
    args = (inp["X"].cuda(), _i32(disp["row_src"], cfg.cap), _i32(disp["offsets"]), _i32(disp["row_dst"], cfg.cap),
            inp["W1"].cuda(), inp["W2"].cuda(), dO.cuda())
    ref = None
    for grid in (0, 1, 2, 7, 40):
        p = problem_of(cfg, sched="auto", grid=grid)
        out = _outputs(cfg)
        moe.expert_backward(p, *args, *out, moe.alloc_backward_workspace(p))
        torch.cuda.synchronize()
        ref = ref or out
        for a, b in zip(ref, out):
            assert torch.equal(a, b), grid


def test_saturated_gates():
    """Gates far out on both sides: the derivative is 0 or 1 there, never NaN."""
    T, d, f = 40, 128, 128
    g = torch.Generator().manual_seed(2)
    X = torch.randn(T, d, generator=g).to(torch.bfloat16)
    W1 = (torch.randn(1, 2 * f, d, generator=g) * 30).to(torch.bfloat16)
    W2 = torch.randn(1, d, f, generator=g).to(torch.bfloat16)
    dO = torch.randn(T, d, generator=g).to(torch.bfloat16)
    p = moe.make_problem(T, d, f, 1, 1, sched="auto")
    z = dict(dtype=torch.bfloat16, device="cuda")
    out = torch.empty(T, d, **z), torch.empty(1, 2 * f, d, **z), torch.empty(1, d, f, **z)
    moe.expert_backward(p, X.cuda(), None, _i32([0, T]), _i32(np.arange(T)), W1.cuda(), W2.cuda(), dO.cuda(), *out,
                        moe.alloc_backward_workspace(p))
    got = [t.double().cpu().numpy() for t in out]
    with np.errstate(over="ignore"):
        ops = X.double().numpy(), dO.double().numpy(), np.array([0, T]), W1.double().numpy(), W2.double().numpy()
        _check(got, backward.expert_backward(*ops), _rounded_reference(*ops), _bounds(*ops), "saturated")


def test_infinite_gradient_stays_in_its_expert():
    cfg, inp, disp, dO = _setup(CASES["odd_tokens"])
    off, e = disp["offsets"], int(np.argmax(disp["counts"]))
    dO[disp["row_dst"][off[e]], 5] = float("inf")
    p = problem_of(cfg, sched="auto")
    out = _outputs(cfg)
    moe.expert_backward(p, inp["X"].cuda(), _i32(disp["row_src"], cfg.cap), _i32(off),
                        _i32(disp["row_dst"], cfg.cap), inp["W1"].cuda(), inp["W2"].cuda(), dO.cuda(), *out,
                        moe.alloc_backward_workspace(p))
    torch.cuda.synchronize()
    dxs, dW1, dW2 = out
    rows = torch.tensor([int(disp["row_dst"][r]) for r in range(disp["A"]) if r != off[e]], device="cuda")
    assert torch.isfinite(dxs[rows]).all()
    for x in range(cfg.E_local):
        assert torch.isfinite(dW1[x]).all() == (x != e) and torch.isfinite(dW2[x]).all() == (x != e)


def test_whole_backward_pass_of_a_layer():
    """layer_forward, then the three gradients in a row, against the fp64 chain on the forward's own bf16 operands.
    Tolerance: the chain's gradients pass three to four roundings to bf16 (dO, dh or a, the row's gradient, the
    output), each at most 2^-8 of its elements: 4 * 2^-8 of the norm."""
    cfg = moe_synth.make_config("tiny", T=512, d=512, f=384, E_global=16, k=4, e_begin=2, e_end=12, num_segments=4,
                                seed=21)
    inp = moe_synth.generate(cfg)
    g = to_gpu(inp)
    p = problem_of(cfg, sched="auto")
    ws = moe.alloc_backward_workspace(p)
    Y = torch.empty(cfg.T, cfg.d, dtype=torch.bfloat16, device="cuda")
    moe.layer_forward(p, g["X"], None, g["logits"], g["W1"], None, g["W2"], None, Y, None, ws)
    v = moe.workspace_views(p, ws)
    dY = torch.randn(cfg.T, cfg.d, generator=torch.Generator().manual_seed(3)).to(torch.bfloat16)
    bf = dict(dtype=torch.bfloat16, device="cuda")
    d_buf, dxs, dX = torch.empty(cfg.cap, cfg.d, **bf), torch.empty(cfg.cap, cfg.d, **bf), torch.empty(cfg.T, cfg.d, **bf)
    dW1, dW2 = torch.empty_like(g["W1"]), torch.empty_like(g["W2"])
    d_w = torch.empty(cfg.T, cfg.k, device="cuda")
    d_l = torch.empty(cfg.T, cfg.E_global, device="cuda")

    def step():
        moe.combine_backward(p, dY.cuda(), v["combine_buf"], v["tok_off"], v["topk_idx"], v["topk_w"], d_buf, d_w, d_l)
        moe.expert_backward(p, g["X"], v["row_src"], v["offsets"], v["row_dst"], g["W1"], g["W2"], d_buf, dxs, dW1,
                            dW2, ws)
        moe.dispatch_backward(p, dxs, v["tok_off"], dX)

    step()
    torch.cuda.synchronize()
    moe.check_workspace(p, ws)
    ref = oracle.moe_layer(inp, cfg)
    idx, w, _ = oracle.route_topk(inp["logits"].numpy(), cfg.k)
    disp = oracle.dispatch(idx, w, cfg.e_begin, cfg.e_end, cfg.num_segments)
    A, rd, tok = disp["A"], disp["row_dst"], disp["row_src"] // cfg.k
    W1, W2, X = (inp[n].double().numpy() for n in ("W1", "W2", "X"))
    O = np.zeros((A, cfg.d))
    for e in range(cfg.E_local):
        r = slice(disp["offsets"][e], disp["offsets"][e + 1])
        h, u = np.split(X[tok[r]] @ W1[e].T, 2, axis=1)
        O[rd[r]] = oracle.round_to_bf16(h / (1 + np.exp(-h)) * u) @ W2[e].T
    r_buf, r_w, r_l = backward.combine_backward(dY.double().numpy(), O, disp["tok_off"], idx, w, cfg.e_begin, cfg.e_end,
                                                cfg.E_global, cfg.num_segments)
    dx, r1, r2 = backward.expert_backward(X[tok], r_buf[rd], disp["offsets"], W1, W2)
    slots = np.zeros_like(dx)
    slots[rd] = dx
    rX = backward.dispatch_backward(slots, disp["tok_off"], cfg.T, cfg.num_segments)
    for name, got, want, tol in (("dX", dX, rX, 4 * B), ("dW1", dW1, r1, 4 * B), ("dW2", dW2, r2, 4 * B),
                                 ("d_buf", d_buf[:A], r_buf, B + 64 * U), ("d_logits", d_l, r_l, B),
                                 ("d_w", d_w, r_w, B)):
        rel = np.linalg.norm(got.double().cpu().numpy() - want) / np.linalg.norm(want)
        print(f"[backward pass] {name}: {rel:.2e}", flush=True)
        assert rel <= tol, (name, rel)
    # the forward's views are untouched, so another pass gives the same bits
    before = [t.clone() for t in (d_buf, d_l, dX, dW1, dW2)]
    step()
    for a, b in zip(before, (d_buf, d_l, dX, dW1, dW2)):
        assert torch.equal(a, b)
    Y2 = torch.empty_like(Y)
    moe.layer_forward(p, g["X"], None, g["logits"], g["W1"], None, g["W2"], None, Y2, None, ws)
    assert torch.equal(Y, Y2)


def test_padded_owner_layout():
    """The rows of owner_gather (zero rows between the owners' groups), row r at slot r: the zero rows change nothing."""
    cfg = moe_synth.make_config("tiny", T=128, d=256, f=128, E_global=8, k=2, e_begin=0, e_end=4, num_segments=4, seed=6)
    inp = moe_synth.generate(cfg)
    idx, w, _ = oracle.route_topk(inp["logits"].numpy(), cfg.k)
    plan = moe.owner_plan(problem_of(cfg), idx, 1, 32, 2)
    R = plan["R"]
    p = problem_of(cfg, sched="auto", row_capacity=R)
    cap = moe.row_capacity(p)
    X = torch.zeros(cap, cfg.d, dtype=torch.bfloat16, device="cuda")
    moe.owner_gather(p, inp["X"].cuda(), None, torch.tensor(plan["row_src"], device="cuda"), X)
    dO = torch.randn(cap, cfg.d, generator=torch.Generator().manual_seed(1)).to(torch.bfloat16)
    dO[torch.tensor(np.flatnonzero(plan["row_src"] < 0))] = 0
    z = dict(dtype=torch.bfloat16, device="cuda")
    out = torch.empty(cap, cfg.d, **z), torch.empty(4, 2 * cfg.f, cfg.d, **z), torch.empty(4, cfg.d, cfg.f, **z)
    ws = moe.alloc_backward_workspace(p)
    moe.expert_backward(p, X, None, _i32(plan["expert_off"]), _i32(np.arange(cap)), inp["W1"].cuda(), inp["W2"].cuda(),
                        dO.cuda(), *out, ws)
    torch.cuda.synchronize()
    moe.check_workspace(p, ws)
    ops = (X.double().cpu().numpy()[:R], dO.double().numpy()[:R], plan["expert_off"], inp["W1"].double().numpy(),
           inp["W2"].double().numpy())
    got = [t.double().cpu().numpy() for t in out]
    _check((got[0][:R], *got[1:]), backward.expert_backward(*ops), _rounded_reference(*ops), _bounds(*ops), "padded")


@pytest.mark.parametrize("bad", ["src", "dst_high", "dst_negative", "offsets"])
def test_device_side_checks(bad):
    cfg, inp, disp, dO = _setup(CASES["odd_tokens"])
    p = problem_of(cfg, sched="auto")
    src, dst, off = _i32(disp["row_src"], cfg.cap), _i32(disp["row_dst"], cfg.cap), _i32(disp["offsets"])
    good = [t.clone() for t in (src, off, dst)]
    if bad == "src":
        src[0] = cfg.T * cfg.k
    elif bad == "dst_high":
        dst[disp["A"] - 1] = cfg.cap
    elif bad == "dst_negative":
        dst[3] = -5
    else:
        off[2] = off[1] - 1
    out = _outputs(cfg)
    ws = moe.alloc_backward_workspace(p)
    tail = (inp["W1"].cuda(), inp["W2"].cuda(), dO.cuda(), *out, ws)
    moe.expert_backward(p, inp["X"].cuda(), src, off, dst, *tail)
    torch.cuda.synchronize()
    with pytest.raises(moe.MoEError) as ei:
        moe.check_workspace(p, ws)
    assert ei.value.status == 1
    for t in out:
        assert torch.all(t == 3.0)
    moe.expert_backward(p, inp["X"].cuda(), *good, *tail)
    torch.cuda.synchronize()
    moe.check_workspace(p, ws)
    assert torch.isfinite(out[1].float()).all() and not torch.all(out[1] == 3.0)


def test_replayed_graph_beside_eager_calls():
    cfg, inp, disp, dO = _setup(CASES["segments"])
    p = problem_of(cfg, sched="auto")
    g = to_gpu(inp)
    src, dst, off = _i32(disp["row_src"], cfg.cap), _i32(disp["row_dst"], cfg.cap), _i32(disp["offsets"])
    d, out, eager = dO.cuda(), _outputs(cfg), _outputs(cfg)
    ws, ws2 = moe.alloc_backward_workspace(p), moe.alloc_backward_workspace(p)
    run = lambda o, s: moe.expert_backward(p, g["X"], src, off, dst, g["W1"], g["W2"], d, *o, s)  # noqa: E731
    run(out, ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run(out, ws)
    for i in range(3):
        d.copy_((dO * (1 + i)).to(torch.bfloat16))
        for t in (*out, *eager):
            t.zero_()
        graph.replay()
        run(eager, ws2)
        torch.cuda.synchronize()
        for a, b in zip(out, eager):
            assert torch.equal(a, b) and a.any()


@pytest.mark.parametrize("change", ["workspace", "dtype", "small", "fp8", "alias"])
def test_refusals(change):
    cfg, inp, disp, dO = _setup(CASES["one_token"])
    p = problem_of(cfg, sched="auto")
    src, dst, off = _i32(disp["row_src"], cfg.cap), _i32(disp["row_dst"], cfg.cap), _i32(disp["offsets"])
    out = list(_outputs(cfg))
    args = [inp["X"].cuda(), src, off, dst, inp["W1"].cuda(), inp["W2"].cuda(), dO.cuda(), *out,
            moe.alloc_backward_workspace(p)]
    err, status = ValueError, None
    if change == "workspace":
        args[-1], err, status = moe.alloc_workspace(p), moe.MoEError, 3
    elif change == "dtype":
        args[0] = args[0].float()
    elif change == "small":
        args[8] = args[8][:, :-1].contiguous()
    elif change == "alias":
        args[7], err, status = args[6], moe.MoEError, 1
    else:
        q = moe.make_problem(128, cfg.d, cfg.f, 4, 2, dtype="fp8_e4m3")
        with pytest.raises(moe.MoEError):
            moe.backward_workspace_size(q)
        p, err, status = q, (moe.MoEError, ValueError), None
    with pytest.raises(err) as ei:
        moe.expert_backward(p, *args)
    assert status is None or ei.value.status == status
    torch.cuda.synchronize()
    assert torch.all(out[1] == 3.0)
