"""The experts' products with 8-bit activation checkpoints: the forward pass
that leaves one, and the gradient that reads it.

Forward: the combine buffer is moe_expert_forward's, bit for bit. A value g of
the checkpoint is off by the sum's error, eg = d u (sum of magnitudes) with u =
2^-24, and by the rounding to the block's grid: half a step, or the distance to
127 steps if that is more. A block's scale is its largest magnitude's binade,
or the next one's if that lies within eg of the border.

Backward: against the formulas at the checkpoint's values, with a bound per
element (b = 2^-8 per rounding to bf16; the hardware's exp2 and reciprocal and
the products around them within 16 u (1 + |g|) of silu and 32 u (1 + |g|) of
its derivative):
  da         a sum of d products: eda = d u (sum of magnitudes)
  a          (16 u (1 + |g|) + b) |a|
  dg         |u D| eda + |da u| 32 u (1 + |g|) + b |dg|
  du         |silu| eda + |da| 16 u (1 + |g|) |silu| + b |du|
  dx, dW     the sum over the products of those errors, n u (sum of magnitudes)
             for n products, one more b
"""
import numpy as np
import pytest
import torch

import expert_grouped_gemm_amd as moe
import moe_synth
import oracle
from moe_cases import problem_of
from oracle import backward, int8

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
    dO = torch.randn(cfg.cap, cfg.d, generator=torch.Generator().manual_seed(seed)).to(torch.bfloat16)
    return cfg, inp, disp, dO


def _codes(rows, cols):
    return (torch.full((rows, cols), 85, dtype=torch.int8, device="cuda"),
            torch.full((rows, cols // 32), 85, dtype=torch.uint8, device="cuda"))


def _quantized(x):
    """x fp64 in MXINT8 by the oracle's codec, on the GPU, and its values."""
    c, s = int8.quantize_mxint8(x)
    return torch.tensor(c).cuda(), torch.tensor(s).cuda(), int8.decode_mxint8(c, s)


def _outputs(cfg):
    z = dict(dtype=torch.bfloat16, device="cuda")
    return (torch.full((cfg.cap, cfg.d), 3.0, **z), torch.full((cfg.E_local, 2 * cfg.f, cfg.d), 3.0, **z),
            torch.full((cfg.E_local, cfg.d, cfg.f), 3.0, **z))


def _products(X, off, W1):
    """g and u of every row, and the bound on an fp32 sum's error."""
    gu, e = np.zeros((X.shape[0], W1.shape[1])), np.zeros((X.shape[0], W1.shape[1]))
    for i in range(W1.shape[0]):
        r = slice(off[i], off[i + 1])
        gu[r] = X[r] @ W1[i].T
        e[r] = X.shape[1] * U * (np.abs(X[r]) @ np.abs(W1[i]).T)
    return gu, e


def _check_checkpoint(codes, scales, gu, err):
    """The kernel's codes and scale bytes against fp64 products."""
    top = np.abs(gu).reshape(gu.shape[0], -1, 32).max(axis=2)
    e_top = err.reshape(gu.shape[0], -1, 32).max(axis=2)
    binade = lambda v: np.maximum(np.frexp(np.maximum(v, 0))[1] + 126, 7)  # noqa: E731
    byte = scales.astype(np.int64)
    assert np.all((byte >= binade(top - e_top)) & (byte <= binade(top + e_top)) | (top <= e_top))
    step = np.exp2(byte - 133.0).repeat(32, 1)
    off = np.abs(int8.decode_mxint8(codes, scales) - gu)
    assert np.all(off <= np.maximum(step / 2, np.abs(gu) - 127 * step) + 2 * err), float((off / step).max())
    assert np.abs(codes.astype(np.int64)).max() <= 127


@pytest.mark.parametrize("kw", [dict(), dict(tiles="narrow"), dict(bf16_combine_buf=True, grid=5)])
@pytest.mark.parametrize("gather", [True, False])
@pytest.mark.parametrize("name", list(CASES))
def test_forward(name, gather, kw):
    print(f"[expert_forward_checkpoint] {name} gather={gather} {kw}", flush=True)
    cfg, inp, disp, _ = _setup(CASES[name])
    A, cap, off = disp["A"], cfg.cap, disp["offsets"]
    p = problem_of(cfg, sched="auto", **kw)
    tok = disp["row_src"] // cfg.k
    Xp = torch.zeros(cap, cfg.d, dtype=torch.bfloat16)
    Xp[:A] = inp["X"][torch.tensor(tok)]
    W1, W2, offs, dst = inp["W1"].cuda(), inp["W2"].cuda(), _i32(off), _i32(disp["row_dst"], cap)
    buf = dict(dtype=torch.bfloat16 if kw.get("bf16_combine_buf") else torch.float32, device="cuda")
    want, got = torch.full((cap, cfg.d), 5.0, **buf), torch.full((cap, cfg.d), 5.0, **buf)
    moe.expert_forward(p, Xp.cuda(), None, offs, dst, W1, None, W2, None, want, moe.alloc_workspace(p))
    gu, gus = _codes(cap, 2 * cfg.f)
    ws = moe.alloc_workspace(p)
    X, src = (inp["X"].cuda(), _i32(disp["row_src"], cap)) if gather else (Xp.cuda(), None)
    moe.expert_forward_checkpoint(p, X, src, offs, dst, W1, W2, gu, gus, got, ws)
    torch.cuda.synchronize()
    moe.check_workspace(p, ws)
    assert torch.equal(want, got)
    gu, gus = gu.cpu().numpy(), gus.cpu().numpy()
    assert np.all(gu[A:] == 85) and np.all(gus[A:] == 85)
    if A:
        _check_checkpoint(gu[:A], gus[:A], *_products(inp["X"].double().numpy()[tok], off, inp["W1"].double().numpy()))


def test_forward_of_bad_values():
    """A token with an infinity or a NaN poisons its own blocks of the checkpoint only; zeros give scale 1."""
    cfg, inp, disp, _ = _setup(CASES["odd_tokens"])
    X = inp["X"].clone()
    X[3, 7], X[5, 0], X[6] = float("inf"), float("nan"), 0.0
    p = problem_of(cfg, sched="auto")
    gu, gus = _codes(cfg.cap, 2 * cfg.f)
    out = torch.zeros(cfg.cap, cfg.d, device="cuda")
    moe.expert_forward_checkpoint(p, X.cuda(), _i32(disp["row_src"], cfg.cap), _i32(disp["offsets"]),
                                  _i32(disp["row_dst"], cfg.cap), inp["W1"].cuda(), inp["W2"].cuda(), gu, gus, out,
                                  moe.alloc_workspace(p))
    tok = disp["row_src"] // cfg.k
    gu, gus = gu.cpu().numpy()[:disp["A"]], gus.cpu().numpy()[:disp["A"]]
    bad = np.isin(tok, [3, 5])
    assert np.all(gus[bad] == 255) and np.all(gu[bad] == 0) and np.all(gus[~bad] != 255)
    assert np.all(gus[tok == 6] == 127) and np.all(gu[tok == 6] == 0)


def _reference(x, do, off, gu, W1, W2):
    """The gradients at given g and u, the same with the roundings to bf16 on the way, and the bounds."""
    f = W2.shape[2]
    exact = [np.zeros_like(x), np.zeros(W1.shape), np.zeros(W2.shape)]
    rounded, tol = [np.zeros_like(t) for t in exact], [np.zeros_like(t) for t in exact]
    for e in range(W1.shape[0]):
        r = slice(off[e], off[e + 1])
        n = off[e + 1] - off[e]
        X, D, w1, w2 = x[r], do[r], W1[e], W2[e]
        g, u = np.split(gu[r], 2, axis=1)
        with np.errstate(over="ignore"):
            s = 1 / (1 + np.exp(-g))
        silu, ds = g * s, s + g * s * (1 - s)
        da, eda = D @ w2, X.shape[1] * U * (np.abs(D) @ np.abs(w2))
        G = U * (1 + np.abs(g))
        a, ea = silu * u, (16 * G + B) * np.abs(silu * u)
        dh = np.concatenate([da * u * ds, da * silu], 1)
        edh = np.concatenate([np.abs(u * ds) * eda + np.abs(da * u) * 32 * G + B * np.abs(da * u * ds),
                              np.abs(silu) * eda + np.abs(da) * 16 * G * np.abs(silu) + B * np.abs(da * silu)], 1)
        m = np.abs(dh) + edh
        for k, (dhk, ak) in enumerate(((dh, a), (oracle.round_to_bf16(dh), oracle.round_to_bf16(a)))):
            to = rounded if k else exact
            to[0][r], to[1][e], to[2][e] = dhk @ w1, dhk.T @ X, D.T @ ak
        tol[0][r] = edh @ np.abs(w1) + 2 * f * U * (m @ np.abs(w1))
        tol[1][e] = edh.T @ np.abs(X) + n * U * (m.T @ np.abs(X))
        tol[2][e] = np.abs(D).T @ ea + n * U * (np.abs(D).T @ (np.abs(a) + ea))
    return exact, rounded, tol


def _check(got, ref, label):
    for name, g, x, rr, tol in zip(("dx", "dW1", "dW2"), got, *ref):
        err = np.abs(g - x)
        assert np.all(err <= tol + B * (np.abs(x) + tol) + 1e-30), (label, name, float((err - tol).max()))
        norm = np.linalg.norm(rr)
        if norm:  # one rounding of each output is left, and roundings on the way that fall the other way
            assert np.linalg.norm(g - rr) <= 1.1 * B * norm, (label, name)


def _gate_up(cfg, A, seed=6):
    """Gate and up values of their own (a gradient from a checkpoint takes what it is given)."""
    gu = np.random.default_rng(seed).normal(size=(cfg.cap, 2 * cfg.f)) * 1.7
    codes, scales, values = _quantized(gu)
    scales[A:] = 255  # rows of no expert are not read
    return codes, scales, values[:A]


@pytest.mark.parametrize("x8", [True, False])
@pytest.mark.parametrize("gather", [True, False])
@pytest.mark.parametrize("name", list(CASES))
def test_backward(name, gather, x8):
    print(f"[expert_backward_checkpoint] {name} gather={gather} x8={x8}", flush=True)
    cfg, inp, disp, dO = _setup(CASES[name])
    A, cap, off = disp["A"], cfg.cap, disp["offsets"]
    dO[A:] = float("nan")
    p = problem_of(cfg, sched="auto")
    tok = disp["row_src"] // cfg.k
    gu, gus, gu_values = _gate_up(cfg, A)
    if x8:
        X, Xs, x = _quantized(inp["X"].double().numpy())
    else:
        X, Xs, x = inp["X"].cuda(), None, inp["X"].double().numpy()
    src = _i32(disp["row_src"], cap)
    if not gather:
        pick = torch.tensor(np.concatenate([tok, np.zeros(cap - A, np.int64)])).cuda()
        X, Xs, src = X[pick], None if Xs is None else Xs[pick], None
        if Xs is not None:
            Xs[A:] = 255
    args = (X, Xs, src, _i32(off), _i32(disp["row_dst"], cap), gu, gus, inp["W1"].cuda(), inp["W2"].cuda(), dO.cuda())
    out = _outputs(cfg)
    ws = moe.alloc_checkpoint_workspace(p)
    ws.fill_(255)
    moe.expert_backward_checkpoint(p, *args, *out, ws)
    torch.cuda.synchronize()
    moe.check_workspace(p, ws)
    dxs, dW1, dW2 = (t.double().cpu().numpy() for t in out)
    ref = _reference(x[tok], dO.double().numpy()[disp["row_dst"]], off, gu_values, inp["W1"].double().numpy(),
                     inp["W2"].double().numpy())
    _check((dxs[disp["row_dst"]], dW1, dW2), ref, name)
    assert np.all(dxs[A:] == 3.0)
    again = _outputs(cfg)
    moe.expert_backward_checkpoint(p, *args, *again, ws)
    for a, b in zip(out, again):
        assert torch.equal(a, b)                 # the same bits on every call


@pytest.mark.parametrize("counts", [[1, 63, 64, 65], [0, 0, 257, 0], [127, 128, 129, 2], [256, 0, 31, 33]])
def test_rows_per_expert_around_the_tile_borders(counts):
    print(f"[checkpoint] counts {counts}", flush=True)
    A, d, f = sum(counts), 256, 128
    off = np.concatenate([[0], np.cumsum(counts)])
    rng = np.random.default_rng(A)
    g = torch.Generator().manual_seed(A)
    p = moe.make_problem(A, d, f, 4, 1, sched="auto")
    X, dO = (torch.randn(A, d, generator=g).to(torch.bfloat16) for _ in range(2))
    W1, W2 = (torch.randn(*s, generator=g).mul_(0.05).to(torch.bfloat16) for s in ((4, 2 * f, d), (4, d, f)))
    dst = rng.permutation(A)
    z = dict(device="cuda")
    (gu, gus), C = _codes(A, 2 * f), torch.empty(A, d, **z)
    ws = moe.alloc_checkpoint_workspace(p)
    moe.expert_forward_checkpoint(p, X.cuda(), None, _i32(off), _i32(dst), W1.cuda(), W2.cuda(), gu, gus, C, ws)
    x, w1, w2 = X.double().numpy(), W1.double().numpy(), W2.double().numpy()
    _check_checkpoint(gu.cpu().numpy(), gus.cpu().numpy(), *_products(x, off, w1))
    z["dtype"] = torch.bfloat16
    out = torch.empty(A, d, **z), torch.empty(4, 2 * f, d, **z), torch.empty(4, d, f, **z)
    moe.expert_backward_checkpoint(p, X.cuda(), None, None, _i32(off), _i32(dst), gu, gus, W1.cuda(), W2.cuda(),
                                   dO.cuda(), *out, ws)
    moe.check_workspace(p, ws)
    dxs, dW1, dW2 = (t.double().cpu().numpy() for t in out)
    values = int8.decode_mxint8(gu.cpu().numpy(), gus.cpu().numpy())
    _check((dxs[dst], dW1, dW2), _reference(x, dO.double().numpy()[dst], off, values, w1, w2), counts)


def test_rows_that_do_not_start_at_zero():
    """offsets[0] > 0: the rows before it belong to no expert."""
    A, d, f, first = 90, 128, 128, 7
    off = np.array([first, 40, 40, A])
    g = torch.Generator().manual_seed(8)
    p = moe.make_problem(A, d, f, 3, 1, sched="auto")
    dO = torch.randn(A, d, generator=g).to(torch.bfloat16)
    W1, W2 = (torch.randn(*s, generator=g).mul_(0.05).to(torch.bfloat16) for s in ((3, 2 * f, d), (3, d, f)))
    rng = np.random.default_rng(8)
    (X, Xs, x), (gu, gus, values) = _quantized(rng.normal(size=(A, d))), _quantized(rng.normal(size=(A, 2 * f)))
    Xs[:first] = 255
    gus[:first] = 255
    z = dict(dtype=torch.bfloat16, device="cuda")
    out = torch.full((A, d), 3.0, **z), torch.empty(3, 2 * f, d, **z), torch.empty(3, d, f, **z)
    ws = moe.alloc_checkpoint_workspace(p)
    moe.expert_backward_checkpoint(p, X, Xs, None, _i32(off), _i32(np.arange(A)), gu, gus, W1.cuda(), W2.cuda(),
                                   dO.cuda(), *out, ws)
    moe.check_workspace(p, ws)
    dxs, dW1, dW2 = (t.double().cpu().numpy() for t in out)
    assert np.all(dxs[:first] == 3.0)
    _check((dxs[first:], dW1, dW2), _reference(x[first:], dO.double().numpy()[first:], off - first, values[first:],
                                               W1.double().numpy(), W2.double().numpy()), "first")


def test_saturated_gates():
    """Gates far out on both sides: the derivative is 0 or 1 there, never NaN."""
    T, d, f = 40, 128, 128
    g = torch.Generator().manual_seed(2)
    W1, W2 = (torch.randn(1, *s, generator=g).to(torch.bfloat16) for s in ((2 * f, d), (d, f)))
    X, dO = (torch.randn(T, d, generator=g).to(torch.bfloat16) for _ in range(2))
    gu, gus, values = _quantized(np.random.default_rng(2).normal(size=(T, 2 * f)) * 300)
    p = moe.make_problem(T, d, f, 1, 1, sched="auto")
    z = dict(dtype=torch.bfloat16, device="cuda")
    out = torch.empty(T, d, **z), torch.empty(1, 2 * f, d, **z), torch.empty(1, d, f, **z)
    moe.expert_backward_checkpoint(p, X.cuda(), None, None, _i32([0, T]), _i32(np.arange(T)), gu, gus, W1.cuda(),
                                   W2.cuda(), dO.cuda(), *out, moe.alloc_checkpoint_workspace(p))
    _check([t.double().cpu().numpy() for t in out],
           _reference(X.double().numpy(), dO.double().numpy(), np.array([0, T]), values, W1.double().numpy(),
                      W2.double().numpy()), "saturated")


def test_training_step_run_together():
    """route -> dispatch -> forward with a checkpoint -> combine, the tokens kept in MXINT8, and back through the
    combine, the experts and the dispatch: every gradient against the formulas at the values that were kept, and
    against the layer's exact gradient with the checkpoint's rounding carried through."""
    cfg = moe_synth.make_config("tiny", T=384, d=512, f=256, E_global=8, k=2, e_begin=1, e_end=7, num_segments=2,
                                seed=3)
    inp = moe_synth.generate(cfg)
    g = {k: v.cuda().contiguous() for k, v in inp.items()}
    p = problem_of(cfg, sched="auto")
    ws = moe.alloc_checkpoint_workspace(p)
    v = moe.workspace_views(p, ws)
    cap = cfg.cap
    moe.route_topk(p, g["logits"], v["topk_idx"], v["topk_w"])
    moe.dispatch(p, g["X"], None, v["topk_idx"], v["topk_w"], v["counts"], v["offsets"], v["row_src"], v["row_dst"],
                 v["tok_off"], v["comb_w"], v["x_perm"], None, ws)
    gu, gus = _codes(cap, 2 * cfg.f)
    moe.expert_forward_checkpoint(p, g["X"], v["row_src"], v["offsets"], v["row_dst"], g["W1"], g["W2"], gu, gus,
                                  v["combine_buf"], ws)
    Y = torch.empty(cfg.T, cfg.d, dtype=torch.bfloat16, device="cuda")
    moe.combine(p, v["combine_buf"], v["tok_off"], v["comb_w"], Y)
    X8, Xs = _codes(cfg.T, cfg.d)
    moe.mxint8_quantize(g["X"], X8, Xs)
    dY = torch.randn(cfg.T, cfg.d, generator=torch.Generator().manual_seed(1)).to(torch.bfloat16).cuda()
    z = dict(dtype=torch.bfloat16, device="cuda")
    dO, dw = torch.zeros(cap, cfg.d, **z), torch.empty(cfg.T, cfg.k, device="cuda")
    dlog = torch.empty(cfg.T, cfg.E_global, device="cuda")
    moe.combine_backward(p, dY, v["combine_buf"], v["tok_off"], v["topk_idx"], v["topk_w"], dO, dw, dlog)
    dxs, dW1, dW2 = _outputs(cfg)
    moe.expert_backward_checkpoint(p, X8, Xs, v["row_src"], v["offsets"], v["row_dst"], gu, gus, g["W1"], g["W2"], dO,
                                   dxs, dW1, dW2, ws)
    dX = torch.empty(cfg.T, cfg.d, **z)
    dX32 = torch.empty(cfg.T, cfg.d, device="cuda")
    moe.dispatch_backward(p, dxs, v["tok_off"], dX, dX32)
    torch.cuda.synchronize()
    moe.check_workspace(p, ws)
    idx, w, _ = oracle.route_topk(inp["logits"].numpy(), cfg.k)
    disp = oracle.dispatch(idx, w, cfg.e_begin, cfg.e_end, cfg.num_segments)
    A, off, dst, tok = disp["A"], disp["offsets"], disp["row_dst"], disp["row_src"] // cfg.k
    W1, W2 = inp["W1"].double().numpy(), inp["W2"].double().numpy()
    values = int8.decode_mxint8(gu.cpu().numpy()[:A], gus.cpu().numpy()[:A])
    x8 = int8.decode_mxint8(X8.cpu().numpy(), Xs.cpu().numpy())
    do = dO.double().cpu().numpy()[dst]
    got = dxs.double().cpu().numpy()[dst], dW1.double().cpu().numpy(), dW2.double().cpu().numpy()
    ref = _reference(x8[tok], do, off, values, W1, W2)
    _check(got, ref, "together")
    want = backward.dispatch_backward(dxs.double().cpu().numpy(), disp["tok_off"], cfg.T, cfg.num_segments)
    got_dX = dX32.double().cpu().numpy()
    assert np.all(np.abs(got_dX - want) <= cfg.k * U * 4 * np.abs(want).max())
    # the exact gradient: g, u and x are off by eg, eu and ex (the checkpoint's rounding, from its own values)
    x = inp["X"].double().numpy()[tok]
    exact = backward.expert_backward(x, do, off, W1, W2)
    gu_x, _ = _products(x, off, W1)
    egu, ex = np.abs(values - gu_x), np.abs(x8[tok] - x)
    step = np.exp2(gus.cpu().numpy()[:A].astype(np.float64) - 133).repeat(32, 1)
    assert np.all(egu <= step + 1e-4)
    for e in range(cfg.E_local):
        r = slice(off[e], off[e + 1])
        ge, u = np.split(values[r], 2, axis=1)
        eg, eu = np.split(egu[r], 2, axis=1)
        s = 1 / (1 + np.exp(-ge))
        silu, ds, da = ge * s, s + ge * s * (1 - s), np.abs(do[r] @ W2[e])
        # |silu'| <= 1.1, |silu''| <= 0.5, to second order in the errors
        edh = np.concatenate([da * (np.abs(ds) * eu + 0.5 * eg * (np.abs(u) + eu)), da * 1.1 * eg], 1)
        dh = np.abs(np.concatenate([da * u * ds, da * silu], 1))
        edx = edh @ np.abs(W1[e])
        edW1 = edh.T @ np.abs(x[r]) + (dh + edh).T @ ex[r]
        edW2 = np.abs(do[r]).T @ (1.1 * eg * (np.abs(u) + eu) + np.abs(silu) * eu)
        for t, wt, extra in ((0, r, edx), (1, e, edW1), (2, e, edW2)):
            tol = ref[2][t][wt] + extra
            assert np.all(np.abs(got[t][wt] - exact[t][wt]) <= tol + B * (np.abs(exact[t][wt]) + tol))


@pytest.mark.parametrize("bad", ["src_high", "dst_negative", "offsets"])
@pytest.mark.parametrize("x8", [True, False])
@pytest.mark.parametrize("T", [77, 1500])
def test_device_side_checks(T, x8, bad):
    cfg, inp, disp, dO = _setup(dict(T=T, d=128, f=128, E_global=2, k=1))
    A, cap = disp["A"], cfg.cap
    p = problem_of(cfg, sched="auto")
    src, dst, off = _i32(disp["row_src"], cap), _i32(disp["row_dst"], cap), _i32(disp["offsets"])
    good = src.clone(), off.clone(), dst.clone()
    if bad == "src_high":
        src[10] = cfg.T * cfg.k
    elif bad == "dst_negative":
        dst[A // 2] = -1
    else:
        off[-1] = cap + 1
    ws = moe.alloc_checkpoint_workspace(p)
    gu, gus = _codes(cap, 2 * cfg.f)
    C = torch.full((cap, cfg.d), 5.0, device="cuda")
    X, W1, W2 = inp["X"].cuda(), inp["W1"].cuda(), inp["W2"].cuda()
    X8 = _quantized(inp["X"].double().numpy())[:2] if x8 else (X, None)
    out = _outputs(cfg)

    def forward(s, o, d):
        moe.expert_forward_checkpoint(p, X, s, o, d, W1, W2, gu, gus, C, ws)

    def backward_(s, o, d):
        moe.expert_backward_checkpoint(p, *X8, s, o, d, gu, gus, W1, W2, dO.cuda(), *out, ws)

    def expect_report():
        with pytest.raises(moe.MoEError) as ei:
            moe.check_workspace(p, ws)
        assert ei.value.status == 1
        moe.check_workspace(p, ws)

    forward(src, off, dst)
    expect_report()
    assert (gu == 85).all() and (gus == 85).all() and (C == 5.0).all()
    backward_(src, off, dst)
    expect_report()
    for t in out:
        assert (t == 3.0).all()
    forward(src, off, dst)  # its rejection is still reported after a backward pass that went well
    backward_(*good)
    expect_report()
    forward(*good)
    backward_(*good)
    moe.check_workspace(p, ws)
    for t in out:
        assert torch.isfinite(t).all()


@pytest.mark.parametrize("T", [300, 1300])
def test_replayed_graph_and_another_stream(T):
    """Both weight-gradient forms; the step captured once, replayed on new tokens and gradients."""
    cfg, inp, disp, dO = _setup(dict(T=T, d=256, f=128, E_global=2, k=1))
    p = problem_of(cfg, sched="auto")
    X, dO, W1, W2 = inp["X"].cuda(), dO.cuda(), inp["W1"].cuda(), inp["W2"].cuda()
    src, off, dst = _i32(disp["row_src"], cfg.cap), _i32(disp["offsets"]), _i32(disp["row_dst"], cfg.cap)
    (gu, gus), (X8, Xs), C = _codes(cfg.cap, 2 * cfg.f), _codes(T, cfg.d), torch.zeros(cfg.cap, cfg.d, device="cuda")
    out, ws = _outputs(cfg), moe.alloc_checkpoint_workspace(p)

    def run(s=None):
        moe.expert_forward_checkpoint(p, X, src, off, dst, W1, W2, gu, gus, C, ws, stream=s)
        moe.mxint8_quantize(X, X8, Xs, stream=s)
        moe.expert_backward_checkpoint(p, X8, Xs, src, off, dst, gu, gus, W1, W2, dO, *out, ws, stream=s)

    run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run()
    side = torch.cuda.Stream()
    for i in range(3):
        X.normal_()
        dO.normal_()
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in (C, gu, gus, *out)]
        for t in (C, gu, gus, *out):
            t.zero_()
        torch.cuda.synchronize()
        run(side if i == 1 else None)
        torch.cuda.synchronize()
        for a, b in zip(got, (C, gu, gus, *out)):
            assert torch.equal(a, b)
    moe.check_workspace(p, ws)


def test_grid_changes_no_bit():
    cfg, inp, disp, dO = _setup(CASES["odd_widths"])
    X8, Xs, _ = _quantized(inp["X"].double().numpy())
    gu, gus, _ = _gate_up(cfg, disp["A"])
    args = (X8, Xs, _i32(disp["row_src"], cfg.cap), _i32(disp["offsets"]), _i32(disp["row_dst"], cfg.cap), gu, gus,
            inp["W1"].cuda(), inp["W2"].cuda(), dO.cuda())
    ref = None
    for grid in (0, 1, 2, 7, 40):
        p = problem_of(cfg, sched="auto", grid=grid)
        out = _outputs(cfg)
        moe.expert_backward_checkpoint(p, *args, *out, moe.alloc_checkpoint_workspace(p))
        torch.cuda.synchronize()
        ref = ref or out
        for a, b in zip(ref, out):
            assert torch.equal(a, b), grid


def test_tile_trace_of_the_forward():
    """Every tile of both launches is recorded, Linear-1's before Linear-2's."""
    cfg, inp, disp, _ = _setup(CASES["segments"])
    p = problem_of(cfg, sched="auto", trace=True, tiles="narrow")
    (gu, gus), C, ws = _codes(cfg.cap, 2 * cfg.f), torch.zeros(cfg.cap, cfg.d, device="cuda"), moe.alloc_workspace(p)
    moe.expert_forward_checkpoint(p, inp["X"].cuda(), _i32(disp["row_src"], cfg.cap), _i32(disp["offsets"]),
                                  _i32(disp["row_dst"], cfg.cap), inp["W1"].cuda(), inp["W2"].cuda(), gu, gus, C, ws)
    torch.cuda.synchronize()
    tr = moe.tile_trace(p, ws)
    bands = int(np.sum((disp["counts"] + 255) // 256))
    assert np.sum(tr["kind"] == 1) == bands * (cfg.f // 64) and np.sum(tr["kind"] == 2) == bands * (cfg.d // 128)
    assert tr["t_end"][tr["kind"] == 1].max() <= tr["t_start"][tr["kind"] == 2].min()


def test_a_poisoned_block_of_the_checkpoint():
    """A NaN scale byte: the row's gradient and its expert's weight gradients are NaN, nothing else."""
    cfg, inp, disp, dO = _setup(CASES["odd_tokens"])
    A, off = disp["A"], disp["offsets"]
    gu, gus, _ = _gate_up(cfg, A)
    e = int(np.argmax(disp["counts"]))
    r = int(off[e])
    gus[r, 0] = 255
    gu[r, :32] = 0
    p = problem_of(cfg, sched="auto")
    out = _outputs(cfg)
    moe.expert_backward_checkpoint(p, inp["X"].cuda(), None, _i32(disp["row_src"], cfg.cap), _i32(off),
                                   _i32(disp["row_dst"], cfg.cap), gu, gus, inp["W1"].cuda(), inp["W2"].cuda(),
                                   dO.cuda(), *out, moe.alloc_checkpoint_workspace(p))
    dxs, dW1, dW2 = (t.cpu() for t in out)
    bad = torch.zeros(cfg.cap, dtype=torch.bool)
    bad[disp["row_dst"][r]] = True
    assert torch.equal(torch.isnan(dxs).all(1), bad) and torch.equal(torch.isnan(dxs).any(1), bad)
    for i in range(cfg.E_local):
        nan1, nan2 = torch.isnan(dW1[i]), torch.isnan(dW2[i])
        if i != e:
            assert not nan1.any() and not nan2.any()
        else:  # gate columns 0 .. 31: their a, dg and du
            assert nan1[:32].all() and nan1[cfg.f:cfg.f + 32].all() and nan2[:, :32].all()
            assert not nan1[32:cfg.f].any() and not nan1[cfg.f + 32:].any() and not nan2[:, 32:].any()


def test_refused_by_the_binding():
    cfg, inp, disp, dO = _setup(CASES["odd_tokens"])
    p = problem_of(cfg, sched="auto")
    src, off, dst = _i32(disp["row_src"], cfg.cap), _i32(disp["offsets"]), _i32(disp["row_dst"], cfg.cap)
    X, W1, W2, dO = inp["X"].cuda(), inp["W1"].cuda(), inp["W2"].cuda(), dO.cuda()
    X8, Xs, _ = _quantized(inp["X"].double().numpy())
    (gu, gus), C, out, ws = _codes(cfg.cap, 2 * cfg.f), torch.zeros(cfg.cap, cfg.d, device="cuda"), _outputs(cfg), \
        moe.alloc_checkpoint_workspace(p)
    for bad in (dict(X=X8), dict(gu=gu[:-1]), dict(gus=gus[:-1]), dict(gu=gu.view(torch.uint8)), dict(C=C.bfloat16())):
        a = dict(dict(X=X, gu=gu, gus=gus, C=C), **bad)
        with pytest.raises(ValueError):
            moe.expert_forward_checkpoint(p, a["X"], src, off, dst, W1, W2, a["gu"], a["gus"], a["C"], ws)
    for bad in (dict(X=X), dict(Xs=None), dict(Xs=Xs[:-1]), dict(gus=gus.char()), dict(gu=gu[:-1])):
        a = dict(dict(X=X8, Xs=Xs, gu=gu, gus=gus), **bad)
        with pytest.raises(ValueError):
            moe.expert_backward_checkpoint(p, a["X"], a["Xs"], src, off, dst, a["gu"], a["gus"], W1, W2, dO, *out, ws)
    with pytest.raises(moe.MoEError) as ei:
        moe.expert_backward_checkpoint(p, X8, Xs, src, off, dst, gu, gus, W1, W2, dO, *out, ws[:moe.workspace_size(p)])
    assert ei.value.status == 3
