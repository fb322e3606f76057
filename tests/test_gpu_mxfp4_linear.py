"""The experts' Linears on MXFP4 rows and weights against fp64 products of the
decoded operands.

Tolerances, per element: a product of two decoded values is exact in fp32, so
a sum of K of them is off by at most K u of the sum of magnitudes (u = 2^-24),
in whatever order. linear2 returns that sum (and one rounding, 2^-8, to a bf16
buffer). linear1: with errors eg, eu of gate and up, |silu'| <= 1.1 and the
hardware's exp2, reciprocal and the products around them within 16 u of silu's
value times (1 + |g|) (an argument's rounding scales with the argument),
  |H - ref| <= 1.1 |u| eg + |silu(g)| eu + 16 u (1 + |g|) |ref| + 2^-8 |ref|.
"""
import numpy as np
import pytest
import torch

import expert_grouped_gemm_amd as moe
import moe_synth
import oracle
from moe_cases import problem_of

pytestmark = pytest.mark.gpu

U, B = 2.0 ** -24, 2.0 ** -8

CASES = {
    "one_token": dict(T=1, d=128, f=128, E_global=4, k=2),
    "half_slices": dict(T=70, d=384, f=128, E_global=8, k=2, e_begin=1, e_end=6),
    "odd_rows": dict(T=333, d=256, f=640, E_global=16, k=4, e_begin=0, e_end=8),
    "bands": dict(T=700, d=512, f=384, E_global=2, k=1),
    "full_bands_long_k": dict(T=600, d=2048, f=1664, E_global=1, k=1),
    "many_tiles": dict(T=1200, d=1024, f=6400, E_global=4, k=2),
    "long_k": dict(T=40, d=7168, f=256, E_global=64, k=8, e_begin=0, e_end=8),
    "empty_experts": dict(T=3, d=640, f=256, E_global=256, k=2, e_begin=0, e_end=128),
    "none_local": dict(T=2, d=128, f=128, E_global=512, k=1, e_begin=511, e_end=512),
}


def _rand_mx(g, *shape):
    codes = torch.randint(0, 256, (*shape[:-1], shape[-1] // 2), generator=g, dtype=torch.uint8)
    scales = torch.randint(118, 128, (*shape[:-1], shape[-1] // 32), generator=g, dtype=torch.uint8)
    return codes, scales


def _decode(c, s):
    return oracle.decode_mxfp4(c.reshape(-1, c.shape[-1]).numpy(), s.reshape(-1, s.shape[-1]).numpy()).reshape(
        *c.shape[:-1], -1)


def _i32(x, cap=None):
    x = np.asarray(x)
    if cap is not None:
        x = np.concatenate([x, np.zeros(cap - x.size, x.dtype)])
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _setup(case, seed=11):
    cfg = moe_synth.make_config("tiny", **{**dict(e_begin=0, e_end=case["E_global"]), **case})
    rng = np.random.default_rng(seed)
    idx, w, _ = oracle.route_topk(rng.normal(size=(cfg.T, cfg.E_global)).astype(np.float32), cfg.k)
    return cfg, oracle.dispatch(idx, w, cfg.e_begin, cfg.e_end), torch.Generator().manual_seed(seed)


def _ref_linear1(X, W1, disp, cfg):
    A, f = disp["A"], cfg.f
    ref, tol = np.zeros((A, f)), np.zeros((A, f))
    for e in range(cfg.E_local):
        r = slice(disp["offsets"][e], disp["offsets"][e + 1])
        x = X[disp["row_src"][r] // cfg.k]
        g, u = np.split(x @ W1[e].T, 2, axis=1)
        eg, eu = np.split(cfg.d * U * (np.abs(x) @ np.abs(W1[e]).T), 2, axis=1)
        silu = g / (1 + np.exp(-g))
        ref[r] = silu * u
        tol[r] = 1.1 * np.abs(u) * eg + np.abs(silu) * eu + (16 * U * (1 + np.abs(g)) + B) * np.abs(ref[r])
    return ref, tol + 1e-30


@pytest.mark.parametrize("tiles", ["auto", "narrow"])
@pytest.mark.parametrize("gather", [True, False])
@pytest.mark.parametrize("name", list(CASES))
def test_linear1(name, gather, tiles):
    print(f"[mxfp4_linear1] {name} gather={gather} {tiles}", flush=True)
    cfg, disp, g = _setup(CASES[name])
    A, cap = disp["A"], cfg.cap
    x, xs = _rand_mx(g, cfg.T, cfg.d)
    w, ws_ = _rand_mx(g, cfg.E_local, 2 * cfg.f, cfg.d)
    p = problem_of(cfg, sched="auto", tiles=tiles)
    H = torch.full((cap, cfg.f), 5.0, dtype=torch.bfloat16, device="cuda")
    ws = moe.alloc_workspace(p)
    rows, src = (x, xs), _i32(disp["row_src"], cap)
    if not gather:
        pick = torch.tensor(np.concatenate([disp["row_src"] // cfg.k, np.zeros(cap - A, np.int64)]))
        rows, src = (x[pick], xs[pick]), None
    moe.mxfp4_linear1(p, rows[0].cuda(), rows[1].cuda(), src, _i32(disp["offsets"]), w.cuda(), ws_.cuda(), H, ws)
    torch.cuda.synchronize()
    moe.check_workspace(p, ws)
    ref, tol = _ref_linear1(_decode(x, xs), _decode(w, ws_), disp, cfg)
    got = H.double().cpu().numpy()
    assert np.all(np.abs(got[:A] - ref) <= tol), np.max(np.abs(got[:A] - ref) - tol)
    assert np.all(got[A:] == 5.0)


@pytest.mark.parametrize("tiles", ["auto", "narrow"])
@pytest.mark.parametrize("bf16_buf", [False, True])
@pytest.mark.parametrize("name", list(CASES))
def test_linear2(name, bf16_buf, tiles):
    print(f"[mxfp4_linear2] {name} bf16_buf={bf16_buf} {tiles}", flush=True)
    cfg, disp, g = _setup(CASES[name])
    A, cap = disp["A"], cfg.cap
    h, hs = _rand_mx(g, cap, cfg.f)
    w, ws_ = _rand_mx(g, cfg.E_local, cfg.d, cfg.f)
    p = problem_of(cfg, sched="auto", tiles=tiles, bf16_combine_buf=bf16_buf)
    C = torch.full((cap, cfg.d), 5.0, dtype=torch.bfloat16 if bf16_buf else torch.float32, device="cuda")
    ws = moe.alloc_workspace(p)
    moe.mxfp4_linear2(p, h.cuda(), hs.cuda(), _i32(disp["offsets"]), _i32(disp["row_dst"], cap), w.cuda(), ws_.cuda(),
                      C, ws)
    torch.cuda.synchronize()
    moe.check_workspace(p, ws)
    H, W = _decode(h, hs), _decode(w, ws_)
    got = C.double().cpu().numpy()
    for e in range(cfg.E_local):
        r = slice(disp["offsets"][e], disp["offsets"][e + 1])
        ref, tol = H[r] @ W[e].T, cfg.f * U * (np.abs(H[r]) @ np.abs(W[e]).T)
        if bf16_buf:
            tol = tol + B * (np.abs(ref) + tol)
        assert np.all(np.abs(got[disp["row_dst"][r]] - ref) <= tol), e
    assert np.all(got[A:] == 5.0)


def test_poisoned_blocks_reach_their_products_only():
    cfg, disp, g = _setup(CASES["odd_rows"])
    x, xs = _rand_mx(g, cfg.T, cfg.d)
    w, ws_ = _rand_mx(g, cfg.E_local, 2 * cfg.f, cfg.d)
    xs[7, 3] = 255                # one block of token 7
    ws_[2, cfg.f + 5, 1] = 255    # the up row of column 5 of local expert 2
    p = problem_of(cfg, sched="auto")
    H = torch.zeros(cfg.cap, cfg.f, dtype=torch.bfloat16, device="cuda")
    moe.mxfp4_linear1(p, x.cuda(), xs.cuda(), _i32(disp["row_src"], cfg.cap), _i32(disp["offsets"]), w.cuda(),
                      ws_.cuda(), H, moe.alloc_workspace(p))
    want = np.zeros((disp["A"], cfg.f), bool)
    want[disp["row_src"] // cfg.k == 7] = True
    want[disp["offsets"][2]:disp["offsets"][3], 5] = True
    np.testing.assert_array_equal(torch.isnan(H).cpu().numpy()[:disp["A"]], want)


def test_w4a4_layer_run_together():
    """quantise -> linear1 -> quantise -> linear2 -> combine on the routing and dispatch of the same layer, each step
    against fp64 of its own inputs and the result against the composition of the decoded steps."""
    cfg = moe_synth.make_config("tiny", T=512, d=512, f=384, E_global=16, k=4, e_begin=2, e_end=12, num_segments=4,
                                seed=9)
    inp = moe_synth.generate(cfg)
    g = {k: v.cuda().contiguous() for k, v in inp.items()}
    p = problem_of(cfg, sched="auto")
    ws = moe.alloc_workspace(p)
    v = moe.workspace_views(p, ws)
    cap, El = cfg.cap, cfg.E_local

    def quant(x):
        c = torch.empty(*x.shape[:-1], x.shape[-1] // 2, dtype=torch.uint8, device="cuda")
        s = torch.empty(*x.shape[:-1], x.shape[-1] // 32, dtype=torch.uint8, device="cuda")
        moe.mxfp4_quantize(x, c, s)
        return c, s

    moe.route_topk(p, g["logits"], v["topk_idx"], v["topk_w"])
    moe.dispatch(p, g["X"], None, v["topk_idx"], v["topk_w"], v["counts"], v["offsets"], v["row_src"], v["row_dst"],
                 v["tok_off"], v["comb_w"], v["x_perm"], None, ws)
    torch.cuda.synchronize()
    A = int(v["offsets"][-1])
    v["row_src"][A:] = 0
    v["row_dst"][A:] = 0
    xq, w1, w2 = quant(g["X"]), quant(g["W1"]), quant(g["W2"])
    H = torch.zeros(cap, cfg.f, dtype=torch.bfloat16, device="cuda")
    moe.mxfp4_linear1(p, *xq, v["row_src"], v["offsets"], *w1, H, ws)
    hq = quant(H)
    moe.mxfp4_linear2(p, *hq, v["offsets"], v["row_dst"], *w2, v["combine_buf"], ws)
    Y = torch.empty(cfg.T, cfg.d, dtype=torch.bfloat16, device="cuda")
    Y32 = torch.empty(cfg.T, cfg.d, device="cuda")
    moe.combine(p, v["combine_buf"], v["tok_off"], v["comb_w"], Y, Y32)
    torch.cuda.synchronize()
    moe.check_workspace(p, ws)
    idx, w, _ = oracle.route_topk(inp["logits"].numpy(), cfg.k)
    disp = oracle.dispatch(idx, w, cfg.e_begin, cfg.e_end, cfg.num_segments)
    ref, tol = _ref_linear1(_decode(*(t.cpu() for t in xq)), _decode(*(t.cpu() for t in w1)), disp, cfg)
    assert np.all(np.abs(H.double().cpu().numpy()[:A] - ref) <= tol)
    hd, w2d = _decode(*(t.cpu() for t in hq)), _decode(*(t.cpu() for t in w2))
    Yref, mag = np.zeros((cfg.T, cfg.d)), np.zeros((cfg.T, cfg.d))
    for e in range(El):
        for r in range(disp["offsets"][e], disp["offsets"][e + 1]):
            a = disp["row_src"][r]
            q, gate = oracle.y_row_of_token(a // cfg.k, cfg.T, cfg.num_segments), float(w.reshape(-1)[a])
            Yref[q] += gate * (w2d[e] @ hd[r])
            mag[q] += gate * (np.abs(w2d[e]) @ np.abs(hd[r]))
    # f products per expert, k gates (fp32, off by 8 u with their softmax) and sums
    assert np.all(np.abs(Y32.double().cpu().numpy() - Yref) <= (cfg.f + cfg.k + 8) * U * mag + 1e-30)


@pytest.mark.parametrize("bad", ["src_high", "src_negative", "dst_high", "offsets"])
def test_device_side_checks(bad):
    cfg, disp, g = _setup(CASES["odd_rows"])
    p = problem_of(cfg, sched="auto")
    x, xs = _rand_mx(g, cfg.T, cfg.d)
    w1, w1s = _rand_mx(g, cfg.E_local, 2 * cfg.f, cfg.d)
    h, hs = _rand_mx(g, cfg.cap, cfg.f)
    w2, w2s = _rand_mx(g, cfg.E_local, cfg.d, cfg.f)
    src, dst, off = _i32(disp["row_src"], cfg.cap), _i32(disp["row_dst"], cfg.cap), _i32(disp["offsets"])
    good = src.clone(), dst.clone(), off.clone()
    if bad == "src_high":
        src[10] = cfg.T * cfg.k
    elif bad == "src_negative":
        src[disp["A"] - 1] = -1
    elif bad == "dst_high":
        dst[disp["A"] // 2] = cfg.cap
    else:
        off[-1] = cfg.cap + 1
    ws = moe.alloc_workspace(p)
    H = torch.full((cfg.cap, cfg.f), 5.0, dtype=torch.bfloat16, device="cuda")
    C = torch.full((cfg.cap, cfg.d), 5.0, device="cuda")

    def one(s, o):
        moe.mxfp4_linear1(p, x.cuda(), xs.cuda(), s, o, w1.cuda(), w1s.cuda(), H, ws)

    def two(t, o):
        moe.mxfp4_linear2(p, h.cuda(), hs.cuda(), o, t, w2.cuda(), w2s.cuda(), C, ws)

    for call, out in ((lambda: one(src, off), H), (lambda: two(dst, off), C)):
        call()
        torch.cuda.synchronize()
        reached = bad == "offsets" or (bad.startswith("src")) == (out is H)
        if reached:
            with pytest.raises(moe.MoEError) as ei:
                moe.check_workspace(p, ws)
            assert ei.value.status == 1
            assert torch.all(out == 5.0)
        else:
            moe.check_workspace(p, ws)
    one(good[0], good[2])
    moe.check_workspace(p, ws)
    assert torch.isfinite(H).all() and not torch.all(H[:disp["A"]] == 5.0)


def test_rows_past_the_last_are_not_looked_at():
    """Indices behind the last row may hold anything."""
    cfg, disp, g = _setup(CASES["half_slices"])
    p = problem_of(cfg, sched="auto")
    x, xs = _rand_mx(g, cfg.T, cfg.d)
    w, ws_ = _rand_mx(g, cfg.E_local, 2 * cfg.f, cfg.d)
    src = _i32(disp["row_src"], cfg.cap)
    src[disp["A"]:] = 2 ** 31 - 1
    ws = moe.alloc_workspace(p)
    H = torch.zeros(cfg.cap, cfg.f, dtype=torch.bfloat16, device="cuda")
    moe.mxfp4_linear1(p, x.cuda(), xs.cuda(), src, _i32(disp["offsets"]), w.cuda(), ws_.cuda(), H, ws)
    moe.check_workspace(p, ws)


def test_grid_and_raster_change_no_bit():
    cfg, disp, g = _setup(CASES["half_slices"])
    (x, xs), (w, ws_) = _rand_mx(g, cfg.T, cfg.d), _rand_mx(g, cfg.E_local, 2 * cfg.f, cfg.d)
    ref = None
    for kw in (dict(), dict(grid=1), dict(grid=2), dict(grid=9), dict(tiles="narrow"), dict(band_major=True)):
        p = problem_of(cfg, sched="auto", **kw)
        H = torch.zeros(cfg.cap, cfg.f, dtype=torch.bfloat16, device="cuda")
        moe.mxfp4_linear1(p, x.cuda(), xs.cuda(), _i32(disp["row_src"], cfg.cap), _i32(disp["offsets"]), w.cuda(),
                          ws_.cuda(), H, moe.alloc_workspace(p))
        torch.cuda.synchronize()
        ref = H if ref is None else ref
        assert torch.equal(ref, H), kw


def test_replayed_graph():
    cfg, disp, g = _setup(CASES["odd_rows"])
    p = problem_of(cfg, sched="auto")
    (x, xs), (w, ws_) = _rand_mx(g, cfg.T, cfg.d), _rand_mx(g, cfg.E_local, 2 * cfg.f, cfg.d)
    x, xs, w, ws_ = (t.cuda() for t in (x, xs, w, ws_))
    src, off, ws = _i32(disp["row_src"], cfg.cap), _i32(disp["offsets"]), moe.alloc_workspace(p)
    H = torch.zeros(cfg.cap, cfg.f, dtype=torch.bfloat16, device="cuda")
    run = lambda: moe.mxfp4_linear1(p, x, xs, src, off, w, ws_, H, ws)  # noqa: E731
    run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run()
    for i in range(3):
        x.random_(0, 256)
        H.zero_()
        graph.replay()
        torch.cuda.synchronize()
        got = H.clone()
        H.zero_()
        run()
        torch.cuda.synchronize()
        assert torch.equal(got, H)
