"""The experts' Linears on 8-bit integers against fp64 products of the operands.

Tolerances, per element: the sums over K are exact integers below 2^31, so an
output is one rounding to fp32 and two products away from its value, 3 u (u =
2^-24; 4 u with the products of those terms). linear1: with such errors of gate
and up, |silu'| <= 1.1 and the hardware's exp2, reciprocal and the products
around them within 16 u of silu's value times (1 + |g|) (an argument's rounding
scales with the argument), the value before its rounding is off by
  e = 4 u (1.1 |u g| + |ref|) + 16 u (1 + |g|) |ref|.
Rounding a value v to bf16 moves it by up to half a step, 2^-8 |v| (met where v
lies just above a power of two), and |v| <= |ref| + e: so by 2^-8 (|ref| + e),
not 2^-8 |ref|.
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
    "one_token_wide": dict(T=1, d=2304, f=1408, E_global=8, k=3),
    "few_tokens": dict(T=5, d=1152, f=2176, E_global=4, k=2),
    "odd_blocks": dict(T=70, d=384, f=128, E_global=8, k=2, e_begin=1, e_end=6),
    "odd_rows": dict(T=333, d=256, f=640, E_global=16, k=4, e_begin=0, e_end=8),
    "bands": dict(T=700, d=512, f=384, E_global=2, k=1),
    "full_bands_long_k": dict(T=600, d=2048, f=1664, E_global=1, k=1),
    "many_tiles": dict(T=1200, d=1024, f=6400, E_global=4, k=2),
    "long_k": dict(T=40, d=7168, f=256, E_global=64, k=8, e_begin=0, e_end=8),
    "empty_experts": dict(T=3, d=640, f=256, E_global=256, k=2, e_begin=0, e_end=128),
    "none_local": dict(T=2, d=128, f=128, E_global=512, k=1, e_begin=511, e_end=512),
}


def _rand(g, *shape):
    codes = torch.randint(-128, 128, shape, generator=g, dtype=torch.int8)
    return codes, torch.rand(shape[:-1], generator=g) * 2e-3 + 1e-4


class _Scaled:
    """Codes and row scales: products sum the whole codes, exactly, before they are scaled (sums of the scaled values
    would leave fp64 noise where a sum is zero)."""

    def __init__(self, c, s):
        self.c, self.s = c.cpu().double().numpy(), s.cpu().double().numpy()

    def __getitem__(self, i):
        part = object.__new__(_Scaled)
        part.c, part.s = self.c[i], self.s[i]
        return part

    def times(self, w):
        return (self.c @ w.c.T) * np.multiply.outer(self.s, w.s)


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
        g, u = np.split(X[disp["row_src"][r] // cfg.k].times(W1[e]), 2, axis=1)
        ref[r] = g / (1 + np.exp(-g)) * u
        tol[r] = 4 * U * (1.1 * np.abs(u * g) + np.abs(ref[r])) + 16 * U * (1 + np.abs(g)) * np.abs(ref[r])
    return ref, tol + B * (np.abs(ref) + tol) + 1e-30


@pytest.mark.parametrize("tiles", ["auto", "narrow"])
@pytest.mark.parametrize("gather", [True, False])
@pytest.mark.parametrize("name", list(CASES))
def test_linear1(name, gather, tiles):
    print(f"[int8_linear1] {name} gather={gather} {tiles}", flush=True)
    cfg, disp, g = _setup(CASES[name])
    A, cap = disp["A"], cfg.cap
    x, xs = _rand(g, cfg.T, cfg.d)
    w, ws_ = _rand(g, cfg.E_local, 2 * cfg.f, cfg.d)
    p = problem_of(cfg, sched="auto", tiles=tiles)
    H = torch.full((cap, cfg.f), 5.0, dtype=torch.bfloat16, device="cuda")
    ws = moe.alloc_workspace(p)
    rows, src = (x, xs), _i32(disp["row_src"], cap)
    if not gather:
        pick = torch.tensor(np.concatenate([disp["row_src"] // cfg.k, np.zeros(cap - A, np.int64)]))
        rows, src = (x[pick], xs[pick]), None
    moe.int8_linear1(p, rows[0].cuda(), rows[1].cuda(), src, _i32(disp["offsets"]), w.cuda(), ws_.cuda(), H, ws)
    torch.cuda.synchronize()
    moe.check_workspace(p, ws)
    ref, tol = _ref_linear1(_Scaled(x, xs), _Scaled(w, ws_), disp, cfg)
    got = H.double().cpu().numpy()
    assert np.all(np.abs(got[:A] - ref) <= tol), np.max(np.abs(got[:A] - ref) - tol)
    assert np.all(got[A:] == 5.0)


@pytest.mark.parametrize("tiles", ["auto", "narrow"])
@pytest.mark.parametrize("bf16_buf", [False, True])
@pytest.mark.parametrize("name", list(CASES))
def test_linear2(name, bf16_buf, tiles):
    print(f"[int8_linear2] {name} bf16_buf={bf16_buf} {tiles}", flush=True)
    cfg, disp, g = _setup(CASES[name])
    A, cap = disp["A"], cfg.cap
    h, hs = _rand(g, cap, cfg.f)
    w, ws_ = _rand(g, cfg.E_local, cfg.d, cfg.f)
    p = problem_of(cfg, sched="auto", tiles=tiles, bf16_combine_buf=bf16_buf)
    C = torch.full((cap, cfg.d), 5.0, dtype=torch.bfloat16 if bf16_buf else torch.float32, device="cuda")
    ws = moe.alloc_workspace(p)
    moe.int8_linear2(p, h.cuda(), hs.cuda(), _i32(disp["offsets"]), _i32(disp["row_dst"], cap), w.cuda(), ws_.cuda(),
                     C, ws)
    torch.cuda.synchronize()
    moe.check_workspace(p, ws)
    H, W = _Scaled(h, hs), _Scaled(w, ws_)
    got = C.double().cpu().numpy()
    for e in range(cfg.E_local):
        r = slice(disp["offsets"][e], disp["offsets"][e + 1])
        ref = H[r].times(W[e])
        tol = 4 * U * np.abs(ref)
        tol += B * (np.abs(ref) + tol) * bf16_buf + 1e-30
        assert np.all(np.abs(got[disp["row_dst"][r]] - ref) <= tol), e
    assert np.all(got[A:] == 5.0)


@pytest.mark.parametrize("T", [3, 40])
@pytest.mark.parametrize("first", [True, False])
def test_longest_sums(first, T):
    """K just below 2^17: sums of -128 x -128 reach 2^31 - 2^21, and of 127 x -128 the same below zero."""
    K = (1 << 17) - 128
    p = moe.make_problem(T, K if first else 128, 128 if first else K, 1, 1, sched="auto")
    x = torch.full((T, K), -128, dtype=torch.int8, device="cuda")
    x[1] = 127
    x[2, ::2] = 127
    w = torch.full((1, 256 if first else 128, K), -128, dtype=torch.int8, device="cuda")
    xs = torch.full((T,), 2.0 ** -16, device="cuda")
    ws_ = torch.full((1, w.shape[1]), 2.0 ** -15, device="cuda")
    sums = x.double().sum(1) * -128 * 2.0 ** -31
    ws, off = moe.alloc_workspace(p), _i32([0, T])
    if first:
        H = torch.empty(T, 128, dtype=torch.bfloat16, device="cuda")
        moe.int8_linear1(p, x, xs, None, off, w, ws_, H, ws)
        ref = sums * sums / (1 + torch.exp(-sums))
        got, tol = H.double(), 2 * B * ref.abs()
    else:
        C = torch.empty(T, 128, device="cuda")
        moe.int8_linear2(p, x, xs, off, _i32(np.arange(T)), w, ws_, C, ws)
        ref, got = sums, C.double()
        tol = 4 * U * ref.abs()
    moe.check_workspace(p, ws)
    assert ((got - ref[:, None]).abs() <= tol[:, None]).all()


@pytest.mark.parametrize("counts", [[1, 7, 8, 9], [0, 15, 16, 17], [31, 0, 32, 33], [0, 0, 64, 0], [65, 1, 0, 300]])
@pytest.mark.parametrize("E", [4, 300])
def test_rows_per_expert_around_the_borders(counts, E):
    """Row counts around the passes of the kernel for few rows (E = 300: the mean says few, whatever the counts) and the
    tiles of the other, offsets that do not start at zero, slots in any order."""
    d, f, first = 384, 256, 3
    A = first + sum(counts)
    off = np.zeros(E + 1, np.int64)
    off[:] = first + sum(counts)
    at = sorted(np.random.default_rng(E).choice(E, 4, replace=False))
    full = np.zeros(E, np.int64)
    full[at] = counts
    off = first + np.concatenate([[0], np.cumsum(full)])
    p = moe.make_problem(A, d, f, E, 1, sched="auto")
    g = torch.Generator().manual_seed(A)
    (x, xs), (w, ws_) = _rand(g, A, d), _rand(g, E, 2 * f, d)
    (h, hs), (w2, w2s) = _rand(g, A, f), _rand(g, E, d, f)
    H = torch.full((A, f), 5.0, dtype=torch.bfloat16, device="cuda")
    C = torch.full((A, d), 5.0, device="cuda")
    ws, dst = moe.alloc_workspace(p), np.random.default_rng(A).permutation(A)
    moe.int8_linear1(p, x.cuda(), xs.cuda(), None, _i32(off), w.cuda(), ws_.cuda(), H, ws)
    moe.int8_linear2(p, h.cuda(), hs.cuda(), _i32(off), _i32(dst), w2.cuda(), w2s.cuda(), C, ws)
    moe.check_workspace(p, ws)
    v = moe.workspace_views(p, ws)
    assert int(v["meta"][0]) == A and int(v["meta"][1]) == sum(-(-c // 256) for c in counts)
    H, C = H.double().cpu().numpy(), C.double().cpu().numpy()
    assert np.all(H[:first] == 5.0) and np.all(C[dst[:first]] == 5.0)
    for e in at:
        r = slice(off[e], off[e + 1])
        gate, u = np.split(_Scaled(x, xs)[r].times(_Scaled(w, ws_)[e]), 2, axis=1)
        ref = gate / (1 + np.exp(-gate)) * u
        tol = 4 * U * (1.1 * np.abs(u * gate) + np.abs(ref)) + 16 * U * (1 + np.abs(gate)) * np.abs(ref)
        assert np.all(np.abs(H[r] - ref) <= tol + B * (np.abs(ref) + tol) + 1e-30), e
        ref = _Scaled(h, hs)[r].times(_Scaled(w2, w2s)[e])
        assert np.all(np.abs(C[dst[r]] - ref) <= 4 * U * np.abs(ref) + 1e-30), e


@pytest.mark.parametrize("name", ["odd_rows", "few_tokens"])
def test_poisoned_scales_reach_their_products_only(name):
    cfg, disp, g = _setup(CASES[name])
    t, e = (7, 2) if name == "odd_rows" else (3, 1)
    x, xs = _rand(g, cfg.T, cfg.d)
    w, ws_ = _rand(g, cfg.E_local, 2 * cfg.f, cfg.d)
    xs[t] = float("nan")              # one token
    x[t] = 0                          # ... as the quantiser leaves a row it cannot hold
    ws_[e, cfg.f + 5] = float("nan")  # the up row of column 5 of one local expert
    p = problem_of(cfg, sched="auto")
    H = torch.zeros(cfg.cap, cfg.f, dtype=torch.bfloat16, device="cuda")
    moe.int8_linear1(p, x.cuda(), xs.cuda(), _i32(disp["row_src"], cfg.cap), _i32(disp["offsets"]), w.cuda(),
                     ws_.cuda(), H, moe.alloc_workspace(p))
    want = np.zeros((disp["A"], cfg.f), bool)
    want[disp["row_src"] // cfg.k == t] = True
    want[disp["offsets"][e]:disp["offsets"][e + 1], 5] = True
    np.testing.assert_array_equal(torch.isnan(H).cpu().numpy()[:disp["A"]], want)


def test_w8a8_layer_run_together():
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
        c = torch.empty(x.shape, dtype=torch.int8, device="cuda")
        s = torch.empty(x.shape[:-1], device="cuda")
        moe.int8_quantize(x, c, s)
        return c, s

    moe.route_topk(p, g["logits"], v["topk_idx"], v["topk_w"])
    moe.dispatch(p, g["X"], None, v["topk_idx"], v["topk_w"], v["counts"], v["offsets"], v["row_src"], v["row_dst"],
                 v["tok_off"], v["comb_w"], v["x_perm"], None, ws)
    xq, w1, w2 = quant(g["X"]), quant(g["W1"]), quant(g["W2"])
    H = torch.zeros(cap, cfg.f, dtype=torch.bfloat16, device="cuda")
    moe.int8_linear1(p, *xq, v["row_src"], v["offsets"], *w1, H, ws)
    hq = quant(H)
    moe.int8_linear2(p, *hq, v["offsets"], v["row_dst"], *w2, v["combine_buf"], ws)
    Y = torch.empty(cfg.T, cfg.d, dtype=torch.bfloat16, device="cuda")
    Y32 = torch.empty(cfg.T, cfg.d, device="cuda")
    moe.combine(p, v["combine_buf"], v["tok_off"], v["comb_w"], Y, Y32)
    torch.cuda.synchronize()
    moe.check_workspace(p, ws)
    idx, w, _ = oracle.route_topk(inp["logits"].numpy(), cfg.k)
    disp = oracle.dispatch(idx, w, cfg.e_begin, cfg.e_end, cfg.num_segments)
    A = disp["A"]
    ref, tol = _ref_linear1(_Scaled(*xq), _Scaled(*w1), disp, cfg)
    assert np.all(np.abs(H.double().cpu().numpy()[:A] - ref) <= tol)
    hd, w2d = _Scaled(*hq), _Scaled(*w2)
    Yref, mag = np.zeros((cfg.T, cfg.d)), np.zeros((cfg.T, cfg.d))
    for e in range(El):
        for r in range(disp["offsets"][e], disp["offsets"][e + 1]):
            a = disp["row_src"][r]
            q, gate = oracle.y_row_of_token(a // cfg.k, cfg.T, cfg.num_segments), float(w.reshape(-1)[a])
            o = gate * hd[r].times(w2d[e])
            Yref[q] += o
            mag[q] += np.abs(o)
    # 4 u per product, k gates (fp32, off by 8 u with their softmax) and sums
    assert np.all(np.abs(Y32.double().cpu().numpy() - Yref) <= (4 + cfg.k + 8) * U * mag + 1e-30)
    # A row of n normal values (n <= 512) has its largest below 4.5 of its standard deviation, so its 8-bit rounding
    # is 4.5 / (127 sqrt 12) = 1.1% of it (X, W1, W2); gate and up are 1.5% off, H (|silu'| <= 1.1) 2.3%, and H's own
    # rounding, of rows whose largest is below 12 deviations, 2.8%: 3.8% with W2's, over all elements.
    exact = oracle.moe_layer(inp, cfg)["Y"]
    assert np.linalg.norm(Yref - exact) <= 0.06 * np.linalg.norm(exact)


@pytest.mark.parametrize("name", ["odd_rows", "few_tokens"])
@pytest.mark.parametrize("bad", ["src_high", "src_negative", "dst_high", "offsets", "not_monotone", "far_apart"])
def test_device_side_checks(bad, name):
    cfg, disp, g = _setup(CASES[name])
    p = problem_of(cfg, sched="auto")
    (x, xs), (w1, w1s) = _rand(g, cfg.T, cfg.d), _rand(g, cfg.E_local, 2 * cfg.f, cfg.d)
    (h, hs), (w2, w2s) = _rand(g, cfg.cap, cfg.f), _rand(g, cfg.E_local, cfg.d, cfg.f)
    src, dst, off = _i32(disp["row_src"], cfg.cap), _i32(disp["row_dst"], cfg.cap), _i32(disp["offsets"])
    good = src.clone(), dst.clone(), off.clone()
    if bad == "src_high":
        src[disp["A"] // 3] = cfg.T * cfg.k
    elif bad == "src_negative":
        src[disp["A"] - 1] = -1
    elif bad == "dst_high":
        dst[disp["A"] // 2] = cfg.cap
    elif bad == "offsets":
        off[-1] = cfg.cap + 1
    elif bad == "far_apart":  # differences that 32 bits do not hold come out small and not negative
        off[:] = 0
        off[1], off[2], off[3] = 2 ** 31 - 1, -2 ** 31, -1
    else:
        off[1] = off[2] + 1
    ws = moe.alloc_workspace(p)
    H = torch.full((cfg.cap, cfg.f), 5.0, dtype=torch.bfloat16, device="cuda")
    C = torch.full((cfg.cap, cfg.d), 5.0, device="cuda")

    def one(s, o):
        moe.int8_linear1(p, x.cuda(), xs.cuda(), s, o, w1.cuda(), w1s.cuda(), H, ws)

    def two(t, o):
        moe.int8_linear2(p, h.cuda(), hs.cuda(), o, t, w2.cuda(), w2s.cuda(), C, ws)

    for call, out in ((lambda: one(src, off), H), (lambda: two(dst, off), C)):
        call()
        torch.cuda.synchronize()
        reached = bad in ("offsets", "not_monotone", "far_apart") or (bad.startswith("src")) == (out is H)
        if reached:
            with pytest.raises(moe.MoEError) as ei:
                moe.check_workspace(p, ws)
            assert ei.value.status == 1
            assert torch.all(out == 5.0)
        else:
            moe.check_workspace(p, ws)
    if not bad.startswith("dst"):  # a rejected Linear-1 is still reported after a Linear-2 that went well
        one(src, off)
        two(good[1], good[2])
        with pytest.raises(moe.MoEError):
            moe.check_workspace(p, ws)
    one(good[0], good[2])
    moe.check_workspace(p, ws)
    assert torch.isfinite(H).all() and not torch.all(H[:disp["A"]] == 5.0)


def test_padded_layout():
    """A row capacity of its own (the owner-aligned layout) on few tokens: every row of the padded experts."""
    T, E, k, d, f, cap = 4, 4, 2, 256, 128, 700
    off = np.array([0, 0, 300, 300, 700])
    p = moe.make_problem(T, d, f, E, k, sched="auto", row_capacity=cap)
    g = torch.Generator().manual_seed(1)
    (x, xs), (w, ws_) = _rand(g, cap, d), _rand(g, E, 2 * f, d)
    H, ws = torch.zeros(cap, f, dtype=torch.bfloat16, device="cuda"), moe.alloc_workspace(p)
    moe.int8_linear1(p, x.cuda(), xs.cuda(), None, _i32(off), w.cuda(), ws_.cuda(), H, ws)
    moe.check_workspace(p, ws)
    for e in (1, 3):
        r = slice(off[e], off[e + 1])
        gate, u = np.split(_Scaled(x, xs)[r].times(_Scaled(w, ws_)[e]), 2, axis=1)
        ref = gate / (1 + np.exp(-gate)) * u
        tol = 4 * U * (1.1 * np.abs(u * gate) + np.abs(ref)) + 16 * U * (1 + np.abs(gate)) * np.abs(ref)
        assert np.all(np.abs(H[r].double().cpu().numpy() - ref) <= tol + B * (np.abs(ref) + tol) + 1e-30), e


@pytest.mark.parametrize("counts", [[12, 7, 8, 9], [0, 15, 16, 17], [31, 0, 32, 33], [0, 0, 64, 0], [65, 1, 0, 100],
                                    [63, 64, 65, 64], [0, 256, 0, 0], [129, 95, 31, 1]])
@pytest.mark.parametrize("d,f", [(128, 256), (640, 128), (1152, 896)])
def test_both_kernels_give_the_same_bits(counts, d, f):
    """At most 64 rows per expert in the mean: a whole grid leaves the tiles of these to the kernel for few rows, a grid
    of 8 workgroups or fewer to the persistent GEMM. Sums of whole numbers are the same in any order."""
    E, A = 4, sum(counts)
    g = torch.Generator().manual_seed(A)
    (x, xs), (w, ws_) = _rand(g, A, d), _rand(g, E, 2 * f, d)
    (h, hs), (w2, w2s) = _rand(g, A, f), _rand(g, E, d, f)
    off, src, dst = np.concatenate([[0], np.cumsum(counts)]), torch.randperm(A, generator=g), torch.randperm(A, generator=g)
    outs = []
    for grid in (0, 8, 2):
        p = moe.make_problem(A, d, f, E, 1, sched="auto", grid=grid)
        ws = moe.alloc_workspace(p).fill_(255)
        H, C = torch.zeros(A, f, dtype=torch.bfloat16, device="cuda"), torch.zeros(A, d, device="cuda")
        moe.int8_linear1(p, x.cuda(), xs.cuda(), _i32(src), _i32(off), w.cuda(), ws_.cuda(), H, ws)
        moe.int8_linear2(p, h.cuda(), hs.cuda(), _i32(off), _i32(dst), w2.cuda(), w2s.cuda(), C, ws)
        moe.check_workspace(p, ws)
        outs.append((H, C))
    for H, C in outs[1:]:
        assert torch.equal(H, outs[0][0]) and torch.equal(C, outs[0][1])
    H, C = (t.double().cpu().numpy() for t in outs[0])
    X, W, Hq, W2 = _Scaled(x, xs), _Scaled(w, ws_), _Scaled(h, hs), _Scaled(w2, w2s)
    for e in range(E):
        r = slice(off[e], off[e + 1])
        gate, u = np.split(X[src[r].numpy()].times(W[e]), 2, axis=1)
        ref = gate / (1 + np.exp(-gate)) * u
        tol = 4 * U * (1.1 * np.abs(u * gate) + np.abs(ref)) + 16 * U * (1 + np.abs(gate)) * np.abs(ref)
        assert np.all(np.abs(H[r] - ref) <= tol + B * (np.abs(ref) + tol) + 1e-30), e
        ref = Hq[r].times(W2[e])
        assert np.all(np.abs(C[dst[r].numpy()] - ref) <= 4 * U * np.abs(ref)), e


@pytest.mark.parametrize("E", [8, 1024])
def test_a_problem_of_any_type_and_schedule(E):
    """The Linears take their operands' type from the call: what the problem names for the layer's own, its schedule and
    its segments do not matter. 1024 local experts are the most there are."""
    T, d, f, k = 128, 256, 128, 2
    g = torch.Generator().manual_seed(E)
    (x, xs), (w, ws_) = _rand(g, T, d), _rand(g, E, 2 * f, d)
    (h, hs), (w2, w2s) = _rand(g, T * k, f), _rand(g, E, d, f)
    idx = torch.stack([torch.randperm(E, generator=g)[:k] for _ in range(T)])
    order = torch.argsort(idx.flatten(), stable=True)
    off = _i32(np.concatenate([[0], np.cumsum(np.bincount(idx.flatten().numpy(), minlength=E))]))
    src, dst = order.to(torch.int32).cuda(), torch.randperm(T * k, generator=g).to(torch.int32).cuda()
    x, xs, w, ws_, h, hs, w2, w2s = (t.cuda() for t in (x, xs, w, ws_, h, hs, w2, w2s))
    outs = []
    for kw in (dict(), dict(dtype="fp8_e4m3", sched="interleaved"), dict(dtype="w4a8_mxfp4", sched="separate", num_segments=4),
               dict(sched="expert_wave", trace=True), dict(dtype="fp8_e4m3", keep_h_f32=True, band_major=True)):
        p = moe.make_problem(T, d, f, E, k, **dict(dict(sched="auto"), **kw))
        H, C = torch.full((T * k, f), 5.0, dtype=torch.bfloat16, device="cuda"), torch.zeros(T * k, d, device="cuda")
        wsp = moe.alloc_workspace(p)
        moe.int8_linear1(p, x, xs, src, off, w, ws_, H, wsp)
        moe.int8_linear2(p, h, hs, off, dst, w2, w2s, C, wsp)
        moe.check_workspace(p, wsp)
        outs.append((H, C))
    for H, C in outs[1:]:
        assert torch.equal(H, outs[0][0]) and torch.equal(C, outs[0][1])
    H, C = (t.double().cpu().numpy() for t in outs[0])
    o = off.cpu().numpy()
    X, W, Hq, W2 = _Scaled(x.cpu(), xs.cpu()), _Scaled(w.cpu(), ws_.cpu()), _Scaled(h.cpu(), hs.cpu()), _Scaled(w2.cpu(), w2s.cpu())
    for e in range(E):
        r = slice(o[e], o[e + 1])
        if o[e] == o[e + 1]:
            continue
        gate, u = np.split(X[src[r].cpu().numpy() // k].times(W[e]), 2, axis=1)
        ref = gate / (1 + np.exp(-gate)) * u
        tol = 4 * U * (1.1 * np.abs(u * gate) + np.abs(ref)) + 16 * U * (1 + np.abs(gate)) * np.abs(ref)
        assert np.all(np.abs(H[r] - ref) <= tol + B * (np.abs(ref) + tol) + 1e-30), e
        ref = Hq[r].times(W2[e])
        assert np.all(np.abs(C[dst[r].cpu().numpy()] - ref) <= 4 * U * np.abs(ref)), e


@pytest.mark.parametrize("name", ["odd_blocks", "empty_experts"])
def test_rows_past_the_last_are_not_looked_at(name):
    """Indices and scales behind the last row may hold anything."""
    cfg, disp, g = _setup(CASES[name])
    A = disp["A"]
    p = problem_of(cfg, sched="auto")
    (x, xs), (w, ws_) = _rand(g, cfg.T, cfg.d), _rand(g, cfg.E_local, 2 * cfg.f, cfg.d)
    src = _i32(disp["row_src"], cfg.cap)
    src[A:] = 2 ** 31 - 1
    ws = moe.alloc_workspace(p)
    H = torch.zeros(cfg.cap, cfg.f, dtype=torch.bfloat16, device="cuda")
    moe.int8_linear1(p, x.cuda(), xs.cuda(), src, _i32(disp["offsets"]), w.cuda(), ws_.cuda(), H, ws)
    moe.check_workspace(p, ws)
    (h, hs), (w2, w2s) = _rand(g, cfg.cap, cfg.f), _rand(g, cfg.E_local, cfg.d, cfg.f)
    hs[A:] = float("nan")
    dst = _i32(disp["row_dst"], cfg.cap)
    dst[A:] = -5
    C = torch.full((cfg.cap, cfg.d), 5.0, device="cuda")
    moe.int8_linear2(p, h.cuda(), hs.cuda(), _i32(disp["offsets"]), dst, w2.cuda(), w2s.cuda(), C, ws)
    moe.check_workspace(p, ws)
    assert torch.isfinite(C).all() and torch.all(C[A:] == 5.0)


@pytest.mark.parametrize("name", ["odd_blocks", "few_tokens"])
def test_grid_and_raster_change_no_bit(name):
    cfg, disp, g = _setup(CASES[name])
    (x, xs), (w, ws_) = _rand(g, cfg.T, cfg.d), _rand(g, cfg.E_local, 2 * cfg.f, cfg.d)
    (h, hs), (w2, w2s) = _rand(g, cfg.cap, cfg.f), _rand(g, cfg.E_local, cfg.d, cfg.f)
    ref = None
    for kw in (dict(), dict(grid=1), dict(grid=2), dict(grid=9), dict(tiles="narrow"), dict(band_major=True)):
        p = problem_of(cfg, sched="auto", **kw)
        H = torch.zeros(cfg.cap, cfg.f, dtype=torch.bfloat16, device="cuda")
        C = torch.zeros(cfg.cap, cfg.d, device="cuda")
        ws = moe.alloc_workspace(p)
        moe.int8_linear1(p, x.cuda(), xs.cuda(), _i32(disp["row_src"], cfg.cap), _i32(disp["offsets"]), w.cuda(),
                         ws_.cuda(), H, ws)
        moe.int8_linear2(p, h.cuda(), hs.cuda(), _i32(disp["offsets"]), _i32(disp["row_dst"], cfg.cap), w2.cuda(),
                         w2s.cuda(), C, ws)
        torch.cuda.synchronize()
        ref = (H, C) if ref is None else ref
        assert torch.equal(ref[0], H) and torch.equal(ref[1], C), kw


@pytest.mark.parametrize("name", ["odd_rows", "few_tokens"])
def test_replayed_graphs_and_another_stream(name):
    """Two graphs on one workspace, replayed in turn, and a call on a stream of the caller's."""
    cfg, disp, g = _setup(CASES[name])
    p = problem_of(cfg, sched="auto")
    x, xs, w, ws_ = (t.cuda() for q in (_rand(g, cfg.T, cfg.d), _rand(g, cfg.E_local, 2 * cfg.f, cfg.d)) for t in q)
    h, hs, w2, w2s = (t.cuda() for q in (_rand(g, cfg.cap, cfg.f), _rand(g, cfg.E_local, cfg.d, cfg.f)) for t in q)
    src, dst = _i32(disp["row_src"], cfg.cap), _i32(disp["row_dst"], cfg.cap)
    off, ws = _i32(disp["offsets"]), moe.alloc_workspace(p)
    H = torch.zeros(cfg.cap, cfg.f, dtype=torch.bfloat16, device="cuda")
    C = torch.zeros(cfg.cap, cfg.d, device="cuda")
    one = lambda s=None: moe.int8_linear1(p, x, xs, src, off, w, ws_, H, ws, stream=s)  # noqa: E731
    two = lambda s=None: moe.int8_linear2(p, h, hs, off, dst, w2, w2s, C, ws, stream=s)  # noqa: E731
    one()
    two()
    torch.cuda.synchronize()
    graphs = []
    for run in (one, two):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            run()
        graphs.append(graph)
    side = torch.cuda.Stream()
    for i in range(3):
        x.random_(-128, 128)
        h.random_(-128, 128)
        H.zero_()
        C.zero_()
        for graph in graphs:
            graph.replay()
        torch.cuda.synchronize()
        got = H.clone(), C.clone()
        H.zero_()
        C.zero_()
        torch.cuda.synchronize()
        s = side if i == 1 else None
        one(s)
        two(s)
        torch.cuda.synchronize()
        assert torch.equal(got[0], H) and torch.equal(got[1], C)
    moe.check_workspace(p, ws)
