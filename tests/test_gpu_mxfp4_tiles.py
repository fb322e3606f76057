"""The MXFP4 Linears' tiles of both widths, with 1 to 8 row blocks, of experts
with one row band and with several, over a K of whole slices and one that ends
in half a slice, against fp64. A small grid makes whole rounds of wide tiles out
of few of them; by default those of so few tiles are all cut in two. References
and bounds are those of test_gpu_mxfp4_linear."""
import numpy as np
import pytest
import torch

import expert_grouped_gemm_amd as moe
import moe_synth
from test_gpu_mxfp4_linear import B, U, _decode, _i32, _rand_mx, _ref_linear1

pytestmark = pytest.mark.gpu

COUNTS = {"single": (20, 50, 90, 120, 150, 180, 220, 256), "several": (276, 306, 346, 376, 406, 436, 476, 768),
          "mixed": (0, 600, 5, 0, 257, 1)}
MOST = (1, 0, 2) * 341 + (130,)     # as many experts as there may be
GRIDS = (2, 8, 40, 0)


def _setup(name, d, f):
    counts = MOST if name == "most" else COUNTS[name]
    A, E = sum(counts), len(counts)
    cfg = moe_synth.make_config("tiny", T=A, d=d, f=f, E_global=E, k=1, e_begin=0, e_end=E)
    rng = np.random.default_rng(A + d + f)
    disp = dict(A=A, offsets=np.concatenate([[0], np.cumsum(counts)]), row_src=rng.permutation(A),
                row_dst=rng.permutation(A))
    return cfg, disp, torch.Generator().manual_seed(A + d + f)


def _problem(cfg, grid, **kw):
    return moe.make_problem(cfg.T, cfg.d, cfg.f, cfg.E_global, 1, sched="auto", grid=grid, **kw)


@pytest.mark.parametrize("name,d,f", [(n, *s) for n in COUNTS for s in ((1152, 640), (1280, 384))]
                         + [("most", 128, 256)])
def test_linear1_tiles(name, d, f):
    cfg, disp, g = _setup(name, d, f)
    (x, xs), (w, ws_) = _rand_mx(g, cfg.T, d), _rand_mx(g, cfg.E_local, 2 * f, d)
    ref, tol = _ref_linear1(_decode(x, xs), _decode(w, ws_), disp, cfg)
    args = x.cuda(), xs.cuda(), _i32(disp["row_src"]), _i32(disp["offsets"]), w.cuda(), ws_.cuda()
    for grid in GRIDS:
        print(f"[mxfp4_linear1 tiles] {name} d={d} f={f} grid={grid}", flush=True)
        p = _problem(cfg, grid)
        ws = moe.alloc_workspace(p)
        H = torch.full((disp["A"], f), 5.0, dtype=torch.bfloat16, device="cuda")
        moe.mxfp4_linear1(p, *args, H, ws)
        torch.cuda.synchronize()
        moe.check_workspace(p, ws)
        assert np.all(np.abs(H.double().cpu().numpy() - ref) <= tol), grid


@pytest.mark.parametrize("bf16_buf", [False, True])
@pytest.mark.parametrize("name,d,f", [(n, *s) for n in COUNTS for s in ((1280, 1152), (768, 1664), (512, 1024))]
                         + [("most", 256, 128)])
def test_linear2_tiles(name, d, f, bf16_buf):
    cfg, disp, g = _setup(name, d, f)
    A, off, dst = disp["A"], disp["offsets"], disp["row_dst"]
    (h, hs), (w, ws_) = _rand_mx(g, A, f), _rand_mx(g, cfg.E_local, d, f)
    H, W = _decode(h, hs), _decode(w, ws_)
    ref, tol = np.zeros((A, d)), np.zeros((A, d))
    for e in range(cfg.E_local):
        r = slice(off[e], off[e + 1])
        ref[dst[r]], tol[dst[r]] = H[r] @ W[e].T, f * U * (np.abs(H[r]) @ np.abs(W[e]).T)
    if bf16_buf:
        tol = tol + B * (np.abs(ref) + tol)
    args = h.cuda(), hs.cuda(), _i32(off), _i32(dst), w.cuda(), ws_.cuda()
    first = None
    for grid in GRIDS:
        print(f"[mxfp4_linear2 tiles] {name} d={d} f={f} bf16_buf={bf16_buf} grid={grid}", flush=True)
        p = _problem(cfg, grid, bf16_combine_buf=bf16_buf)
        ws = moe.alloc_workspace(p)
        C = torch.full((A, d), 5.0, dtype=torch.bfloat16 if bf16_buf else torch.float32, device="cuda")
        moe.mxfp4_linear2(p, *args, C, ws)
        torch.cuda.synchronize()
        moe.check_workspace(p, ws)
        assert np.all(np.abs(C.double().cpu().numpy() - ref) <= tol), grid
        first = C if first is None else first
        assert torch.equal(first, C), grid           # the grid changes no bit


@pytest.mark.parametrize("dtype", ["fp8_e4m3", "w4a8_mxfp4"])
def test_a_problem_of_another_operand_type(dtype):
    """Of the problem's dtype nothing is used: the same bits as with bf16."""
    counts, d, f = (100, 28), 384, 256
    g = torch.Generator().manual_seed(1)
    (x, xs), (w, ws_) = _rand_mx(g, 128, d), _rand_mx(g, 2, 2 * f, d)
    off = _i32(np.concatenate([[0], np.cumsum(counts)]))
    res = []
    for t in ("bf16", dtype):
        p = moe.make_problem(128, d, f, 2, 1, sched="auto", dtype=t)
        ws = moe.alloc_workspace(p)
        H = torch.zeros(128, f, dtype=torch.bfloat16, device="cuda")
        moe.mxfp4_linear1(p, x.cuda(), xs.cuda(), None, off, w.cuda(), ws_.cuda(), H, ws)
        moe.check_workspace(p, ws)
        res.append(H)
    assert torch.equal(*res) and res[0].any()
