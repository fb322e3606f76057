"""Captured calls of the 8-bit integer products and the checkpoints: nothing of
the rows' distribution is read on the host, so that a graph captured with one
serves every other; two graphs share a workspace."""
import numpy as np
import pytest
import torch

import expert_grouped_gemm_amd as moe

pytestmark = pytest.mark.gpu


def _i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


def _captured(run):
    run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run()
    return graph


def _splits(T, k, E, rng):
    """Offsets that leave experts empty, give one all rows, one row each, or end before the last row."""
    A = T * k
    yield np.concatenate([[0], np.full(E, A)])
    yield np.concatenate([np.zeros(E), [A]])
    yield np.concatenate([np.zeros(E - 1), [A // 2], [A // 2 + 1]])
    yield np.zeros(E + 1)
    yield np.concatenate([[0], np.sort(rng.integers(0, A + 1, E))])


@pytest.mark.parametrize("T", [96, 1400])
@pytest.mark.parametrize("x8", [True, False])
def test_checkpoint_graphs_serve_any_distribution(T, x8):
    E, k, d, f = 4, 1, 256, 384
    p = moe.make_problem(T, d, f, E, k, sched="auto")
    g = torch.Generator().manual_seed(T)
    bf = dict(dtype=torch.bfloat16, device="cuda")
    X, dO, W1, W2 = (torch.randn(*s, generator=g).to(torch.bfloat16).cuda() for s in ((T, d), (T, d), (E, 2 * f, d), (E, d, f)))
    W1 *= 0.05
    W2 *= 0.05
    off, src, dst = _i32(np.arange(E + 1) * (T // E)), _i32(np.arange(T)), _i32(np.arange(T))
    X8, Xs = torch.empty(T, d, dtype=torch.int8, device="cuda"), torch.empty(T, d // 32, dtype=torch.uint8, device="cuda")
    moe.mxint8_quantize(X, X8, Xs)
    gu, gus = torch.zeros(T, 2 * f, dtype=torch.int8, device="cuda"), torch.full((T, f // 16), 127, dtype=torch.uint8, device="cuda")
    C, ws = torch.zeros(T, d, device="cuda"), moe.alloc_checkpoint_workspace(p)
    out = torch.zeros(T, d, **bf), torch.zeros(E, 2 * f, d, **bf), torch.zeros(E, d, f, **bf)
    everything = (C, gu, gus, *out)

    def forward():
        moe.expert_forward_checkpoint(p, X, src, off, dst, W1, W2, gu, gus, C, ws)

    def backward():
        moe.expert_backward_checkpoint(p, X8 if x8 else X, Xs if x8 else None, src, off, dst, gu, gus, W1, W2, dO, *out, ws)

    one, two = _captured(forward), _captured(backward)
    rng = np.random.default_rng(T)
    for split in _splits(T, k, E, rng):
        print(f"[graphs] {split.astype(int).tolist()}", flush=True)
        off.copy_(_i32(split))
        src.copy_(_i32(rng.permutation(T)))
        dst.copy_(_i32(rng.permutation(T)))
        for t in everything:
            t.fill_(1)
        one.replay()
        two.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in everything]
        for t in everything:
            t.fill_(1)
        forward()
        backward()
        moe.check_workspace(p, ws)
        for a, b in zip(got, everything):
            assert torch.equal(a, b)
        counts = np.diff(split).astype(int)
        for e in range(E):  # an expert without rows has gradients of zero
            assert bool(out[1][e].any()) == bool(counts[e]) and bool(out[2][e].any()) == bool(counts[e])
        rows = torch.zeros(T, dtype=torch.bool, device="cuda")
        rows[dst[int(split[0]):int(split[-1])].long()] = True
        assert torch.equal((C != 1).any(1), rows) and torch.equal((out[0] != 1).any(1), rows)


@pytest.mark.parametrize("E_global", [4, 64])
def test_int8_graphs_serve_any_distribution(E_global):
    """Both kernels: 96 rows of 4 experts (24 each in the mean), and of a share of 64."""
    T, k, E, d, f = 96, 1, 4, 256, 384
    p = moe.make_problem(T, d, f, E_global, k, 0, E, sched="auto")
    g = torch.Generator().manual_seed(E_global)

    def rand(*s):
        return (torch.randint(-128, 128, s, generator=g, dtype=torch.int8).cuda(),
                (torch.rand(s[:-1], generator=g) * 2e-3 + 1e-4).cuda())

    (x, xs), (w, ws1), (h, hs), (w2, ws2) = rand(T, d), rand(E, 2 * f, d), rand(T, f), rand(E, d, f)
    off, src, dst = _i32(np.arange(E + 1) * (T // E)), _i32(np.arange(T)), _i32(np.arange(T))
    H, C = torch.zeros(T, f, dtype=torch.bfloat16, device="cuda"), torch.zeros(T, d, device="cuda")
    ws = moe.alloc_workspace(p)

    def run():
        moe.int8_linear1(p, x, xs, src, off, w, ws1, H, ws)
        moe.int8_linear2(p, h, hs, off, dst, w2, ws2, C, ws)

    graph = _captured(run)
    rng = np.random.default_rng(E_global)
    for split in _splits(T, k, E, rng):
        print(f"[graphs] {split.astype(int).tolist()}", flush=True)
        off.copy_(_i32(split))
        src.copy_(_i32(rng.permutation(T)))
        dst.copy_(_i32(rng.permutation(T)))
        H.fill_(1)
        C.fill_(1)
        graph.replay()
        torch.cuda.synchronize()
        got = H.clone(), C.clone()
        H.fill_(1)
        C.fill_(1)
        run()
        moe.check_workspace(p, ws)
        assert torch.equal(got[0], H) and torch.equal(got[1], C)
        for e in range(E):  # exact sums: the products in 64 bits, scaled
            r = slice(int(split[e]), int(split[e + 1]))
            ref = (h[r].double() @ w2[e].double().T) * hs[r].double()[:, None] * ws2[e].double()[None]
            assert bool(((C[dst[r].long()].double() - ref).abs() <= 4 * 2.0 ** -24 * ref.abs()).all()), e
        rows = torch.zeros(T, dtype=torch.bool, device="cuda")
        rows[dst[int(split[0]):int(split[-1])].long()] = True
        assert torch.equal((C != 1).any(1), rows)
