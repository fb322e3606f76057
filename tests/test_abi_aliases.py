"""Outputs that share bytes with an input, or with another output, of the
gradients, the MXFP4 codec and the MXFP4 Linears: refused on the host, before
anything is enqueued. The addresses are made up and never dereferenced."""
import ctypes
import os

import pytest

import expert_grouped_gemm_amd as moe


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(moe.LIB_PATH):
        from expert_grouped_gemm_amd import build
        build.build()
    return moe.lib()


T, d, f, E, k = 64, 128, 256, 4, 2
CAP = T * k
P = moe.make_problem(T, d, f, E, k)
INVALID = 1

# name: (arguments' names and bytes in the order of the call, outputs), the workspace and stream apart
_BACKWARD_WS = 1 << 24
CALLS = {
    "moe_combine_backward": ([("dY", 2 * T * d), ("buf", 4 * CAP * d), ("tok_off", 4 * (T + 1)), ("idx", 4 * T * k),
                              ("w", 4 * T * k), ("d_buf", 2 * CAP * d), ("d_w", 4 * T * k), ("d_logits", 4 * T * E)],
                             ("d_buf", "d_w", "d_logits")),
    "moe_dispatch_backward": ([("dxs", 2 * CAP * d), ("tok_off", 4 * (T + 1)), ("dX", 2 * T * d), ("dX32", 4 * T * d)],
                              ("dX", "dX32")),
    "moe_expert_backward": ([("X", 2 * T * d), ("row_src", 4 * CAP), ("offsets", 4 * (E + 1)), ("row_dst", 4 * CAP),
                             ("W1", 4 * E * f * d), ("W2", 2 * E * d * f), ("dO", 2 * CAP * d), ("dxs", 2 * CAP * d),
                             ("dW1", 4 * E * f * d), ("dW2", 2 * E * d * f)], ("dxs", "dW1", "dW2")),
    "moe_mxfp4_linear1": ([("X", T * d // 2), ("Xs", T * d // 32), ("row_src", 4 * CAP), ("offsets", 4 * (E + 1)),
                           ("W1", E * f * d), ("W1s", E * f * d // 16), ("H", 2 * CAP * f)], ("H",)),
    "moe_mxfp4_linear2": ([("H", CAP * f // 2), ("Hs", CAP * f // 32), ("offsets", 4 * (E + 1)), ("row_dst", 4 * CAP),
                           ("W2", E * d * f // 2), ("W2s", E * d * f // 32), ("C", 4 * CAP * d)], ("C",)),
}
WITH_WORKSPACE = ("moe_expert_backward", "moe_mxfp4_linear1", "moe_mxfp4_linear2")


def _pairs():
    for fn, (args, outs) in CALLS.items():
        names = [n for n, _ in args]
        for o in outs:
            for other in names:
                if other != o:
                    yield fn, o, other


def _call(L, fn, at):
    args = [ctypes.c_void_p(at[n]) for n, _ in CALLS[fn][0]]
    if fn in WITH_WORKSPACE:
        args += [ctypes.c_void_p(1 << 40), ctypes.c_size_t(_BACKWARD_WS)]
    return getattr(L, fn)(ctypes.byref(P), *args, None)


@pytest.mark.parametrize("where", ["same", "last_bytes", "inside"])
@pytest.mark.parametrize("fn,out,other", list(_pairs()))
def test_shared_bytes_are_refused(L, fn, out, other, where):
    size = dict(CALLS[fn][0])
    at = {n: (1 + i) << 30 for i, (n, _) in enumerate(CALLS[fn][0])}
    if where == "same":
        at[out] = at[other]
    elif where == "last_bytes":        # the output starts in the other's last 16 bytes
        at[out] = at[other] + (size[other] - 1) // 16 * 16
    else:                              # the other starts in the output's last 16 bytes
        at[out] = at[other] - (size[out] - 1) // 16 * 16
    assert _call(L, fn, at) == INVALID


@pytest.mark.parametrize("fn,out", [(fn, o) for fn in WITH_WORKSPACE for o in CALLS[fn][1]])
def test_outputs_over_the_workspaces_tables_are_refused(L, fn, out):
    """The error words and the band tables lie at the workspace's start, the gradient's intermediates at its end."""
    at = {n: (1 + i) << 30 for i, (n, _) in enumerate(CALLS[fn][0])}
    at[out] = 1 << 40
    assert _call(L, fn, at) == INVALID
    if fn == "moe_expert_backward":
        at[out] = (1 << 40) + moe.workspace_size(P)
        assert _call(L, fn, at) == INVALID


@pytest.mark.parametrize("fp32", [0, 1])
def test_codec_in_place_is_refused(L, fp32):
    rows, cols = 8, 96
    n = rows * cols
    xb, cb, sb = n * (4 if fp32 else 2), n // 2, n // 32
    X = 1 << 30
    far = ((2 << 30), (3 << 30))
    for codes, scales in ((X, far[1]), (X + xb - 16, far[1]), (X - cb + 16, far[1]), (far[0], X), (far[0], X + xb - 1),
                          (far[0], X - sb + 1), (far[0], far[0]), (far[0], far[0] + cb - 1)):
        ptr = [ctypes.c_void_p(v) for v in (X, codes, scales)]
        assert L.moe_mxfp4_quantize(ptr[0], fp32, rows, cols, ptr[1], ptr[2], None) == INVALID, (codes, scales)
    for codes, scales in ((X, far[1]), (X + xb - 16, far[1]), (X - cb + 16, far[1]), (far[0], X), (far[0], X + xb - 1),
                          (far[0], X - sb + 1)):
        ptr = [ctypes.c_void_p(v) for v in (codes, scales, X)]
        assert L.moe_mxfp4_dequantize(ptr[0], ptr[1], rows, cols, ptr[2], fp32, None) == INVALID, (codes, scales)
