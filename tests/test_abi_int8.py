"""Calls of the 8-bit integer codecs, the Linears on 8-bit integers and the
checkpoint calls that are refused on the host, before anything is enqueued.
The addresses are made up and never dereferenced."""
import ctypes
import os

import pytest

import expert_grouped_gemm_amd as moe

OK, INVALID, UNSUPPORTED, TOO_SMALL = 0, 1, 2, 3
T, d, f, E, k = 64, 128, 256, 4, 2
CAP = T * k
P = moe.make_problem(T, d, f, E, k)
WS, WS_BYTES = 1 << 40, 1 << 24

# name: (arguments' names and bytes in the order of the call, outputs, those that may be null)
CALLS = {
    "moe_int8_linear1": ([("X", T * d), ("Xs", 4 * T), ("row_src", 4 * CAP), ("offsets", 4 * (E + 1)),
                          ("W1", E * 2 * f * d), ("W1s", E * 2 * f * 4), ("H", 2 * CAP * f)], ("H",), ("row_src",)),
    "moe_int8_linear2": ([("H", CAP * f), ("Hs", 4 * CAP), ("offsets", 4 * (E + 1)), ("row_dst", 4 * CAP),
                          ("W2", E * d * f), ("W2s", 4 * E * d), ("C", 4 * CAP * d)], ("C",), ()),
    "moe_expert_forward_checkpoint": ([("X", 2 * T * d), ("row_src", 4 * CAP), ("offsets", 4 * (E + 1)),
                                       ("row_dst", 4 * CAP), ("W1", 4 * E * f * d), ("W2", 2 * E * d * f),
                                       ("gu", 2 * CAP * f), ("gus", CAP * f // 16), ("C", 4 * CAP * d)],
                                      ("gu", "gus", "C"), ("row_src",)),
    "moe_expert_backward_checkpoint": ([("X", T * d), ("Xs", T * d // 32), ("row_src", 4 * CAP),
                                        ("offsets", 4 * (E + 1)), ("row_dst", 4 * CAP), ("gu", 2 * CAP * f),
                                        ("gus", CAP * f // 16), ("W1", 4 * E * f * d), ("W2", 2 * E * d * f),
                                        ("dO", 2 * CAP * d), ("dxs", 2 * CAP * d), ("dW1", 4 * E * f * d),
                                        ("dW2", 2 * E * d * f)], ("dxs", "dW1", "dW2"), ("Xs", "row_src")),
}
INDICES = ("row_src", "row_dst", "offsets")


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(moe.LIB_PATH):
        from expert_grouped_gemm_amd import build
        build.build()
    return moe.lib()


def _at(fn):
    return {n: (1 + i) << 30 for i, (n, _) in enumerate(CALLS[fn][0])}


def _call(L, fn, at, p=P, ws=WS, ws_bytes=WS_BYTES):
    args = [ctypes.c_void_p(at[n]) for n, _ in CALLS[fn][0]]
    return getattr(L, fn)(ctypes.byref(p), *args, ctypes.c_void_p(ws), ctypes.c_size_t(ws_bytes), None)


def _pairs():
    for fn, (args, outs, _) in CALLS.items():
        for o in outs:
            for other, _ in args:
                if other != o:
                    yield fn, o, other


@pytest.mark.parametrize("where", ["same", "last_bytes", "inside"])
@pytest.mark.parametrize("fn,out,other", list(_pairs()))
def test_shared_bytes_are_refused(L, fn, out, other, where):
    size, at = dict(CALLS[fn][0]), _at(fn)
    if where == "same":
        at[out] = at[other]
    elif where == "last_bytes":        # the output starts in the other's last 16 bytes
        at[out] = at[other] + (size[other] - 1) // 16 * 16
    else:                              # the other starts in the output's last 16 bytes
        at[out] = at[other] - (size[out] - 1) // 16 * 16
    assert _call(L, fn, at) == INVALID


@pytest.mark.parametrize("fn,name", [(fn, n) for fn, (args, _, _) in CALLS.items() for n, _ in args])
def test_operands_over_what_the_call_writes_in_the_workspace(L, fn, name):
    """The error words and the band tables at its start; H (forward) and the intermediates at its end (backward)."""
    at = _at(fn)
    at[name] = WS
    assert _call(L, fn, at) == INVALID
    if fn == "moe_expert_forward_checkpoint":
        at[name] = WS + moe.workspace_layout(P).h
        assert _call(L, fn, at) == INVALID
    if fn == "moe_expert_backward_checkpoint":
        at[name] = WS + moe.workspace_size(P)
        assert _call(L, fn, at) == INVALID


@pytest.mark.parametrize("fn,name", [(fn, n) for fn, (args, _, _) in CALLS.items() for n, _ in args])
def test_null_and_misaligned_operands(L, fn, name):
    at = _at(fn)
    at[name] += 8
    if name not in INDICES:
        assert _call(L, fn, at) == INVALID
    at[name] = 0
    if name not in CALLS[fn][2]:
        assert _call(L, fn, at) == INVALID


@pytest.mark.parametrize("fn", list(CALLS))
def test_workspace_and_problem(L, fn):
    at = _at(fn)
    need = moe.checkpoint_workspace_size(P) if fn == "moe_expert_backward_checkpoint" else moe.workspace_size(P)
    assert _call(L, fn, at, ws_bytes=need - 1) == TOO_SMALL
    assert _call(L, fn, at, ws=0) == INVALID
    assert _call(L, fn, at, ws=WS + 16) == INVALID
    assert _call(L, fn, at, p=moe.make_problem(T, 100, f, E, k)) == UNSUPPORTED
    if "checkpoint" in fn:
        assert _call(L, fn, at, p=moe.make_problem(128, d, f, E, k, dtype="fp8_e4m3")) == UNSUPPORTED


def test_integer_sums_past_32_bits_are_refused(L):
    """K = 2^17 codes of -128 against -128 sum to 2^31."""
    wide = 1 << 17
    assert _call(L, "moe_int8_linear1", _at("moe_int8_linear1"), p=moe.make_problem(2, wide, f, E, k)) == UNSUPPORTED
    assert _call(L, "moe_int8_linear2", _at("moe_int8_linear2"), p=moe.make_problem(2, d, wide, E, k)) == UNSUPPORTED


def test_checkpoint_workspace(L):
    assert L.moe_checkpoint_workspace_size(None) == 0
    assert L.moe_checkpoint_workspace_size(ctypes.byref(moe.make_problem(128, d, f, E, k, dtype="fp8_e4m3"))) == 0
    assert L.moe_checkpoint_workspace_size(ctypes.byref(moe.make_problem(2, 1 << 21, 128, 1, 1))) == 0
    # it holds a, dh and the token rows, but no fp32 gate and up values
    inner = CAP * (2 * f + 4 * f + 2 * d)
    size = moe.checkpoint_workspace_size(P) - moe.workspace_size(P)
    assert inner <= size <= inner + 1024
    assert moe.checkpoint_workspace_size(P) < moe.backward_workspace_size(P)


@pytest.mark.parametrize("codec,unit,scale_bytes", [("int8", 16, lambda r, c: 4 * r), ("mxint8", 32, lambda r, c: r * c // 32)])
@pytest.mark.parametrize("fp32", [0, 1])
def test_codecs(L, codec, unit, scale_bytes, fp32):
    quantize, dequantize = getattr(L, f"moe_{codec}_quantize"), getattr(L, f"moe_{codec}_dequantize")
    rows, cols = 8, 96
    n, sb = rows * cols, scale_bytes(8, 96)
    xb = n * (4 if fp32 else 2)
    X, A, S = 1 << 30, 2 << 30, 3 << 30
    ptr = ctypes.c_void_p

    def both(x, codes, scales, r=rows, c=cols):
        return {quantize(ptr(x), fp32, r, c, ptr(codes), ptr(scales), None),
                dequantize(ptr(codes), ptr(scales), r, c, ptr(x), fp32, None)}

    for codes, scales in ((X, S), (X + xb - 16, S), (X - n + 16, S), (A, X), (A, X + xb - 4), (A, X - sb + 4)):
        assert both(X, codes, scales) == {INVALID}, (codes, scales)
    for codes, scales in ((A, A), (A, A + n - 4)):  # outputs of the quantiser over each other
        assert quantize(ptr(X), fp32, rows, cols, ptr(codes), ptr(scales), None) == INVALID
    assert both(0, A, S) == both(X, 0, S) == both(X, A, 0) == {INVALID}
    assert both(X + 8, A, S) == both(X, A + 8, S) == {INVALID}
    if codec == "int8":
        assert both(X, A, S + 2) == {INVALID}
    assert both(X, A, S, r=-1) == both(X, A, S, c=0) == {INVALID}
    assert both(X, A, S, c=unit + unit // 2) == {UNSUPPORTED}
    assert both(X, A, S, r=1 << 40, c=1 << 20) == {UNSUPPORTED}
    assert both(0, 0, 0, r=0) == {OK}
