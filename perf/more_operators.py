"""Cases, plain forms and calls of the experts' 8-bit integer products and of the 8-bit activation checkpoints.

A case names an operator (`op`) and the share's shape: T tokens of width d,
E experts of which [e_begin, e_begin + E_l) are local, k experts per token,
S destination segments of the output rows, expert width f, and `zipf` > 0 for
a router that favours some experts. The quantisers' cases are rows x cols.

With `own` false, `run` computes an operator with elementary torch operations
in fp32; with `own` true it makes the package's calls on the same inputs.
"""
import math
import random

import torch

own = False


# ---------------------------------------------------------------- the cases
def listed():
    share = dict(d=7168, f=2048, E=256, k=8, e_begin=0, E_l=32, S=8, zipf=0.0)
    mixtral = dict(d=4096, f=14336, E=8, k=2, e_begin=0, E_l=8, S=1, zipf=0.0)
    return [
        # the tokens of one decoding step
        dict(name="int8-quant-decode", op="int8_quantize", rows=16, cols=7168, fp32=False),
        # the SwiGLU rows of a prefill through wide experts
        dict(name="int8-quant-prefill", op="int8_quantize", rows=16384, cols=14336, fp32=False),
        # one token through wide experts: two experts' weights
        dict(name="int8-linear1-token", op="int8_linear1", T=1, **mixtral),
        # a prefill-sized batch through a fine-grained share
        dict(name="int8-linear1-share", op="int8_linear1", T=4096, **share),
        # a decoding step through the share: the weights' bytes
        dict(name="int8-linear2-decode", op="int8_linear2", **dict(share, T=64, S=1), bf16_buf=False),
        # prefill through wide experts: the matrix units
        dict(name="int8-linear2-mixtral", op="int8_linear2", T=8192, **mixtral, bf16_buf=False),
        # the tokens of the smallest layer the package is configured with: launch latency
        dict(name="mxint8-quant-tiny", op="mxint8_quantize", rows=64, cols=128, fp32=False),
        # the tokens of a long batch, kept for the backward pass
        dict(name="mxint8-quant-tokens", op="mxint8_quantize", rows=32768, cols=7168, fp32=False),
        # the forward pass of a few odd tokens: ragged bands, experts without rows
        dict(name="checkpoint-fwd-small", op="checkpoint_forward", T=201, d=384, f=640, E=16, k=2, e_begin=3, E_l=9,
             S=1, zipf=1.2),
        # the forward pass of a training step on the share
        dict(name="checkpoint-fwd-share", op="checkpoint_forward", T=4096, **share),
        # its backward pass: weights and their gradients streamed once against ~128 rows per expert
        dict(name="checkpoint-bwd-share", op="checkpoint_backward", T=4096, **share, x8=True),
        # wide experts with thousands of rows, the tokens still at hand in bf16: the matrix units
        dict(name="checkpoint-bwd-mixtral", op="checkpoint_backward", T=8192, **mixtral, x8=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _expected_rows(case):
    """Local assignments of a batch, in the mean (of 200 sampled tokens where the router is skewed)."""
    T, E, k, e0, El = (case[x] for x in ("T", "E", "k", "e_begin", "E_l"))
    if case["zipf"] == 0 or El == E:
        return T * k * El / E
    r, local = random.Random(0), 0
    for _ in range(200):
        logits = [r.gauss(0, 1) - case["zipf"] * math.log(e + 1) for e in range(E)]
        top = sorted(range(E), key=lambda e: -logits[e])[:k]
        local += sum(e0 <= e < e0 + El for e in top)
    return T * local / 200


def draw(rng):
    op = rng.choice(["int8_quantize", "int8_linear1", "int8_linear2", "mxint8_quantize", "checkpoint_forward",
                     "checkpoint_backward"])
    if op.endswith("quantize"):
        unit = 16 if op == "int8_quantize" else 32
        cols = unit * _log(rng, 4, 14336 // unit)
        fp32 = rng.random() < 0.5
        return dict(op=op, rows=_log(rng, 1, max(2, min(65536, (16384 if fp32 else 32768) * 7168 // cols))), cols=cols,
                    fp32=fp32)
    E = rng.choice([4, 8, 16, 64, 160, 256])
    k = rng.randint(1, min(8, E))
    E_l = max(1, E // rng.choice([1, 1, 2, 8]))
    case = dict(op=op, d=128 * _log(rng, 1, 56), f=128 * _log(rng, 1, 112), E=E, k=k,
                e_begin=rng.randint(0, E - E_l), E_l=E_l, zipf=rng.choice([0.0, 0.0, 1.2]))
    if case["zipf"] > 0:  # the share that holds the favoured experts
        case["e_begin"] = rng.randint(0, min(3, E - E_l))
    weights = (32 * 7168 * 2048 if op.startswith("checkpoint") else 8 * 4096 * 14336)
    while E_l * case["d"] * case["f"] > weights:
        case["f"] = max(128, case["f"] // 256 * 128)
        if case["f"] == 128 and E_l * case["d"] * 128 > weights:
            case["d"] = case["d"] // 256 * 128
    flops = 16384 * 4096 * 14336 // (8 if op == "checkpoint_forward" else 1) // (case["d"] * case["f"] * min(k, E_l))
    case["T"] = _log(rng, 1, max(2, min(8192, flops // 2, 2 ** 30 // (max(case["d"], case["f"]) * k))))
    if op == "int8_linear2":
        case["bf16_buf"] = rng.random() < 0.5
    if op == "checkpoint_backward":
        case["x8"] = rng.random() < 0.6
    if _expected_rows(case) < 32:  # a few tokens: every expert local, so that there are rows
        case.update(e_begin=0, E_l=E)
        while E * case["d"] * case["f"] > 8 * 4096 * 14336:
            case["f"] = max(128, case["f"] // 256 * 128)
            if case["f"] == 128:
                case["d"] = max(128, case["d"] // 256 * 128)
    s = rng.choice([1, 2, 8])
    case["S"] = s if case["T"] % s == 0 else 1
    return case


# ------------------------------------------------------- inputs, from a seed
def _rand(g, *shape, std=1.0, dtype=torch.bfloat16):
    out = torch.empty(shape, dtype=dtype, device="cuda")
    flat = out.view(-1)
    for a in range(0, flat.numel(), 1 << 28):  # bounds the fp32 draws in flight
        n = min(1 << 28, flat.numel() - a)
        flat[a:a + n] = torch.randn(n, generator=g, device="cuda").mul_(std)
    return out


def _rows_of(case, g):
    """The routing and dispatch of one batch: what route_topk and dispatch leave behind."""
    T, E, k, e0, El, S = (case[x] for x in ("T", "E", "k", "e_begin", "E_l", "S"))
    logits = torch.randn(T, E, generator=g, device="cuda")
    if case["zipf"] > 0:
        logits -= case["zipf"] * torch.log(torch.arange(1, E + 1, device="cuda", dtype=torch.float32))
    idx = torch.topk(logits, k, dim=1).indices
    t = torch.arange(T, device="cuda")
    q = (t % S) * (T // S) + t // S
    local = (idx >= e0) & (idx < e0 + El)
    per_row = torch.zeros(T, dtype=torch.int64, device="cuda")
    per_row[q] = local.sum(1)
    tok_off = torch.cat([per_row.new_zeros(1), per_row.cumsum(0)])
    slot = tok_off[q][:, None] + local.cumsum(1) - 1
    a = torch.arange(T * k, device="cuda")[local.view(-1)]
    order = torch.argsort(idx.view(-1)[a], stable=True)
    row_src, row_dst = a[order], slot.view(-1)[a][order]
    counts = torch.bincount(idx.view(-1)[a] - e0, minlength=El)
    offsets = torch.cat([counts.new_zeros(1), counts.cumsum(0)])
    cap = T * min(k, El)

    def padded(x):  # as the library hands it over: cap entries, those behind the last row unused
        return torch.cat([x, x.new_zeros(cap - x.numel())]).to(torch.int32)

    return dict(A=int(a.numel()), cap=cap, row_src=padded(row_src), row_dst=padded(row_dst),
                offsets=offsets.to(torch.int32), bounds=offsets.tolist())


def _slots(g, A, cap, width, std):
    out = torch.zeros(cap, width, dtype=torch.bfloat16, device="cuda")
    out[:A] = _rand(g, A, width, std=std)
    return out


def _int8(g, amax, *shape):
    """Codes and scales as normal rows quantised by their largest value have them."""
    codes = torch.empty(shape, dtype=torch.int8, device="cuda")
    flat = codes.view(-1)
    for a in range(0, flat.numel(), 1 << 28):
        n = min(1 << 28, flat.numel() - a)
        flat[a:a + n] = torch.randn(n, generator=g, device="cuda").mul_(32).round_().clamp_(-127, 127)
    scales = (1 + 0.2 * torch.randn(shape[:-1], generator=g, device="cuda").clamp(-3, 3)) * (amax / 127)
    return codes, scales


def _mxint8(g, std, rows, used, cols):
    """MXINT8 codes and scales of normal values in the first `used` of `rows` rows."""
    codes = torch.zeros(rows, cols, dtype=torch.int8, device="cuda")
    scales = torch.full((rows, cols // 32), 127, dtype=torch.uint8, device="cuda")
    step = max(1, (1 << 27) // cols)
    for a in range(0, used, step):
        b = min(used, a + step)
        x = _rand(g, b - a, cols, std=std, dtype=torch.float32).view(b - a, cols // 32, 32)
        e = torch.frexp(x.abs().amax(2)).exponent - 1
        codes[a:b] = torch.ldexp(x, 6 - e[..., None]).round_().clamp_(-127, 127).view(b - a, cols)
        scales[a:b] = (e + 127).to(torch.uint8)
    return codes, scales


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    op = case["op"]
    if op.endswith("quantize"):
        x = _rand(g, case["rows"], case["cols"], dtype=torch.float32 if case["fp32"] else torch.bfloat16)
        # channels of unlike size, as activations have them
        x *= torch.exp2(1.5 * torch.randn(case["cols"], generator=g, device="cuda")).to(x.dtype)
        st = dict(x=x)
    else:
        st = _rows_of(case, g)
        T, d, f, El, A, cap = case["T"], case["d"], case["f"], case["E_l"], st["A"], st["cap"]
        if op == "int8_linear1":
            (st["x"], st["xs"]), (st["w"], st["ws"]) = _int8(g, 4.0, T, d), _int8(g, 0.08, El, 2 * f, d)
        elif op == "int8_linear2":
            (st["x"], st["xs"]), (st["w"], st["ws"]) = _int8(g, 4.0, cap, f), _int8(g, 0.08, El, d, f)
        else:
            st.update(W1=_rand(g, El, 2 * f, d, std=0.02), W2=_rand(g, El, d, f, std=0.02))
            if op == "checkpoint_forward" or not case["x8"]:
                st.update(X=_rand(g, T, d), xs=None)
            else:
                st["X"], st["xs"] = _mxint8(g, 1.0, T, T, d)
            if op == "checkpoint_backward":
                st["gu8"], st["gus"] = _mxint8(g, 0.02 * math.sqrt(d), cap, A, 2 * f)
                st["dO"] = _slots(g, A, cap, d, 0.02)
    st["case"] = dict(case)
    _buffers(st)
    if own:
        _plan(st)
    return st


def _buffers(st):
    """The output buffers a program keeps from step to step. Row buffers have the row capacity; the rows behind the
    batch's last are left as they are."""
    c, op = st["case"], st["case"]["op"]

    def new(*shape, dtype=torch.bfloat16):
        return torch.zeros(shape, dtype=dtype, device="cuda")

    if op.endswith("quantize"):
        st["out"] = new(c["rows"], c["cols"], dtype=torch.float32 if op == "int8_quantize" else torch.bfloat16)
        return
    d, f, El, cap = c["d"], c["f"], c["E_l"], st["cap"]
    if op == "int8_linear1":
        st["out"] = new(cap, f)
    elif op == "int8_linear2":
        st["out"] = new(cap, d, dtype=torch.bfloat16 if c["bf16_buf"] else torch.float32)
    elif op == "checkpoint_forward":
        st.update(out=new(cap, d), gu=new(cap, 2 * f))
    else:
        st.update(dxs=new(cap, d), dW1=new(El, 2 * f, d), dW2=new(El, d, f))


# ------------------------------------------------------------- the own calls
def _plan(st):
    """What a program keeps from step to step besides its buffers: the problem, the workspace, and room for codes."""
    import expert_grouped_gemm_amd as moe
    c, op = st["case"], st["case"]["op"]

    def codes(rows, cols, scale_shape, scale_dtype):
        return (torch.zeros(rows, cols, dtype=torch.int8, device="cuda"),
                torch.zeros(scale_shape, dtype=scale_dtype, device="cuda"))

    if op == "int8_quantize":
        st["codes"], st["scales"] = codes(c["rows"], c["cols"], (c["rows"],), torch.float32)
        return
    if op == "mxint8_quantize":
        st["codes"], st["scales"] = codes(c["rows"], c["cols"], (c["rows"], c["cols"] // 32), torch.uint8)
        return
    p = moe.make_problem(c["T"], c["d"], c["f"], c["E"], c["k"], c["e_begin"], c["e_begin"] + c["E_l"],
                         num_segments=c["S"], sched="auto",
                         bf16_combine_buf=op == "checkpoint_forward" or c.get("bf16_buf", False))
    st["p"] = p
    if op == "checkpoint_backward":
        st["workspace"] = moe.alloc_checkpoint_workspace(p)
    else:
        st["workspace"] = moe.alloc_workspace(p)
    if op == "checkpoint_forward":
        st["gu8"], st["gus"] = codes(st["cap"], 2 * c["f"], (st["cap"], c["f"] // 16), torch.uint8)


def _own(st):
    import expert_grouped_gemm_amd as moe
    op = st["case"]["op"]
    if op == "int8_quantize":
        moe.int8_quantize(st["x"], st["codes"], st["scales"])
        moe.int8_dequantize(st["codes"], st["scales"], st["out"])
        return [st["out"]]
    if op == "mxint8_quantize":
        moe.mxint8_quantize(st["x"], st["codes"], st["scales"])
        moe.mxint8_dequantize(st["codes"], st["scales"], st["out"])
        return [st["out"]]
    p = st["p"]
    if op == "int8_linear1":
        moe.int8_linear1(p, st["x"], st["xs"], st["row_src"], st["offsets"], st["w"], st["ws"], st["out"],
                         st["workspace"])
        return [st["out"]]
    if op == "int8_linear2":
        moe.int8_linear2(p, st["x"], st["xs"], st["offsets"], st["row_dst"], st["w"], st["ws"], st["out"],
                         st["workspace"])
        return [st["out"]]
    if op == "checkpoint_forward":
        moe.expert_forward_checkpoint(p, st["X"], st["row_src"], st["offsets"], st["row_dst"], st["W1"], st["W2"],
                                      st["gu8"], st["gus"], st["out"], st["workspace"])
        moe.mxint8_dequantize(st["gu8"][:st["A"]], st["gus"][:st["A"]], st["gu"][:st["A"]])
        return [st["out"], st["gu"]]
    moe.expert_backward_checkpoint(p, st["X"], st["xs"], st["row_src"], st["offsets"], st["row_dst"], st["gu8"],
                                   st["gus"], st["W1"], st["W2"], st["dO"], st["dxs"], st["dW1"], st["dW2"],
                                   st["workspace"])
    return [st["dxs"], st["dW1"], st["dW2"]]


# ------------------------------------------------------------ the plain forms
def _int8_values(x):
    """What 8-bit integers with a scale for each row keep of x: the scale is the row's largest magnitude / 127, a code
    127 x over that magnitude, rounded to nearest even. In 64 bits up to the code: ratios of bf16 values often lie
    halfway between two codes."""
    x = x.double()
    amax = x.abs().amax(1, keepdim=True)
    scale = torch.where(amax > 0, (amax / 127).float(), 1.0)
    return torch.round(x * 127 / torch.where(amax > 0, amax, 1.0)).float() * scale


def _pow2(e):
    """2^e in fp32, exactly, for whole e from -126 to 127."""
    return ((e.to(torch.int32) + 127) << 23).view(torch.float32)


def _mxint8_values(x):
    """What MXINT8 keeps of x [R, K]: per 32 along K a scale 2^floor(log2 amax) (2^-120 at least), and elements of
    that scale / 64, rounded to nearest even, at most 127 in magnitude."""
    R, K = x.shape
    b = x.float().view(R, K // 32, 32)
    amax = b.abs().amax(2, keepdim=True)
    e = torch.where(amax > 0, (torch.frexp(amax).exponent - 1).clamp(min=-120), 0)
    return (torch.round(b * _pow2(6 - e)).clamp(-127, 127) * _pow2(e - 6)).view(R, K)


def _decode(codes, scales):
    """MXINT8 codes and E8M0 scales as fp32 values."""
    R, K = codes.shape
    step = _pow2(scales.to(torch.int32) - 133)
    return (codes.float().view(R, K // 32, 32) * step[..., None]).view(R, K)


def _plain(st):
    c = st["case"]
    op = c["op"]
    if op == "int8_quantize":
        st["out"].copy_(_int8_values(st["x"]))
        return [st["out"]]
    if op == "mxint8_quantize":
        st["out"].copy_(_mxint8_values(st["x"]))
        return [st["out"]]
    A, El, k, f = st["A"], c["E_l"], c["k"], c["f"]
    src, dst, bounds = st["row_src"][:A].long(), st["row_dst"][:A].long(), st["bounds"]
    if op == "int8_linear1":
        out = st["out"]
        for e in range(El):
            r = slice(bounds[e], bounds[e + 1])
            tok = src[r] // k
            y = (st["x"][tok].float() @ st["w"][e].float().t()) * st["xs"][tok][:, None] * st["ws"][e]
            gate, up = y.chunk(2, 1)
            out[r] = (gate * torch.sigmoid(gate) * up).to(torch.bfloat16)
        return [out]
    if op == "int8_linear2":
        out = st["out"]
        for e in range(El):
            r = slice(bounds[e], bounds[e + 1])
            y = (st["x"][r].float() @ st["w"][e].float().t()) * st["xs"][r][:, None] * st["ws"][e]
            out[dst[r]] = y.to(out.dtype)
        return [out]
    if op == "checkpoint_forward":
        out, gu = st["out"], st["gu"]
        for e in range(El):
            r = slice(bounds[e], bounds[e + 1])
            y = st["X"][src[r] // k].float() @ st["W1"][e].float().t()
            gu[r] = _mxint8_values(y).to(torch.bfloat16)
            gate, up = y.chunk(2, 1)
            out[dst[r]] = ((gate * torch.sigmoid(gate) * up) @ st["W2"][e].float().t()).to(torch.bfloat16)
        return [out, gu]
    dxs, dW1, dW2 = st["dxs"], st["dW1"], st["dW2"]
    X = st["X"].float() if st["xs"] is None else _decode(st["X"], st["xs"])
    for e in range(El):
        r = slice(bounds[e], bounds[e + 1])
        x, do = X[src[r] // k], st["dO"][dst[r]].float()
        w1, w2 = st["W1"][e].float(), st["W2"][e].float()
        gate, up = _decode(st["gu8"][r], st["gus"][r]).chunk(2, 1)
        s = torch.sigmoid(gate)
        act, da = gate * s * up, do @ w2
        dh = torch.cat([da * up * s * (1 + gate * (1 - s)), da * gate * s], 1)
        dxs[dst[r]] = (dh @ w1).to(torch.bfloat16)
        dW1[e] = dh.t() @ x
        dW2[e] = do.t() @ act
    return [dxs, dW1, dW2]


def run(state):
    return _own(state) if own else _plain(state)


# ------------------------------------------------------- the work of one pass
def work(case):
    c, op = case, case["op"]
    if op.endswith("quantize"):
        n = c["rows"] * c["cols"]
        scales = 4 * c["rows"] if op == "int8_quantize" else n // 32
        # the values in, codes and scales out and in again, the values they stand for out
        return {"bytes": n * (4 if c["fp32"] else 2) + 2 * (n + scales) + n * (4 if op == "int8_quantize" else 2),
                "flops": 0}
    T, d, f, El, k = c["T"], c["d"], c["f"], c["E_l"], c["k"]
    A = _expected_rows(c)
    reached = El * (1 - (1 - min(1.0, k / c["E"])) ** T)  # experts with a row: only their weights are read
    if op == "int8_linear1":
        return {"bytes": T * (d + 4) + reached * 2 * f * (d + 4) + 2 * A * f, "flops": 4 * A * d * f}
    if op == "int8_linear2":
        return {"bytes": A * (f + 4) + reached * d * (f + 4) + A * d * (2 if c["bf16_buf"] else 4),
                "flops": 2 * A * d * f}
    gu = A * 2 * f * 33 / 32
    if op == "checkpoint_forward":
        # the checkpoint out, and in again for the values it stands for
        return {"bytes": 2 * T * d + 2 * reached * 3 * d * f + 2 * gu + 4 * A * f + 2 * A * d, "flops": 6 * A * d * f}
    return {"bytes": T * d * (33 / 32 if c["x8"] else 2) + gu + 4 * A * d + 2 * 6 * El * d * f,
            "flops": 12 * A * d * f}


# ----------------------------------------------- the definitions, in 64 bits
def _mx_exact(x):
    """x fp64 [R, K] on the MXINT8 grid of its blocks."""
    b = x.unflatten(1, (-1, 32))
    top = b.abs().amax(2, keepdim=True)
    expo = torch.floor(torch.log2(torch.where(top > 0, top, 1.0)))
    # the logarithm's rounding, put right at the borders
    expo = expo - (torch.exp2(expo) > top).double() * (top > 0) + (torch.exp2(expo + 1) <= top).double()
    unit = torch.exp2(expo.clamp(min=-120) - 6)
    return (torch.clamp((b / unit).round(), -127, 127) * unit).flatten(1)


def _mx_values(codes, scales):
    return codes.double() * torch.exp2(scales.double() - 133).repeat_interleave(32, 1)


def exact(case, seed):
    st = prepare(case, seed)
    c, op = case, case["op"]
    if op.endswith("quantize"):
        out = torch.empty(c["rows"], c["cols"], dtype=torch.float64, device="cuda")
        for a in range(0, c["rows"], 4096):
            x = st["x"][a:a + 4096].double()
            if op == "mxint8_quantize":
                out[a:a + 4096] = _mx_exact(x)
            else:
                amax = x.abs().amax(1, keepdim=True)
                halves = torch.where(amax > 0, 254 * x.abs() / amax, 0.0)  # in half codes, exact where it is whole
                code = torch.div(halves + 1, 2, rounding_mode="floor")
                code = code - ((halves == 2 * code - 1) & (code % 2 == 1)).double()  # a tie goes to the even one
                out[a:a + 4096] = torch.sign(x) * code * amax / 127
        return [out]
    A, d, f, El, k, cap = st["A"], c["d"], c["f"], c["E_l"], c["k"], st["cap"]
    tok, dst, b = st["row_src"][:A].long() // k, st["row_dst"][:A].long(), st["bounds"]
    if 12 * A * d * f > 4e13:
        return None

    def zeros(*shape):
        return torch.zeros(shape, dtype=torch.float64, device="cuda")

    if op == "int8_linear1" or op == "int8_linear2":
        first = op == "int8_linear1"
        out = zeros(cap, f if first else d)
        for e in range(El):
            rows = torch.arange(b[e], b[e + 1], device="cuda")
            at = tok[rows] if first else rows
            x = st["x"][at].double() * st["xs"][at].double()[:, None]
            w = st["w"][e].double() * st["ws"][e].double()[:, None]
            if first:
                g, u = torch.mm(x, w[:f].t()), torch.mm(x, w[f:].t())
                out[rows] = g / (1 + torch.exp(-g)) * u
            else:
                out[dst[rows]] = torch.mm(x, w.t())
        return [out]
    if op == "checkpoint_forward":
        out, gu = zeros(cap, d), zeros(cap, 2 * f)
        for e in range(El):
            rows = torch.arange(b[e], b[e + 1], device="cuda")
            x, w1 = st["X"][tok[rows]].double(), st["W1"][e].double()
            g, u = torch.mm(x, w1[:f].t()), torch.mm(x, w1[f:].t())
            gu[rows, :f], gu[rows, f:] = _mx_exact(g), _mx_exact(u)
            out[dst[rows]] = torch.mm(g / (1 + torch.exp(-g)) * u, st["W2"][e].double().t())
        return [out, gu]
    X = st["X"].double() if st["xs"] is None else _mx_values(st["X"], st["xs"])
    gu = _mx_values(st["gu8"][:A], st["gus"][:A])
    dxs, dW1, dW2 = zeros(cap, d), zeros(El, 2 * f, d), zeros(El, d, f)
    for e in range(El):
        rows = torch.arange(b[e], b[e + 1], device="cuda")
        x, do = X[tok[rows]], st["dO"][dst[rows]].double()
        wg, wu = st["W1"][e, :f].double(), st["W1"][e, f:].double()
        g, u = gu[rows, :f], gu[rows, f:]
        sig = 1 / (1 + torch.exp(-g))
        da = torch.mm(do, st["W2"][e].double())
        dg, du = da * u * (sig + g * sig * (1 - sig)), da * g * sig
        dxs[dst[rows]] = torch.mm(dg, wg) + torch.mm(du, wu)
        dW1[e, :f], dW1[e, f:] = torch.mm(dg.t(), x), torch.mm(du.t(), x)
        dW2[e] = torch.mm(do.t(), g * sig * u)
    return [dxs, dW1, dW2]
