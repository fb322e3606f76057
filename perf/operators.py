"""Cases, plain forms and calls of the expert layer's backward pass and its MXFP4 products.

A case names an operator (`op`) and the share's shape: T tokens of width d,
E experts of which [e_begin, e_begin + E_l) are local, k experts per token,
S destination segments of the output rows, expert width f, and `zipf` > 0 for
a router that favours some experts. The quantiser's cases are rows x cols.

With `own` false, `run` computes an operator with elementary torch operations
in fp32; with `own` true it makes the package's calls on the same inputs.
"""
import math
import random

import torch

own = False


# ---------------------------------------------------------------- the cases
def listed():
    share = dict(T=4096, d=7168, E=256, k=8, e_begin=0, E_l=32, S=8, zipf=0.0)
    mixtral = dict(d=4096, f=14336, E=8, k=2, e_begin=0, E_l=8, S=1, zipf=0.0)
    return [
        # the smallest layer the package is configured with: launch latency
        dict(name="combine-bwd-tiny", op="combine_backward", T=64, d=128, E=4, k=2, e_begin=0, E_l=4, S=1, zipf=0.0,
             bf16_buf=False, logits=True),
        # a fine-grained share (32 of 256 experts) in a training step
        dict(name="combine-bwd-share", op="combine_backward", **share, bf16_buf=False, logits=True),
        dict(name="dispatch-bwd-share", op="dispatch_backward", **share),
        # long sequences, a skewed router, every expert local
        dict(name="dispatch-bwd-skewed", op="dispatch_backward", T=32768, d=2048, E=64, k=4, e_begin=0, E_l=64, S=1,
             zipf=1.2),
        # a few odd tokens: ragged bands, experts without rows
        dict(name="expert-bwd-small", op="expert_backward", T=201, d=384, f=640, E=16, k=2, e_begin=3, E_l=9, S=1,
             zipf=1.2),
        # weights and their gradients streamed once against ~128 rows per expert
        dict(name="expert-bwd-share", op="expert_backward", **share, f=2048),
        # wide experts with thousands of rows: the matrix units
        dict(name="expert-bwd-mixtral", op="expert_backward", T=8192, **mixtral),
        # the tokens of one decoding step
        dict(name="mxfp4-quant-decode", op="mxfp4_quantize", rows=16, cols=7168, fp32=False),
        # one expert's gate and up weights out of fp32 master weights
        dict(name="mxfp4-quant-weights", op="mxfp4_quantize", rows=28672, cols=4096, fp32=True),
        # a decoding step through the share: the weights' bytes
        dict(name="mxfp4-linear1-decode", op="mxfp4_linear1", **dict(share, T=64, S=1), f=2048),
        # a training- or prefill-sized batch through the share
        dict(name="mxfp4-linear2-share", op="mxfp4_linear2", **share, f=2048, bf16_buf=False),
        # prefill through wide experts: the matrix units
        dict(name="mxfp4-linear1-mixtral", op="mxfp4_linear1", T=8192, **mixtral),
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
    op = rng.choice(["combine_backward", "dispatch_backward", "expert_backward", "mxfp4_quantize", "mxfp4_linear1",
                     "mxfp4_linear2"])
    if op == "mxfp4_quantize":
        cols = 32 * _log(rng, 4, 448)
        return dict(op=op, rows=_log(rng, 1, max(2, min(65536, 28672 * 4096 // cols))), cols=cols,
                    fp32=rng.random() < 0.5)
    E = rng.choice([4, 8, 16, 64, 160, 256])
    k = rng.randint(1, min(8, E))
    E_l = max(1, E // rng.choice([1, 1, 2, 8]))
    case = dict(op=op, d=128 * _log(rng, 1, 56), E=E, k=k, e_begin=rng.randint(0, E - E_l), E_l=E_l,
                zipf=rng.choice([0.0, 0.0, 1.2]))
    if case["zipf"] > 0:  # the share that holds the favoured experts
        case["e_begin"] = rng.randint(0, min(3, E - E_l))
    rows = case["d"] * min(k, E_l)
    if op in ("combine_backward", "dispatch_backward"):
        # at most the gathered bytes of the largest listed cases
        case["T"] = _log(rng, 1, max(2, min(32768, 131072 * 2048 // (2 * rows))))
        if op == "combine_backward":
            case.update(bf16_buf=rng.random() < 0.5, logits=rng.random() < 0.7)
    else:
        case["f"] = 128 * _log(rng, 1, 112)
        while E_l * case["d"] * case["f"] > 8 * 4096 * 14336:
            case["f"] = max(128, case["f"] // 256 * 128)
        flops = 16384 * 4096 * 14336 // (case["d"] * case["f"] * min(k, E_l))
        case["T"] = _log(rng, 1, max(2, min(8192, flops // 2, 2 ** 30 // (max(case["d"], case["f"]) * k))))
        if op == "mxfp4_linear2":
            case["bf16_buf"] = rng.random() < 0.5
    if _expected_rows(case) < 32:  # a few tokens: every expert local, so that there are rows
        case.update(e_begin=0, E_l=E)
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
    top, idx = torch.topk(logits, k, dim=1)
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

    return dict(A=int(a.numel()), cap=cap, topk_idx=idx.to(torch.int32).contiguous(),
                topk_w=torch.softmax(top, 1).contiguous(), tok_off=tok_off.to(torch.int32), row_src=padded(row_src),
                row_dst=padded(row_dst), offsets=offsets.to(torch.int32), bounds=offsets.tolist())


def _slots(g, case, A, cap, width, std, dtype):
    out = torch.zeros(cap, width, dtype=dtype, device="cuda")
    out[:A] = _rand(g, A, width, std=std, dtype=dtype)
    return out


def _mxfp4(g, mid, *shape):
    """Codes and scales as quantised normal values have them: every code, scales within an octave of 2^(mid - 127)."""
    codes = torch.randint(0, 256, shape[:-1] + (shape[-1] // 2,), generator=g, device="cuda", dtype=torch.uint8)
    scales = torch.randint(mid - 1, mid + 2, shape[:-1] + (shape[-1] // 32,), generator=g, device="cuda",
                           dtype=torch.uint8)
    return codes, scales


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    op = case["op"]
    if op == "mxfp4_quantize":
        x = _rand(g, case["rows"], case["cols"], dtype=torch.float32 if case["fp32"] else torch.bfloat16)
        # channels of unlike size, as weights and activations have them
        x *= torch.exp2(4 * torch.randn(case["cols"], generator=g, device="cuda")).to(x.dtype)
        st = dict(x=x)
    else:
        st = _rows_of(case, g)
        T, d, El, A, cap = case["T"], case["d"], case["E_l"], st["A"], st["cap"]
        f = case.get("f", 0)
        if op == "combine_backward":
            st.update(dY=_rand(g, T, d, std=0.02), buf=_slots(
                g, case, A, cap, d, 0.3, torch.bfloat16 if case["bf16_buf"] else torch.float32))
        elif op == "dispatch_backward":
            st.update(dxs=_slots(g, case, A, cap, d, 0.02, torch.bfloat16))
        elif op == "expert_backward":
            st.update(X=_rand(g, T, d), dO=_slots(g, case, A, cap, d, 0.02, torch.bfloat16),
                      W1=_rand(g, El, 2 * f, d, std=0.02), W2=_rand(g, El, d, f, std=0.02))
        elif op == "mxfp4_linear1":
            (st["x"], st["xs"]), (st["w"], st["ws"]) = _mxfp4(g, 125, T, d), _mxfp4(g, 118, El, 2 * f, d)
        else:
            (st["x"], st["xs"]), (st["w"], st["ws"]) = _mxfp4(g, 123, cap, f), _mxfp4(g, 118, El, d, f)
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

    if op == "mxfp4_quantize":
        st["out"] = new(c["rows"], c["cols"])
        return
    T, d, El, cap, f = c["T"], c["d"], c["E_l"], st["cap"], c.get("f", 0)
    if op == "combine_backward":
        st.update(d_buf=new(cap, d), d_w=new(T, c["k"], dtype=torch.float32),
                  d_logits=new(T, c["E"], dtype=torch.float32) if c["logits"] else None)
    elif op == "dispatch_backward":
        st["dX"] = new(T, d)
    elif op == "expert_backward":
        st.update(dxs=new(cap, d), dW1=new(El, 2 * f, d), dW2=new(El, d, f))
    elif op == "mxfp4_linear1":
        st["out"] = new(cap, f)
    else:
        st["out"] = new(cap, d, dtype=torch.bfloat16 if c["bf16_buf"] else torch.float32)


# ------------------------------------------------------------- the own calls
def _plan(st):
    """What a program keeps from step to step besides its buffers: the problem and the workspace."""
    import expert_grouped_gemm_amd as moe
    c, op = st["case"], st["case"]["op"]
    if op == "mxfp4_quantize":
        R, C = c["rows"], c["cols"]
        st.update(codes=torch.empty(R, C // 2, dtype=torch.uint8, device="cuda"),
                  scales=torch.empty(R, C // 32, dtype=torch.uint8, device="cuda"))
        return
    p = moe.make_problem(c["T"], c["d"], c.get("f", 128), c["E"], c["k"], c["e_begin"], c["e_begin"] + c["E_l"],
                         num_segments=c["S"], sched="auto", bf16_combine_buf=c.get("bf16_buf", False))
    st["p"] = p
    if op == "expert_backward":
        st["workspace"] = moe.alloc_backward_workspace(p)
    elif op.startswith("mxfp4"):
        st["workspace"] = moe.alloc_workspace(p)


def _own(st):
    import expert_grouped_gemm_amd as moe
    op = st["case"]["op"]
    if op == "mxfp4_quantize":
        moe.mxfp4_quantize(st["x"], st["codes"], st["scales"])
        moe.mxfp4_dequantize(st["codes"], st["scales"], st["out"])
        return [st["out"]]
    p = st["p"]
    if op == "combine_backward":
        moe.combine_backward(p, st["dY"], st["buf"], st["tok_off"], st["topk_idx"], st["topk_w"], st["d_buf"],
                             st["d_w"], st["d_logits"])
        return [st["d_buf"], st["d_w"]] + ([] if st["d_logits"] is None else [st["d_logits"]])
    if op == "dispatch_backward":
        moe.dispatch_backward(p, st["dxs"], st["tok_off"], st["dX"])
        return [st["dX"]]
    if op == "expert_backward":
        moe.expert_backward(p, st["X"], st["row_src"], st["offsets"], st["row_dst"], st["W1"], st["W2"], st["dO"],
                            st["dxs"], st["dW1"], st["dW2"], st["workspace"])
        return [st["dxs"], st["dW1"], st["dW2"]]
    if op == "mxfp4_linear1":
        moe.mxfp4_linear1(p, st["x"], st["xs"], st["row_src"], st["offsets"], st["w"], st["ws"], st["out"],
                          st["workspace"])
    else:
        moe.mxfp4_linear2(p, st["x"], st["xs"], st["offsets"], st["row_dst"], st["w"], st["ws"], st["out"],
                          st["workspace"])
    return [st["out"]]


# ------------------------------------------------------------ the plain forms
def _row_of_token(T, S):
    t = torch.arange(T, device="cuda")
    return (t % S) * (T // S) + t // S


def _pow2(e):
    """2^e in fp32, exactly, for whole e from -127 to 127."""
    e = e.to(torch.int32)
    return torch.where(e > -127, (e + 127) << 23, 1 << 22).to(torch.int32).view(torch.float32)


def _quantized(x):
    """The values MXFP4 keeps of x [R, K]: per 32 along K a scale 2^(floor(log2 amax) - 2) and E2M1 elements,
    rounded to nearest even, at most 6 scales."""
    R, K = x.shape
    b = x.float().view(R, K // 32, 32)
    amax = b.abs().amax(2, keepdim=True)
    e = (torch.frexp(amax).exponent - 3).clamp(-127, 127)
    scale = _pow2(torch.where(amax > 0, e, 0))
    y = (b / scale).abs()
    step = torch.where(y < 2, 0.5, torch.where(y < 4, 1.0, 2.0))
    v = torch.clamp(torch.round(y / step) * step, max=6.0)
    return (torch.copysign(v, b) * scale).view(R, K)


def _decode(codes, scales):
    """MXFP4 codes (even element in the low nibble) and E8M0 scales as fp32 values."""
    R, K = codes.shape[0], codes.shape[1] * 2
    nib = torch.stack([codes & 15, codes >> 4], -1).view(R, K).to(torch.int64)
    table = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6, -0.0, -0.5, -1, -1.5, -2, -3, -4, -6], device="cuda")
    unit = _pow2(scales.to(torch.int32) - 127)
    return (table[nib].view(R, K // 32, 32) * unit[..., None]).view(R, K)


def _plain(st):
    c = st["case"]
    op = c["op"]
    if op == "mxfp4_quantize":
        st["out"].copy_(_quantized(st["x"]))
        return [st["out"]]
    A, T, d, El, k = st["A"], c["T"], c["d"], c["E_l"], c["k"]
    if op == "combine_backward":
        q = _row_of_token(T, c["S"])
        idx, w = st["topk_idx"].long(), st["topk_w"]
        local = (idx >= c["e_begin"]) & (idx < c["e_begin"] + El)
        slot = st["tok_off"].long()[q][:, None] + local.cumsum(1) - 1
        dY = st["dY"].float()[q]
        d_w = (st["buf"][torch.where(local, slot, 0)].float() * dY[:, None, :]).sum(2) * local
        st["d_buf"][slot[local]] = (w[:, :, None] * dY[:, None, :])[local].to(torch.bfloat16)
        res = [st["d_buf"], d_w]
        if c["logits"]:
            dl = w * (d_w - (w * d_w).sum(1, keepdim=True))
            res.append(torch.zeros(T, c["E"], device="cuda").scatter_add_(1, idx, dl))
        return res
    if op == "dispatch_backward":
        q = _row_of_token(T, c["S"])
        off = st["tok_off"].long()
        slot = off[q][:, None] + torch.arange(min(k, El), device="cuda")
        mine = slot < off[q + 1][:, None]
        rows = st["dxs"][torch.where(mine, slot, 0)].float()
        return [(rows * mine[:, :, None]).sum(1).to(torch.bfloat16)]
    src, dst, bounds = st["row_src"][:A].long(), st["row_dst"][:A].long(), st["bounds"]
    if op == "expert_backward":
        dxs, dW1, dW2 = st["dxs"], st["dW1"], st["dW2"]
        for e in range(El):
            r = slice(bounds[e], bounds[e + 1])
            x, do = st["X"][src[r] // k].float(), st["dO"][dst[r]].float()
            w1, w2 = st["W1"][e].float(), st["W2"][e].float()
            gate, up = (x @ w1.t()).chunk(2, 1)
            s = torch.sigmoid(gate)
            act, da = gate * s * up, do @ w2
            dh = torch.cat([da * up * s * (1 + gate * (1 - s)), da * gate * s], 1)
            dxs[dst[r]] = (dh @ w1).to(torch.bfloat16)
            dW1[e] = dh.t() @ x
            dW2[e] = do.t() @ act
        return [dxs, dW1, dW2]
    if op == "mxfp4_linear1":
        x = _decode(st["x"], st["xs"])
        out = st["out"]
        for e in range(El):
            r = slice(bounds[e], bounds[e + 1])
            gate, up = (x[src[r] // k] @ _decode(st["w"][e], st["ws"][e]).t()).chunk(2, 1)
            out[r] = (gate * torch.sigmoid(gate) * up).to(torch.bfloat16)
        return [out]
    out = st["out"]
    for e in range(El):
        r = slice(bounds[e], bounds[e + 1])
        out[dst[r]] = (_decode(st["x"][r], st["xs"][r]) @ _decode(st["w"][e], st["ws"][e]).t()).to(out.dtype)
    return [out]


def run(state):
    return _own(state) if own else _plain(state)


# ------------------------------------------------------- the work of one pass
def work(case):
    c, op = case, case["op"]
    if op == "mxfp4_quantize":
        n = c["rows"] * c["cols"]
        # the values in, codes and scales out and in again, the values they stand for out
        return {"bytes": n * (4 if c["fp32"] else 2) + 2 * n * 17 // 32 + 2 * n, "flops": 0}
    T, d, El, k, f = c["T"], c["d"], c["E_l"], c["k"], c.get("f", 0)
    A = _expected_rows(c)
    if op == "combine_backward":
        buf = 2 if c["bf16_buf"] else 4
        return {"bytes": 2 * T * d + A * d * (buf + 2) + 12 * T * k + (4 * T * c["E"] if c["logits"] else 0),
                "flops": 3 * A * d}
    if op == "dispatch_backward":
        return {"bytes": 2 * A * d + 2 * T * d, "flops": A * d}
    if op == "expert_backward":
        return {"bytes": 2 * T * d + 4 * A * d + 2 * 6 * El * d * f, "flops": 16 * A * d * f}
    reached = El * (1 - (1 - min(1.0, k / c["E"])) ** T)  # experts with a row: only their weights are read
    if op == "mxfp4_linear1":
        return {"bytes": (T * d + reached * 2 * f * d) * 17 / 32 + 2 * A * f, "flops": 4 * A * d * f}
    return {"bytes": (A * f + reached * f * d) * 17 / 32 + A * d * (2 if c["bf16_buf"] else 4), "flops": 2 * A * d * f}


# ----------------------------------------------- the definitions, in 64 bits
def exact(case, seed):
    st = prepare(case, seed)
    c, op = case, case["op"]
    e2m1 = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64, device="cuda")

    def two_to(n):  # the exponent field of an fp64 value
        return ((n.long() + 1023) << 52).view(torch.float64)

    def values(codes, scales):  # one row block of MXFP4 in fp64
        n = codes.shape[1] * 2
        nib = torch.empty(codes.shape[0], n, dtype=torch.long, device="cuda")
        nib[:, 0::2], nib[:, 1::2] = (codes % 16).long(), (codes // 16).long()
        mag = e2m1[nib % 8] * (1 - 2 * (nib // 8)).double()
        return mag * two_to(scales.long() - 127).repeat_interleave(32, 1)

    if op == "mxfp4_quantize":
        out = torch.empty(case["rows"], case["cols"], dtype=torch.float64, device="cuda")
        bounds = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], dtype=torch.float64, device="cuda")
        for a in range(0, case["rows"], 4096):
            x = st["x"][a:a + 4096].double()
            blocks = x.unflatten(1, (-1, 32))
            top = blocks.abs().amax(2)
            expo = torch.floor(torch.log2(torch.where(top > 0, top, 1.0))).long()
            # the logarithm's rounding, put right at the borders
            expo = expo - (two_to(expo) > top).long() + (two_to(expo + 1) <= top).long()
            unit = two_to(torch.where(top > 0, (expo - 2).clamp(-127, 127), 0))[:, :, None]
            y = blocks.abs() / unit
            code = torch.bucketize(y, bounds)  # a tie stays below ...
            for tie in (0.75, 1.75, 3.5):      # ... but for those whose even code is above
                code = code + (y == tie)
            out[a:a + 4096] = (torch.sign(blocks) * e2m1[code] * unit).flatten(1)
        return [out]
    A, T, d, El, k = st["A"], c["T"], c["d"], c["E_l"], c["k"]
    src, dst, b = st["row_src"][:A].long(), st["row_dst"][:A].long(), st["bounds"]
    tok, S = src // k, c["S"]
    row = (tok % S) * (T // S) + tok // S  # output row of each local assignment
    step = max(1, (1 << 28) // d)          # rows of fp64 in flight
    if op == "combine_backward":
        w = st["topk_w"].double()
        d_buf = torch.zeros(st["cap"], d, dtype=torch.float64, device="cuda")
        d_w = torch.zeros(T * k, dtype=torch.float64, device="cuda")
        for a in range(0, A, step):
            r = slice(a, min(A, a + step))
            dy = st["dY"][row[r]].double()
            d_buf[dst[r]] = w.view(-1)[src[r]][:, None] * dy
            d_w[src[r]] = (st["buf"][dst[r]].double() * dy).sum(1)
        d_w = d_w.view(T, k)
        res = [d_buf, d_w]
        if c["logits"]:
            # the softmax's Jacobian, diag(w) - w w^T, applied to the gate gradients
            jac = torch.diag_embed(w) - w[:, :, None] * w[:, None, :]
            dl = torch.zeros(T, c["E"], dtype=torch.float64, device="cuda")
            dl.scatter_add_(1, st["topk_idx"].long(), (jac * d_w[:, None, :]).sum(2))
            res.append(dl)
        return res
    if op == "dispatch_backward":
        dX = torch.zeros(T, d, dtype=torch.float64, device="cuda")
        for a in range(0, A, step):
            r = slice(a, min(A, a + step))
            dX.index_add_(0, tok[r], st["dxs"][dst[r]].double())
        return [dX]
    f = c["f"]
    if op == "expert_backward":
        if 16 * A * d * f > 4e13:
            return None
        dxs = torch.zeros(st["cap"], d, dtype=torch.float64, device="cuda")
        dW1 = torch.zeros(El, 2 * f, d, dtype=torch.float64, device="cuda")
        dW2 = torch.zeros(El, d, f, dtype=torch.float64, device="cuda")
        for e in range(El):
            lo, hi = b[e], b[e + 1]
            x, do = st["X"][tok[lo:hi]].double(), st["dO"][dst[lo:hi]].double()
            wg, wu, w2 = st["W1"][e, :f].double(), st["W1"][e, f:].double(), st["W2"][e].double()
            g, u = torch.mm(x, wg.t()), torch.mm(x, wu.t())
            sig = 1 / (1 + torch.exp(-g))
            da = torch.mm(do, w2)
            dg, du = da * u * (sig + g * sig * (1 - sig)), da * g * sig
            dxs[dst[lo:hi]] = torch.mm(dg, wg) + torch.mm(du, wu)
            dW1[e, :f], dW1[e, f:] = torch.mm(dg.t(), x), torch.mm(du.t(), x)
            dW2[e] = torch.mm(do.t(), g * sig * u)
        return [dxs, dW1, dW2]
    out = torch.zeros(st["cap"], f if op == "mxfp4_linear1" else d, dtype=torch.float64, device="cuda")
    for e in range(El):
        lo, hi = b[e], b[e + 1]
        w = values(st["w"][e], st["ws"][e])
        if op == "mxfp4_linear1":
            x = values(st["x"][tok[lo:hi]], st["xs"][tok[lo:hi]])
            g, u = torch.mm(x, w[:f].t()), torch.mm(x, w[f:].t())
            out[lo:hi] = g / (1 + torch.exp(-g)) * u
        else:
            out[dst[lo:hi]] = torch.mm(values(st["x"][lo:hi], st["xs"][lo:hi]), w.t())
    return [out]
