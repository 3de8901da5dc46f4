"""The expert stage between dispatch and combine, and the way back through it.

Four operators, each in its plain form (elementary torch operations in 32 bits) and as the calls a
user makes of combine_moe_get_amd:

  forward   experts_matmul: products grouped by expert over ragged rows, bf16 or int8, plain or with
            the SwiGLU gate; int8 rows come from dispatch or are quantised in the call
  backward  experts_matmul_dgrad and experts_matmul_wgrad: the gradients of the rows and of the weights
  mxfp4     quantize_rows and experts_matmul on microscaled 4-bit floats (e2m1 codes, one power of two
            per 32 of them)
  combine   combine_grad: the gradients of the weighted combine (rows, routing weights, special experts)
"""
import math

import torch

own = False

DEV = "cuda"

# ---- cases -------------------------------------------------------------------------------------


def _expert(name, kind, T, K, E, inf, outf, gated=False, dtype="bf16", quant=False, skew=0.5, grad32=False):
    """T tokens, K experts each of E; inf: contraction; outf: columns of the result; skew: spread of
    the experts' popularity (standard deviation of its logarithm)."""
    c = {"kind": kind, "T": T, "K": K, "E": E, "inf": inf, "outf": outf, "gated": gated, "dtype": dtype,
         "quant": quant, "skew": skew, "grad32": grad32}
    return dict(c, name=name) if name else c


def _combine(name, T, H, K, E, C=0, Kc=0, masked=0.0):
    c = {"kind": "combine", "T": T, "H": H, "K": K, "E": E, "C": C, "Kc": Kc, "masked": masked}
    return dict(c, name=name) if name else c


def listed():
    return [
        # one token of a chat: its eight experts' gate and up weights are read once
        _expert("one token, gated", "forward", 1, 8, 64, 4096, 1024, gated=True, skew=0.0),
        # one rank's share of a 4096-token decode batch over 32 ranks: 8 experts, about 128 rows each
        _expert("rank decode, down", "forward", 1024, 1, 8, 2048, 7168, skew=0.2),
        # a prefill batch on 64 experts, gate and up products
        _expert("prefill, gated", "forward", 4096, 8, 64, 7168, 1024, gated=True),
        # the same share of a decode batch as dispatch sends it in dynamic int8
        _expert("rank decode, int8 gated", "forward", 1024, 1, 8, 7168, 2048, gated=True, dtype="int8", skew=0.2),
        # odd sizes: the second product of an int8 layer, its rows quantised between the two
        _expert("odd rows, int8 down", "forward", 771, 8, 33, 2064, 4104, dtype="int8", quant=True, skew=1.0),
        # a fine-tuning step on a small batch and small experts
        _expert("small step", "backward", 100, 4, 16, 1024, 512, grad32=True),
        # odd sizes in training
        _expert("odd step", "backward", 1021, 3, 13, 1048, 2056, skew=1.0),
        # a training step of 4096 tokens, top-8
        _expert("training step", "backward", 4096, 8, 32, 4096, 2048),
        # decode of 16 sequences on 4-bit weights
        _expert("decode, 4-bit gated", "mxfp4", 16, 8, 64, 7168, 2048, gated=True, dtype="mxfp4", quant=True),
        # prefill on 4-bit weights
        _expert("prefill, 4-bit gated", "mxfp4", 4096, 8, 32, 4096, 2048, gated=True, dtype="mxfp4", quant=True),
        # the combine's gradient at one rank's batch and at a whole prefill batch with special experts
        _combine("combine gradient, 128", 128, 7168, 8, 256),
        _combine("combine gradient, special", 4096, 4096, 8, 128, C=2, Kc=2, masked=0.1),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["forward", "forward", "backward", "mxfp4", "combine"])
    K = rng.choice([1, 2, 3, 4, 6, 8])
    if kind == "combine":
        E = rng.choice([16, 64, 128, 256])
        special = rng.random() < 0.5
        T = _log(rng, 2, 4096)
        return _combine(None, T if T <= 512 else T // 16 * 16, 8 * _log(rng, 8, 896), K, E, rng.randint(1, 3) if special else 0,
                        rng.randint(0, 3) if special else 0, rng.choice([0.0, 0.1, 0.5]))
    E = max(K, _log(rng, 1, 64))
    T = _log(rng, 1, 4096) if kind != "backward" else _log(rng, 16, 4096)
    dtype = "mxfp4" if kind == "mxfp4" else rng.choice(["bf16", "bf16", "int8"]) if kind == "forward" else "bf16"
    step = {"bf16": 8, "int8": 16, "mxfp4": 32}[dtype]
    inf, outf = step * (_log(rng, 128, 7168) // step), 8 * _log(rng, 16, 512)
    gated = kind != "backward" and rng.random() < 0.5
    # no dearer than the largest listed ones
    nw = outf * (2 if gated else 1)
    while T * K * inf * nw > 32768 * 4096 * 2048:
        T = (T + 1) // 2
    while E > K and E * inf * nw > 32 * 4096 * 2048:
        E = max(K, E // 2)
    return _expert(None, kind, T, K, E, inf, outf, gated, dtype, dtype == "mxfp4" or (dtype == "int8" and rng.random() < 0.5),
                   rng.choice([0.0, 0.5, 1.0]), kind == "backward" and rng.random() < 0.5)


def _weight_rows(case):
    return case["outf"] * (2 if case["gated"] else 1)


def work(case):
    T, K, E = case["T"], case["K"], case["E"]
    if case["kind"] == "combine":
        n = T * K * (1 - case["masked"]) * E / (E + case["C"] + case["Kc"])
        H = case["H"]
        extra = 2 * T * H * 2 if case["C"] + case["Kc"] else 0
        return {"bytes": int(n * H * 4 + T * H * 2 + T * K * 16 + extra + case["Kc"] * H * 18), "flops": int(3 * T * K * H)}
    rows, nw, k = T * K, _weight_rows(case), case["inf"]
    hit = E * (1 - (1 - K / E) ** T)  # experts that get a row
    if case["kind"] == "backward":
        w32 = 4 if case["grad32"] else 2
        return {"bytes": int(rows * (nw + 2 * k) * 2 + hit * nw * k * 2 + E * nw * k * w32), "flops": 4 * rows * nw * k}
    size = {"bf16": 2, "int8": 1, "mxfp4": 17 / 32}[case["dtype"]]
    return {"bytes": int(rows * k * (2 if case["quant"] else size) + hit * nw * k * size + rows * case["outf"] * 2),
            "flops": 2 * rows * nw * k}


# ---- inputs ------------------------------------------------------------------------------------


def _normal(g, *shape, scale=1.0):
    return torch.randn(*shape, generator=g, device=DEV, dtype=torch.bfloat16).mul_(scale)


def _mx_round(v):
    """The nearest of 0, 0.5, 1, 1.5, 2, 3, 4, 6 (ties to the even code), sign kept, for float v."""
    a = v.abs()
    step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0))
    return torch.copysign((torch.round(a / step) * step).clamp(max=6.0), v)


def _mx_parts(x):
    """x [.., H] float -> (rounded elements [.., H/32, 32], exponent of their scale [.., H/32])."""
    b = x.unflatten(-1, (-1, 32))
    amax = b.abs().amax(-1)
    e = (torch.frexp(amax)[1] - 3).clamp(-127, 127)
    e = torch.where(amax == 0, -127, e)
    return _mx_round(torch.ldexp(b, -e[..., None].float())), e


def _mx_pack(x):
    """(codes [.., H/2], scales [.., H/32]) of x: two e2m1 codes a byte, the even element low."""
    r, e = _mx_parts(x.float())
    a = r.abs()
    code = torch.where(a < 2, a * 2, torch.where(a < 4, a + 2, a / 2 + 4)).to(torch.uint8)
    code = (code | (torch.signbit(r).to(torch.uint8) << 3)).flatten(-2)
    return code[..., 0::2] | (code[..., 1::2] << 4), (e + 127).to(torch.uint8)


def _route(case, g):
    """Receive rows of T tokens on K different experts each, expert-major: (rows, offsets [E + 1])."""
    T, K, E = case["T"], case["K"], case["E"]
    pop = torch.randn(E, generator=g, device=DEV) * case["skew"]
    gumbel = -torch.log(-torch.log(torch.rand(T, E, generator=g, device=DEV).clamp(1e-7, 1 - 1e-7)))
    counts = torch.bincount((pop + gumbel).topk(K, dim=1).indices.flatten(), minlength=E)
    off = torch.zeros(E + 1, dtype=torch.int32, device=DEV)
    off[1:] = counts.cumsum(0)
    return T * K, off, int(counts.max())


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(int(seed))
    if case["kind"] == "combine":
        return _prepare_combine(case, g)
    n, off, cap = _route(case, g)
    E, k, nw = case["E"], case["inf"], _weight_rows(case)
    s = {"case": case, "n": n, "off": off, "cap": cap}
    if case["kind"] == "backward":
        s["x"], s["dy"] = _normal(g, n, k), _normal(g, n, nw)
        s["w"] = _normal(g, E, nw, k, scale=k ** -0.5)
        return s
    x = _normal(g, n, k)
    if case["dtype"] == "bf16":
        s["x"], s["w"] = x, _normal(g, E, nw, k, scale=k ** -0.5)
    elif case["dtype"] == "int8":
        s["w"] = torch.empty(E, nw, k, dtype=torch.int8, device=DEV)
        for e in range(E):  # weights quantised once, one scale per output channel
            s["w"][e] = _normal(g, nw, k, scale=30.0).round().clamp(-127, 127).to(torch.int8)
        s["ws"] = (0.5 + torch.rand(E, nw, generator=g, device=DEV)) * (k ** -0.5 / 30)
        if case["quant"]:
            s["x"] = x
        else:
            amax = x.float().abs().amax(1)
            s["x"], s["xs"] = torch.round(x.float() * (127 / amax)[:, None]).to(torch.int8), amax / 127
    else:
        s["x"] = x
        s["w"] = torch.empty(E, nw, k // 2, dtype=torch.uint8, device=DEV)
        s["ws"] = torch.empty(E, nw, k // 32, dtype=torch.uint8, device=DEV)
        for e in range(E):  # weights quantised once
            s["w"][e], s["ws"][e] = _mx_pack(_normal(g, nw, k, scale=k ** -0.5))
    return s


def _prepare_combine(case, g):
    T, H, K, E, C, Kc = (case[v] for v in ("T", "H", "K", "E", "C", "Kc"))
    ids = torch.rand(T, E + C + Kc, generator=g, device=DEV).topk(K, dim=1).indices.to(torch.int32)
    mask = (torch.rand(T, generator=g, device=DEV) >= case["masked"]).to(torch.uint8) if case["masked"] else None
    sent = ids < E
    if mask is not None:
        sent &= mask[:, None] > 0
    # rows in the order of (expert, token, slot); the rows behind the last stay as they are (zero)
    key = torch.where(sent, ids, E).flatten().long()
    order = torch.argsort(key, stable=True)
    place = torch.empty_like(order)
    place[order] = torch.arange(T * K, device=DEV)
    s = {"case": case, "ids": ids, "mask": mask, "dst": torch.where(sent, place.view(T, K), -1).to(torch.int32),
         "w": torch.softmax(torch.randn(T, K, generator=g, device=DEV), 1), "go": _normal(g, T, H),
         "y": _normal(g, T * K, H), "gy": torch.zeros(T * K, H, dtype=torch.bfloat16, device=DEV)}
    if C + Kc:
        s["x"] = _normal(g, T, H)
    if Kc:
        s["a1"], s["a2"], s["v"] = _normal(g, Kc, H), _normal(g, Kc, H), _normal(g, Kc, H)
    return s


# ---- one pass ----------------------------------------------------------------------------------


def run(state):
    kind = state["case"]["kind"]
    if own:
        return _own_combine(state) if kind == "combine" else _own_backward(state) if kind == "backward" else _own_forward(state)
    return _plain_combine(state) if kind == "combine" else _plain_backward(state) if kind == "backward" else _plain_forward(state)


def _own_forward(s):
    import combine_moe_get_amd as mg

    c = s["case"]
    shape = mg.make_experts_shape(s["n"], c["E"], c["inf"], c["outf"])
    x, xs = s["x"], s.get("xs")
    if c["quant"]:
        x, xs = mg.quantize_rows(x, mg.ROWS_MXFP4 if c["dtype"] == "mxfp4" else mg.ROWS_INT8)
    return mg.experts_matmul(shape, x, s["w"], s["off"], row_scales=xs, w_scales=s.get("ws"),
                             act=mg.ACT_SWIGLU if c["gated"] else mg.ACT_NONE)


def _own_backward(s):
    import combine_moe_get_amd as mg

    c = s["case"]
    shape = mg.make_experts_shape(s["n"], c["E"], c["inf"], c["outf"])
    dx = mg.experts_matmul_dgrad(shape, s["dy"], s["w"], s["off"])
    dw = mg.experts_matmul_wgrad(shape, s["dy"], s["x"], s["off"], dtype=torch.float32 if c["grad32"] else torch.bfloat16)
    return {"dx": dx, "dw": dw}


def _own_combine(s):
    import combine_moe_get_amd as mg

    c = s["case"]
    shape = mg.make_shape(c["T"], c["H"], c["K"], c["E"], 1 if c["T"] <= 512 else 16, 0, c["C"], c["Kc"])
    g = mg.combine_grad(shape, s["go"], s["y"], s["ids"], s["w"], s["dst"], x_active_mask=s["mask"], ori_x=s.get("x"),
                        const_alpha1=s.get("a1"), const_alpha2=s.get("a2"), const_v=s.get("v"), grad_expert_out=s["gy"])
    out = {"y": g.grad_expert_out, "w": g.grad_topk_weights}
    if c["C"] + c["Kc"]:
        out["x"] = g.grad_ori_x
    if c["Kc"]:
        out["a1"], out["a2"], out["v"] = g.grad_alpha1, g.grad_alpha2, g.grad_v
    return out


def _padded(s, t):
    """Rows t [n, X] as float [E, cap, X], rows past an expert's count zero."""
    at = torch.arange(s["cap"], device=DEV)
    first, count = s["off"][:-1, None].long(), (s["off"][1:] - s["off"][:-1])[:, None]
    return torch.where((at < count)[..., None], t[(first + at).clamp(max=s["n"] - 1)].float(), 0.0)


def _ragged(s, t):
    """The rows of t [E, cap, X] that stand for receive rows, in their order: [n, X]."""
    r = torch.arange(s["n"], device=DEV)
    e = torch.searchsorted(s["off"][1:].long(), r, right=True)
    return t[e, r - s["off"][e].long()]


def _plain_forward(s):
    c = s["case"]
    x, w = s["x"].float() if c["dtype"] != "mxfp4" else s["x"], s["w"]
    if c["dtype"] == "mxfp4":
        r, e = _mx_parts(x.float())
        x = torch.ldexp(r, e[..., None].float()).flatten(-2)
        w = _mx_values(w, s["ws"])
    elif c["quant"]:
        amax = x.abs().amax(1)
        dyn = torch.where(amax > 0, 127 / amax, 0.0)
        x, xs = torch.round(x * dyn[:, None]).clamp(-127, 127), torch.where(amax > 0, 1 / dyn, 0.0)
    elif c["dtype"] == "int8":
        xs = s["xs"]
    y = torch.bmm(_padded(s, x), w.float().transpose(1, 2))
    if c["dtype"] == "int8":
        y = y * s["ws"][:, None, :]
    y = _ragged(s, y)
    if c["dtype"] == "int8":
        y = y * xs[:, None]
    if c["gated"]:
        gate, up = y.chunk(2, dim=1)
        y = gate / (1 + torch.exp(-gate)) * up
    return y.bfloat16()


def _mx_values(codes, scales):
    """The float values of packed e2m1 codes [.., H/2] with scales [.., H/32]."""
    grid = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6, -0.0, -0.5, -1, -1.5, -2, -3, -4, -6], device=DEV)
    v = torch.stack((grid[(codes & 15).long()], grid[(codes >> 4).long()]), -1).flatten(-2)
    return torch.ldexp(v.unflatten(-1, (-1, 32)), (scales.float() - 127)[..., None]).flatten(-2)


def _plain_backward(s):
    dy, x = _padded(s, s["dy"]), _padded(s, s["x"])
    dx = _ragged(s, torch.bmm(dy, s["w"].float()))
    dw = torch.bmm(dy.transpose(1, 2), x)
    return {"dx": dx.bfloat16(), "dw": dw if s["case"]["grad32"] else dw.bfloat16()}


def _plain_combine(s):
    c, n = s["case"], s["y"].shape[0]
    T, H, E, C, Kc = c["T"], c["H"], c["E"], c["C"], c["Kc"]
    go, dst = s["go"].float(), s["dst"].long()
    w = s["w"]
    sent = dst >= 0
    gy = torch.zeros(n + 1, H, device=DEV)  # the last row takes the slots that have none
    gy[torch.where(sent, dst, n)] = w[..., None] * go[:, None, :]
    y = torch.cat((s["y"].float(), torch.zeros(1, H, device=DEV)))
    moe = y[torch.where(sent, dst, n)]
    out = {"y": gy[:n].bfloat16()}
    if C + Kc:
        live = torch.ones(T, 1, dtype=torch.bool, device=DEV) if s["mask"] is None else s["mask"][:, None] > 0
        x = s["x"].float()
        ids = torch.where(live, s["ids"], -1)
        copied = (ids >= E) & (ids < E + C)
        moe = moe + copied[..., None] * x[:, None, :]
        share = (w * copied).sum(1, keepdim=True)
        if Kc:
            a1, a2, v = s["a1"].float(), s["a2"].float(), s["v"].float()
            const = (ids >= E + C)[..., None] & (ids[..., None] - E - C == torch.arange(Kc, device=DEV))  # [T, K, Kc]
            wc = (w[..., None] * const).sum(1)  # weight of each constant expert in each token
            moe = moe + torch.where(const.any(-1, keepdim=True),
                                    (const.float() @ a1) * x[:, None, :] + const.float() @ (a2 * v), 0.0)
            share = share + wc @ a1
            g = wc.t() @ go
            out["a1"], out["a2"], out["v"] = wc.t() @ (go * x), v * g, a2 * g
        out["x"] = (share * go).bfloat16()
    out["w"] = (moe * go[:, None, :]).sum(-1)
    return out


# ---- the definitions in 64 bits ----------------------------------------------------------------


def exact(case, seed):
    s = prepare(case, seed)
    if case["kind"] == "combine":
        return _exact_combine(s)
    off = s["off"].tolist()
    spans = [(e, off[e], off[e + 1]) for e in range(case["E"])]
    if case["kind"] == "backward":
        dx = torch.empty(s["n"], case["inf"], dtype=torch.float64, device=DEV)
        dw = torch.zeros(s["w"].shape, dtype=torch.float64, device=DEV)
        for e, lo, hi in spans:
            dx[lo:hi] = s["dy"][lo:hi].double() @ s["w"][e].double()
            dw[e] = s["dy"][lo:hi].double().t() @ s["x"][lo:hi].double()
        return {"dx": dx, "dw": dw}
    y = torch.empty(s["n"], case["outf"], dtype=torch.float64, device=DEV)
    for e, lo, hi in spans:
        if hi == lo:
            continue
        x = s["x"][lo:hi].double()
        scale = None
        if case["dtype"] == "mxfp4":
            x, w = _exact_mx(x), _exact_unpack(s["w"][e], s["ws"][e])
        else:
            w = s["w"][e].double()
        if case["dtype"] == "int8":
            if case["quant"]:
                # the codes' own arithmetic is binary32 by definition: 127 / amax, the product and 1 / dyn each rounded
                f = s["x"][lo:hi].float()
                dyn = 127 / f.abs().amax(1, keepdim=True)
                x, scale = torch.round(f * dyn).double(), (1 / dyn).double()
            else:
                scale = s["xs"][lo:hi, None].double()
            w = w * s["ws"][e][:, None].double()
        z = x @ w.t()
        if scale is not None:
            z = z * scale
        if case["gated"]:
            z = z[:, : case["outf"]] * torch.sigmoid(z[:, : case["outf"]]) * z[:, case["outf"]:]
        y[lo:hi] = z
    return y


def _exact_mx(x):
    """x [r, H] double -> the values of its e2m1 codes: the scale from log2, the codes from the grid's midpoints."""
    grid = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64, device=DEV)
    mid = (grid[1:] + grid[:-1]) / 2
    b = x.view(x.shape[0], -1, 32)
    scale = torch.exp2((torch.floor(torch.log2(b.abs().amax(-1, keepdim=True))) - 2).clamp(min=-127))
    a = b.abs() / scale
    down, up = torch.bucketize(a, mid), torch.bucketize(a, mid, right=True)
    code = torch.where(down % 2 == 0, down, up)  # on a midpoint the two differ: the even one
    return (torch.sign(b) * grid[code] * scale).view_as(x)


def _exact_unpack(codes, scales):
    c = torch.stack((codes & 15, codes >> 4), -1).flatten(-2).long()
    m, ex = c & 1, (c >> 1) & 3
    v = torch.where(ex == 0, m * 0.5, (1 + m * 0.5) * torch.exp2((ex - 1).double()))
    v = torch.where(c >= 8, -v, v).double()
    return (v.view(v.shape[0], -1, 32) * torch.exp2(scales.double() - 127)[..., None]).view_as(v)


def _exact_combine(s):
    c, n = s["case"], s["y"].shape[0]
    T, H, K, E, C, Kc = (c[v] for v in ("T", "H", "K", "E", "C", "Kc"))
    go, w = s["go"].double(), s["w"].double()
    out = {"y": torch.zeros(n, H, dtype=torch.float64, device=DEV), "w": torch.zeros(T, K, dtype=torch.float64, device=DEV)}
    if C + Kc:
        x, out["x"] = s["x"].double(), torch.zeros(T, H, dtype=torch.float64, device=DEV)
    if Kc:
        a1, a2, v = s["a1"].double(), s["a2"].double(), s["v"].double()
        out["a1"], out["a2"], out["v"] = (torch.zeros(Kc, H, dtype=torch.float64, device=DEV) for _ in range(3))
    live = torch.ones(T, dtype=torch.bool, device=DEV) if s["mask"] is None else s["mask"] > 0
    for j in range(K):
        t = torch.nonzero(s["dst"][:, j] >= 0).flatten()
        row = s["dst"][t, j].long()
        out["y"][row] = w[t, j, None] * go[t]
        out["w"][t, j] = (go[t] * s["y"][row].double()).sum(1)
        for i in range(C + Kc):
            t = torch.nonzero(live & (s["ids"][:, j] == E + i)).flatten()
            if i < C:
                out["w"][t, j] = (go[t] * x[t]).sum(1)
                out["x"][t] += w[t, j, None] * go[t]
            else:
                k = i - C
                out["w"][t, j] = (go[t] * (a1[k] * x[t] + a2[k] * v[k])).sum(1)
                out["x"][t] += w[t, j, None] * go[t] * a1[k]
                out["a1"][k] += (w[t, j, None] * go[t] * x[t]).sum(0)
                out["a2"][k] += (w[t, j, None] * go[t]).sum(0) * v[k]
                out["v"][k] += (w[t, j, None] * go[t]).sum(0) * a2[k]
    return out
