"""The router, its balance loss and the gate of a layer that trains.

Three operators, each in its plain form (elementary torch operations in 32 bits, in 64 where scores are
compared or long sums taken) and as the calls a user makes of combine_moe_get_amd:

  route  route: the ids and weights of each token's experts from the router's logits; softmax or
         sigmoid scores, with a bias that only the choice sees, with groups of experts
  loss   balance_loss and route_grad: counts and probability sums per segment, the balance and z losses,
         and the gradient of the logits through the chosen weights and both losses
  gate   swiglu and swiglu_grad: silu(g) u with routing weights; for the way back 8-bit codes are kept
         (or the bf16 values), from which the gradients and the gate's result are made again
"""
import math

import torch

own = False

DEV = "cuda"

# ---- cases -------------------------------------------------------------------------------------


def _route(name, T, E, K, score="softmax", dtype="fp32", bias=False, groups=1, keep=1, two=False, renorm=True,
           scale=1.0, masked=0.0, down=0):
    """groups: groups of experts, keep: how many of them a token may use, two: a group's score is the sum of its two
    best keys, else its best; masked: share of padding tokens; down: experts whose logits are -inf."""
    c = {"kind": "route", "T": T, "E": E, "K": K, "score": score, "dtype": dtype, "bias": bias, "groups": groups,
         "keep": keep, "two": two, "renorm": renorm, "scale": scale, "masked": masked, "down": down}
    return dict(c, name=name) if name else c


def _loss(name, T, E, K, score="softmax", dtype="fp32", renorm=True, scale=1.0, segments=1, z=0.0, masked=0.0):
    """segments: equal runs of tokens that are balanced each for itself; z: coefficient of the z loss."""
    c = {"kind": "loss", "T": T, "E": E, "K": K, "score": score, "dtype": dtype, "renorm": renorm, "scale": scale,
         "segments": segments, "z": z, "masked": masked}
    return dict(c, name=name) if name else c


def _gate(name, rows, E, I, step="train", weights=True, skew=0.5, P=1, slack=0):
    """I: columns of the result; step: "train" (forward with 8-bit codes, backward from them), "forward" alone, or
    "backward" from bf16; P, slack: ranks and the spare rows of each one's window (compact rows if P is 1)."""
    c = {"kind": "gate", "rows": rows, "E": E, "I": I, "step": step, "weights": weights, "skew": skew, "P": P, "slack": slack}
    return dict(c, name=name) if name else c


def listed():
    return [
        # one rank's share of a decode batch: every step waits for these ids
        _route("decode, 128 tokens", 128, 256, 8),
        # a prefill batch, sigmoid scores, four of eight groups by their two best, a bias that evens the load
        _route("prefill, biased groups", 4096, 256, 8, score="sigmoid", bias=True, groups=8, keep=4, two=True, scale=2.5),
        # padded batch, 128 experts and six special ones, two experts out of service
        _route("padded, special experts", 8191, 134, 6, dtype="bf16", renorm=False, masked=0.1, down=2),
        # the largest batch, groups by their best expert
        _route("16384 tokens, groups", 16384, 256, 8, groups=8, keep=4),
        # a fine-tuning step on a small batch
        _loss("small step", 100, 33, 4, score="sigmoid"),
        # a training batch balanced over the whole
        _loss("training step", 4096, 64, 8, dtype="bf16", z=1e-3),
        # sequences of 256 tokens balanced each for itself, padded
        _loss("sequences", 16384, 256, 8, score="sigmoid", scale=2.5, segments=64, masked=0.1),
        # one token's rows on eight experts: serving, no gradient
        _gate("one token", 8, 8, 1024, step="forward"),
        # a small batch's step
        _gate("small step, 8-bit", 400, 16, 512),
        # odd rows and columns, experts of very different size
        _gate("odd rows, 8-bit", 6168, 33, 2056, skew=1.0),
        # a training step of 4096 tokens, top-8
        _gate("training step, 8-bit", 32768, 32, 2048),
        # the way back from bf16 values, rows in windows of eight ranks
        _gate("windows, bf16 kept", 8192, 64, 4096, step="backward", weights=False, P=8, slack=100),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["route", "loss", "gate"])
    if kind == "gate":
        I = 8 * _log(rng, 8, 896)
        E, step = rng.choice([8, 16, 64, 128]), rng.choice(["train", "train", "forward", "backward"])
        P = rng.choice([1, 1, 4])
        rows = max(1, _log(rng, 1, min(32768, 32768 * 2048 // I)) // P) * P
        return _gate(None, rows, E, I, step, rng.random() < 0.6, rng.choice([0.0, 0.5, 1.0]), P, rng.randint(0, 64) if P > 1 else 0)
    T, E = _log(rng, 1, 16384), rng.choice([8, 16, 33, 64, 96, 128, 134, 160, 256])
    K, score, dtype = rng.choice([1, 2, 3, 4, 6, 8]), rng.choice(["softmax", "sigmoid"]), rng.choice(["fp32", "bf16"])
    masked = rng.choice([0.0, 0.0, 0.1, 0.5])
    renorm, scale = rng.random() < 0.6, rng.choice([1.0, 2.5])
    if kind == "loss":
        segments = rng.choice([1, 1, 4, 16])
        return _loss(None, (T + segments - 1) // segments * segments, E, K, score, dtype, renorm, scale, segments,
                     rng.choice([0.0, 1e-3]), masked)
    groups = rng.choice([1, 1, 4, 8]) if E % 8 == 0 and E >= 64 else 1
    keep = rng.randint(1, groups) if groups == 1 or E // groups >= K else groups
    return _route(None, T, E, K, score, dtype, rng.random() < 0.5, groups, keep, groups > 1 and rng.random() < 0.5, renorm,
                  scale, masked, rng.choice([0, 0, 1, 3]))


def _size(case):
    return 4 if case["dtype"] == "fp32" else 2


def work(case):
    if case["kind"] == "gate":
        rows, I = case["rows"], case["I"]
        blocks = 2 * ((I + 127) // 128)
        # forward: h0, weights in, the result out, codes and scales out; backward: d, codes or h0 in, grad, h, dw out
        fwd = rows * (4 * I + 2 * I + 4 * case["weights"])
        codes = rows * (2 * I + 4 * blocks)
        bwd = rows * (2 * I + 4 * I + 2 * I + 8 * case["weights"])
        b = {"train": fwd + bwd + 2 * codes, "forward": fwd, "backward": bwd + rows * 4 * I}[case["step"]]
        return {"bytes": b, "flops": rows * I * {"train": 30, "forward": 6, "backward": 16}[case["step"]]}
    T, E, K = case["T"], case["E"], case["K"]
    if case["kind"] == "route":
        return {"bytes": T * E * _size(case) + T * K * 8, "flops": 6 * T * E}
    return {"bytes": 2 * T * E * _size(case) + T * K * 8 + case["segments"] * E * 8, "flops": 20 * T * E}


# ---- inputs ------------------------------------------------------------------------------------


def _logits(case, g):
    """Logits of a router in training: experts of different popularity, tokens of different certainty."""
    T, E = case["T"], case["E"]
    l = torch.randn(T, E, generator=g, device=DEV) * (0.5 + torch.rand(T, 1, generator=g, device=DEV))
    l += 0.5 * torch.randn(E, generator=g, device=DEV)
    return l if case["dtype"] == "fp32" else l.bfloat16()


def _mask(case, g):
    if not case["masked"]:
        return None
    return (torch.rand(case["T"], generator=g, device=DEV) >= case["masked"]).to(torch.uint8)


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(int(seed))
    if case["kind"] == "gate":
        return _prepare_gate(case, g)
    s = {"case": case, "logits": _logits(case, g), "mask": _mask(case, g)}
    T, E, K = case["T"], case["E"], case["K"]
    if case["kind"] == "route":
        if case["down"]:
            s["logits"][:, torch.randperm(E, generator=g, device=DEV)[:case["down"]]] = -math.inf
        s["bias"] = 0.1 * torch.randn(E, generator=g, device=DEV) if case["bias"] else None
        return s
    ids = s["logits"].float().sort(dim=1, descending=True, stable=True).indices[:, :K].to(torch.int32)
    s["ids"] = ids if s["mask"] is None else torch.where(s["mask"][:, None] > 0, ids, -1)
    s["gw"] = torch.randn(T, K, generator=g, device=DEV) / T  # of a loss that is a mean over tokens
    s["gl"] = torch.ones(2, device=DEV)
    return s


def _prepare_gate(case, g):
    E, I, P = (case[v] for v in ("E", "I", "P"))
    each, L = case["rows"] // P, E // P  # as many rows on every rank
    n = P * each
    pop = torch.softmax(torch.randn(P, L, generator=g, device=DEV) * case["skew"], 1)
    e = torch.multinomial(pop, each, replacement=True, generator=g) + L * torch.arange(P, device=DEV)[:, None]
    off = torch.zeros(E + 1, dtype=torch.int32, device=DEV)
    off[1:] = torch.bincount(e.flatten(), minlength=E).cumsum(0)
    stride = each + case["slack"] if P > 1 else 0
    rows = P * stride if stride else n
    s = {"case": case, "off": off, "rows": rows, "stride": stride}
    # where each row in use lies
    r = torch.arange(n, device=DEV)
    if stride:
        r = r // each * stride + r % each
    s["used"] = r
    s["h0"] = torch.randn(rows, 2 * I, generator=g, device=DEV, dtype=torch.bfloat16)
    s["w"] = torch.rand(rows, generator=g, device=DEV) if case["weights"] else None
    if case["step"] != "forward":
        s["dh"] = torch.randn(rows, I, generator=g, device=DEV, dtype=torch.bfloat16)
    # results that the program keeps; rows of no expert stay as they are
    b = dict(dtype=torch.bfloat16, device=DEV)
    s["h"], s["again"] = torch.zeros(rows, I, **b), torch.zeros(rows, I, **b)
    s["gh0"], s["gw"] = torch.zeros(rows, 2 * I, **b), torch.zeros(rows, device=DEV)
    return s


# ---- one pass ----------------------------------------------------------------------------------


def run(state):
    kind = state["case"]["kind"]
    if own:
        return {"route": _own_route, "loss": _own_loss, "gate": _own_gate}[kind](state)
    return {"route": _plain_route, "loss": _plain_loss, "gate": _plain_gate}[kind](state)


def _shape(mg, c):
    return mg.make_route_shape(c["T"], c["E"], c["K"], score=mg.SCORE_SOFTMAX if c["score"] == "softmax" else mg.SCORE_SIGMOID,
                               renormalize=c["renorm"], scale=c["scale"], groups=c.get("groups", 1), topk_groups=c.get("keep", 1),
                               group_score=mg.GROUP_TOP2 if c.get("two") else mg.GROUP_MAX)


def _own_route(s):
    import combine_moe_get_amd as mg

    r = mg.route(_shape(mg, s["case"]), s["logits"], bias=s["bias"], x_active_mask=s["mask"])
    return {"ids": r.topk_idx, "w": r.topk_weights}


def _own_loss(s):
    import combine_moe_get_amd as mg

    c = s["case"]
    shape, balance = _shape(mg, c), mg.make_balance(segments=c["segments"], balance_coef=1e-2, z_coef=c["z"])
    b = mg.balance_loss(shape, balance, s["logits"], s["ids"], x_active_mask=s["mask"])
    gl = mg.route_grad(shape, s["logits"], s["ids"], grad_topk_weights=s["gw"], balance=balance, balance_loss=b,
                       grad_losses=s["gl"], x_active_mask=s["mask"])
    return {"losses": b.losses, "counts": b.counts, "sums": b.prob_sums, "tokens": b.segment_tokens, "grad": gl}


def _own_gate(s):
    import combine_moe_get_amd as mg

    c = s["case"]
    shape = mg.make_experts_shape(s["rows"], c["E"], c["I"], 8, c["P"], s["stride"])
    out = {}
    if c["step"] != "backward":
        f = mg.swiglu(s["h0"], row_weights=s["w"], checkpoint=c["step"] == "train", shape=shape, expert_offsets=s["off"],
                      out=s["h"])
        out["h"] = f.out
    if c["step"] != "forward":
        kept = dict(h0=s["h0"]) if c["step"] == "backward" else dict(codes=f.codes, scales=f.scales)
        g = mg.swiglu_grad(s["dh"], **kept, row_weights=s["w"], shape=shape, expert_offsets=s["off"], out=s["again"],
                           grad_h0=s["gh0"], grad_row_weights=s["gw"] if c["weights"] else None)
        out["again"], out["gh0"] = g.out, g.grad_h0
        if c["weights"]:
            out["gw"] = g.grad_row_weights
    return out


def _plain_scores(c, l, ok):
    """The logarithm of the scores of l [T, E]; -inf where not ok."""
    if c["score"] == "sigmoid":
        q = l.clamp(max=0) - torch.log(1 + torch.exp(-l.abs()))
    else:
        m = torch.where(ok, l, -math.inf).amax(1, keepdim=True)
        m = torch.where(m > -math.inf, m, 0.0)
        q = l - m - torch.log(torch.where(ok, torch.exp(l - m), 0.0).sum(1, keepdim=True))
    return torch.where(ok, q, -math.inf)


def _plain_route(s):
    c = s["case"]
    T, E, K, G = c["T"], c["E"], c["K"], c["groups"]
    l = s["logits"].float()
    ok = l > -math.inf
    if s["mask"] is not None:
        ok = ok & (s["mask"][:, None] > 0)
    key = l.double()
    if s["bias"] is not None or c["two"]:  # scores next to one another: compared in 64 bits
        key = torch.exp(_plain_scores(c, key, ok))
        if s["bias"] is not None:
            key = key + s["bias"].double()
    key = torch.where(ok, key, -math.inf)
    if G > 1:
        k = key.view(T, G, E // G)
        if c["two"]:
            top = k.sort(dim=2, descending=True).values
            score = top[..., 0] + torch.where(top[..., 1] > -math.inf, top[..., 1], 0.0)
        else:
            score = k.amax(2)
        first = score.sort(dim=1, descending=True, stable=True).indices[:, : c["keep"]]
        kept = (first[:, :, None] == torch.arange(G, device=DEV)).any(1)
        key = torch.where(kept[:, :, None], k, -math.inf).view(T, E)
    key, ids = key.sort(dim=1, descending=True, stable=True)
    key, ids = key[:, :K], ids[:, :K]
    some = key > -math.inf
    q = torch.where(some, _plain_scores(c, l, ok).gather(1, ids), -math.inf)
    if c["renorm"]:
        m = q.amax(1, keepdim=True)
        w = torch.where(some, torch.exp(q - torch.where(m > -math.inf, m, 0.0)), 0.0)
        w = w / torch.where(some.any(1, keepdim=True), w.sum(1, keepdim=True), 1.0)
    else:
        w = torch.exp(q)
    return {"ids": torch.where(some, ids, -1).to(torch.int32), "w": w * c["scale"]}


def _plain_loss(s):
    c = s["case"]
    T, E, K, S = c["T"], c["E"], c["K"], c["segments"]
    l, ids, gw = s["logits"].float(), s["ids"].long(), s["gw"]
    ok = l > -math.inf
    if s["mask"] is not None:
        ok = ok & (s["mask"][:, None] > 0)
    live = ok.any(1)
    chosen = ids[..., None] == torch.arange(E, device=DEV)  # [T, K, E]
    counts = chosen.view(S, -1, E).sum(1)
    tokens = live.view(S, -1).sum(1)
    logq = _plain_scores(c, l, ok)
    m = torch.where(live[:, None], logq.amax(1, keepdim=True), 0.0)
    e = torch.exp(logq - m)
    p = e / torch.where(live[:, None], e.sum(1, keepdim=True), 1.0)
    sums = p.double().view(S, -1, E).sum(1)
    per = torch.where(tokens > 0, 1e-2 * E / (S * K * tokens.double().clamp(min=1) ** 2), 0.0)[:, None]
    balance = (per * counts * sums).sum()
    soft = torch.exp(_plain_scores({"score": "softmax"}, l, ok)) if c["score"] == "sigmoid" else p
    ml = torch.where(live, torch.where(ok, l, -math.inf).amax(1), 0.0)
    lse = ml + torch.log(torch.where(live, torch.where(ok, torch.exp(l - ml[:, None]), 0.0).sum(1), 1.0))
    total = tokens.sum().clamp(min=1)
    z = c["z"] * (lse.double() ** 2).sum() / total

    # gradient: of the logarithms of the scores, then of the logits
    slope = torch.where(ok, 1 / (1 + torch.exp(l)), 0.0) if c["score"] == "sigmoid" else None  # 1 - sigmoid
    some = ids >= 0
    q = torch.where(some, logq.gather(1, ids.clamp(min=0)), -math.inf)
    if c["renorm"]:
        mq = torch.where(some.any(1, keepdim=True), q.amax(1, keepdim=True), 0.0)
        w = torch.exp(q - mq)
        w = w / torch.where(some.any(1, keepdim=True), w.sum(1, keepdim=True), 1.0)
        a = c["scale"] * w * (gw - (w * gw).sum(1, keepdim=True))
    else:
        a = c["scale"] * torch.exp(q) * gw
    a = torch.where(some, a, 0.0)
    grad = (chosen * a[..., None]).sum(1)
    if c["score"] == "softmax" and not c["renorm"]:
        grad = grad - p * a.sum(1, keepdim=True)
    A = (s["gl"][0] * per * (counts - counts.double().mean(1, keepdim=True))).float().repeat_interleave(T // S, 0)
    grad = grad + p * (A - (A * p).sum(1, keepdim=True))
    if slope is not None:
        grad = grad * slope
    grad = grad + s["gl"][1] * (2 * c["z"] * lse / total)[:, None] * soft
    return {"losses": torch.stack((balance, z)).float(), "counts": counts.to(torch.int32), "sums": sums.float(),
            "tokens": tokens.to(torch.int32), "grad": grad.to(s["logits"].dtype)}


def _blocks(x):
    """x [rows, I] in blocks of 128: [rows, blocks, 128], the last one filled up with zeros."""
    n = (x.shape[1] + 127) // 128
    out = torch.zeros(x.shape[0], n * 128, device=DEV)
    out[:, : x.shape[1]] = x
    return out.view(x.shape[0], n, 128)


def _through_8_bits(x):
    """What the codes of x [rows, I] stand for: each operation rounded once, as the codes are defined."""
    b = _blocks(x)
    dyn = 127 / b.abs().amax(2, keepdim=True)
    code = torch.round(b * dyn).clamp(-127, 127)
    return (code * (1 / dyn)).flatten(1)[:, : x.shape[1]]


def _plain_gate(s):
    c, r, I = s["case"], s["used"], s["case"]["I"]
    h0 = s["h0"][r].float()
    w = s["w"][r, None] if c["weights"] else torch.ones(len(r), 1, device=DEV)
    out = {}
    g, u = h0[:, :I], h0[:, I:]
    if c["step"] != "backward":
        s["h"][r] = (w * (g / (1 + torch.exp(-g)) * u)).bfloat16()
        out["h"] = s["h"]
    if c["step"] == "forward":
        return out
    if c["step"] == "train":
        g, u = _through_8_bits(g), _through_8_bits(u)
    d = s["dh"][r].float()
    sig = 1 / (1 + torch.exp(-g))
    act = g * sig
    s["again"][r] = (w * (act * u)).bfloat16()
    s["gh0"][r] = torch.cat((w * d * u * sig * (1 + g * (1 - sig)), w * d * act), 1).bfloat16()
    out["again"], out["gh0"] = s["again"], s["gh0"]
    if c["weights"]:
        s["gw"][r] = (d * act * u).sum(1)
        out["gw"] = s["gw"]
    return out


# ---- the definitions in 64 bits ----------------------------------------------------------------


def exact(case, seed):
    s = prepare(case, seed)
    return {"route": _exact_route, "loss": _exact_loss, "gate": _exact_gate}[case["kind"]](s)


def _exact_p(c, l):
    """Scores of the logits l [T, E] in 64 bits (-inf: none), and those divided by their sum."""
    e = torch.sigmoid(l) if c["score"] == "sigmoid" else torch.softmax(l, 1)
    return e, e / e.sum(1, keepdim=True)


def _best(key):
    """The largest of each row and the lowest place that has it."""
    m = key.max(-1, keepdim=True).values
    at = torch.where(key == m, torch.arange(key.shape[-1], device=DEV), key.shape[-1]).min(-1).values
    return m[..., 0], at


def _exact_route(s):
    c = s["case"]
    T, E, K, G = c["T"], c["E"], c["K"], c["groups"]
    l = s["logits"].double()
    ids = torch.full((T, K), -1, dtype=torch.int32, device=DEV)
    w = torch.zeros(T, K, dtype=torch.float64, device=DEV)
    t = torch.arange(T, device=DEV) if s["mask"] is None else torch.nonzero(s["mask"]).flatten()
    if len(t) == 0:
        return {"ids": ids, "w": w}
    l = l[t]
    score = _exact_p(c, l)[0]
    gone = l == -math.inf
    if s["bias"] is not None:
        key = score + s["bias"].double()
    else:
        key = score if c["two"] else l
    key = key.masked_fill(gone, -math.inf)
    if G > 1:
        k, use = key.reshape(len(t), G, E // G), torch.zeros(len(t), G, dtype=torch.bool, device=DEV)
        one, at = _best(k)
        if c["two"]:
            two = _best(k.scatter(2, at[..., None], -math.inf))[0]
            one = one + two.masked_fill(two == -math.inf, 0.0)
        for _ in range(c["keep"]):
            _, at = _best(one)
            use.scatter_(1, at[:, None], True)
            one = one.scatter(1, at[:, None], -math.inf)
        key = k.masked_fill(~use[..., None], -math.inf).reshape(len(t), E)
    for j in range(K):
        m, at = _best(key)
        some = m > -math.inf
        ids[t[some], j] = at[some].to(torch.int32)
        w[t[some], j] = score.gather(1, at.clamp(max=E - 1)[:, None])[some, 0]
        key = key.scatter(1, at.clamp(max=E - 1)[:, None], -math.inf)
    if c["renorm"]:
        w = w / w.sum(1, keepdim=True).clamp(min=1e-300)
    return {"ids": ids, "w": w * c["scale"]}


def _exact_loss(s):
    """The losses as functions of the logits, their gradient from the derivative of each step."""
    c = s["case"]
    T, E, K, S = c["T"], c["E"], c["K"], c["segments"]
    live = torch.ones(T, dtype=torch.bool, device=DEV) if s["mask"] is None else s["mask"] > 0
    l, ids = s["logits"].double(), s["ids"].long()
    score, p = _exact_p(c, l)
    n = T // S
    counts = torch.zeros(S, E, dtype=torch.int64, device=DEV)
    sums = torch.zeros(S, E, dtype=torch.float64, device=DEV)
    tokens = torch.zeros(S, dtype=torch.int64, device=DEV)
    ds = torch.zeros(T, E, dtype=torch.float64, device=DEV)  # of the scores, through the weights
    dp = torch.zeros(T, E, dtype=torch.float64, device=DEV)  # of the probabilities, through the balance loss
    balance = torch.zeros((), dtype=torch.float64, device=DEV)
    for g in range(S):
        at = slice(g * n, (g + 1) * n)
        i = ids[at].flatten()
        counts[g] = torch.bincount(i[i >= 0], minlength=E)
        sums[g] = p[at][live[at]].sum(0)
        tokens[g] = live[at].sum()
        if tokens[g] > 0:
            f = counts[g] / (K * tokens[g]) * E
            balance += 1e-2 * (f * sums[g] / tokens[g]).sum() / S
            dp[at] = s["gl"][0].double() * 1e-2 * f / tokens[g] / S
    total = tokens.sum().clamp(min=1)
    lse = torch.logsumexp(l, 1)
    z = c["z"] * lse[live].square().sum() / total
    some = ids >= 0
    q = torch.where(some, score.gather(1, ids.clamp(min=0)), 0.0)
    dw = torch.where(some, s["gw"].double(), 0.0) * c["scale"]
    if c["renorm"]:
        whole = q.sum(1, keepdim=True).clamp(min=1e-300)
        dw = torch.where(some, (dw - (dw * q).sum(1, keepdim=True) / whole) / whole, 0.0)
    ds.scatter_add_(1, ids.clamp(min=0), dw)
    if c["score"] == "sigmoid":  # p = score / sum of scores
        ds += (dp - (dp * p).sum(1, keepdim=True)) / score.sum(1, keepdim=True)
        grad = ds * score * torch.sigmoid(-l)
    else:
        ds += dp
        grad = p * (ds - (ds * p).sum(1, keepdim=True))
    grad += s["gl"][1].double() * c["z"] * 2 * lse[:, None] / total * torch.softmax(l, 1)
    grad[~live] = 0
    return {"losses": torch.stack((balance, z)), "counts": counts.to(torch.int32), "sums": sums,
            "tokens": tokens.to(torch.int32), "grad": grad}


def _exact_codes(x):
    """x [rows, I] -> the values of its codes. The codes' own arithmetic is binary32 by definition: 127 / amax, the product
    and the reciprocal each rounded."""
    out = torch.empty(x.shape, dtype=torch.float64, device=DEV)
    for lo in range(0, x.shape[1], 128):
        b = x[:, lo:lo + 128].float()
        dyn = 127 / b.abs().max(1, keepdim=True).values
        out[:, lo:lo + 128] = torch.round(b * dyn).double() * (1 / dyn).double()
    return out


def _exact_gate(s):
    c, I = s["case"], s["case"]["I"]
    out, rows = {}, s["rows"]
    names = {"train": ("h", "again", "gh0"), "forward": ("h",), "backward": ("again", "gh0")}[c["step"]]
    for k in names:
        out[k] = torch.zeros(rows, 2 * I if k == "gh0" else I, dtype=torch.float64, device=DEV)
    if c["weights"] and c["step"] != "forward":
        out["gw"] = torch.zeros(rows, dtype=torch.float64, device=DEV)
    for r in s["used"].split(4096):
        g, u = s["h0"][r, :I].double(), s["h0"][r, I:].double()
        w = s["w"][r].double()[:, None] if c["weights"] else 1.0
        if "h" in out:
            out["h"][r] = w * torch.sigmoid(g) * g * u
        if c["step"] == "forward":
            continue
        if c["step"] == "train":
            g, u = _exact_codes(s["h0"][r, :I]), _exact_codes(s["h0"][r, I:])
        d, sig = s["dh"][r].double(), torch.sigmoid(g)
        out["again"][r] = w * sig * g * u
        out["gh0"][r, :I] = w * d * u * (sig + g * sig * torch.sigmoid(-g))
        out["gh0"][r, I:] = w * d * sig * g
        if "gw" in out:
            out["gw"][r] = (d * sig * g * u).sum(1)
    return out
