"""Helpers of the router's tests: the definitions in 64 bits (numpy) and tolerances that follow from the arithmetic."""
import numpy as np

STEP32 = 2.0 ** -23  # a whole step of fp32, relative: bounds one operation however it rounds
TINY = 2.0 ** -120
SOFTMAX, SIGMOID = 0, 1
MAX, TOP2 = 0, 1
FLT_MAX = float(np.finfo(np.float32).max)


def usable(l):
    """Logits that count, in 64 bits: NaN as -inf, +inf as the largest finite fp32."""
    l = np.asarray(l, np.float64)
    return np.where(np.isnan(l), -np.inf, np.minimum(l, FLT_MAX))


def scores(l, score):
    """s of usable logits [T, E]; 0 where there is none."""
    ok = l > -np.inf
    with np.errstate(over="ignore", invalid="ignore"):
        if score == SIGMOID:
            return np.where(ok, np.exp(np.minimum(l, 0)) / (1 + np.exp(-np.abs(l))), 0.0)
        m = l.max(1, keepdims=True)
        m = np.where(m > -np.inf, m, 0.0)
        e = np.where(ok, np.exp(l - m), 0.0)
        return e / np.where(e.sum(1, keepdims=True) > 0, e.sum(1, keepdims=True), 1.0)


def log_scores(l, score):
    ok = l > -np.inf
    with np.errstate(over="ignore", invalid="ignore", divide="ignore"):
        if score == SIGMOID:
            q = np.minimum(l, 0) - np.log1p(np.exp(-np.abs(l)))
        else:
            m = l.max(1, keepdims=True)
            m = np.where(m > -np.inf, m, 0.0)
            s = np.where(ok, np.exp(l - m), 0.0).sum(1, keepdims=True)
            q = l - m - np.log(np.where(s > 0, s, 1.0))
    return np.where(ok, q, -np.inf)


def live(l, mask):
    a = (l > -np.inf).any(1)
    return a if mask is None else a & (np.asarray(mask) > 0)


def choose(l, K, score, bias=None, mask=None, groups=1, keep=1, group_score=MAX):
    """ids [T, K]: by sorting each token's (key, id) pairs."""
    T, E = l.shape
    wide = bias is not None or (group_score == TOP2 and keep < groups)
    s = scores(l, score)
    on = live(l, mask)
    ids = np.full((T, K), -1, np.int32)
    per = E // groups
    for t in range(T):
        if not on[t]:
            continue
        key = {}
        for e in range(E):
            if not l[t, e] > -np.inf:
                continue
            k = s[t, e] if wide else l[t, e]
            if bias is not None:
                if not bias[e] > -np.inf:
                    continue
                k = k + float(bias[e])
            key[e] = k
        if keep < groups:
            g = {}
            for e, k in key.items():
                g.setdefault(e // per, []).append(k)
            val = {i: sum(sorted(v, reverse=True)[:2 if group_score == TOP2 else 1]) for i, v in g.items()}
            best = sorted(val, key=lambda i: (-val[i], i))[:keep]
            key = {e: k for e, k in key.items() if e // per in best}
        order = sorted(key, key=lambda e: (-key[e], e))[:K]
        ids[t, :len(order)] = order
    return ids


def weights(l, ids, score, renorm, scale):
    """(weights [T, K], tolerances): the exponential of a difference d of logarithms, each rounded to fp32, is good to
    (|d| + |q| + |max q| + 8) steps; the sum of K such and the division add K + 4; of E for the softmax over all."""
    T, K = ids.shape
    q = np.where(ids >= 0, np.take_along_axis(log_scores(l, score), np.maximum(ids, 0), 1), -np.inf)
    raw = np.where(ids >= 0, np.take_along_axis(l, np.maximum(ids, 0), 1), 0.0)
    if renorm:
        m = q.max(1, keepdims=True)
        m = np.where(m > -np.inf, m, 0.0)
        with np.errstate(invalid="ignore"):
            e = np.exp(q - m)
        s = e.sum(1, keepdims=True)
        w = e / np.where(s > 0, s, 1.0)
    else:
        w = np.exp(q)
    spread = np.abs(np.where(ids >= 0, raw, 0.0)).max(1, keepdims=True) + np.abs(np.where(l > -np.inf, l, 0.0)).max(1, keepdims=True)
    w = np.where(ids >= 0, w * scale, 0.0)
    # where the exponential itself is below what fp32 holds it may be 0
    return w, np.abs(w) * (2 * np.minimum(spread, 200.0) + l.shape[1] / 8 + K + 16) * STEP32 + abs(scale) * TINY


def losses(l, ids, score, S, bc, zc, mask=None):
    """dict of losses [2], counts, sums, tokens."""
    T, E = l.shape
    K = ids.shape[1]
    on = live(l, mask)
    n = T // S
    p = probabilities(l, score, on)
    counts, sums, tokens = np.zeros((S, E), np.int64), np.zeros((S, E)), np.zeros(S, np.int64)
    bal = 0.0
    for g in range(S):
        r = np.arange(g * n, (g + 1) * n)[on[g * n:(g + 1) * n]]
        tokens[g] = len(r)
        sums[g] = p[r].sum(0)
        i = ids[r].ravel()
        i = i[(i >= 0) & (i < E)]
        np.add.at(counts[g], i, 1)
        if len(r):
            bal += bc / S * E / (K * len(r) ** 2) * (counts[g] * sums[g]).sum()
    total = tokens.sum()
    z = zc / total * (lse(l, on)[on] ** 2).sum() if total else 0.0
    return dict(losses=np.array([bal, z]), counts=counts, sums=sums, tokens=tokens)


def probabilities(l, score, on):
    """Scores divided by their sum, by their logarithms (so that small ones do not vanish)."""
    q = log_scores(l, score)
    m = np.where(on, q.max(1), 0.0)[:, None]
    with np.errstate(invalid="ignore"):
        e = np.where((q > -np.inf) & on[:, None], np.exp(q - m), 0.0)
    s = e.sum(1, keepdims=True)
    return e / np.where(s > 0, s, 1.0)


def lse(l, on):
    m = np.where(on, l.max(1), 0.0)
    with np.errstate(invalid="ignore", divide="ignore", over="ignore"):
        return np.where(on, m + np.log(np.where(l > -np.inf, np.exp(l - m[:, None]), 0.0).sum(1)), 0.0)


def grad(l, ids, score, renorm, scale, gw=None, S=1, bc=0.0, zc=0.0, gl=(1.0, 1.0), counts=None, tokens=None, mask=None):
    """(gradient of the logits, magnitudes that its rounding is relative to)."""
    T, E = l.shape
    K = ids.shape[1]
    on = live(l, mask)
    s = np.where(on[:, None], scores(l, score), 0.0)
    p = probabilities(l, score, on)
    d, mag = np.zeros((T, E)), np.zeros((T, E))
    if gw is not None:
        use = (ids >= 0) & (ids < E) & on[:, None]
        at = np.where(use, ids, 0)
        q = np.where(use, np.take_along_axis(log_scores(l, score), at, 1), -np.inf)
        use &= q > -np.inf
        g = np.where(use, gw, 0.0)
        if renorm:
            m = np.where(use.any(1), q.max(1), 0.0)[:, None]
            with np.errstate(invalid="ignore"):
                e = np.where(use, np.exp(q - m), 0.0)
            w = e / np.where(e.sum(1, keepdims=True) > 0, e.sum(1, keepdims=True), 1.0)
            mean = (w * g).sum(1, keepdims=True)
            a = scale * w * (g - mean)
            am = abs(scale) * w * (np.abs(g) + (w * np.abs(g)).sum(1, keepdims=True))
        else:
            a = scale * np.where(use, np.exp(q), 0.0) * g
            am = np.abs(a)
        rows = np.repeat(np.arange(T), K)
        np.add.at(d, (rows, at.ravel()), np.where(use, a, 0.0).ravel())
        np.add.at(mag, (rows, at.ravel()), np.where(use, am, 0.0).ravel())
        if score == SOFTMAX and not renorm:
            d -= s * a.sum(1, keepdims=True)
            mag += s * am.sum(1, keepdims=True)
    if counts is not None:
        n = T // S
        f = np.array([gl[0] * bc * E / (S * K * t ** 2) if t else 0.0 for t in tokens])
        A = np.repeat(f[:, None] * counts, n, 0)
        d += p * (A - (A * p).sum(1, keepdims=True))
        top = np.repeat(np.abs(f)[:, None] * (counts + np.array([K * t / E for t in tokens])[:, None]), n, 0)
        mag += p * (top + (top * p).sum(1, keepdims=True))
    if score == SIGMOID:
        with np.errstate(over="ignore"):
            slope = np.where(l > -np.inf, 1 / (1 + np.exp(np.minimum(l, 700.0))), 0.0)
        d, mag = d * slope, mag * slope
    if counts is not None and zc:
        total = max(int(np.sum(tokens)), 1)
        z = gl[1] * 2 * zc * lse(l, on)[:, None] / total * np.where(on[:, None], scores(l, SOFTMAX), 0.0)
        d, mag = d + z, mag + np.abs(z)
    return d, mag


def grad_tol(mag, d, l, bf16):
    """An exponential is good to (2 |l| + 8) steps; the sums over the ids and slots add E / 8 (eight lanes' values and the
    folds of 64 lanes are added one after the other) and 32 for the rest; half a step of the result's type at the end."""
    E = l.shape[1]
    spread = np.abs(np.where(l > -np.inf, l, 0.0)).max(1, keepdims=True)
    err = mag * (4 * np.minimum(spread, 200.0) + E / 8 + 64) * STEP32 + 2.0 ** -126
    return err + (2.0 ** -8 if bf16 else 2.0 ** -24) * (np.abs(d) + err)
