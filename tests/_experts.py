"""Helpers of the expert-stage tests: ragged row layouts, references in 64 bits on the CPU and
tolerances that follow from the arithmetic (one rounding to the output's type, one to fp32 per addition)."""
import numpy as np
import torch

import combine_moe_get_amd as mg

DEV = torch.device("cuda:0")
E2M1 = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6, -0.0, -0.5, -1, -1.5, -2, -3, -4, -6])
BF16_HALF = 2.0 ** -8  # half a step of bf16, relative
STEP32 = 2.0 ** -23    # a whole step of fp32, relative: bounds an addition however it rounds
TINY = 2.0 ** -126


def offsets(counts):
    off = np.zeros(len(counts) + 1, np.int32)
    off[1:] = np.cumsum(counts)
    return off


class Rows:
    """Rows of experts in a buffer of `rows`: compact, or P windows of `stride` rows."""

    def __init__(self, counts, extra=3, P=1, slack=None):
        self.counts, self.E, self.P = list(counts), len(counts), P
        self.off = offsets(counts)
        L = self.E // P
        if slack is None:
            self.stride, self.rows = 0, int(self.off[-1]) + extra
            self.first = self.off[:-1].astype(np.int64)
        else:
            self.stride = max(int(self.off[(r + 1) * L] - self.off[r * L]) for r in range(P)) + slack
            self.rows = self.stride * P + extra
            self.first = np.array([(e // L) * self.stride + self.off[e] - self.off[e // L * L] for e in range(self.E)])
        self.used = np.zeros(self.rows, bool)
        for f, c in zip(self.first, self.counts):
            self.used[f:f + c] = True

    def shape(self, k, n):
        return mg.make_experts_shape(self.rows, self.E, k, n, self.P, self.stride)

    def spans(self):
        return [(e, int(f), int(f) + c) for e, (f, c) in enumerate(zip(self.first, self.counts))]

    def dev_off(self):
        return torch.from_numpy(self.off).to(DEV)


def bf16(rng, *shape, scale=1.0):
    return (torch.from_numpy(rng.standard_normal(shape, dtype=np.float32)) * scale).bfloat16()


def f64(t):
    return t.double().numpy()


def poison(t, used):
    """t with the rows of no expert NaN (or 255): they must not be read."""
    t = t.clone()
    t[torch.from_numpy(~used)] = float("nan") if t.dtype.is_floating_point else 127 if t.dtype == torch.int8 else 255
    return t


def canary(rows, n):
    return torch.full((rows, n), -7.0, dtype=torch.bfloat16, device=DEV)


def check(got, ref, tol, used, what, left=-7.0):
    """Rows in use within tol of ref; the others as they were."""
    got = got.cpu().double().numpy()
    assert np.all(got[~used] == left), f"{what}: rows of no expert were written"
    g, r, t = got[used], ref[used], tol[used]
    bad = ~(np.abs(g - r) <= t)
    if bad.any():
        i = np.unravel_index(np.argmax(np.where(np.isnan(g), np.inf, np.abs(g - r) / t)), g.shape)
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.size} values off; worst at {i}: got {g[i]} want {r[i]} "
                             f"allowed {t[i]}")


def unpack_mx(codes, scales):
    c = codes.astype(np.uint8)
    v = np.stack((E2M1[c & 15], E2M1[c >> 4]), -1).reshape(c.shape[:-1] + (-1,))
    s = np.where(scales == 255, np.nan, 2.0 ** (scales.astype(np.float64) - 127))
    return (v.reshape(v.shape[:-1] + (-1, 32)) * s[..., None]).reshape(v.shape)


def quant_mx(x):
    """The definition in 64 bits: x [.., K] float64 -> (codes [.., K / 2], scales [.., K / 32])."""
    b = x.reshape(x.shape[:-1] + (-1, 32))
    amax = np.abs(b).max(-1)
    fine = np.isfinite(amax)
    with np.errstate(divide="ignore", invalid="ignore"):
        e = np.floor(np.log2(np.where(fine & (amax > 0), amax, 1.0)))
        # log2 may round up to a whole number just below a power of two
        e = np.where(2.0 ** e > np.where(amax > 0, amax, 1.0), e - 1, e)
    s = np.where(amax > 0, np.maximum(e - 2, -127), -127)
    a = np.where(fine[..., None], np.abs(b) / 2.0 ** s[..., None], 0.0)
    dist = np.abs(a[..., None] - E2M1[:8])
    near = dist.min(-1, keepdims=True)
    even = np.arange(8) % 2
    code = np.argmin(np.where(dist == near, even, 9), -1)  # the nearest; of two, the even code
    code = np.where(fine[..., None], code | (np.signbit(b).astype(np.int64) << 3), 0)
    code = code.reshape(x.shape).astype(np.uint8)
    scale = np.where(fine, s + 127, 255).astype(np.uint8)
    return code[..., 0::2] | (code[..., 1::2] << 4), scale


def product(rows, x, w, gated, extra=1.0):
    """(reference, tolerance) of the products of x [rows, K] and w [E, Nw, K] in float64, for fp32 sums:
    K additions of at most a step of fp32 each of the sum of magnitudes, then half a bf16 step."""
    n = w.shape[1] // 2 if gated else w.shape[1]
    ref = np.zeros((rows.rows, n))
    tol = np.ones((rows.rows, n))
    K = w.shape[2]
    for e, lo, hi in rows.spans():
        if hi == lo:
            continue
        y = x[lo:hi] @ w[e].T
        err = extra * (K + 8) * STEP32 * (np.abs(x[lo:hi]) @ np.abs(w[e]).T)
        if gated:
            y, err = gate(y, err)
        ref[lo:hi] = y
        tol[lo:hi] = err + BF16_HALF * (np.abs(y) + err) + TINY
    return ref, tol


def gate(y, err):
    """silu(g) u of y = [g | u] known to within err: |silu'| <= 1.1, and silu itself to within
    (|g| + 8) steps of fp32, from the exponential of a rounded argument."""
    n = y.shape[1] // 2
    g, u, eg, eu = y[:, :n], y[:, n:], err[:, :n], err[:, n:]
    with np.errstate(over="ignore"):
        s = g / (1 + np.exp(-g))
    es = 1.1 * eg + (np.abs(g) + 8) * STEP32 * np.abs(s)
    return s * u, np.abs(s) * eu + es * (np.abs(u) + eu)
