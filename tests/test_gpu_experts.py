"""The products grouped by expert and their gradients against 64-bit references: ragged sizes (experts
with no row, with one, with several tiles), odd features, compact rows and windows, every type, the gate,
rows of no expert poisoned on the way in and untouched on the way out."""
import numpy as np
import pytest
import torch

import combine_moe_get_amd as mg
from tests import _experts as X

pytestmark = pytest.mark.gpu

RAGGED = [
    [1],
    [0, 0, 5, 0],
    [1, 0, 2, 3, 16, 17, 0],
    [15, 33, 64, 1, 0, 31],
    [130, 0, 127, 128, 1, 300],
    [700, 3],
]
# (K, N): odd sizes, less than a tile, more than one
FEATURES = [(8, 8), (64, 24), (136, 136), (1000, 264), (192, 520)]


def _counts_id(c):
    return "-".join(map(str, c))


@pytest.mark.parametrize("gated", [False, True], ids=["plain", "gated"])
@pytest.mark.parametrize("K,N", FEATURES)
@pytest.mark.parametrize("counts", RAGGED, ids=_counts_id)
def test_bf16(counts, K, N, gated):
    print(f"[experts bf16] {counts} K={K} N={N} gated={gated}", flush=True)
    r = np.random.default_rng([1, K, N, sum(counts)])
    rows = X.Rows(counts)
    x, w = X.bf16(r, rows.rows, K), X.bf16(r, rows.E, N * (2 if gated else 1), K, scale=K ** -0.5)
    ref, tol = X.product(rows, X.f64(x), X.f64(w), gated)
    out = X.canary(rows.rows, N)
    mg.experts_matmul(rows.shape(K, N), X.poison(x, rows.used).to(X.DEV), w.to(X.DEV), rows.dev_off(),
                      act=mg.ACT_SWIGLU if gated else mg.ACT_NONE, out=out)
    X.check(out, ref, tol, rows.used, "bf16")


@pytest.mark.parametrize("scales", ["both", "rows", "channels", "none"])
@pytest.mark.parametrize("gated", [False, True], ids=["plain", "gated"])
@pytest.mark.parametrize("K,N", [(16, 8), (144, 136), (1008, 264)])
@pytest.mark.parametrize("counts", RAGGED[2:5], ids=_counts_id)
def test_int8(counts, K, N, gated, scales):
    print(f"[experts int8] {counts} K={K} N={N} gated={gated} scales={scales}", flush=True)
    r = np.random.default_rng([2, K, N, sum(counts)])
    rows = X.Rows(counts)
    nw = N * (2 if gated else 1)
    x = torch.from_numpy(r.integers(-127, 128, (rows.rows, K)).astype(np.int8))
    w = torch.from_numpy(r.integers(-128, 128, (rows.E, nw, K)).astype(np.int8))
    unit = 1 / (70.0 * 70.0 * K ** 0.5)
    xs = (r.uniform(0.5, 2, rows.rows) * unit).astype(np.float32) if scales in ("both", "rows") else None
    ws = (r.uniform(0.5, 2, (rows.E, nw)) * (1 if scales == "both" else unit)).astype(np.float32) \
        if scales in ("both", "channels") else None
    ref, tol = np.zeros((rows.rows, N)), np.ones((rows.rows, N))
    for e, lo, hi in rows.spans():
        y = (x[lo:hi].long().numpy() @ w[e].long().numpy().T).astype(np.float64)  # exact
        if ws is not None:
            y = y * ws[e].astype(np.float64)
        if xs is not None:
            y = y * xs[lo:hi, None].astype(np.float64)
        err = 2 * X.STEP32 * np.abs(y)  # the sum and the two scalings, half a step each
        if gated:
            y, err = X.gate(y, err)
        ref[lo:hi] = y
        tol[lo:hi] = err + X.BF16_HALF * (np.abs(y) + err) + X.TINY
    # without scales the gate works on whole numbers up to 127 * 128 * K: silu(g) u is still finite
    out = X.canary(rows.rows, N)
    d = lambda a: None if a is None else torch.from_numpy(a).to(X.DEV)  # noqa: E731
    mg.experts_matmul(rows.shape(K, N), X.poison(x, rows.used).to(X.DEV), w.to(X.DEV), rows.dev_off(), d(xs), d(ws),
                      mg.ACT_SWIGLU if gated else mg.ACT_NONE, out)
    X.check(out, ref, tol, rows.used, "int8")


def test_int8_largest_sum_is_exact():
    # every product -128 * 127 over the longest row: the int32 sum holds it
    K, N = 65536, 8
    x = torch.full((2, K), 127, dtype=torch.int8, device=X.DEV)
    w = torch.full((1, N, K), -128, dtype=torch.int8, device=X.DEV)
    off = torch.tensor([0, 2], dtype=torch.int32, device=X.DEV)
    out = mg.experts_matmul(mg.make_experts_shape(2, 1, K, N), x, w, off)
    want = torch.tensor(-128.0 * 127 * K, dtype=torch.float64).bfloat16()
    assert torch.all(out.cpu() == want)


@pytest.mark.parametrize("gated", [False, True], ids=["plain", "gated"])
@pytest.mark.parametrize("K,N", [(32, 8), (96, 24), (128, 72), (288, 136), (640, 264), (1056, 264), (2048, 136)])
@pytest.mark.parametrize("counts", RAGGED, ids=_counts_id)
def test_mxfp4(counts, K, N, gated):
    print(f"[experts mxfp4] {counts} K={K} N={N} gated={gated}", flush=True)
    r = np.random.default_rng([3, K, N, sum(counts)])
    rows = X.Rows(counts)
    nw = N * (2 if gated else 1)
    x = r.integers(0, 256, (rows.rows, K // 2)).astype(np.uint8)
    w = r.integers(0, 256, (rows.E, nw, K // 2)).astype(np.uint8)
    xs = r.integers(121, 131, (rows.rows, K // 32)).astype(np.uint8)
    ws = (r.integers(119, 128, (rows.E, nw, K // 32)) - int(np.log2(K) / 2)).astype(np.uint8)
    ref, tol = X.product(rows, X.unpack_mx(x, xs), X.unpack_mx(w, ws), gated)
    out = X.canary(rows.rows, N)
    t = torch.from_numpy
    mg.experts_matmul(rows.shape(K, N), X.poison(t(x), rows.used).to(X.DEV), t(w).to(X.DEV), rows.dev_off(),
                      X.poison(t(xs), rows.used).to(X.DEV), t(ws).to(X.DEV), mg.ACT_SWIGLU if gated else mg.ACT_NONE, out)
    X.check(out, ref, tol, rows.used, "mxfp4")


@pytest.mark.parametrize("K", [320, 384, 640])  # the last with scales that fill 16 bytes a row and a part
@pytest.mark.parametrize("rows_of", [1, 40, 200])
def test_mxfp4_nan_scale_reaches_its_own_sums_only(rows_of, K):
    N = 72
    r = np.random.default_rng(4)
    t = torch.from_numpy
    x, w = r.integers(0, 256, (rows_of, K // 2)).astype(np.uint8), r.integers(0, 256, (1, N, K // 2)).astype(np.uint8)
    xs, ws = np.full((rows_of, K // 32), 127, np.uint8), np.full((1, N, K // 32), 120, np.uint8)
    xs[rows_of // 2, -1] = 255  # the last block of a row
    xs[rows_of // 3, 0] = 255   # the first of another
    ws[0, 5, 3] = 255
    ws[0, 9, 0] = 255
    off = torch.tensor([0, rows_of], dtype=torch.int32, device=X.DEV)
    out = mg.experts_matmul(mg.make_experts_shape(rows_of, 1, K, N), t(x).to(X.DEV), t(w).to(X.DEV), off, t(xs).to(X.DEV),
                            t(ws).to(X.DEV)).cpu()
    nan = torch.zeros(rows_of, N, dtype=torch.bool)
    nan[[rows_of // 2, rows_of // 3]] = True
    nan[:, [5, 9]] = True
    assert torch.equal(torch.isnan(out), nan)


def test_mxfp4_scales_at_odd_addresses():
    K, N, rows = 256, 136, 70
    r = np.random.default_rng(13)
    t = torch.from_numpy
    x, w = r.integers(0, 256, (rows, K // 2)).astype(np.uint8), r.integers(0, 256, (1, N, K // 2)).astype(np.uint8)
    xs, ws = r.integers(121, 131, (rows, K // 32)).astype(np.uint8), r.integers(112, 120, (1, N, K // 32)).astype(np.uint8)
    off = torch.tensor([0, rows], dtype=torch.int32, device=X.DEV)
    shape, xd, wd = mg.make_experts_shape(rows, 1, K, N), t(x).to(X.DEV), t(w).to(X.DEV)
    want = mg.experts_matmul(shape, xd, wd, off, t(xs).to(X.DEV), t(ws).to(X.DEV))

    def odd(a, by):  # the same values, `by` bytes behind an aligned address
        buf = torch.empty(a.size + by, dtype=torch.uint8, device=X.DEV)
        buf[by:] = t(a).flatten().to(X.DEV)
        return buf[by:].view(a.shape)

    for i, j in ((1, 0), (0, 3), (2, 1)):
        assert torch.equal(mg.experts_matmul(shape, xd, wd, off, odd(xs, i), odd(ws, j)), want)


def test_misaligned_rows_are_refused():
    s = mg.make_experts_shape(4, 1, 64, 24)
    x = torch.zeros(4 * 64 + 4, dtype=torch.bfloat16, device=X.DEV)[4:].view(4, 64)
    w = torch.zeros(1, 24, 64, dtype=torch.bfloat16, device=X.DEV)
    off = torch.tensor([0, 4], dtype=torch.int32, device=X.DEV)
    with pytest.raises(mg.MoeGetError):
        mg.experts_matmul(s, x, w, off)
    with pytest.raises(ValueError, match="contiguous"):
        mg.experts_matmul(s, torch.zeros(64, 4, dtype=torch.bfloat16, device=X.DEV).t(), w, off)
    with pytest.raises(ValueError, match="elements"):
        mg.experts_matmul(s, torch.zeros(3, 64, dtype=torch.bfloat16, device=X.DEV), w, off)
    with pytest.raises(TypeError):
        mg.experts_matmul(s, w.view(24, 64)[:4].float(), w, off)
    with pytest.raises(TypeError):
        mg.experts_matmul(s, w.view(24, 64)[:4], w, off.long())
    with pytest.raises(ValueError, match="scales"):
        mg.experts_matmul(s, w.view(24, 64)[:4], w, off, row_scales=torch.ones(4, device=X.DEV))
    with pytest.raises(ValueError, match="device"):
        mg.experts_matmul(s, w.view(24, 64)[:4], w, off.cpu())


@pytest.mark.parametrize("rows_of", [1, 40, 200])
def test_bf16_infinities_and_nan_stay_in_their_sums(rows_of):
    K, N = 200, 72
    r = np.random.default_rng(5)
    x, w = X.bf16(r, rows_of, K), X.bf16(r, 1, N, K)
    x[rows_of // 2, K - 1] = float("nan")
    w[0, 7, 0] = float("inf")
    off = torch.tensor([0, rows_of], dtype=torch.int32, device=X.DEV)
    out = mg.experts_matmul(mg.make_experts_shape(rows_of, 1, K, N), x.to(X.DEV), w.to(X.DEV), off).cpu()
    assert torch.isnan(out[rows_of // 2]).all()
    rest = torch.cat((out[: rows_of // 2], out[rows_of // 2 + 1:]))
    assert torch.isfinite(rest[:, torch.arange(N) != 7]).all()
    first = torch.cat((x[: rows_of // 2, 0], x[rows_of // 2 + 1:, 0])).float()
    assert torch.equal(rest[:, 7].float(), first * float("inf"))


WINDOWS = [([3, 0, 5, 20], 2, 4), ([0, 0, 1, 140, 0, 7], 3, 0), ([70, 130, 0, 0], 4, 1)]


@pytest.mark.parametrize("counts,P,slack", WINDOWS)
def test_windows(counts, P, slack):
    print(f"[experts windows] {counts} P={P} slack={slack}", flush=True)
    K, N = 160, 136
    r = np.random.default_rng([6, sum(counts)])
    rows = X.Rows(counts, P=P, slack=slack)
    x, w = X.bf16(r, rows.rows, K), X.bf16(r, rows.E, N, K, scale=K ** -0.5)
    ref, tol = X.product(rows, X.f64(x), X.f64(w), False)
    out = X.canary(rows.rows, N)
    mg.experts_matmul(rows.shape(K, N), X.poison(x, rows.used).to(X.DEV), w.to(X.DEV), rows.dev_off(), out=out)
    X.check(out, ref, tol, rows.used, "windows")
    _backward(rows, K, N, r, torch.float32)


def _backward(rows, K, N, r, dtype):
    x, w = X.bf16(r, rows.rows, K), X.bf16(r, rows.E, N, K, scale=K ** -0.5)
    dy = X.bf16(r, rows.rows, N)
    shape, off = rows.shape(K, N), rows.dev_off()
    dyd, xd = X.poison(dy, rows.used).to(X.DEV), X.poison(x, rows.used).to(X.DEV)
    # to the rows: the product with the weights' other index
    wt = np.ascontiguousarray(X.f64(w).transpose(0, 2, 1))
    ref, tol = X.product(rows, X.f64(dy), wt, False)
    dx = X.canary(rows.rows, K)
    mg.experts_matmul_dgrad(shape, dyd, w.to(X.DEV), off, out=dx)
    X.check(dx, ref, tol, rows.used, "dgrad")
    # to the weights
    dw = torch.full((rows.E, N, K), -7.0, dtype=dtype, device=X.DEV)
    mg.experts_matmul_wgrad(shape, dyd, xd, off, out=dw)
    ref, tol = np.zeros((rows.E, N, K)), np.zeros((rows.E, N, K))
    for e, lo, hi in rows.spans():
        a, b = X.f64(dy[lo:hi]), X.f64(x[lo:hi])
        ref[e] = a.T @ b
        err = (hi - lo + 8) * X.STEP32 * (np.abs(a).T @ np.abs(b))
        tol[e] = err + (X.BF16_HALF * (np.abs(ref[e]) + err) if dtype == torch.bfloat16 else 0)
        if hi == lo:
            assert np.all(tol[e] == 0)  # zeros, exactly
    every = np.ones(rows.E, bool)
    X.check(dw, ref, tol + np.where(tol > 0, X.TINY, 0), every, "wgrad")


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("K,N", FEATURES)
@pytest.mark.parametrize("counts", RAGGED, ids=_counts_id)
def test_gradients(counts, K, N, dtype):
    print(f"[experts gradients] {counts} K={K} N={N} {dtype}", flush=True)
    _backward(X.Rows(counts), K, N, np.random.default_rng([7, K, N, sum(counts)]), dtype)


def test_gradients_against_differences():
    """<grad, direction> against central differences of the products in 64 bits.  The sum is linear in
    x and in w, so a difference has no error of its own but 64-bit rounding; the gradients' errors are at
    most half a bf16 step of each element (and fp32 sums), so the dot product's at most that of its terms."""
    K, N, counts = 72, 40, [5, 0, 18, 33]
    r = np.random.default_rng(8)
    rows = X.Rows(counts, extra=0)
    x, w, dy = X.bf16(r, rows.rows, K), X.bf16(r, 4, N, K), X.bf16(r, rows.rows, N)
    shape, off = rows.shape(K, N), rows.dev_off()
    dx = X.f64(mg.experts_matmul_dgrad(shape, dy.to(X.DEV), w.to(X.DEV), off).cpu())
    dw = X.f64(mg.experts_matmul_wgrad(shape, dy.to(X.DEV), x.to(X.DEV), off).cpu())

    def loss(x64, w64):
        return sum(float((x64[lo:hi] @ w64[e].T * X.f64(dy)[lo:hi]).sum()) for e, lo, hi in rows.spans())

    x64, w64 = X.f64(x), X.f64(w)
    for i in range(4):
        vx, vw = r.standard_normal(x64.shape), r.standard_normal(w64.shape)
        got, allowed = (dx * vx).sum(), (np.abs(dx * vx)).sum() * 2 * X.BF16_HALF
        want = (loss(x64 + vx, w64) - loss(x64 - vx, w64)) / 2
        assert abs(got - want) <= allowed
        got, allowed = (dw * vw).sum(), (np.abs(dw * vw)).sum() * 2 * X.BF16_HALF
        want = (loss(x64, w64 + vw) - loss(x64, w64 - vw)) / 2
        assert abs(got - want) <= allowed


@pytest.mark.parametrize("counts,K,N", [([2000, 1, 900], 512, 768), ([300] * 9, 1024, 1288), ([9] * 40, 2048, 264),
                                        ([1] * 100 + [0] * 28, 520, 72)])
def test_larger(counts, K, N):
    """Several tiles each way, every operator, on one layout."""
    print(f"[experts larger] {counts[:4]}.. K={K} N={N}", flush=True)
    r = np.random.default_rng([9, K, N])
    rows = X.Rows(counts)
    x, w = X.bf16(r, rows.rows, K), X.bf16(r, rows.E, N, K, scale=K ** -0.5)
    ref, tol = X.product(rows, X.f64(x), X.f64(w), False)
    out = X.canary(rows.rows, N)
    mg.experts_matmul(rows.shape(K, N), X.poison(x, rows.used).to(X.DEV), w.to(X.DEV), rows.dev_off(), out=out)
    X.check(out, ref, tol, rows.used, "bf16")
    _backward(rows, K, N, r, torch.bfloat16)


# counts, N: several tiles for each workgroup that is resident, for every tile shape that the sizes select
SHAPES = {
    "16 rows": ([8, 0, 15, 3] * 24, 1544),
    "64 rows": ([40, 64, 65, 0] * 24, 1544),
    "128 rows": ([100, 129, 1, 130] * 24, 1544),
    "few tiles": ([129, 260, 7, 300], 1032),
    "256 rows": ([700, 513, 256, 1, 999, 0, 1500, 300] * 2, 3080),
}


@pytest.mark.parametrize("gated", [False, True], ids=["plain", "gated"])
@pytest.mark.parametrize("row_type", ["bf16", "int8", "mxfp4", "mxfp4, odd rows of scales"])
@pytest.mark.parametrize("name", list(SHAPES))
def test_tile_shapes(name, row_type, gated):
    counts, N = SHAPES[name]
    K = {"bf16": 416, "int8": 400, "mxfp4": 384}.get(row_type, 416)
    N = N // 2 // 8 * 8 if gated else N
    print(f"[experts shapes] {name} {row_type} gated={gated} N={N} K={K}", flush=True)
    r = np.random.default_rng([11, N, K])
    rows = X.Rows(counts)
    nw = N * (2 if gated else 1)
    t = torch.from_numpy
    xs = ws = None
    if row_type == "bf16":
        x, w = X.bf16(r, rows.rows, K), X.bf16(r, rows.E, nw, K, scale=K ** -0.5)
        x64, w64 = X.f64(x), X.f64(w)
    elif row_type == "int8":
        x, w = (t(r.integers(-127, 128, s, dtype=np.int8)) for s in ((rows.rows, K), (rows.E, nw, K)))
        xs, ws = (t(r.uniform(0.5, 2, s).astype(np.float32) / 70) for s in ((rows.rows,), (rows.E, nw)))
        ws /= K ** 0.5
        x64, w64 = X.f64(x) * X.f64(xs)[:, None], X.f64(w) * X.f64(ws)[..., None]
    else:
        x, w = (t(r.integers(0, 256, s, dtype=np.uint8)) for s in ((rows.rows, K // 2), (rows.E, nw, K // 2)))
        xs = t(r.integers(122, 129, (rows.rows, K // 32), dtype=np.uint8))
        ws = t(r.integers(116, 123, (rows.E, nw, K // 32), dtype=np.uint8))
        x64, w64 = X.unpack_mx(x.numpy(), xs.numpy()), X.unpack_mx(w.numpy(), ws.numpy())
    ref, tol = X.product(rows, x64, w64, gated)
    d = lambda a: None if a is None else a.to(X.DEV)  # noqa: E731
    xd, wd, xsd, wsd = d(X.poison(x, rows.used)), d(w), d(xs), d(ws)
    outs = []
    for _ in range(2):
        out = X.canary(rows.rows, N)
        mg.experts_matmul(rows.shape(K, N), xd, wd, rows.dev_off(), xsd, wsd,
                          mg.ACT_SWIGLU if gated else mg.ACT_NONE, out)
        outs.append(out)
    X.check(outs[0], ref, tol, rows.used, name)
    assert torch.equal(outs[0], outs[1]), "the same call twice"


@pytest.mark.parametrize("name", list(SHAPES))
def test_tile_shapes_of_gradients(name):
    counts, N = SHAPES[name]
    print(f"[experts shapes] {name} gradients", flush=True)
    _backward(X.Rows(counts), 416 if N < 2000 else 1040, N // 2 // 8 * 8, np.random.default_rng(12), torch.bfloat16)


def test_many_experts():
    counts = [(e * 7) % 5 for e in range(2048)]
    rows = X.Rows(counts)
    r = np.random.default_rng(10)
    K, N = 64, 16
    x, w = X.bf16(r, rows.rows, K), X.bf16(r, rows.E, N, K, scale=K ** -0.5)
    ref, tol = X.product(rows, X.f64(x), X.f64(w), False)
    out = X.canary(rows.rows, N)
    mg.experts_matmul(rows.shape(K, N), x.to(X.DEV), w.to(X.DEV), rows.dev_off(), out=out)
    X.check(out, ref, tol, rows.used, "2048 experts")
    _backward(rows, K, N, r, torch.bfloat16)


@pytest.mark.parametrize("off", [[0, 5, 3, 9, 9], [0, 4000, 4001, 4002, 5000], [-5, 3, 700, 2, 6], [7, 7, 7, 7, 7]])
@pytest.mark.parametrize("stride", [0, 5])
def test_offsets_that_make_no_sense_touch_nothing_outside(off, stride):
    """Offsets that do not ascend or pass the buffer: the calls return, and guard rows around every
    buffer keep their values."""
    rows, K, N = 10, 64, 72
    shape = mg.make_experts_shape(rows, 4, K, N, 2 if stride else 1, stride)
    offd = torch.tensor(off, dtype=torch.int32, device=X.DEV)
    x = torch.ones(rows, K, dtype=torch.bfloat16, device=X.DEV)
    w = torch.ones(4, N, K, dtype=torch.bfloat16, device=X.DEV)
    dy = torch.ones(rows, N, dtype=torch.bfloat16, device=X.DEV)
    out, dx = X.canary(rows + 4, N), X.canary(rows + 4, K)
    mg.experts_matmul(shape, x, w, offd, out=out[2:-2])
    mg.experts_matmul_dgrad(shape, dy, w, offd, out=dx[2:-2])
    dw = mg.experts_matmul_wgrad(shape, dy, x, offd)
    torch.cuda.synchronize()
    for t in (out, dx):
        assert torch.all(t[:2] == -7) and torch.all(t[-2:] == -7)
    assert torch.all((dw >= 0) & (dw <= rows))


def test_beyond_4_gib():
    """Rows and weights whose byte offsets pass 32 bits: the last window's rows, the last expert's weights."""
    K, N, E, stride = 8192, 8192, 40, 7500
    counts = [2] + [0] * (E - 2) + [21]
    r = np.random.default_rng(14)
    rows = E * stride  # 4.9 GB of bf16
    shape = mg.make_experts_shape(rows, E, K, N, E, stride)
    off = torch.from_numpy(X.offsets(counts)).to(X.DEV)
    lo = (E - 1) * stride
    x = torch.zeros(rows, K, dtype=torch.bfloat16, device=X.DEV)
    w = torch.zeros(E, N, K, dtype=torch.bfloat16, device=X.DEV)  # 5.4 GB
    assert x.numel() * 2 > 1 << 32 and w.numel() * 2 > 1 << 32
    x1, w1, dy1 = X.bf16(r, 21, K), X.bf16(r, N, K, scale=K ** -0.5), X.bf16(r, 21, N)
    x[lo:lo + 21], w[-1] = x1.to(X.DEV), w1.to(X.DEV)
    one = X.Rows([21], extra=0)
    out = torch.zeros(rows, N, dtype=torch.bfloat16, device=X.DEV)
    mg.experts_matmul(shape, x, w, off, out=out)
    ref, tol = X.product(one, X.f64(x1), X.f64(w1)[None], False)
    X.check(out[lo:lo + 21], ref, tol, one.used, "forward")
    assert not out[lo + 21:].any() and not out[:lo].any()
    out[lo:lo + 21] = dy1.to(X.DEV)
    dx = mg.experts_matmul_dgrad(shape, out, w, off, out=torch.zeros_like(x))
    ref, tol = X.product(one, X.f64(dy1), X.f64(w1).T[None], False)
    X.check(dx[lo:lo + 21], ref, tol, one.used, "dgrad")
    del dx
    dw = mg.experts_matmul_wgrad(shape, out, x, off, out=w)
    a, b = X.f64(dy1), X.f64(x1)
    err = 29 * X.STEP32 * (np.abs(a).T @ np.abs(b))
    X.check(dw[-1], a.T @ b, err + X.BF16_HALF * (np.abs(a.T @ b) + err) + X.TINY, np.ones(N, bool), "wgrad")
    assert not dw[:-1].any()
    del dw, w, out
    for row_type in (mg.ROWS_INT8, mg.ROWS_MXFP4):
        codes, scales = mg.quantize_rows(x, row_type)
        want = mg.quantize_rows(x1.to(X.DEV), row_type)
        assert torch.equal(codes[lo:lo + 21], want[0]) and torch.equal(scales[lo:lo + 21], want[1])


def test_no_rows():
    shape = mg.make_experts_shape(0, 3, 64, 24)
    off = torch.zeros(4, dtype=torch.int32, device=X.DEV)
    x = torch.empty(0, 64, dtype=torch.bfloat16, device=X.DEV)
    w = torch.ones(3, 24, 64, dtype=torch.bfloat16, device=X.DEV)
    dy = torch.empty(0, 24, dtype=torch.bfloat16, device=X.DEV)
    assert mg.experts_matmul(shape, x, w, off).shape == (0, 24)
    assert mg.experts_matmul_dgrad(shape, dy, w, off).shape == (0, 64)
    assert torch.all(mg.experts_matmul_wgrad(shape, dy, x, off) == 0)
