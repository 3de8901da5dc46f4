"""Row quantization: int8 codes and scales, and microscaled 4-bit floats, bit for bit against their
definitions (binary32 for int8, as its formula says; 64 bits for the 4-bit floats)."""
import numpy as np
import pytest
import torch

import combine_moe_get_amd as mg
from tests import _experts as X

pytestmark = pytest.mark.gpu


def _int8(x):
    """x float32 [rows, K] -> codes, scales; each operation rounded once to binary32."""
    amax = np.abs(x).max(1)
    with np.errstate(divide="ignore", invalid="ignore", over="ignore"):
        dyn = np.where(amax > 0, np.float32(127) / amax, np.float32(0)).astype(np.float32)
        p = np.rint(x * dyn[:, None])
        code = np.clip(np.where(np.isnan(p), 0, p), -127, 127).astype(np.int8)
        return code, np.where(amax > 0, np.float32(1) / dyn, np.float32(0)).astype(np.float32)


@pytest.mark.parametrize("rows,K", [(1, 16), (3, 48), (7, 1040), (64, 2048), (5, 8192), (2, 65536), (1000, 272)])
def test_int8(rows, K):
    r = np.random.default_rng([1, rows, K])
    x = X.bf16(r, rows, K)
    x *= torch.from_numpy(np.exp(r.uniform(-8, 8, (rows, 1)))).bfloat16()
    if rows > 2:
        x[1] = 0
        x[2, 1:] = 0  # one value alone
    codes, scales = mg.quantize_rows(x.to(X.DEV), mg.ROWS_INT8)
    c, s = _int8(x.float().numpy())
    assert np.array_equal(codes.cpu().numpy(), c)
    assert np.array_equal(scales.cpu().numpy(), s)


@pytest.mark.parametrize("rows,K", [(1, 32), (3, 96), (7, 1056), (64, 2048), (3, 65536), (1000, 288)])
def test_mxfp4(rows, K):
    r = np.random.default_rng([2, rows, K])
    x = X.bf16(r, rows, K)
    x *= torch.from_numpy(np.exp(r.uniform(-8, 8, (rows, 1)))).bfloat16()
    codes, scales = mg.quantize_rows(x.to(X.DEV), mg.ROWS_MXFP4)
    c, s = X.quant_mx(X.f64(x))
    assert np.array_equal(scales.cpu().numpy(), s)
    assert np.array_equal(codes.cpu().numpy(), c)


def test_mxfp4_every_value_against_every_scale():
    """All finite bf16 magnitudes beside amaxes of every exponent: ties, subnormals, zeros of both signs,
    values that saturate."""
    bits = np.arange(0x7f80, dtype=np.uint16)
    blocks = []
    for top in np.arange(0, 0x7f80, 61, dtype=np.uint16):
        v = bits[bits <= top][-31 * 40:]  # the values within reach of this amax
        v = np.concatenate((v, np.zeros((-len(v)) % 31, np.uint16))).reshape(-1, 31)
        blocks.append(np.concatenate((v, np.full((len(v), 1), top, np.uint16)), 1))
    b = np.concatenate(blocks)
    b = b | (np.random.default_rng(3).integers(0, 2, b.shape).astype(np.uint16) << 15)
    x = torch.from_numpy(b.view(np.int16)).view(torch.bfloat16)
    codes, scales = mg.quantize_rows(x.to(X.DEV), mg.ROWS_MXFP4)
    c, s = X.quant_mx(X.f64(x))
    assert np.array_equal(scales.cpu().numpy(), s)
    assert np.array_equal(codes.cpu().numpy(), c)


def test_mxfp4_hand_case():
    # amax 6: scale 1; 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5 lie between two values: the even code
    v = [6, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5, -0.25, -0.75, -1.25, -1.75, -2.5, -3.5, -5, -6, 0, -0.0, 0.5, 1, 1.5, 2,
         3, 4, 0.26, 0.24, 2.6, 2.4, 5.1, 4.9, 3.4, 3.6]
    want = [7, 0, 2, 2, 4, 4, 6, 6, 8, 10, 10, 12, 12, 14, 14, 15, 0, 8, 1, 2, 3, 4, 5, 6, 1, 0, 5, 4, 7, 6, 5, 6]
    x = torch.tensor([v, [7.75] + [0.0] * 31, [8.0] + [0.0] * 31]).bfloat16()
    codes, scales = mg.quantize_rows(x.to(X.DEV), mg.ROWS_MXFP4)
    codes = codes.cpu().numpy()
    assert [int(q) for b in codes[0] for q in (b & 15, b >> 4)] == want
    assert scales.cpu().flatten().tolist() == [127, 127, 128]  # 7.75 saturates at 6, 8 begins the next power
    assert codes[1, 0] == 7 and codes[2, 0] == 6


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_mxfp4_not_finite(bad):
    x = torch.ones(2, 96)
    x[1, 40] = bad
    codes, scales = mg.quantize_rows(x.bfloat16().to(X.DEV), mg.ROWS_MXFP4)
    assert scales.cpu().tolist() == [[125, 125, 125], [125, 255, 125]]
    assert torch.all(codes.cpu()[1, 16:32] == 0) and torch.all(codes.cpu()[0] == codes.cpu()[0, 0])


@pytest.mark.parametrize("P,slack", [(1, None), (2, 3), (4, 0)])
@pytest.mark.parametrize("row_type", [mg.ROWS_INT8, mg.ROWS_MXFP4])
def test_only_rows_of_experts(row_type, P, slack):
    K = 96
    rows = X.Rows([5, 0, 1, 9], P=P, slack=slack)
    r = np.random.default_rng(4)
    x = X.bf16(r, rows.rows, K)
    mx = row_type == mg.ROWS_MXFP4
    codes = torch.full((rows.rows, K // 2 if mx else K), 77, dtype=torch.uint8 if mx else torch.int8, device=X.DEV)
    scales = torch.full((rows.rows, 3) if mx else (rows.rows,), 77, dtype=torch.uint8 if mx else torch.float32, device=X.DEV)
    mg.quantize_rows(X.poison(x, rows.used).to(X.DEV), row_type, codes, scales, rows.shape(K, 8), rows.dev_off())
    c, s = X.quant_mx(X.f64(x)) if mx else _int8(x.float().numpy())
    codes, scales = codes.cpu().numpy(), scales.cpu().numpy()
    assert np.array_equal(codes[rows.used], c[rows.used]) and np.array_equal(scales[rows.used], s[rows.used])
    assert np.all(codes[~rows.used] == 77) and np.all(scales[~rows.used] == 77)


def test_weights_and_nothing():
    r = np.random.default_rng(5)
    w = X.bf16(r, 3, 5, 64)
    codes, scales = mg.quantize_rows(w.to(X.DEV), mg.ROWS_MXFP4)
    assert codes.shape == (3, 5, 32) and scales.shape == (3, 5, 2)
    c, s = X.quant_mx(X.f64(w))
    assert np.array_equal(codes.cpu().numpy(), c) and np.array_equal(scales.cpu().numpy(), s)
    codes, scales = mg.quantize_rows(torch.empty(0, 64, dtype=torch.bfloat16, device=X.DEV), mg.ROWS_INT8)
    assert codes.shape == (0, 64) and scales.shape == (0,)
