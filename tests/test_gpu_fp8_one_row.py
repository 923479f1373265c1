"""A single row has no row stride: operands and outputs that are one row of a tensor whose rows are no whole
16-byte pieces apart are taken."""

import pytest
import torch

pytestmark = pytest.mark.gpu

import moe_prefill_nvfp4_gb300 as moe  # noqa: E402

from test_gpu_fp8 import assert_product, codes, dequant_blocks64, dequant_rows64, product64, quantize_ref, rand, weights  # noqa: E402


@pytest.fixture(autouse=True)
def _no_device_error():
    moe.moe_get_device_error()
    yield
    assert moe.moe_get_device_error() == 0


def row_of(dtype, cols, stride, fill):
    """Row 0 of three rows `stride` elements apart, and all of them as bytes."""
    t = torch.full((3, stride), fill, dtype=torch.uint8 if dtype == torch.float8_e4m3fn else dtype, device="cuda")
    return t.view(dtype)[:1, :cols], t


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("k", [5, 200, 256, 1031])
def test_quantise_one_row(k, dtype):
    x = rand((3, k + 3), k, 1.0, dtype)[:1, :k]
    qr, sr = quantize_ref(x, 1)
    for f in (moe.moe_fp8_quantize_rows, moe.moe_fp8_quantize_blocks):
        out, flat = row_of(torch.float8_e4m3fn, k, k + 7, 0x55)
        q, s = f(x, out=out)
        assert (codes(q) == qr).all() and (s.cpu().numpy() == sr).all()
        assert (flat[0, k:] == 0x55).all() and (flat[1:] == 0x55).all()


@pytest.mark.parametrize("c_dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("n,k", [(1, 100), (7, 200), (130, 257), (513, 500)])
def test_gemm_one_row(n, k, c_dtype):
    a, _ = row_of(torch.float8_e4m3fn, k, k + 9, 0x7F)  # (NaN codes beside the row)
    _, sa = moe.moe_fp8_quantize_rows(rand((1, k), n + k), out=a)
    w, sw = moe.moe_fp8_quantize_blocks(rand((n, k), n + k + 1, 0.05))
    out, flat = row_of(c_dtype, n, n + 3, 3.0)
    moe.moe_fp8_gemm(a, sa, w, sw, out=out, c_dtype=c_dtype)
    ref, mags = product64(dequant_rows64(a, sa), dequant_blocks64(w, sw))
    assert_product(out, ref, mags, k)
    assert (flat[0, n:] == 3).all() and (flat[1:] == 3).all()


@pytest.mark.parametrize("rows", [1, 40, 300])
def test_gemm_one_weight_row(rows):
    k = 300
    a, sa = moe.moe_fp8_quantize_rows(rand((rows, k), 5))
    w, _ = row_of(torch.float8_e4m3fn, k, k + 5, 0x7F)
    _, sw = moe.moe_fp8_quantize_blocks(rand((1, k), 6), out=w)
    ref, mags = product64(dequant_rows64(a, sa), dequant_blocks64(w, sw))
    assert_product(moe.moe_fp8_gemm(a, sa, w, sw, c_dtype=torch.float32), ref, mags, k)


def test_grouped_one_row():
    n, k, inter = 128, 200, 128
    a, _ = row_of(torch.float8_e4m3fn, k, k + 9, 0x7F)
    _, sa = moe.moe_fp8_quantize_rows(rand((1, k), 7), out=a)
    w, sw = weights(2, n, k, 8)
    off = torch.tensor([0, 0, 1], dtype=torch.int32, device="cuda")
    out, _ = row_of(torch.bfloat16, n, n + 5, 3.0)
    moe.moe_fp8_grouped_gemm(a, sa, w, sw, off, 1, out=out)
    ref, mags = product64(dequant_rows64(a, sa), dequant_blocks64(w[1], sw[1]))
    assert_product(out, ref, mags, k)
    w, sw = weights(2, 2 * inter, k, 9)
    act, flat = row_of(torch.float8_e4m3fn, inter, inter + 3, 0x55)
    want, scales = moe.moe_fp8_grouped_gemm_swiglu(a, sa, w, sw, off, 1)
    _, s = moe.moe_fp8_grouped_gemm_swiglu(a, sa, w, sw, off, 1, out=act)
    assert (codes(act) == codes(want)).all() and torch.equal(s, scales)
    assert (flat[0, inter:] == 0x55).all() and (flat[1:] == 0x55).all()
