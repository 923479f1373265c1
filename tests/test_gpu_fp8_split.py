"""Products of few wide tiles around the length from which a cluster shares a tile's k blocks (18 of them)."""

import pytest
import torch

pytestmark = pytest.mark.gpu

import moe_prefill_nvfp4_gb300 as moe  # noqa: E402

from test_gpu_fp8 import assert_product, dequant_blocks64, dequant_rows64, grouped64, grouped_case, product64, rand  # noqa: E402


@pytest.fixture(autouse=True)
def _no_device_error():
    moe.moe_get_device_error()
    yield
    assert moe.moe_get_device_error() == 0


@pytest.mark.parametrize("c_dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("k", [2176, 2177, 2304, 2500, 2944])
@pytest.mark.parametrize("r,n", [(130, 256), (333, 1500), (1100, 1001)])  # four CTAs to a tile, four, two
def test_gemm(r, n, k, c_dtype):
    a, sa = moe.moe_fp8_quantize_rows(rand((r, k), r + k))
    w, sw = moe.moe_fp8_quantize_blocks(rand((n, k), r + k + 1, 0.05))
    got = moe.moe_fp8_gemm(a, sa, w, sw, c_dtype=c_dtype)
    ref, mags = product64(dequant_rows64(a, sa), dequant_blocks64(w, sw))
    assert_product(got, ref, mags, k)
    assert torch.equal(moe.moe_fp8_gemm(a, sa, w, sw, c_dtype=c_dtype), got)


@pytest.mark.parametrize("gather", [False, True], ids=["sorted", "gathered"])
@pytest.mark.parametrize("k", [2176, 2300])
def test_grouped(k, gather):
    c = grouped_case([150, 0, 131, 1], 270, k, gather, k)
    got = moe.moe_fp8_grouped_gemm(c["a"], c["sa"], c["w"], c["sw"], c["offsets"], c["slots"], gather_ids=c["ids"],
                                   c_dtype=torch.float32)
    ref, mags = grouped64(c)
    assert_product(got, ref, mags, k)
