"""Offsets whose 32-bit differences wrap: recorded, nothing read or written (FP8 products)."""

import pytest
import torch

pytestmark = pytest.mark.gpu

import moe_prefill_nvfp4_gb300 as moe  # noqa: E402

from test_gpu_fp8 import grouped_case  # noqa: E402

TOP, LOW = 2 ** 31 - 1, -(2 ** 31)


@pytest.mark.parametrize("counts", [[1, 2, 1, 0], [200, 100, 90, 0]], ids=["few-rows", "wide"])
@pytest.mark.parametrize("gather", [False, True], ids=["sorted", "gathered"])
@pytest.mark.parametrize("steps", [[0, 2 ** 30, LOW + 5, -1000, 4], [0, TOP, LOW, -1, 4], [0, 2 ** 30, LOW, LOW + 2 ** 30, 0],
                                   [0, 1, TOP, TOP, 4], [0, -1, 0, 1, 4], [0, 0, 0, 0, TOP]])
def test_wrapping_offsets_write_nothing(counts, gather, steps):
    c = grouped_case(counts, 256, 256, gather, 6)
    off = torch.tensor(steps, dtype=torch.int32, device="cuda")
    out = torch.full((c["slots"], 256), 2.0, dtype=torch.bfloat16, device="cuda")
    moe.moe_fp8_grouped_gemm(c["a"], c["sa"], c["w"], c["sw"], off, c["slots"], gather_ids=c["ids"], out=out)
    assert moe.moe_get_device_error() == 2
    codes = torch.full((c["slots"], 128), 0x55, dtype=torch.uint8, device="cuda")
    scales = torch.full((c["slots"], 1), -1.0, device="cuda")
    moe.moe_fp8_grouped_gemm_swiglu(c["a"], c["sa"], c["w"], c["sw"], off, c["slots"], gather_ids=c["ids"],
                                    out=codes.view(torch.float8_e4m3fn), scales=scales)
    assert moe.moe_get_device_error() == 2
    assert (out == 2).all() and (codes == 0x55).all() and (scales == -1).all()
