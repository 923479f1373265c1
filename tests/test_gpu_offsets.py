"""Offsets whose 32-bit differences wrap: recorded, nothing read or written (NVFP4 products)."""

import pytest
import torch

pytestmark = pytest.mark.gpu

import moe_prefill_nvfp4_gb300 as moe  # noqa: E402
from synth import inputs as S  # noqa: E402

from gpu_helpers import bf16_dev, upload  # noqa: E402

TOP, LOW = 2 ** 31 - 1, -(2 ** 31)


@pytest.fixture(autouse=True)
def _no_device_error():
    moe.moe_get_device_error()
    yield
    moe.moe_debug_set_gemm_kernel(moe.MOE_GEMM_KERNEL_AUTO)
    assert moe.moe_get_device_error() == 0


@pytest.mark.parametrize("call", ["single", "pair", "swiglu-single", "swiglu-pair", "gemv", "gemv-swiglu"])
@pytest.mark.parametrize("steps", [[0, 2 ** 30, LOW + 5, -1000, 4], [0, TOP, LOW, -1, 4], [0, 2 ** 30, LOW, LOW + 2 ** 30, 0],
                                   [0, TOP, TOP, LOW, LOW + 1]])
def test_wrapping_offsets_write_nothing(call, steps):
    c = S.make_gemm_case(T=40, E=4, k=2, N=512, K=512, seed=5)
    proj = upload(c.w)
    R = c.T * c.k
    a = torch.cat([bf16_dev(c.x)] * 2)  # rows in expert order, no gather
    off = torch.tensor(steps, dtype=torch.int32, device="cuda")
    half = call.startswith("swiglu") or call.endswith("swiglu")
    out = torch.full((R, 256 if half else 512), 7.0, dtype=torch.bfloat16, device="cuda")
    if call.startswith("gemv"):
        f = moe.moe_w4a16_grouped_gemv_swiglu if half else moe.moe_w4a16_grouped_gemv
        f(a, proj.table, off, R, out=out)
    else:
        f = moe.moe_w4a16_grouped_gemm_swiglu if half else moe.moe_w4a16_grouped_gemm
        with moe.gemm_kernel(moe.MOE_GEMM_KERNEL_PAIR if call.endswith("pair") else moe.MOE_GEMM_KERNEL_SINGLE):
            f(a, proj.table, off, R, out=out)
    assert moe.moe_get_device_error() == 2
    assert (out == 7).all()
    proj.close()
