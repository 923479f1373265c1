"""Expert-parallel parts of an FP8 layer that has a shared expert: their results add up to the whole layer's."""

import pytest
import torch

pytestmark = pytest.mark.gpu

import moe_prefill_nvfp4_gb300 as moe  # noqa: E402
from moe_prefill_nvfp4_gb300 import fp8  # noqa: E402

from test_gpu_fp8 import rand  # noqa: E402
from test_gpu_fp8_path import make  # noqa: E402


def test_parts_with_a_shared_expert_add_up():
    tokens, experts, top_k, hidden, inter = 64, 8, 3, 512, 128
    gu, dn = make(experts, hidden, inter, 30)
    sg, sd = make(1, hidden, 256, 60)
    shared = fp8.Fp8SharedExpert(fp8.Fp8Weight.quantise(sg[0]), fp8.Fp8Weight.quantise(sd[0]))
    x, logits = rand((tokens, hidden), 5), rand((tokens, experts), 6, 1.0, torch.float32)
    g, d = fp8.Fp8Weight.quantise(gu), fp8.Fp8Weight.quantise(dn)
    whole = fp8.Fp8Experts(g, d, top_k, shared=shared).forward(x, logits=logits).double()
    routed = fp8.Fp8Experts(g, d, top_k).forward(x, logits=logits).double()
    total, mags = torch.zeros_like(whole), torch.zeros_like(whole)
    for first, count in ((0, 5), (5, 3)):
        sub = slice(first, first + count)
        part = fp8.Fp8Experts(fp8.Fp8Weight(g.q[sub], g.s[sub]), fp8.Fp8Weight(d.q[sub], d.s[sub]), top_k,
                              num_experts=experts, first=first, shared=shared if first == 0 else None)
        y = part.forward(x, logits=logits).double()
        total += y
        mags += y.abs()
    # the parts' and the whole's rounding to BF16: half a unit each, 2^-9 of the magnitude
    assert ((total - whole).abs() <= 2.0 ** -8 * (mags + whole.abs())).all()
    assert float((whole - routed).norm() / whole.norm()) > 0.3  # the shared expert is a good part of it
    assert moe.moe_get_device_error() == 0


def test_shared_expert_without_tokens():
    sg, sd = make(1, 256, 128, 70)
    shared = fp8.Fp8SharedExpert(fp8.Fp8Weight.quantise(sg[0]), fp8.Fp8Weight.quantise(sd[0]))
    y = shared.forward(*moe.moe_fp8_quantize_rows(rand((0, 256), 1)))
    assert y.shape == (0, 256) and y.dtype == torch.bfloat16
    assert moe.moe_get_device_error() == 0
