"""The FP8 experts' chunk path (fp8.py): its stages joined as they are used, against FP64 and against the
unquantised experts.

Against FP64 with the path's own codes: the routed sum of the down products, which the path rounds to
BF16 before and after the combine -- half a unit of each term and of the sum, 2^-8 of the magnitudes
covers both with the FP32 sums' own error.

Against the unquantised experts: x, gate/up weight, activation and down weight are each off by at most
2^-4 relative, uniformly spread at worst (RMS 2^-4 / sqrt 3 = 0.036); four independent such errors make
0.072 of the norm.
"""

import pytest
import torch

pytestmark = pytest.mark.gpu

import moe_prefill_nvfp4_gb300 as moe  # noqa: E402
from moe_prefill_nvfp4_gb300 import fp8  # noqa: E402

from test_gpu_fp8 import dequant_blocks64, dequant_rows64, rand  # noqa: E402


@pytest.fixture(autouse=True)
def _no_device_error():
    moe.moe_get_device_error()
    yield
    assert moe.moe_get_device_error() == 0


def make(experts, hidden, inter, seed):
    gu = torch.stack([rand((2 * inter, hidden), seed + e, hidden ** -0.5) for e in range(experts)])
    dn = torch.stack([rand((hidden, inter), seed + 500 + e, inter ** -0.5) for e in range(experts)])
    return gu, dn


@pytest.mark.parametrize("tokens,experts,top_k,hidden,inter", [(1, 16, 4, 512, 256), (37, 6, 2, 520, 128),
                                                             (300, 12, 3, 1000, 384)])
def test_routed_experts(tokens, experts, top_k, hidden, inter):
    gu, dn = make(experts, hidden, inter, tokens)
    x, logits = rand((tokens, hidden), 1), rand((tokens, experts), 2, 1.0, torch.float32)
    layer = fp8.Fp8Experts(fp8.Fp8Weight.quantise(gu), fp8.Fp8Weight.quantise(dn), top_k)
    out = layer.forward(x, logits=logits)
    # FP64 down products and combine of the path's own activation codes
    ids, wts = moe.moe_route_topk(logits, top_k)
    order = moe.moe_sort_by_expert(ids, experts)
    q, s = moe.moe_fp8_quantize_rows(x)
    aq, a_s = moe.moe_fp8_grouped_gemm_swiglu(q, s, layer.gate_up.q, layer.gate_up.s, order["expert_offsets"], tokens * top_k,
                                              gather_ids=order["sorted_token_ids"])
    act, w = dequant_rows64(aq, a_s), dequant_blocks64(layer.down.q, layer.down.s)
    e = order["sorted_expert_ids"].long().cpu()
    y = torch.stack([w[e[p]] @ act[p] for p in range(tokens * top_k)])
    mag = torch.stack([w[e[p]].abs() @ act[p].abs() for p in range(tokens * top_k)])
    at, wt = order["token_to_perm"].long().cpu(), wts.double().cpu()
    ref = (y[at] * wt[..., None]).sum(1)
    tol = 2.0 ** -8 * (y[at].abs() * wt[..., None]).sum(1) + 2.0 ** -8 * ref.abs() + 2.0 ** -15 * (mag[at] * wt[..., None]).sum(1)
    assert ((out.double().cpu() - ref).abs() <= tol).all()
    plain = fp8._reference(x, logits, gu, dn, top_k, 7.0)
    assert float((out.float() - plain).norm() / plain.norm()) < 0.072


def test_router_shared_and_stream():
    tokens, experts, top_k, hidden, inter = 130, 8, 2, 640, 256
    gu, dn = make(experts, hidden, inter, 9)
    sg, sd = make(1, hidden, 384, 20)
    shared = fp8.Fp8SharedExpert(fp8.Fp8Weight.quantise(sg[0]), fp8.Fp8Weight.quantise(sd[0]))
    x, w_router = rand((tokens, hidden), 3), rand((experts, hidden), 4, 0.05)
    layer = fp8.Fp8Experts(fp8.Fp8Weight.quantise(gu), fp8.Fp8Weight.quantise(dn), top_k, shared=shared)
    out = layer.forward(x, w_router=w_router)
    alone = fp8.Fp8Experts(layer.gate_up, layer.down, top_k).forward(x, w_router=w_router)
    add = shared.forward(*moe.moe_fp8_quantize_rows(x))
    both = alone.double() + add.double()
    assert ((out.double() - both).abs() <= 2.0 ** -7 * (alone.double().abs() + add.double().abs())).all()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        again = layer.forward(x, w_router=w_router, stream=side)
    side.synchronize()
    assert torch.equal(again, out)


def test_expert_parallel_parts_add_up():
    """Two ranks' parts (experts 0-4 and 5-7) sum to the whole: each slot's product is made by one of them."""
    tokens, experts, top_k, hidden, inter = 64, 8, 3, 512, 128
    gu, dn = make(experts, hidden, inter, 30)
    x, logits = rand((tokens, hidden), 5), rand((tokens, experts), 6, 1.0, torch.float32)
    g, d = fp8.Fp8Weight.quantise(gu), fp8.Fp8Weight.quantise(dn)
    whole = fp8.Fp8Experts(g, d, top_k).forward(x, logits=logits).double()
    total = torch.zeros_like(whole)
    mags = torch.zeros_like(whole)
    for first, count in ((0, 5), (5, 3)):
        sub = slice(first, first + count)
        part = fp8.Fp8Experts(fp8.Fp8Weight(g.q[sub], g.s[sub]), fp8.Fp8Weight(d.q[sub], d.s[sub]), top_k,
                              num_experts=experts, first=first).forward(x, logits=logits).double()
        total += part
        mags += part.abs()
    assert ((total - whole).abs() <= 2.0 ** -8 * (mags + whole.abs())).all()  # the parts' and the whole's rounding
    assert float(mags.abs().max()) > 0


def test_refuses_both_or_no_routing():
    g = fp8.Fp8Weight.quantise(rand((2, 256, 256), 1))
    layer = fp8.Fp8Experts(g, fp8.Fp8Weight.quantise(rand((2, 256, 128), 2)), 1)
    x = rand((4, 256), 3)
    with pytest.raises(ValueError):
        layer.forward(x)
    with pytest.raises(ValueError):
        layer.forward(x, logits=torch.zeros(4, 3, device="cuda"))
