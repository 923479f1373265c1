"""GPU tests of calls at the edges of what the decode-step operators allow: ties and masked experts, results in the place of
their inputs, rows past 32-bit offsets (bounds: few_helpers, test_gpu_rms_norm)."""

import pytest
import torch

pytestmark = pytest.mark.gpu

import moe_prefill_nvfp4_gb300 as moe  # noqa: E402

from few_helpers import assert_near, logits_of, rand  # noqa: E402
from test_gpu_few_calls import Any, KINDS  # noqa: E402
from test_gpu_rms_norm import check  # noqa: E402

BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(autouse=True)
def _no_device_error():
    moe.moe_get_device_error()
    yield
    assert moe.moe_get_device_error() == 0


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("experts", [16, 100, 200, 300])
def test_ties_go_to_the_lower_expert(kind, experts):
    """Equal logits, of a router and given: the experts picked are the first ones, or the first of those on top."""
    layer = Any(kind, experts, 512, 256, 4)
    x, w = rand((5, 512), 3), rand((1, 512), 5, 0.05).expand(experts, -1).contiguous()
    first = torch.zeros(5, experts, device="cuda")
    first[:, :4] = 1.0
    want = layer.run(x, logits=first)
    assert torch.equal(layer.run(x, logits=torch.zeros_like(first)), want)
    assert torch.equal(layer.run(x, w_router=w), want)
    bias = torch.zeros(experts, device="cuda")
    bias[7::3] = 1.0  # (selection only: the weights stay those of equal logits)
    some = torch.zeros_like(first)
    some[:, [7, 10, 13, 16] if experts > 16 else [7, 10, 13, 0]] = 1.0
    assert torch.equal(layer.run(x, logits=torch.zeros_like(first), router_bias=bias), layer.run(x, logits=some))


@pytest.mark.parametrize("kind", KINDS)
def test_masked_experts(kind):
    """Logits of -inf: fewer experts left than there are picks (the others have no weight), one, and none (NaN, in that row)."""
    layer = Any(kind, 100, 512, 256, 4)
    x, logits = rand((6, 512), 3), logits_of(6, 100, 4)
    for t, left in enumerate(([5, 70, 71, 99, 3], [2, 98], [64], [0, 1, 2], [90])):
        keep = logits[t, left].clone()
        logits[t] = -float("inf")
        logits[t, left] = keep
    out = layer.run(x, logits=logits)
    assert_near(out, *layer.ref(x, logits))
    logits[2] = -float("inf")
    again = layer.run(x, logits=logits)
    assert again[2].isnan().all()
    for t in (0, 1, 3, 4, 5):
        assert torch.equal(again[t], out[t])


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("routed_by", ["w_router", "logits"])
@pytest.mark.parametrize("tokens", [1, 16])
def test_result_in_the_place_of_x(kind, routed_by, tokens):
    layer = Any(kind, 40, 1024, 512, 4)
    x = rand((tokens, 1024), 3)
    how = dict(w_router=rand((40, 1024), 5, 0.05)) if routed_by == "w_router" else dict(logits=logits_of(tokens, 40, 4))
    want = layer.run(x, **how)
    for _ in range(20):
        y = x.clone()
        assert layer.run(y, out=y, **how) is y
        assert torch.equal(y, want)


@pytest.mark.parametrize("k", [256, 250])
def test_norm_past_32_bit_offsets(k):
    """Rows whose last elements lie past 2^32 bytes and 2^31 elements, of every operand and output."""
    rows, ld = 450_000, 5120
    wide = lambda dtype: torch.zeros(rows * ld, dtype=dtype, device="cuda").view(rows, ld)  # noqa: E731
    x, r, y = wide(BF16)[:, ld - 256:][:, :k], wide(BF16)[:, 512:512 + k], wide(BF16)[:, :k]
    q = wide(torch.uint8).view(torch.float8_e4m3fn)[:, 1024:1024 + k]
    s = torch.zeros(rows, 5000, device="cuda")[:, 3000:3002]
    some = torch.cat([torch.arange(0, 40), torch.arange(rows - 2000, rows), torch.tensor([209_715, 209_716, 419_430, 419_431])]).cuda()
    x[some], r[some] = rand((len(some), k), 1, 0.5), rand((len(some), k), 2, 2.0)
    x0, r0, w = x[some], r[some], 1 + rand((k,), 3, 0.3)
    moe.moe_fp8_add_rms_norm(x, w, r, eps=1e-5, normed=y, residual_out=r, out=q, scales=s)
    codes = q.view(torch.uint8)[some].contiguous().view(torch.float8_e4m3fn)
    check(x0, w, r0, 1e-5, codes, s[some].contiguous(), r[some], y[some])
