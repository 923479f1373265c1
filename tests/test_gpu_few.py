"""GPU tests of the whole layers for a few tokens against FP64 (bounds: few_helpers)."""

import pytest
import torch

pytestmark = pytest.mark.gpu

import moe_prefill_nvfp4_gb300 as moe  # noqa: E402

from few_helpers import Fp8Layer, W4Layer, assert_near, logits_of, rand  # noqa: E402


@pytest.fixture(autouse=True)
def _no_device_error():
    moe.moe_get_device_error()
    yield
    assert moe.moe_get_device_error() == 0


# tokens, experts, top_k, hidden, inter, shared
FP8 = [(1, 1, 1, 128, 128, 0), (1, 8, 2, 256, 128, 0), (2, 16, 4, 1024, 256, 0), (3, 33, 5, 1152, 640, 384),
       (5, 3, 3, 2176, 1152, 128), (8, 64, 8, 2048, 768, 0), (9, 4, 2, 640, 384, 256), (16, 6, 3, 512, 128, 1280),
       (16, 160, 8, 1280, 256, 0), (13, 300, 8, 384, 128, 0), (7, 512, 32, 256, 128, 0), (16, 32, 32, 256, 256, 128)]


@pytest.mark.parametrize("tokens,experts,top_k,hidden,inter,shared", FP8)
def test_fp8(tokens, experts, top_k, hidden, inter, shared):
    layer = Fp8Layer(experts, hidden, inter, tokens, shared)
    x, logits = rand((tokens, hidden), 1), logits_of(tokens, experts, 2)
    ref, tol = layer.ref(x, logits, top_k)
    out = layer.run(x, top_k, logits=logits)
    assert out.shape == (tokens, hidden) and out.dtype == torch.bfloat16
    assert_near(out, ref, tol)
    assert torch.equal(layer.run(x, top_k, logits=logits), out)


W4 = [(1, 1, 1, 256, 256), (1, 8, 2, 256, 256), (2, 16, 4, 1024, 512), (3, 33, 5, 1280, 768), (5, 3, 3, 2304, 1280),
      (8, 64, 8, 2048, 768), (9, 4, 2, 768, 256), (16, 6, 3, 512, 256), (16, 160, 8, 1280, 256), (13, 300, 8, 512, 256),
      (7, 512, 32, 256, 256), (16, 32, 32, 256, 256)]


@pytest.mark.parametrize("tokens,experts,top_k,hidden,inter", W4)
def test_w4(tokens, experts, top_k, hidden, inter):
    layer = W4Layer(experts, hidden, inter, top_k, tokens)
    x, logits = rand((tokens, hidden), 1), logits_of(tokens, experts, 2)
    ref, tol = layer.ref(x, logits)
    out = layer.run(x, logits=logits)
    assert out.shape == (tokens, hidden) and out.dtype == torch.bfloat16
    assert_near(out, ref, tol)
    assert torch.equal(layer.run(x, logits=logits), out)
