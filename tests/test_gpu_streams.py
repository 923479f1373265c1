"""Workspaces that a call allocates itself, on a stream that is not torch's current one."""

import pytest
import torch

pytestmark = pytest.mark.gpu

import moe_prefill_nvfp4_gb300 as moe  # noqa: E402

from test_gpu_fp8 import rand  # noqa: E402
from test_gpu_fp8_streams import occupy, overwrite  # noqa: E402


@pytest.fixture(autouse=True)
def _no_device_error():
    moe.moe_get_device_error()
    yield
    assert moe.moe_get_device_error() == 0


def busy_stream():
    """A stream with some 10 ms of copies, its memory allocated before."""
    side = torch.cuda.Stream()
    held = [occupy(1)]
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        held.append(occupy())
    return side, held


@pytest.mark.parametrize("tokens", [7, 900])
def test_sort_on_a_busy_stream(tokens):
    ids = rand((tokens, 24), tokens, 1.0, torch.float32).topk(4, 1).indices.int()
    want = moe.moe_sort_by_expert(ids, 24)
    side, held = busy_stream()
    got = moe.moe_sort_by_expert(ids, 24, stream=side)
    fill = overwrite()  # of what the current stream's pool has free
    torch.cuda.synchronize()
    for key, t in want.items():
        assert torch.equal(got[key], t), key
    del held, fill


def test_shared_expert_on_a_busy_stream():
    x = rand((130, 256), 1)
    w = [rand((384, 256), 2, 0.06), rand((384, 256), 3, 0.06), rand((256, 384), 4, 0.05)]
    want = moe.moe_shared_expert_forward(x, *w)
    side, held = busy_stream()
    got = moe.moe_shared_expert_forward(x, *w, stream=side)
    fill = overwrite()
    torch.cuda.synchronize()
    assert torch.equal(got, want)
    del held, fill
