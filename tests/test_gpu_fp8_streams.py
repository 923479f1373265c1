"""The FP8 chunk path on a stream that is not torch's current one: same bits as on the current stream, whatever
the current stream does meanwhile."""

import pytest
import torch

pytestmark = pytest.mark.gpu

import moe_prefill_nvfp4_gb300 as moe  # noqa: E402
from moe_prefill_nvfp4_gb300 import fp8  # noqa: E402

from test_gpu_fp8 import rand  # noqa: E402
from test_gpu_fp8_path import make  # noqa: E402


@pytest.fixture(autouse=True)
def _no_device_error():
    moe.moe_get_device_error()
    yield
    assert moe.moe_get_device_error() == 0


def occupy(copies=24):
    """Queues some 10 ms of copies on the current stream."""
    a = torch.empty(1 << 30, dtype=torch.uint8, device="cuda")
    b = torch.empty_like(a)
    for _ in range(copies):
        b.copy_(a)
    return a, b


def overwrite():
    """Takes what the current stream's pool has free, in the sizes that a small chunk allocates, and fills it."""
    return [torch.full((1 << p,), 0x7F, dtype=torch.uint8, device="cuda") for p in range(9, 21) for _ in range(6)]


@pytest.mark.parametrize("busy", ["current", "side"])
@pytest.mark.parametrize("tokens", [3, 130])
def test_forward_on_a_stream_that_is_not_current(tokens, busy):
    """Current stream busy: what the forward queued there would come too late.  Side busy: what the forward
    dropped to the current stream's pool would be overwritten before its use."""
    experts, top_k, hidden, inter = 8, 2, 640, 256
    gu, dn = make(experts, hidden, inter, 9)
    sg, sd = make(1, hidden, 384, 20)
    shared = fp8.Fp8SharedExpert(fp8.Fp8Weight.quantise(sg[0]), fp8.Fp8Weight.quantise(sd[0]))
    layer = fp8.Fp8Experts(fp8.Fp8Weight.quantise(gu), fp8.Fp8Weight.quantise(dn), top_k, shared=shared)
    x, w_router = rand((tokens, hidden), 3), rand((experts, hidden), 4, 0.05)
    want = layer.forward(x, w_router=w_router)  # (and blocks of every size for the current stream's pool)
    alone = shared.forward(*moe.moe_fp8_quantize_rows(x))
    codes = moe.moe_fp8_quantize_rows(x)
    side = torch.cuda.Stream()
    held = [occupy(1)]  # (memory for the copies, before anything is timed against them)
    torch.cuda.synchronize()
    if busy == "current":
        held.append(occupy())
    else:
        with torch.cuda.stream(side):
            held.append(occupy())
    assert not side.query() or busy == "current"
    got = layer.forward(x, w_router=w_router, stream=side)
    part = shared.forward(*codes, stream=side)
    held.append(overwrite())
    torch.cuda.synchronize()
    assert torch.equal(got, want) and torch.equal(part, alone)


def test_result_dropped_by_the_current_stream():
    """A result of a side stream that the current stream still reads when it is dropped keeps its memory."""
    gu, dn = make(4, 512, 128, 11)
    layer = fp8.Fp8Experts(fp8.Fp8Weight.quantise(gu), fp8.Fp8Weight.quantise(dn), 2)
    x, logits = rand((64, 512), 5), rand((64, 4), 6, 1.0, torch.float32)
    want = layer.forward(x, logits=logits)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    y = layer.forward(x, logits=logits, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    held = occupy()
    kept = y.clone()  # behind the copies
    del y
    with torch.cuda.stream(side):
        fill = overwrite()
    torch.cuda.synchronize()
    assert torch.equal(kept, want)
    del held, fill


def test_out_on_a_stream_that_is_not_current():
    gu, dn = make(4, 512, 128, 12)
    layer = fp8.Fp8Experts(fp8.Fp8Weight.quantise(gu), fp8.Fp8Weight.quantise(dn), 2)
    x, logits = rand((40, 512), 7), rand((40, 4), 8, 1.0, torch.float32)
    want = layer.forward(x, logits=logits)
    out = torch.zeros_like(want)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    assert layer.forward(x, logits=logits, out=out, stream=side) is out
    side.synchronize()
    assert torch.equal(out, want)


@pytest.mark.parametrize("given", [False, True], ids=["current", "given"])
def test_captured_on_a_stream(given):
    """A forward with a shared expert captured into a graph, the stream current or given as well."""
    gu, dn = make(4, 512, 128, 13)
    sg, sd = make(1, 512, 128, 21)
    shared = fp8.Fp8SharedExpert(fp8.Fp8Weight.quantise(sg[0]), fp8.Fp8Weight.quantise(sd[0]))
    layer = fp8.Fp8Experts(fp8.Fp8Weight.quantise(gu), fp8.Fp8Weight.quantise(dn), 2, shared=shared)
    x, logits = rand((40, 512), 9), rand((40, 4), 10, 1.0, torch.float32)
    want = layer.forward(x, logits=logits)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        got = layer.forward(x, logits=logits, stream=side if given else None)
    for _ in range(2):
        got.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(got, want)
