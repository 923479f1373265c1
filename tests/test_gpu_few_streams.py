"""Direct calls of the norm and the few-token layers on a stream that is not torch's current one, whose own work is
still queued: neither its temporaries, just dropped, nor the call's results may get the other's values."""

import pytest
import torch

pytestmark = pytest.mark.gpu

import moe_prefill_nvfp4_gb300 as moe  # noqa: E402

from few_helpers import Fp8Layer, W4Layer, logits_of, rand  # noqa: E402
from test_gpu_fp8_streams import occupy  # noqa: E402


@pytest.fixture(autouse=True)
def _no_device_error():
    moe.moe_get_device_error()
    yield
    assert moe.moe_get_device_error() == 0


def fp8_call():
    layer, x, logits = Fp8Layer(16, 1024, 512), rand((5, 1024), 3), logits_of(5, 16, 4)
    ws = moe.moe_few_workspace_bytes(moe.MoePrefillConfig(hidden=1024, moe_intermediate=512, num_experts=16, top_k=4), 5, True)
    return (lambda **kw: (layer.run(x, 4, logits=logits, **kw),)), [ws, 5 * 1024 * 2]


def w4_call():
    layer, x, logits = W4Layer(16, 1024, 512, 4), rand((5, 1024), 3), logits_of(5, 16, 4)
    return (lambda **kw: (layer.run(x, logits=logits, **kw),)), [moe.moe_few_workspace_bytes(layer.cfg, 5, False), 5 * 1024 * 2]


def norm_call():
    x, r, w = rand((300, 2048), 1), rand((300, 2048), 2), rand((2048,), 3)
    return (lambda **kw: moe.moe_fp8_add_rms_norm(x, w, r, normed=True, **kw)), [300 * 2048, 300 * 16 * 4, 300 * 2048 * 2]


def quantiser_call():
    x = rand((300, 2048), 1)
    return (lambda **kw: moe.moe_fp8_quantize_rows(x, **kw)), [300 * 2048, 300 * 16 * 4]


def same(a, b):
    return torch.equal(a.contiguous().view(torch.uint8), b.contiguous().view(torch.uint8))


@pytest.mark.parametrize("make", [fp8_call, w4_call, norm_call, quantiser_call])
def test_direct_call_while_the_current_stream_is_busy(make):
    run, sizes = make()
    want = run()
    side = torch.cuda.Stream()
    bytes_of = lambda n, v: torch.full((n,), v, dtype=torch.uint8, device="cuda")  # noqa: E731
    read = [bytes_of(n, 5) for n in sizes for _ in range(4)]
    written = [bytes_of(n, 6) for n in sizes for _ in range(4)]
    copies = [torch.empty_like(t) for t in read]
    held = [occupy(1)]
    torch.cuda.synchronize()
    held.append(occupy())
    for c, t in zip(copies, read):
        c.copy_(t)  # reads a temporary, behind the copies
    for t in written:
        t.fill_(9)  # writes one
    del read, written, t
    got = [run(stream=side) for _ in range(3)]
    torch.cuda.synchronize()
    assert all((c == 5).all() for c in copies)
    for g in got:
        assert all(same(a, b) for a, b in zip(g, want))
    del held


@pytest.mark.parametrize("make", [fp8_call, w4_call, norm_call])
def test_dropped_while_the_current_stream_reads(make):
    """A result that the current stream still reads when it is dropped keeps its memory from the side stream's next calls."""
    run, _ = make()
    want = run()
    side = torch.cuda.Stream()
    held = [occupy(1)]
    torch.cuda.synchronize()
    got = run(stream=side)
    torch.cuda.current_stream().wait_stream(side)
    held.append(occupy())
    kept = [g.clone() for g in got]
    del got
    with torch.cuda.stream(side):
        held.append([torch.full((1 << p,), 0x7F, dtype=torch.uint8, device="cuda") for p in range(9, 22) for _ in range(6)])
    torch.cuda.synchronize()
    assert all(same(a, b) for a, b in zip(kept, want))
    del held


@pytest.mark.parametrize("make", [fp8_call, w4_call, norm_call])
def test_captured_with_a_given_stream(make):
    run, _ = make()
    want = run()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        got = run(stream=side)
    for _ in range(2):
        for g in got:
            (g.view(torch.uint8) if g.dtype == torch.float8_e4m3fn else g).zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(same(a, b) for a, b in zip(got, want))
