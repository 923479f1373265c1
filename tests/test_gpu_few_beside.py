"""GPU tests of the few-token layers beside other kernels that take tensor memory on the same SMs (library products, the
chunk path's): every call finishes, with the bits that it has alone."""

import pytest
import torch

pytestmark = pytest.mark.gpu

import moe_prefill_nvfp4_gb300 as moe  # noqa: E402

from few_helpers import Fp8Layer, W4Layer, logits_of, rand  # noqa: E402


@pytest.fixture(autouse=True)
def _no_device_error():
    moe.moe_get_device_error()
    yield
    assert moe.moe_get_device_error() == 0


def library_products():
    pairs = [(rand((m, k), 1), rand((k, n), 2)) for m, n, k in ((4096, 4096, 4096), (2048, 2048, 256), (128, 8192, 1024), (8192, 128, 64))]

    def run():
        for a, b in pairs:
            a @ b

    return run


def fp8_products():
    a, sa = moe.moe_fp8_quantize_rows(rand((40, 2048), 3))
    w, sw = (t[0] for t in Fp8Layer(1, 2048, 1024, 4).gu)
    out = moe.moe_fp8_gemm(a, sa, w, sw)
    return lambda: moe.moe_fp8_gemm(a, sa, w, sw, out=out)


@pytest.mark.parametrize("kind", ["fp8", "w4"])
@pytest.mark.parametrize("other", [library_products, fp8_products])
def test_beside_other_products(kind, other):
    layer = Fp8Layer(48, 2048, 768) if kind == "fp8" else W4Layer(48, 2048, 768, 8)
    run = (lambda x, **kw: layer.run(x, 8, **kw)) if kind == "fp8" else layer.run
    xs = [(rand((t, 2048), t), logits_of(t, 48, t + 50)) for t in (1, 4, 16)]
    want = [run(x, logits=lg) for x, lg in xs]
    beside = other()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    outs = []
    for _ in range(60):
        with torch.cuda.stream(streams[0]):
            outs.append([run(x, logits=lg) for x, lg in xs])
        with torch.cuda.stream(streams[1]):
            for _ in range(3):
                beside()
    torch.cuda.synchronize()
    for got in outs:
        assert all(torch.equal(g, w) for g, w in zip(got, want))
