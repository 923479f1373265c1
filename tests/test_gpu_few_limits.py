"""Waits of the few-token layers that run out, by a limit shorter than what they wait for: the kernel records
MOE_DEVERR_TIMEOUT, waits for its copies and MMAs, gives its tensor memory back and returns, and the next call is right.
Nothing is withheld from any wait: with the usual limit the same calls end by themselves."""

import time

import pytest
import torch

pytestmark = pytest.mark.gpu

import moe_prefill_nvfp4_gb300 as moe  # noqa: E402

from few_helpers import Fp8Layer, W4Layer, logits_of, rand  # noqa: E402

TIMEOUT = 3


@pytest.fixture(autouse=True)
def _restore():
    moe.moe_get_device_error()
    yield
    moe.moe_debug_set_wait_limit_ns(0)
    assert moe.moe_get_device_error() == 0


def layer_of(kind):
    if kind == "fp8":
        layer = Fp8Layer(48, 2048, 768, shared=256)
        return lambda x, **kw: layer.run(x, 8, **kw)
    return W4Layer(48, 2048, 768, 8).run


@pytest.mark.parametrize("kind", ["fp8", "w4"])
@pytest.mark.parametrize("tokens", [1, 16])
def test_waits_run_out_and_the_kernel_returns(kind, tokens):
    run = layer_of(kind)
    x, logits = rand((tokens, 2048), 3), logits_of(tokens, 48, 4)
    want = run(x, logits=logits)
    for limit in (1, 1, 2_000, 5_000, 10_000, 20_000, 40_000):
        moe.moe_debug_set_wait_limit_ns(limit)
        t0 = time.perf_counter()
        out = run(x, logits=logits)
        code = moe.moe_get_device_error()
        assert time.perf_counter() - t0 < 5.0
        # (the first activations need some 10 us of weights: a limit of 1 ns is always too short for them)
        assert code == TIMEOUT if limit == 1 else code in (0, TIMEOUT)
        assert code == TIMEOUT or torch.equal(out, want)
        moe.moe_debug_set_wait_limit_ns(0)
        for _ in range(3):
            assert torch.equal(run(x, logits=logits), want)
        assert moe.moe_get_device_error() == 0


@pytest.mark.parametrize("kind", ["fp8", "w4"])
def test_other_kernels_after_waits_that_ran_out(kind):
    """Shared memory and tensor memory of the CTAs that gave up go to others: many calls in a row, then both formats."""
    runs = [layer_of(kind), layer_of("w4" if kind == "fp8" else "fp8")]
    x, logits = rand((16, 2048), 3), logits_of(16, 48, 4)
    want = [run(x, logits=logits) for run in runs]
    moe.moe_debug_set_wait_limit_ns(1)
    for _ in range(30):
        runs[0](x, logits=logits)
    moe.moe_debug_set_wait_limit_ns(0)
    got = [run(x, logits=logits) for _ in range(5) for run in runs]
    assert moe.moe_get_device_error() == TIMEOUT
    for i, g in enumerate(got):
        assert torch.equal(g, want[i % 2])


def test_norm_under_a_limit_of_its_own():
    x, r, w = rand((4000, 5120), 1), rand((4000, 5120), 2), rand((5120,), 3)
    want = moe.moe_fp8_add_rms_norm(x, w, r, normed=True)
    moe.moe_debug_set_wait_limit_ns(50_000_000)
    got = moe.moe_fp8_add_rms_norm(x, w, r, normed=True)
    assert moe.moe_get_device_error() == 0
    for a, b in zip(got, want):
        assert torch.equal(a.contiguous().view(torch.uint8), b.contiguous().view(torch.uint8))
