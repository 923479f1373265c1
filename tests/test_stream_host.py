"""A call that is given a stream makes its outputs and workspaces on it (no GPU: torch's stream context and the
library are stand-ins).  From the current stream's pool it could get memory that work queued there still uses."""

import contextlib
import ctypes

import pytest
import torch

from moe_prefill_nvfp4_gb300 import _lib

BF16, F32, I32, U8 = torch.bfloat16, torch.float32, torch.int32, torch.uint8


class Side:
    cuda_stream = 1234
    entered = False


class Library:
    """Every call succeeds; sizes are 256 bytes."""

    def __getattr__(self, name):
        return lambda *args: 256 if "bytes" in name else 0


class Handle:
    handle, N, K = ctypes.c_void_p(1), 256, 256


@pytest.fixture
def side(monkeypatch):
    """The stream; side.made: whether it was the current one, for each allocation and each result that was recorded."""
    s = Side()
    s.made, s.recorded = [], 0

    @contextlib.contextmanager
    def on(stream):
        stream.entered = True
        yield
        stream.entered = False

    empty = torch.empty

    def noted(*args, **kw):
        s.made.append(s.entered)
        return empty(*args, **kw)

    class Module:
        def __getattr__(self, name):
            return lambda *args: noted(1)

    def record(result, stream):
        assert stream is s and not s.entered  # for the caller's stream
        s.recorded += 1
        return result

    monkeypatch.setattr(torch.cuda, "Stream", Side)
    monkeypatch.setattr(torch.cuda, "stream", on)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda *device: Side)
    monkeypatch.setattr(torch, "empty", noted)
    monkeypatch.setattr(_lib, "_need", lambda *args: None)
    monkeypatch.setattr(_lib, "lib", Library)
    monkeypatch.setattr(_lib, "_FP8", Module())
    monkeypatch.setattr(_lib, "_result", record, raising=False)
    yield s


def z(dtype, *shape):
    return torch.zeros(*shape, dtype=dtype)


CFG = _lib.MoePrefillConfig(hidden=256, moe_intermediate=256, num_experts=4, top_k=2)
CALLS = {
    "moe_router_logits": lambda st: _lib.moe_router_logits(z(BF16, 3, 256), z(BF16, 4, 256), stream=st),
    "moe_route_topk": lambda st: _lib.moe_route_topk(z(F32, 3, 4), 2, None, True, 1.0, None, None, st),
    "moe_sort_by_expert": lambda st: _lib.moe_sort_by_expert(z(I32, 3, 2), 4, stream=st),
    "moe_sort_by_expert_noalloc": lambda st: _lib.moe_sort_by_expert_noalloc(z(I32, 3, 2), 4, stream=st),
    "moe_w4a16_grouped_gemm_swiglu": lambda st: _lib.moe_w4a16_grouped_gemm_swiglu(z(BF16, 6, 256), Handle, z(I32, 5), 6, stream=st),
    "moe_w4a16_grouped_gemv": lambda st: _lib.moe_w4a16_grouped_gemv(z(BF16, 6, 256), Handle, z(I32, 5), 6, stream=st),
    "moe_w4a16_grouped_gemv_swiglu": lambda st: _lib.moe_w4a16_grouped_gemv_swiglu(z(BF16, 6, 256), Handle, z(I32, 5), 6, stream=st),
    "moe_w4a16_grouped_gemm": lambda st: _lib.moe_w4a16_grouped_gemm(z(BF16, 6, 256), Handle, z(I32, 5), 6, stream=st),
    "moe_dequant_nvfp4": lambda st: _lib.moe_dequant_nvfp4(z(U8, 4, 8), z(U8, 4, 1), 1.0, stream=st),
    "moe_swiglu_clamp": lambda st: _lib.moe_swiglu_clamp(z(BF16, 3, 8), z(BF16, 3, 8), 7.0, stream=st),
    "moe_combine_indexed": lambda st: _lib.moe_combine_indexed(z(BF16, 6, 256), z(I32, 3, 2), z(F32, 3, 2), stream=st),
    "moe_shared_expert_forward": lambda st: _lib.moe_shared_expert_forward(z(BF16, 3, 256), *[z(BF16, 256, 256)] * 3, stream=st),
    "moe_fp8_quantize_rows": lambda st: _lib.moe_fp8_quantize_rows(z(BF16, 3, 256), stream=st),
    "moe_fp8_quantize_blocks": lambda st: _lib.moe_fp8_quantize_blocks(z(BF16, 3, 256), stream=st),
    "moe_fp8_gemm": lambda st: _lib.moe_fp8_gemm(*[z(F32, 3, 256)] * 4, stream=st),
    "moe_fp8_grouped_gemm": lambda st: _lib.moe_fp8_grouped_gemm(*[z(F32, 3, 256)] * 4, z(I32, 5), 6, stream=st),
    "moe_fp8_grouped_gemm_swiglu": lambda st: _lib.moe_fp8_grouped_gemm_swiglu(*[z(F32, 3, 256)] * 4, z(I32, 5), 6, stream=st),
    "moe_fp8_add_rms_norm": lambda st: _lib.moe_fp8_add_rms_norm(z(BF16, 3, 256), z(BF16, 256), stream=st),
    "moe_fp8_few_forward": lambda st: _lib.moe_fp8_few_forward(z(BF16, 3, 256), z(F32, 4, 512, 256), z(F32, 4, 4, 2), z(F32, 4, 256, 256),
                                                               z(F32, 4, 2, 2), 2, logits=z(F32, 3, 4), stream=st),
    "moe_w4a16_few_forward": lambda st: _lib.moe_w4a16_few_forward(CFG, z(BF16, 3, 256), Handle, Handle, logits=z(F32, 3, 4), stream=st),
}


@pytest.mark.parametrize("name", list(CALLS))
def test_allocations_are_on_the_given_stream(side, name):
    CALLS[name](side)
    assert side.made and all(side.made)
    assert side.recorded == 1 and not side.entered


def test_without_a_stream_nothing_is_entered(side):
    for call in CALLS.values():
        call(None)
    assert side.made and not any(side.made) and side.recorded == 0


@pytest.mark.parametrize("args", [dict(x=None), dict(x=None, rows=None, logits=None), dict(x=torch.zeros(256))])
def test_bad_arguments_reach_the_binding_with_a_stream(side, monkeypatch, args):
    """... which refuses them as without one: nothing looks into them before."""
    seen = []
    monkeypatch.setattr(_lib, "_FP8", type("Module", (), {"few_fp8": lambda self, x, *rest: seen.append(x)})())
    _lib.moe_fp8_few_forward(**{**dict(x=None, w_gate_up=z(F32, 4, 512, 256), s_gate_up=z(F32, 4, 4, 2), w_down=z(F32, 4, 256, 256),
                                       s_down=z(F32, 4, 2, 2), top_k=2, stream=side), **args})
    assert len(seen) == 1 and (seen[0] is args["x"])
