"""Host logic of the FP8 chunk path (fp8.py) without a GPU: the library's calls are replaced by stand-ins."""

import contextlib

import pytest
import torch

from moe_prefill_nvfp4_gb300 import fp8


class Side:
    """A stand-in for a stream: knows whether torch's current stream is this one."""

    cuda_stream = 1234
    entered = False


@pytest.fixture
def calls(monkeypatch):
    """Stand-ins of torch's stream context and of the library's calls; the list has (name, stream given, whether
    torch's current stream was that stream)."""
    log = []

    @contextlib.contextmanager
    def on(stream):
        before, stream.entered = stream.entered, True
        yield
        stream.entered = before

    def note(name, result):
        def call(*args, **kw):
            stream = kw.get("stream")
            log.append((name, stream, stream is None or stream.entered))
            return result(*args)

        return call

    arange = torch.arange

    def noted_arange(*args, **kw):
        log.append(("arange", None, Side.current is None or Side.current.entered))
        return arange(*args, **kw)

    codes = lambda r, k: (torch.zeros(r, k).to(torch.float8_e4m3fn), torch.ones(r, -(-k // 128)))  # noqa: E731
    monkeypatch.setattr(torch.cuda, "Stream", Side)
    monkeypatch.setattr(torch.cuda, "stream", on)
    monkeypatch.setattr(torch, "arange", noted_arange)
    monkeypatch.setattr(fp8, "_result", lambda t, stream: t, raising=False)
    for name, result in dict(
            moe_router_logits=lambda x, w: torch.zeros(x.shape[0], w.shape[0]),
            moe_route_topk=lambda logits, k, *a: (torch.zeros(logits.shape[0], k, dtype=torch.int32),
                                                  torch.zeros(logits.shape[0], k)),
            moe_sort_by_expert=lambda ids, e: dict(expert_offsets=None, sorted_token_ids=None, token_to_perm=None),
            moe_fp8_quantize_rows=lambda x: codes(*x.shape),
            moe_fp8_grouped_gemm_swiglu=lambda a, s, w, ws, off, r: codes(r, w.shape[1] // 2),
            moe_fp8_grouped_gemm=lambda a, s, w, ws, off, r: torch.zeros(r, w.shape[1]),
            moe_fp8_gemm=lambda a, s, w, ws: torch.zeros(a.shape[0], w.shape[0]),
            moe_combine_indexed=lambda y, perm, wts, shared: torch.zeros(1)).items():
        monkeypatch.setattr(fp8.moe, name, note(name, result))
    return log


def weight(*shape):
    scales = shape[:-2] + (-(-shape[-2] // 128), -(-shape[-1] // 128))
    return fp8.Fp8Weight(torch.zeros(*shape).to(torch.float8_e4m3fn), torch.ones(scales))


@pytest.mark.parametrize("given", ["stream", "none"])
@pytest.mark.parametrize("routed_by", ["logits", "w_router"])
def test_everything_of_a_forward_is_on_its_stream(calls, given, routed_by):
    """Allocations and torch's own kernels follow the current stream: with a stream that is not current they
    would not be ordered with the calls that are given it."""
    Side.current = Side() if given == "stream" else None
    shared = fp8.Fp8SharedExpert(weight(256, 64), weight(64, 128))
    layer = fp8.Fp8Experts(weight(4, 256, 64), weight(4, 64, 128), top_k=2, shared=shared)
    how = dict(logits=torch.zeros(3, 4)) if routed_by == "logits" else dict(w_router=torch.zeros(4, 64))
    layer.forward(torch.zeros(3, 64), stream=Side.current, **how)
    names = [name for name, _, _ in calls]
    assert {"moe_route_topk", "moe_sort_by_expert", "moe_fp8_quantize_rows", "moe_fp8_gemm", "moe_combine_indexed"} <= set(names)
    assert all(stream is Side.current for name, stream, _ in calls if name != "arange")
    assert all(current for _, _, current in calls), calls
    assert Side.current is None or not Side.current.entered


def test_everything_of_the_shared_expert_is_on_its_stream(calls):
    Side.current = Side()
    shared = fp8.Fp8SharedExpert(weight(256, 64), weight(64, 128))
    shared.forward(torch.zeros(3, 64).to(torch.float8_e4m3fn), torch.ones(3, 1), Side.current)
    assert len(calls) >= 2 and all(current for _, _, current in calls), calls


def test_shared_expert_is_in_one_part_only():
    """The parts' results are added: a shared expert in each of them would count as often."""
    shared = fp8.Fp8SharedExpert(weight(256, 64), weight(64, 128))
    parts = weight(4, 256, 64), weight(4, 64, 128)
    with pytest.raises(ValueError, match="shared"):
        fp8.Fp8Experts(*parts, top_k=2, num_experts=8, first=4, shared=shared)
    assert fp8.Fp8Experts(*parts, top_k=2, num_experts=8, first=0, shared=shared).shared is shared
    assert fp8.Fp8Experts(*parts, top_k=2, num_experts=8, first=4).shared is None


@pytest.mark.parametrize("shape", [(128,), (2, 3, 128, 128), (1, 1, 2, 128, 128)])
def test_weight_of_another_rank_is_refused(shape):
    with pytest.raises(ValueError, match="w: need"):
        fp8.Fp8Weight.quantise(torch.zeros(shape))


def test_shared_expert_without_tokens(calls):
    Side.current = None
    shared = fp8.Fp8SharedExpert(weight(256, 64), weight(64, 128))
    assert shared.forward(torch.zeros(0, 64).to(torch.float8_e4m3fn), torch.ones(0, 1)).shape == (0, 64)
