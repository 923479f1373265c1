"""Routed and shared experts with FP8 weights and activations (E4M3, one FP32 scale per 128 elements).

The chunk path of a checkpoint whose experts are stored in block-scaled FP8 instead of NVFP4: routing,
sort and combine are the library's usual calls; the products are the FP8 ones.

    logits -> top-k -> expert sort -> quantise x by rows -> gate/up product with SwiGLU and quantisation
           -> down product -> weighted combine (+ shared expert)

Between gate/up and down only codes and scales go to memory.  The step before it, residual addition and RMS norm,
gives the quantised rows too (``moe_fp8_add_rms_norm``), and a few tokens take the whole layer in one call
(``forward_few``).  ``python -m moe_prefill_nvfp4_gb300.fp8`` runs a chunk and a few tokens of random weights and
prints their times and distances from the same experts in FP32.
"""

from __future__ import annotations

from typing import Optional

import torch

from . import _lib as moe
from ._lib import _on, _result

__all__ = ["Fp8Weight", "Fp8SharedExpert", "Fp8Experts"]


class Fp8Weight:
    """Codes (E4M3) and scales of a weight, [N, K] and [ceil(N/128), ceil(K/128)], or of one weight per expert,
    both with the experts in front.  ``quantise`` makes them from BF16 or FP32, at load."""

    def __init__(self, q: torch.Tensor, s: torch.Tensor):
        self.q, self.s = q, s

    @classmethod
    def quantise(cls, w: torch.Tensor) -> "Fp8Weight":
        if w.dim() not in (2, 3):
            raise ValueError(f"w: need [N, K] or [experts, N, K], got {tuple(w.shape)}")
        lead, (n, k) = w.shape[:-2], w.shape[-2:]
        q = torch.empty(*lead, n, -(-k // 16) * 16, dtype=torch.float8_e4m3fn, device=w.device)[..., :k]
        s = torch.empty(*lead, -(-n // 128), -(-k // 128), dtype=torch.float32, device=w.device)
        if w.dim() == 2:
            moe.moe_fp8_quantize_blocks(w, out=q, scales=s)
        for e in range(w.shape[0] if w.dim() == 3 else 0):
            moe.moe_fp8_quantize_blocks(w[e], out=q[e], scales=s[e])
        return cls(q, s)


class Fp8SharedExpert:
    """A dense SwiGLU MLP: gate_up [2I, H] (gate rows first), down [H, I].  ``limit``: as for ``Fp8Experts``."""

    def __init__(self, gate_up: Fp8Weight, down: Fp8Weight, limit: float = 7.0):
        self.gate_up, self.down, self.limit = gate_up, down, limit

    def forward(self, q: torch.Tensor, s: torch.Tensor, stream=None) -> torch.Tensor:
        """BF16 [T, H] of quantised rows.  The gate/up product runs as one expert that has every row.
        ``stream``: as for ``Fp8Experts.forward``."""
        tokens = q.shape[0]
        with _on(stream):
            rows = torch.arange(0, 2 * tokens, max(tokens, 1), dtype=torch.int32, device=q.device)  # [0, T]
            act = moe.moe_fp8_grouped_gemm_swiglu(q, s, self.gate_up.q[None], self.gate_up.s[None], rows, tokens,
                                                  limit=self.limit, stream=stream)
            y = moe.moe_fp8_gemm(*act, self.down.q, self.down.s, stream=stream)
        return _result(y, stream)


class Fp8Experts:
    """E routed experts, gate_up [count, 2I, H] and down [count, H, I]: all of them, or the ``count`` experts
    from ``first`` on of ``num_experts`` (expert parallelism: the others' part of the result is zero, and the
    caller adds the ranks' results; the shared expert, which is in one of them only, goes with expert 0).
    Gates are clamped to at most ``limit`` and ups to +-``limit`` before the SwiGLU; float("inf") clamps nothing."""

    def __init__(self, gate_up: Fp8Weight, down: Fp8Weight, top_k: int, num_experts: Optional[int] = None, first: int = 0,
                 limit: float = 7.0, renormalize: bool = True, routed_scale: float = 1.0,
                 shared: Optional[Fp8SharedExpert] = None):
        if shared is not None and first != 0:
            raise ValueError(f"shared: the results of all parts are added, only the one with first = 0 has it (got {first})")
        self.gate_up, self.down, self.top_k, self.first, self.limit = gate_up, down, top_k, first, limit
        self.num_experts = gate_up.q.shape[0] if num_experts is None else num_experts
        self.renormalize, self.routed_scale, self.shared = renormalize, routed_scale, shared

    def forward(self, x: torch.Tensor, w_router: Optional[torch.Tensor] = None, logits: Optional[torch.Tensor] = None,
                router_bias: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None, stream=None,
                rows: Optional[tuple] = None) -> torch.Tensor:
        """BF16 [T, H] of a chunk x BF16 [T, H], routed by ``logits`` FP32 [T, E] or by ``w_router`` BF16 [E, H].
        ``rows``: the codes and scales of x where it is quantised already (``moe_fp8_add_rms_norm``).

        With ``stream`` everything runs on it, temporaries and a new result are allocated on it, and nothing waits
        for the current stream: the caller has the inputs ready on ``stream``, keeps them until it is done, and
        waits for it before it uses the result elsewhere."""
        if (w_router is None) == (logits is None):
            raise ValueError("forward: exactly one of w_router and logits")
        # (the gathers and the combine go by x's tokens: rows of fewer tokens would be read past their end)
        if rows is not None and (len(rows) != 2 or rows[0].shape != x.shape or rows[1].shape[0] != x.shape[0]):
            raise ValueError(f"rows: need codes {tuple(x.shape)} and their scales, got {[tuple(t.shape) for t in rows]}")
        with _on(stream):
            if logits is None:
                logits = moe.moe_router_logits(x, w_router, stream=stream)
            if logits.shape != (x.shape[0], self.num_experts):
                raise ValueError(f"logits: need {(x.shape[0], self.num_experts)}, got {tuple(logits.shape)}")
            y = self._chunk(x, logits, router_bias, out, stream, rows)
        return y if out is not None else _result(y, stream)

    def forward_few(self, x: Optional[torch.Tensor], w_router: Optional[torch.Tensor] = None,
                    logits: Optional[torch.Tensor] = None, router_bias: Optional[torch.Tensor] = None,
                    out: Optional[torch.Tensor] = None, stream=None, rows: Optional[tuple] = None,
                    ws: Optional[torch.Tensor] = None) -> torch.Tensor:
        """The same layer for at most ``MOE_FEW_MAX_TOKENS`` tokens in one call (``moe_fp8_few_forward``), as a decode
        step has them: its sums have an order of their own, and nothing but the result is rounded to BF16.  x may be
        None with ``rows`` and ``logits``.  ``ws``: a workspace of this call's own (``moe_few_workspace_bytes``)."""
        shared = self.shared
        parts = None if shared is None else (shared.gate_up.q, shared.gate_up.s, shared.down.q, shared.down.s)
        with _on(stream):
            y = moe.moe_fp8_few_forward(x, self.gate_up.q, self.gate_up.s, self.down.q, self.down.s, self.top_k, w_router, logits,
                                        router_bias, self.limit, self.renormalize, self.routed_scale, self.num_experts,
                                        self.first, parts, None if shared is None else shared.limit, rows, ws, out, stream)
        return y if out is not None else _result(y, stream)

    def _chunk(self, x, logits, router_bias, out, stream, rows) -> torch.Tensor:
        ids, wts = moe.moe_route_topk(logits, self.top_k, router_bias, self.renormalize, self.routed_scale, stream=stream)
        order = moe.moe_sort_by_expert(ids, self.num_experts, stream=stream)
        slots = ids.numel()
        q, s = rows if rows is not None else moe.moe_fp8_quantize_rows(x, stream=stream)
        act = moe.moe_fp8_grouped_gemm_swiglu(q, s, self.gate_up.q, self.gate_up.s, order["expert_offsets"], slots,
                                              limit=self.limit, gather_ids=order["sorted_token_ids"], first=self.first,
                                              stream=stream)
        y = moe.moe_fp8_grouped_gemm(*act, self.down.q, self.down.s, order["expert_offsets"], slots, first=self.first,
                                     stream=stream)
        shared = self.shared.forward(q, s, stream) if self.shared is not None else None
        return moe.moe_combine_indexed(y, order["token_to_perm"], wts, shared, out=out, stream=stream)


def _reference(x, logits, gate_up, down, top_k, limit):
    """The same experts in FP32 torch operations (unquantised weights)."""
    w, ids = logits.softmax(-1).topk(top_k, -1)
    w = w / w.sum(-1, keepdim=True)
    inter, out = down.shape[2], torch.zeros_like(x, dtype=torch.float32)
    for e in range(gate_up.shape[0]):
        t, slot = (ids == e).nonzero(as_tuple=True)
        y = x[t].float() @ gate_up[e].float().t()
        act = torch.nn.functional.silu(y[:, :inter].clamp(max=limit)) * y[:, inter:].clamp(-limit, limit)
        out.index_add_(0, t, (act @ down[e].float().t()) * w[t, slot, None])
    return out


def main(tokens: int = 256, hidden: int = 2048, inter: int = 768, experts: int = 64, top_k: int = 8, few: int = 4) -> None:
    g = torch.Generator(device="cuda").manual_seed(0)
    rand = lambda *shape: torch.randn(*shape, generator=g, device="cuda", dtype=torch.bfloat16)  # noqa: E731
    x, logits = rand(tokens, hidden), rand(tokens, experts).float()
    gate_up, down = rand(experts, 2 * inter, hidden) * hidden ** -0.5, rand(experts, hidden, inter) * inter ** -0.5
    layer = Fp8Experts(Fp8Weight.quantise(gate_up), Fp8Weight.quantise(down), top_k)
    few = min(few, tokens)
    # a decode step: the residual stream through the norm, which also quantises, to the router and the experts
    residual, w_norm, w_router = rand(few, hidden), 1 + 0.1 * rand(hidden), rand(experts, hidden) * hidden ** -0.5

    def step():
        q, s, _, normed = moe.moe_fp8_add_rms_norm(x[:few], w_norm, residual, normed=True)
        return normed, layer.forward_few(normed, w_router, rows=(q, s))

    def report(what, run, y, ref):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            run()
        for _ in range(3):
            graph.replay()
        start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        start.record()
        for _ in range(20):
            graph.replay()
        end.record()
        torch.cuda.synchronize()
        print(f"{what}, {experts} experts, top-{top_k}: {start.elapsed_time(end) / 20 * 1e3:.1f} us, "
              f"{float((y.float() - ref).norm() / ref.norm()):.3f} of the unquantised experts' norm apart, "
              f"device error {moe.moe_get_device_error()}")

    y = layer.forward(x, logits=logits)
    report(f"{tokens} tokens", lambda: layer.forward(x, logits=logits), y,
           _reference(x, logits, gate_up, down, top_k, layer.limit))
    normed, y = step()
    report(f"norm and layer of {few} tokens", step, y,
           _reference(normed, moe.moe_router_logits(normed, w_router), gate_up, down, top_k, layer.limit))


if __name__ == "__main__":
    main()
