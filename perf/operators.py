"""The FP8 expert operators as cases that can be timed: E4M3 codes with one FP32 scale for each 128
elements of an activation row and for each 128 x 128 block of a weight.

    quantize_rows    activation rows (BF16 or FP32) -> codes and a scale per row and 128 columns
    quantize_blocks  a weight -> codes and a scale per 128 x 128 block
    gemm             dense product of quantised rows with a quantised weight (shared expert, projections)
    grouped          the routed experts' product over expert-sorted rows (down projection)
    grouped_swiglu   gate/up product, clamped SwiGLU, and the result quantised for the down projection

With ``own`` false `run` computes them in plain torch operations in FP32; with ``own`` true it calls the
framework.  `exact` is the definition in FP64.
"""

import math
import random  # noqa: F401  (the type of draw's argument)

import torch

own = False

BLOCK = 128
E4M3_MAX = 448.0
AMAX_FLOOR = 2.0 ** -100  # smallest magnitude a scale is derived from: 448 / it stays finite in FP32
LIMIT = 7.0


# ------------------------------------------------------------------------------------------ cases


def listed():
    return [
        # one token's hidden state on its way into the experts (decode): launch latency
        dict(name="rows_decode", op="quantize_rows", rows=1, k=5120, dtype="bf16"),
        # a prefill chunk's hidden states at the GLM width: memory bandwidth
        dict(name="rows_chunk", op="quantize_rows", rows=8192, k=5120, dtype="bf16"),
        # a small weight of odd sizes held in FP32, quantised when it is loaded
        dict(name="blocks_odd", op="quantize_blocks", n=1000, k=777, dtype="f32"),
        # one expert's down projection, quantised when it is loaded
        dict(name="blocks_expert", op="quantize_blocks", n=5120, k=1536, dtype="bf16"),
        # the shared expert's down projection for one token
        dict(name="gemm_decode", op="gemm", rows=1, n=5120, k=1536, out="bf16"),
        # a ragged chunk against a weight of odd sizes, result kept in FP32
        dict(name="gemm_ragged", op="gemm", rows=333, n=1500, k=2000, out="f32"),
        # the shared expert's gate projection over a whole chunk: tensor-core rate
        dict(name="gemm_chunk", op="gemm", rows=8192, n=1536, k=5120, out="bf16"),
        # down projection of the eight experts of one token: weight streaming
        dict(name="down_decode", op="grouped", tokens=1, experts=160, top_k=8, n=5120, k=1536, skew=0.1, idle=0, out="bf16"),
        # down projection of a long chunk, some experts without a row
        dict(name="down_chunk", op="grouped", tokens=8192, experts=160, top_k=8, n=5120, k=1536, skew=0.1, idle=16, out="bf16"),
        # gate/up of a few tokens in flight (batched decode)
        dict(name="gate_up_decode", op="grouped_swiglu", tokens=4, experts=160, top_k=8, inter=1536, k=5120, skew=0.1, idle=0),
        # gate/up of a 256-row chunk of the smaller block (64 experts)
        dict(name="gate_up_256", op="grouped_swiglu", tokens=256, experts=64, top_k=8, inter=768, k=2048, skew=0.3, idle=0),
        # gate/up of a long chunk at the GLM sizes: tensor-core rate
        dict(name="gate_up_chunk", op="grouped_swiglu", tokens=8192, experts=160, top_k=8, inter=1536, k=5120, skew=0.1, idle=0),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["quantize_rows", "quantize_blocks", "gemm", "gemm", "grouped", "grouped", "grouped_swiglu", "grouped_swiglu"])
    if op == "quantize_rows":
        return dict(op=op, rows=_log_int(rng, 1, 8192), k=_log_int(rng, 128, 5120), dtype=rng.choice(["bf16", "f32"]))
    if op == "quantize_blocks":
        return dict(op=op, n=_log_int(rng, 128, 5120), k=_log_int(rng, 128, 1536), dtype=rng.choice(["bf16", "f32"]))
    if op == "gemm":
        return dict(op=op, rows=_log_int(rng, 1, 8192), n=_log_int(rng, 128, 1536), k=_log_int(rng, 256, 5120),
                    out=rng.choice(["bf16", "f32"]))
    experts = _log_int(rng, 8, 160)
    case = dict(op=op, tokens=_log_int(rng, 1, 8192), experts=experts, top_k=rng.randint(1, 8),
                skew=rng.choice([0.0, 0.1, 0.3]), idle=rng.choice([0, 0, experts // 10]))
    if op == "grouped":
        return dict(case, n=_log_int(rng, 256, 5120), k=_log_int(rng, 256, 1536), out=rng.choice(["bf16", "f32"]))
    return dict(case, inter=BLOCK * rng.randint(2, 12), k=_log_int(rng, 256, 5120))


def _active_experts(case):
    """How many experts have a row, on average, where all are equally likely."""
    e = case["experts"] - case["idle"]
    return e * (1.0 - (1.0 - case["top_k"] / e) ** case["tokens"])


def work(case):
    op = case["op"]
    g = -(-case["k"] // BLOCK)
    if op in ("quantize_rows", "quantize_blocks"):
        size = 2 if case["dtype"] == "bf16" else 4
        lines, scales = (case["rows"], case["rows"] * g) if op == "quantize_rows" else (case["n"], -(-case["n"] // BLOCK) * g)
        return {"bytes": lines * case["k"] * (size + 1) + 4 * scales, "flops": 3 * lines * case["k"]}
    if op == "gemm":
        m, n, k = case["rows"], case["n"], case["k"]
        out = 2 if case["out"] == "bf16" else 4
        return {"bytes": m * k + n * k + 4 * g * (m + -(-n // BLOCK)) + m * n * out, "flops": 2 * m * n * k}
    slots = case["tokens"] * case["top_k"]
    n = case["n"] if op == "grouped" else 2 * case["inter"]
    rows_in = slots if op == "grouped" else case["tokens"]
    read = rows_in * (case["k"] + 4 * g) + _active_experts(case) * (n * case["k"] + 4 * g * -(-n // BLOCK)) + 4 * slots
    if op == "grouped":
        written = slots * n * (2 if case["out"] == "bf16" else 4)
    else:
        written = slots * (case["inter"] + 4 * (case["inter"] // BLOCK))
    return {"bytes": read + written, "flops": 2 * slots * n * case["k"]}


# ------------------------------------------------------------------------------------------ plain forms


def _pad_cols(x, k):
    return torch.nn.functional.pad(x, (0, -(-k // BLOCK) * BLOCK - k))


def _quantize_groups(groups):
    """groups [..., m] FP32 sharing one scale along the last axis -> (codes, scale [..., 1])."""
    amax = groups.abs().amax(-1, keepdim=True)
    # a group with a value that is not finite has no scale
    amax = torch.where(amax.isfinite(), amax.clamp_min(AMAX_FLOOR), torch.full_like(amax, float("nan")))
    return (groups * (E4M3_MAX / amax)).to(torch.float8_e4m3fn), amax / E4M3_MAX


def _quantize_rows(x):
    r, k = x.shape
    q, s = _quantize_groups(_pad_cols(x.float(), k).view(r, -1, BLOCK))
    return q.view(r, -1)[:, :k], s.squeeze(-1)


def _quantize_blocks(w):
    n, k = w.shape
    nb, g = -(-n // BLOCK), -(-k // BLOCK)
    p = torch.nn.functional.pad(w.float(), (0, g * BLOCK - k, 0, nb * BLOCK - n))
    p = p.view(nb, BLOCK, g, BLOCK).transpose(1, 2).reshape(nb, g, BLOCK * BLOCK)
    q, s = _quantize_groups(p)
    q = q.view(nb, g, BLOCK, BLOCK).transpose(1, 2).reshape(nb * BLOCK, g * BLOCK)
    return q[:n, :k], s.squeeze(-1)


def _dequantize_rows(q, s, dtype=torch.float32):
    k = q.shape[-1]
    return q.to(dtype) * s.to(dtype).repeat_interleave(BLOCK, -1)[..., :k]


def _dequantize_blocks(q, s, dtype=torch.float32):
    n, k = q.shape[-2:]
    return q.to(dtype) * s.to(dtype).repeat_interleave(BLOCK, -1)[..., :k].repeat_interleave(BLOCK, -2)[..., :n, :]


def _swiglu(y, inter):
    gate, up = y[..., :inter].clamp(max=LIMIT), y[..., inter:].clamp(-LIMIT, LIMIT)
    return gate / (1.0 + torch.exp(-gate)) * up


def _grouped_plain(st):
    """Expert-sorted product [R, N] in FP32.  Few slots take each slot's own expert weight; otherwise
    every expert's rows are padded to the longest expert's."""
    offsets, experts = st["offsets"], st["sorted_experts"].long()
    slots = experts.numel()
    rows = _dequantize_rows(st["a"], st["a_scales"])
    if st["gather"] is not None:
        rows = rows[st["gather"].long()]
    if 2 * slots <= offsets.numel() - 1:
        w = st["w"].view(torch.uint8)[experts].view(torch.float8_e4m3fn)
        return torch.bmm(rows[:, None], _dequantize_blocks(w, st["w_scales"][experts]).transpose(1, 2))[:, 0]
    at = offsets[:-1, None].long() + torch.arange(st["longest"], device=rows.device)
    inside = at < offsets[1:, None]
    padded = rows[at.clamp(max=slots - 1)] * inside[..., None]
    y = torch.bmm(padded, _dequantize_blocks(st["w"], st["w_scales"]).transpose(1, 2))
    return y[experts, torch.arange(slots, device=rows.device) - offsets[experts].long()]


# ------------------------------------------------------------------------------------------ inputs


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed) * 2 + 1)
    return g


def _activations(g, r, k, dtype):
    """Hidden states: normal, with a few channels of a much larger scale, as residual streams have."""
    x = torch.randn(r, k, generator=g, device="cuda")
    loud = torch.rand(k, generator=g, device="cuda") < 0.01
    return (x * torch.where(loud, 12.0, 1.0)).to(dtype)


def _own_layout_rows(q, s):
    """Codes with rows 16 bytes apart at least and scales column by column: what quantize_rows returns."""
    r, k = q.shape
    buf = torch.empty(r, -(-k // 16) * 16, dtype=torch.float8_e4m3fn, device=q.device)
    buf[:, :k] = q
    return buf[:, :k], s.t().contiguous().t()


def _weight(g, e, n, k):
    """[e, n, k] codes and [e, n/128, k/128] scales of normal weights, rows of whole 16 bytes."""
    q = torch.zeros(e, n, -(-k // 16) * 16, dtype=torch.float8_e4m3fn, device="cuda")
    s = torch.empty(e, -(-n // BLOCK), -(-k // BLOCK), device="cuda")
    for i in range(e):
        qi, s[i] = _quantize_blocks(torch.randn(n, k, generator=g, device="cuda") * k ** -0.5)
        q[i, :, :k] = qi
    return q[..., :k], s


def _route(g, case):
    """Expert-sorted slots of a top-k routing over logits N(0, 1) + a bias per expert; `idle` experts get none."""
    t, e, k = case["tokens"], case["experts"], case["top_k"]
    logits = torch.randn(t, e, generator=g, device="cuda") + case["skew"] * torch.randn(e, generator=g, device="cuda")
    logits[:, torch.randperm(e, generator=g, device="cuda")[: case["idle"]]] = -1e30
    ids = logits.topk(k, dim=1).indices.reshape(-1)
    experts, order = torch.sort(ids, stable=True)
    counts = torch.bincount(ids, minlength=e)
    offsets = torch.cat([counts.new_zeros(1), counts.cumsum(0)]).int()
    return (order // k).int(), experts.int(), offsets, int(counts.max())


def _dtype(name):
    return torch.bfloat16 if name == "bf16" else torch.float32


def prepare(case, seed):
    g, op = _gen(seed), case["op"]
    st = dict(case)
    if op == "quantize_rows":
        st["x"] = _activations(g, case["rows"], case["k"], _dtype(case["dtype"]))
        return st
    if op == "quantize_blocks":
        st["x"] = (torch.randn(case["n"], case["k"], generator=g, device="cuda") * case["k"] ** -0.5).to(_dtype(case["dtype"]))
        return st
    if op == "gemm":
        st["a"], st["a_scales"] = _own_layout_rows(*_quantize_rows(_activations(g, case["rows"], case["k"], torch.bfloat16)))
        w, s = _weight(g, 1, case["n"], case["k"])
        st["w"], st["w_scales"] = w[0], s[0]
        return st
    tokens, st["sorted_experts"], st["offsets"], st["longest"] = _route(g, case)
    slots = tokens.numel()
    # the gate/up product gathers the tokens' rows, the down product's rows are in expert order already
    rows = case["tokens"] if op == "grouped_swiglu" else slots
    st["gather"] = tokens if op == "grouped_swiglu" else None
    st["slots"] = slots
    st["a"], st["a_scales"] = _own_layout_rows(*_quantize_rows(_activations(g, rows, case["k"], torch.bfloat16)))
    n = 2 * case["inter"] if op == "grouped_swiglu" else case["n"]
    st["w"], st["w_scales"] = _weight(g, case["experts"], n, case["k"])
    return st


# ------------------------------------------------------------------------------------------ one pass


def run(st):
    op = st["op"]
    if own:
        import moe_prefill_nvfp4_gb300 as moe

        if op == "quantize_rows":
            q, s = moe.moe_fp8_quantize_rows(st["x"])
            return {"q": q, "s": s}
        if op == "quantize_blocks":
            q, s = moe.moe_fp8_quantize_blocks(st["x"])
            return {"q": q, "s": s}
        if op == "gemm":
            return moe.moe_fp8_gemm(st["a"], st["a_scales"], st["w"], st["w_scales"], c_dtype=_dtype(st["out"]))
        if op == "grouped":
            return moe.moe_fp8_grouped_gemm(st["a"], st["a_scales"], st["w"], st["w_scales"], st["offsets"], st["slots"],
                                            c_dtype=_dtype(st["out"]))
        q, s = moe.moe_fp8_grouped_gemm_swiglu(st["a"], st["a_scales"], st["w"], st["w_scales"], st["offsets"], st["slots"],
                                               limit=LIMIT, gather_ids=st["gather"])
        return {"q": q, "s": s}
    if op == "quantize_rows":
        q, s = _quantize_rows(st["x"])
        return {"q": q, "s": s}
    if op == "quantize_blocks":
        q, s = _quantize_blocks(st["x"])
        return {"q": q, "s": s}
    if op == "gemm":
        y = _dequantize_rows(st["a"], st["a_scales"]) @ _dequantize_blocks(st["w"], st["w_scales"]).t()
        return y.to(_dtype(st["out"]))
    y = _grouped_plain(st)
    if op == "grouped":
        return y.to(_dtype(st["out"]))
    q, s = _quantize_rows(_swiglu(y, st["inter"]))
    return {"q": q, "s": s}


# ------------------------------------------------------------------------------------------ the definition in 64 bits


def _round_e4m3_64(v):
    """Nearest E4M3 value (ties to even), by magnitude: steps of 2^(e-3) for 2^e <= |v|, e >= -6."""
    exponent = torch.frexp(v)[1].clamp(min=-5) - 1
    step = torch.ldexp(torch.ones_like(v), exponent - 3)
    return torch.clamp(torch.round(v / step) * step, -E4M3_MAX, E4M3_MAX)


def _quantize_exact(x, rows_per_scale):
    """FP64 codes and scales of x [n, k], `rows_per_scale` x 128 elements to a scale."""
    n, k = x.shape
    s = torch.empty(-(-n // rows_per_scale), -(-k // BLOCK), dtype=torch.float64, device=x.device)
    q = torch.empty_like(x)
    for j in range(s.shape[1]):
        cols = slice(j * BLOCK, min(k, (j + 1) * BLOCK))
        part = x[:, cols]
        high = part.abs().amax(1)
        if rows_per_scale > 1:
            high = torch.stack([c.amax() for c in high.split(rows_per_scale)])
        s[:, j] = high.clamp_min(AMAX_FLOOR) / E4M3_MAX
        q[:, cols] = _round_e4m3_64(part / s[:, j].repeat_interleave(rows_per_scale)[:n, None])
    return {"q": q, "s": s}


def exact(case, seed):
    st, op = prepare(case, seed), case["op"]
    f64 = torch.float64
    if op == "quantize_rows":
        return _quantize_exact(st["x"].to(f64), 1)
    if op == "quantize_blocks":
        return _quantize_exact(st["x"].to(f64), BLOCK)

    def product(a, a_scales, w, w_scales):
        y = torch.zeros(a.shape[0], w.shape[0], dtype=f64, device=a.device)
        for j in range(a_scales.shape[1]):
            cols = slice(j * BLOCK, (j + 1) * BLOCK)
            part = a[:, cols].to(f64) @ w[:, cols].to(f64).t()
            by_row = w_scales[:, j].to(f64).repeat_interleave(BLOCK)[: w.shape[0]]
            y += part * a_scales[:, j].to(f64)[:, None] * by_row[None]
        return y

    if op == "gemm":
        return product(st["a"], st["a_scales"], st["w"], st["w_scales"])
    bounds = st["offsets"].tolist()
    parts = []
    for e in range(case["experts"]):
        lo, hi = bounds[e], bounds[e + 1]
        if hi > lo:
            at = st["gather"][lo:hi].long() if st["gather"] is not None else torch.arange(lo, hi, device="cuda")
            a = st["a"].view(torch.uint8)[at].view(torch.float8_e4m3fn)
            parts.append(product(a, st["a_scales"][at], st["w"][e], st["w_scales"][e]))
    y = torch.cat(parts)
    if op == "grouped":
        return y
    gate, up = y[:, : st["inter"]].clamp(max=LIMIT), y[:, st["inter"]:].clamp(-LIMIT, LIMIT)
    return _quantize_exact(gate / (1.0 + torch.exp(-gate)) * up, 1)
