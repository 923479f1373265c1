"""Operators of a transformer block's expert layer as cases that can be timed, next to the FP8 and NVFP4 products:

    norm      residual addition, root-mean-square norm, and its result as E4M3 codes with one FP32 scale per 128
              columns (the experts' operand), beside the sum and the result in BF16 (the router's operand)
    few_fp8   a whole layer of FP8 experts for a few tokens, whose rows the norm has quantised: routing, gate/up
              products with SwiGLU and quantiser, down products, weighted sum (and a shared expert)
    few_w4    a whole layer of NVFP4 experts (W4A16) for a few tokens

With ``own`` false `run` computes them in plain torch operations in FP32; with ``own`` true it calls the
framework.  `exact` is the definition in FP64.
"""

import math
import random  # noqa: F401  (the type of draw's argument)

import torch

own = False

BLOCK = 128
E4M3_MAX = 448.0
AMAX_FLOOR = 2.0 ** -100  # smallest magnitude a scale is derived from
LIMIT = 7.0
EPS = 1e-6


# ------------------------------------------------------------------------------------------ cases


def listed():
    return [
        # one token between attention and experts (decode): launch latency
        dict(name="norm_decode", op="norm", rows=1, k=5120, x="bf16", res="bf16", w="bf16", normed=True),
        # a ragged batch, a width that ends inside a group, the residual stream kept in FP32
        dict(name="norm_ragged", op="norm", rows=333, k=2000, x="bf16", res="f32", w="f32", normed=True),
        # a prefill chunk, its router's operand included: memory bandwidth
        dict(name="norm_chunk", op="norm", rows=8192, k=5120, x="bf16", res="bf16", w="bf16", normed=True),
        # a prefill chunk's first norm: no residual yet, codes alone
        dict(name="norm_first", op="norm", rows=2048, k=5120, x="bf16", res="none", w="bf16", normed=False),
        # one token in flight: the weights of its eight experts are the work
        dict(name="fp8_one", op="few_fp8", tokens=1, experts=160, top_k=8, hidden=5120, inter=1536, shared=0, routed_by="router", bias=False),
        # four sequences in flight, the smaller block
        dict(name="fp8_four", op="few_fp8", tokens=4, experts=64, top_k=8, hidden=2048, inter=768, shared=0, routed_by="router", bias=False),
        # a batch of sixteen: most of the experts have a row or two
        dict(name="fp8_sixteen", op="few_fp8", tokens=16, experts=160, top_k=8, hidden=5120, inter=1536, shared=0, routed_by="router", bias=False),
        # drafted tokens to verify, odd sizes, a shared expert, selection with a bias
        dict(name="fp8_shared", op="few_fp8", tokens=5, experts=33, top_k=3, hidden=1152, inter=640, shared=384, routed_by="logits", bias=True),
        # one token in flight, weights in four bits
        dict(name="w4_one", op="few_w4", tokens=1, experts=160, top_k=8, hidden=5120, inter=1536, shared=0, routed_by="router", bias=False),
        # four sequences in flight, the smaller block
        dict(name="w4_four", op="few_w4", tokens=4, experts=64, top_k=8, hidden=2048, inter=768, shared=0, routed_by="router", bias=False),
        # a batch of sixteen
        dict(name="w4_sixteen", op="few_w4", tokens=16, experts=160, top_k=8, hidden=5120, inter=1536, shared=0, routed_by="router", bias=False),
        # drafted tokens, odd sizes, a shared expert's result to add, selection with a bias
        dict(name="w4_shared", op="few_w4", tokens=7, experts=33, top_k=3, hidden=1280, inter=512, shared=1, routed_by="logits", bias=True),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "few_fp8", "few_fp8", "few_w4", "few_w4"])
    if op == "norm":
        return dict(op=op, rows=_log_int(rng, 1, 8192), k=_log_int(rng, 128, 5120), x=rng.choice(["bf16", "bf16", "f32"]),
                    res=rng.choice(["none", "bf16", "bf16", "f32"]), w=rng.choice(["bf16", "f32"]), normed=rng.choice([True, False]))
    piece = BLOCK if op == "few_fp8" else 256
    experts = _log_int(rng, 8, 160)
    inter = piece * _log_int(rng, 1, 1536 // piece)
    shared = rng.choice([0, 0, 1])
    return dict(op=op, tokens=_log_int(rng, 1, 16), experts=experts, top_k=rng.randint(1, 8), hidden=piece * _log_int(rng, 2, 5120 // piece),
                inter=inter, shared=shared * (BLOCK * rng.randint(1, 6) if op == "few_fp8" else 1),
                routed_by=rng.choice(["router", "logits"]), bias=rng.choice([True, False]))


_SIZE = {"none": 0, "bf16": 2, "f32": 4}


def work(case):
    if case["op"] == "norm":
        r, k = case["rows"], case["k"]
        each = _SIZE[case["x"]] + 2 * _SIZE[case["res"]] + 1 + (2 if case["normed"] else 0)
        return {"bytes": r * k * each + 4 * r * -(-k // BLOCK) + k * _SIZE[case["w"]], "flops": 8 * r * k}
    t, e, k, h, i, sh = (case[n] for n in ("tokens", "experts", "top_k", "hidden", "inter", "shared"))
    active = e * (1.0 - (1.0 - k / e) ** t)  # experts with a row, on average, where all are equally likely
    per = 3 * h * i  # weights of an expert
    if case["op"] == "few_fp8":
        weights = active * (per + 4 * per / BLOCK ** 2) + 3 * h * sh * (1 + 4 / BLOCK ** 2)
        flops = 2 * t * (k * per + 3 * h * sh)
    else:
        weights = active * per * (0.5 + 1 / 16) + 2 * t * h * sh
        flops = 2 * t * k * per
    routing = 2 * e * h if case["routed_by"] == "router" else 4 * t * e
    flops += 2 * t * e * h if case["routed_by"] == "router" else 0
    rows = t * (h + 4 * h // BLOCK + (2 * h if case["routed_by"] == "router" else 0)) if case["op"] == "few_fp8" else 2 * t * h
    return {"bytes": weights + routing + rows + 2 * t * h + (4 * e if case["bias"] else 0), "flops": flops}


# ------------------------------------------------------------------------------------------ plain forms


def _quantize_groups(groups):
    """groups [..., 128] FP32 sharing a scale -> (codes, scale [..., 1])."""
    amax = groups.abs().amax(-1, keepdim=True)
    # a group with a value that is not finite has no scale
    amax = torch.where(amax.isfinite(), amax.clamp_min(AMAX_FLOOR), torch.full_like(amax, float("nan")))
    return (groups * (E4M3_MAX / amax)).to(torch.float8_e4m3fn), amax / E4M3_MAX


def _quantize_rows(x):
    r, k = x.shape
    padded = torch.nn.functional.pad(x.float(), (0, -(-k // BLOCK) * BLOCK - k))
    q, s = _quantize_groups(padded.view(r, -1, BLOCK))
    return q.view(r, -1)[:, :k], s.squeeze(-1)


def _rows_again(q, s):
    return q.float() * s.repeat_interleave(BLOCK, -1)[..., : q.shape[-1]]


def _blocks_again(q, s):
    """Weights [..., n, k] of codes and scales [..., n/128, k/128], n and k multiples of 128."""
    lead, (n, k) = q.shape[:-2], q.shape[-2:]
    w = q.float().view(*lead, n // BLOCK, BLOCK, k // BLOCK, BLOCK) * s.view(*lead, n // BLOCK, 1, k // BLOCK, 1)
    return w.view(*lead, n, k)


def _nvfp4_again(packed, scales, scale2):
    """Weights [..., n, k] of packed E2M1 codes [..., n, k/2], E4M3 scales [..., n, k/16] (as bytes) and one FP32
    number each."""
    codes = torch.stack([packed & 15, packed >> 4], -1).flatten(-2).long()
    values = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], device=packed.device)
    v = torch.cat([values, -values])[codes]
    return v * scales.view(torch.float8_e4m3fn).float().repeat_interleave(16, -1) * scale2[..., None, None]


def _swiglu(y):
    gate, up = y.chunk(2, -1)
    gate, up = gate.clamp(max=LIMIT), up.clamp(-LIMIT, LIMIT)
    return gate / (1.0 + torch.exp(-gate)) * up


def _topk(st):
    """Experts and weights of each token, [T, k].  The logits' sums in 64 bits: two of them may lie close together."""
    logits = st["logits"] if st["w_router"] is None else (st["x"].double() @ st["w_router"].double().t()).float()
    keys = logits if st["router_bias"] is None else logits + st["router_bias"]
    ids = torch.sort(keys, dim=-1, descending=True, stable=True).indices[:, : st["top_k"]]  # ties to the lower expert
    picked = logits.gather(1, ids)
    e = torch.exp(picked - picked.amax(-1, keepdim=True))
    return ids, e / e.sum(-1, keepdim=True)


def _norm_plain(st):
    x, r, w = st["x"], st["residual"], st["weight"]
    h = x.float() if r is None else x.float() + r.float()
    y = h * torch.rsqrt((h * h).mean(-1, keepdim=True) + EPS) * w.float()
    q, s = _quantize_rows(y)
    return {"q": q, "s": s, "h": None if r is None else h.to(r.dtype), "y": y.to(torch.bfloat16) if st["normed"] else None}


def _mlp_fp8(rows, gate_up, down):
    """SwiGLU MLPs, one for each row [n, h] or one for all of them; their activations are quantised."""
    def product(v, w):
        return v @ w.t() if w.dim() == 2 else torch.bmm(w, v[..., None])[..., 0]

    act = _swiglu(product(rows, _blocks_again(*gate_up)))
    return product(_rows_again(*_quantize_rows(act)), _blocks_again(*down))


def _few_fp8_plain(st):
    ids, wts = _topk(st)
    slots = ids.flatten()
    of = lambda w: (w[0].view(torch.uint8)[slots].view(torch.float8_e4m3fn), w[1][slots])  # noqa: E731
    rows = _rows_again(*st["rows"])
    y = _mlp_fp8(rows.repeat_interleave(ids.shape[1], 0), of(st["gate_up"]), of(st["down"]))
    out = (y.view(*ids.shape, -1) * wts[..., None]).sum(1)
    if st["shared_weights"] is not None:
        out = out + _mlp_fp8(rows, *st["shared_weights"])
    return out.to(torch.bfloat16)


def _few_w4_plain(st):
    ids, wts = _topk(st)
    slots = ids.flatten()
    of = lambda w: _nvfp4_again(*(t[slots] for t in w))  # noqa: E731
    rows = st["x"].float().repeat_interleave(ids.shape[1], 0)
    act = _swiglu(torch.bmm(of(st["gate_up"]), rows[..., None])[..., 0])
    y = torch.bmm(of(st["down"]), act[..., None])[..., 0]
    out = (y.view(*ids.shape, -1) * wts[..., None]).sum(1)
    if st["shared_out"] is not None:
        out = out + st["shared_out"].float()
    return out.to(torch.bfloat16)


# ------------------------------------------------------------------------------------------ inputs


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed) * 2 + 1)
    return g


def _dtype(name):
    return torch.bfloat16 if name == "bf16" else torch.float32


def _activations(g, r, k, dtype):
    """Hidden states: normal, with a few channels of a much larger scale, as residual streams have."""
    x = torch.randn(r, k, generator=g, device="cuda")
    loud = torch.rand(k, generator=g, device="cuda") < 0.01
    return (x * torch.where(loud, 12.0, 1.0)).to(dtype)


def _fp8_weight(g, n, k):
    w = torch.randn(n, k, generator=g, device="cuda") * k ** -0.5
    p = w.view(n // BLOCK, BLOCK, k // BLOCK, BLOCK).transpose(1, 2)
    q, s = _quantize_groups(p.reshape(n // BLOCK, k // BLOCK, BLOCK * BLOCK))
    return q.view_as(p).transpose(1, 2).reshape(n, k), s.squeeze(-1)


def _nvfp4_weight(g, n, k):
    """Packed codes, E4M3 block scales and the tensor's scale of a normal weight: nearest codes, the block's largest
    magnitude at 6."""
    w = torch.randn(n, k // 16, 16, generator=g, device="cuda") * k ** -0.5
    top = w.abs().amax(-1, keepdim=True)
    scale2 = top.amax() / (6.0 * E4M3_MAX)
    s = (top / (6.0 * scale2)).to(torch.float8_e4m3fn)
    v = w / (s.float() * scale2).clamp_min(1e-30)
    between = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device="cuda")
    code = (torch.bucketize(v.abs(), between) + 8 * (v < 0)).to(torch.uint8).view(n, k // 2, 2)
    return code[..., 0] | (code[..., 1] << 4), s.view(torch.uint8).view(n, k // 16), scale2


def prepare(case, seed):
    g, st = _gen(seed), dict(case)
    if case["op"] == "norm":
        r, k = case["rows"], case["k"]
        # a block's output is smaller than the stream that it is added to
        st["x"] = (_activations(g, r, k, torch.float32) * 0.3).to(_dtype(case["x"]))
        st["residual"] = None if case["res"] == "none" else _activations(g, r, k, _dtype(case["res"]))
        st["weight"] = (1.0 + 0.2 * torch.randn(k, generator=g, device="cuda")).to(_dtype(case["w"]))
        return st
    t, e, h, i = case["tokens"], case["experts"], case["hidden"], case["inter"]
    st["x"] = _activations(g, t, h, torch.bfloat16)
    by_router = case["routed_by"] == "router"
    st["w_router"] = (torch.randn(e, h, generator=g, device="cuda") * h ** -0.5).bfloat16() if by_router else None
    st["logits"] = None if by_router else torch.randn(t, e, generator=g, device="cuda")
    st["router_bias"] = 0.3 * torch.randn(e, generator=g, device="cuda") if case["bias"] else None
    make = _fp8_weight if case["op"] == "few_fp8" else _nvfp4_weight
    for name, n, k in (("gate_up", 2 * i, h), ("down", h, i)):
        st[name] = tuple(torch.stack(parts) for parts in zip(*(make(g, n, k) for _ in range(e))))
    if case["op"] == "few_fp8":
        st["rows"] = _quantize_rows(st["x"])
        sh = case["shared"]
        st["shared_weights"] = (_fp8_weight(g, 2 * sh, h), _fp8_weight(g, h, sh)) if sh else None
        return st
    st["shared_out"] = torch.randn(t, h, generator=g, device="cuda").bfloat16() if case["shared"] else None
    if own:  # the tables of the experts' weights that a program makes when it loads them
        import moe_prefill_nvfp4_gb300 as moe

        st["cfg"] = moe.MoePrefillConfig(hidden=h, moe_intermediate=i, num_experts=e, top_k=case["top_k"], swiglu_limit=LIMIT,
                                         renormalize=1, routed_scale=1.0)
        st["tables"] = [moe.ExpertTable(list(st[name][0]), list(st[name][1]), st[name][2].tolist(), n, k)
                        for name, n, k in (("gate_up", 2 * i, h), ("down", h, i))]
    return st


# ------------------------------------------------------------------------------------------ one pass


def run(st):
    op = st["op"]
    if own:
        import moe_prefill_nvfp4_gb300 as moe

        if op == "norm":
            q, s, h, y = moe.moe_fp8_add_rms_norm(st["x"], st["weight"], st["residual"], eps=EPS, normed=st["normed"])
            return {"q": q, "s": s, "h": h, "y": y}
        routing = dict(w_router=st["w_router"], logits=st["logits"], router_bias=st["router_bias"])
        if op == "few_fp8":
            shared = st["shared_weights"] and (*st["shared_weights"][0], *st["shared_weights"][1])
            return moe.moe_fp8_few_forward(st["x"], *st["gate_up"], *st["down"], st["top_k"], rows=st["rows"],
                                           limit=LIMIT, shared=shared, **routing)
        return moe.moe_w4a16_few_forward(st["cfg"], st["x"], *st["tables"], shared_out=st["shared_out"], **routing)
    if op == "norm":
        return _norm_plain(st)
    return _few_fp8_plain(st) if op == "few_fp8" else _few_w4_plain(st)


# ------------------------------------------------------------------------------------------ the definition in 64 bits


def _round_e4m3_64(v):
    """Nearest E4M3 value (ties to even), by magnitude: steps of 2^(e-3) for 2^e <= |v|, e >= -6."""
    exponent = torch.frexp(v)[1].clamp(min=-5) - 1
    step = torch.ldexp(torch.ones_like(v), exponent - 3)
    return torch.clamp(torch.round(v / step) * step, -E4M3_MAX, E4M3_MAX)


def _codes_exact(x):
    """E4M3 values and scales of x [n, k], 128 columns to a scale."""
    s = torch.stack([c.abs().amax(1) for c in x.split(BLOCK, 1)], 1).clamp_min(AMAX_FLOOR) / E4M3_MAX
    parts = zip(x.split(BLOCK, 1), s.split(1, 1))
    return torch.cat([_round_e4m3_64(c / one) for c, one in parts], 1), s


def _rounded_exact(x):
    q, s = _codes_exact(x)
    return torch.cat([c * one for c, one in zip(q.split(BLOCK, 1), s.split(1, 1))], 1)


def _product_exact(x, st, name, e):
    """x [n, k] times expert e's weight, transposed; of the shared expert's (name: a pair of tensors) with e None."""
    if st["op"] == "few_fp8":
        q, s = name if e is None else (st[name][0][e], st[name][1][e])
        w = torch.cat([torch.cat([b.double() * c.double() for b, c in zip(line.split(BLOCK, 1), row)], 1)
                       for line, row in zip(q.split(BLOCK), s)])
        return x @ w.t()
    packed, scales, scale2 = (t[e] for t in st[name])
    bits = torch.stack([packed % 16, packed // 16], 2).reshape(packed.shape[0], -1).double()
    size = bits % 8
    # codes 0..3 are halves, then two binades with one bit each
    size = torch.where(size < 4, size / 2, torch.where(size < 6, size - 2, 2 * size - 8))
    v = torch.where(bits < 8, size, -size).view(packed.shape[0], -1, 16)
    return x @ (v * scales.view(torch.float8_e4m3fn).double()[..., None]).flatten(1).t() * scale2.double()


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "norm":
        h = st["x"].double() + (0.0 if st["residual"] is None else st["residual"].double())
        y = h / torch.sqrt(torch.einsum("rk,rk->r", h, h) / case["k"] + EPS)[:, None] * st["weight"].double()
        q, s = _codes_exact(y)
        return {"q": q, "s": s, "h": None if st["residual"] is None else h, "y": y if case["normed"] else None}
    x = st["x"].double()
    logits = st["logits"].double() if case["routed_by"] == "logits" else x @ st["w_router"].double().t()
    keys = logits if st["router_bias"] is None else logits + st["router_bias"].double()
    fp8 = case["op"] == "few_fp8"
    out = torch.zeros_like(x)
    if fp8:
        q, s = st["rows"]
        x = torch.cat([c.double() * one.double() for c, one in zip(q.split(BLOCK, 1), s.split(1, 1))], 1)
    held = {}
    for t in range(case["tokens"]):
        order = sorted(range(case["experts"]), key=lambda e, line=keys[t].tolist(): (-line[e], e))[: case["top_k"]]
        share = torch.softmax(logits[t, order], 0)
        for n, e in enumerate(order):
            held.setdefault(e, []).append((t, share[n]))

    def mlp(rows, gate_up, down, e):
        y = _product_exact(rows, st, gate_up, e)
        half = y.shape[1] // 2
        gate, up = y[:, :half].clamp(max=LIMIT), y[:, half:].clamp(-LIMIT, LIMIT)
        act = gate * torch.sigmoid(gate) * up
        return _product_exact(_rounded_exact(act) if fp8 else act, st, down, e)

    for e, rows in held.items():
        at = [t for t, _ in rows]
        out[at] += mlp(x[at], "gate_up", "down", e) * torch.stack([share for _, share in rows])[:, None]
    if fp8 and st["shared_weights"] is not None:
        out += mlp(x, *st["shared_weights"], None)
    if not fp8 and st["shared_out"] is not None:
        out += st["shared_out"].double()
    return out
