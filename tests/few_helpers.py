"""Layers of experts for a few tokens in FP64, with how far an FP32 evaluation may be from them.

A sum over k columns: the products are exact in FP32 (E4M3 and E2M1 x E4M3 codes, FP16 values), a group of 128 is
added in the MMA, each addition off by at most 2^-23 of the sum of magnitudes (truncation allowed); then KB groups
by FMAs and eight warps' parts by additions, 2^-24 each, and the scales' product:
    (128 * 2^-23 + (KB + 12) * 2^-24) * sum |a w|.
NVFP4: a value is the sum of six pieces of at most 2 significant bits, each the rest of the ones before it rounded.
A piece that is not zero is at most twice its rest (zero could be chosen too), leaves no more than the rest itself, and from
the second on at most a half of a step where the step is an eighth of the rest's or less: the magnitudes add up to at most 5
times the value's, 2 + 2 + 2 / 8 + ... .  A block of 256 is added in the MMA, then the six by FMAs, KB blocks by FMAs, and
at most KB slices by additions:
    5 * (256 * 2^-23 + (2 KB + 8) * 2^-24) * sum |a w|.
The activation silu(g) u: 1.1 |u| dg + |silu(g)| du + 2^-20 |act| (|silu'| <= 1.1; the clamps do not widen).
FP8: a quantised activation is its code times its scale; the scale is off as its group's largest activation is, and
a value that lies that close to the middle between two codes may get either.
NVFP4: what the pieces leave of a value is at most 2^-15 s, s the power of two with 3 s < max <= 6 s of its 16 columns, so
2^-15 / 3 of the largest magnitude of those; or, where s is below 2^-14 of that of the block of 256, 2^-29 / 3 of its largest;
or, where all are below 2^-115, 2^-133 (s >= 2^-118).
The weighted sum: the weights to 2^-20 (exponentials, their sum, a division), k + 1 additions; one rounding to BF16, 2^-8,
or below 2^-126, where BF16 numbers are 2^-133 apart, 2^-134.
"""

import torch

import moe_prefill_nvfp4_gb300 as moe

from test_gpu_fp8 import dequant_blocks64, dequant_rows64, rand, weights  # noqa: F401


def sum_bound(k):
    return 128 * 2.0 ** -23 + (-(-k // 128) + 12) * 2.0 ** -24


def sum_bound_pieces(k):
    return 5 * (256 * 2.0 ** -23 + (2 * -(-k // 256) + 8) * 2.0 ** -24)


def step_e4m3(v):
    """Distance of neighbouring E4M3 numbers at magnitude v."""
    return torch.ldexp(torch.ones_like(v), torch.frexp(v.clamp(min=2.0 ** -6))[1] - 4)


def quantised64(a, da):
    """Activations [n, I] and their bounds through the row quantiser: values and bounds."""
    n, inter = a.shape
    g, dg = a.view(n, -1, 128), da.view(n, -1, 128)
    amax = g.abs().amax(-1, keepdim=True).clamp(min=2.0 ** -100)
    s, ds = amax / 448, dg.amax(-1, keepdim=True) / 448 + amax * 2.0 ** -23 / 448
    v = g / s
    dv = dg / s + v.abs() * (ds / s + 2.0 ** -22)
    step = step_e4m3(v.abs() + dv)
    code = torch.round(v.abs() / step_e4m3(v.abs())) * step_e4m3(v.abs()) * v.sign()
    code = code.clamp(-448, 448)
    frac = v.abs() / step_e4m3(v.abs())
    near = ((frac - frac.floor() - 0.5).abs() * step_e4m3(v.abs()) <= dv) | (dv > step / 4)
    # (at a binade's lower end the middle between two codes lies half a smaller step below)
    near |= (torch.frexp(v.abs() + dv)[1] != torch.frexp(v.abs() - dv)[1]) & (v.abs() > 2.0 ** -6)
    bound = code.abs() * ds + torch.where(near, step * (s + ds) + dv * s, torch.zeros_like(v))
    return (code * s).view(n, inter), bound.view(n, inter)


def pieces64(a, da):
    """Values [n, K] and their bounds as sums of six pieces."""
    n, k = a.shape
    of16 = (a.abs() + da).view(n, -1, 16).amax(-1, keepdim=True).expand(n, k // 16, 16).reshape(n, k)
    of256 = (a.abs() + da).view(n, -1, 256).amax(-1, keepdim=True).expand(n, k // 256, 256).reshape(n, k)
    return a, da + of16 * (2.0 ** -15 / 3) + of256 * (2.0 ** -29 / 3) + 2.0 ** -133


def mlp64(rows, gate_up, down, limit, through, drows=None, bound=sum_bound):
    """SwiGLU MLP of FP64 weights on rows [n, H]: (y, bound)."""
    inter = down.shape[1]
    y, mag = rows @ gate_up.t(), rows.abs() @ gate_up.abs().t()
    dy = bound(rows.shape[1]) * mag
    if drows is not None:
        dy = dy + drows @ gate_up.abs().t()
    g, u = y[:, :inter].clamp(max=limit), y[:, inter:].clamp(-limit, limit)
    silu = g / (1 + torch.exp(-g))
    act = silu * u
    dact = 1.1 * u.abs() * dy[:, :inter] + silu.abs() * dy[:, inter:] + 1.1 * dy[:, :inter] * dy[:, inter:] + 2.0 ** -20 * act.abs()
    a, da = through(act, dact)
    return a @ down.t(), da @ down.abs().t() + bound(inter) * (a.abs() @ down.abs().t())


def layer64(rows, ids, wts, gate_up, down, limit, through, shared=None, held=None, drows=None, bound=sum_bound):
    """(out, tolerance of a BF16 result) of FP64 rows [T, H]; gate_up(e), down(e): FP64 weights of expert e; shared:
    (y, bound) to add; held: the experts that count."""
    out, tol = torch.zeros_like(rows), torch.zeros_like(rows)
    k = ids.shape[1]
    for e in ids.unique().tolist():
        if held is not None and e not in held:
            continue
        t, s = (ids == e).nonzero(as_tuple=True)
        y, dy = mlp64(rows[t], gate_up(e), down(e), limit, through, None if drows is None else drows[t], bound)
        w = wts[t, s].double()[:, None]
        out.index_add_(0, t, y * w)
        tol.index_add_(0, t, dy * w.abs() + (2.0 ** -20 + (k + 1) * 2.0 ** -24) * (y * w).abs())
    if shared is not None:
        out, tol = out + shared[0], tol + shared[1]
    return out, tol * (1 + 2.0 ** -8) + out.abs() * 2.0 ** -8 + 2.0 ** -134


def assert_near(got, ref, tol):
    d = (got.double() - ref).abs()
    bad = ~(d <= tol)
    assert not bad.any(), (int(bad.sum()), torch.nonzero(bad)[:4].tolist(), d[bad][:4].tolist(), tol[bad][:4].tolist(),
                           float(((got.double() - ref).norm() / ref.norm())))


def logits_of(tokens, experts, seed):
    return rand((tokens, experts), seed, 1.0, torch.float32)


class Fp8Layer:
    def __init__(self, experts, hidden, inter, seed=0, shared=0):
        self.gu, self.dn = weights(experts, 2 * inter, hidden, seed), weights(experts, hidden, inter, seed + 1000)
        self.shared = None
        if shared:
            (gq, gs), (dq, ds) = weights(1, 2 * shared, hidden, seed + 2000), weights(1, hidden, shared, seed + 2001)
            self.shared = (gq[0], gs[0], dq[0], ds[0])
        self.experts = experts

    def weight(self, which, e):
        return dequant_blocks64(which[0][e], which[1][e]).cuda()

    def ref(self, x, logits, top_k, limit=7.0, shared_limit=None, bias=None, renormalize=True, scale=1.0, held=None,
            rows=None, with_shared=True):
        ids, wts = moe.moe_route_topk(logits, top_k, bias, renormalize, scale)
        q, s = rows if rows is not None else moe.moe_fp8_quantize_rows(x)
        r = dequant_rows64(q, s).cuda()
        sh = None
        if self.shared is not None and with_shared:
            sh = mlp64(r, dequant_blocks64(*self.shared[:2]).cuda(), dequant_blocks64(*self.shared[2:]).cuda(),
                       limit if shared_limit is None else shared_limit, quantised64)
        return layer64(r, ids.long(), wts, lambda e: self.weight(self.gu, e), lambda e: self.weight(self.dn, e), limit,
                       quantised64, sh, held)

    def run(self, x, top_k, **kw):
        return moe.moe_fp8_few_forward(x, *self.gu, *self.dn, top_k, shared=self.shared, **kw)


VALUES = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6, 0, -0.5, -1, -1.5, -2, -3, -4, -6], dtype=torch.float64)


def nvfp4(n, k, seed):
    """Random codes and block scales of about unit spread over k^1/2, and the tensor's scale."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    packed = torch.randint(0, 256, (n, k // 2), generator=g, device="cuda").to(torch.uint8)
    scales = torch.rand(n, k // 16, generator=g, device="cuda") * 1.5 + 0.25
    scales[torch.rand(n, k // 16, generator=g, device="cuda") < 0.02] = 0.0
    return packed, scales.to(torch.float8_e4m3fn).view(torch.uint8), 0.37 * k ** -0.5 * (1 + seed % 3)


def dequant_nvfp4(packed, scales, scale2):
    codes = torch.stack([packed & 15, packed >> 4], -1).flatten(-2).long()
    return VALUES.cuda()[codes] * scales.view(torch.float8_e4m3fn).double().repeat_interleave(16, -1) * float(torch.tensor(scale2).float())


class W4Layer:
    def __init__(self, experts, hidden, inter, top_k, seed=0, absent=(), limit=7.0, **cfg):
        self.gu = [nvfp4(2 * inter, hidden, seed + e) for e in range(experts)]
        self.dn = [nvfp4(hidden, inter, seed + 1000 + e) for e in range(experts)]
        self.absent, self.limit = absent, limit
        table = lambda w, n, k: moe.ExpertTable(*([None if e in absent else w[e][i] for e in range(experts)] for i in (0, 1)),  # noqa: E731
                                                [v[2] for v in w], n, k)
        self.tables = table(self.gu, 2 * inter, hidden), table(self.dn, hidden, inter)
        self.cfg = moe.MoePrefillConfig(hidden=hidden, moe_intermediate=inter, num_experts=experts, top_k=top_k, swiglu_limit=limit,
                                        **{**dict(renormalize=1, routed_scale=1.0), **cfg})
        self.top_k, self.held = top_k, [e for e in range(experts) if e not in absent]

    def ref(self, x, logits, bias=None, shared_out=None):
        ids, wts = moe.moe_route_topk(logits, self.top_k, bias, bool(self.cfg.renormalize), self.cfg.routed_scale)
        sh = None if shared_out is None else (shared_out.double(), 2.0 ** -24 * shared_out.double().abs())
        rows = x.double()
        return layer64(rows, ids.long(), wts, lambda e: dequant_nvfp4(*self.gu[e]), lambda e: dequant_nvfp4(*self.dn[e]),
                       self.limit, pieces64, sh, self.held, pieces64(rows, torch.zeros_like(rows))[1], sum_bound_pieces)

    def run(self, x, **kw):
        return moe.moe_w4a16_few_forward(self.cfg, x, *self.tables, **kw)
