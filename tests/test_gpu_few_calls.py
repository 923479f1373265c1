"""GPU tests of the calls that the few-token layers allow: routing by a router, given rows, parts of the experts,
workspaces, streams, graphs, values that are not finite, and a decode step from the norm on (bounds: few_helpers)."""

import pytest
import torch

pytestmark = pytest.mark.gpu

import moe_prefill_nvfp4_gb300 as moe  # noqa: E402
from moe_prefill_nvfp4_gb300 import fp8  # noqa: E402

from few_helpers import Fp8Layer, W4Layer, assert_near, dequant_rows64, logits_of, rand  # noqa: E402
from test_gpu_rms_norm import check  # noqa: E402

BF16, F32, F8 = torch.bfloat16, torch.float32, torch.float8_e4m3fn


@pytest.fixture(autouse=True)
def _no_device_error():
    moe.moe_get_device_error()
    yield
    assert moe.moe_get_device_error() == 0


KINDS = ["fp8", "w4"]


def same(a, b):
    return torch.equal(a.contiguous().view(torch.uint8), b.contiguous().view(torch.uint8))


class Any:
    """Either kind of layer behind one call."""

    def __init__(self, kind, experts=16, hidden=1024, inter=512, top_k=4, seed=0, **kw):
        self.kind, self.top_k, self.experts, self.hidden, self.inter = kind, top_k, experts, hidden, inter
        self.layer = Fp8Layer(experts, hidden, inter, seed, **kw) if kind == "fp8" else W4Layer(experts, hidden, inter, top_k, seed, **kw)

    def run(self, x, **kw):
        return self.layer.run(x, self.top_k, **kw) if self.kind == "fp8" else self.layer.run(x, **kw)

    def ref(self, x, logits, **kw):
        return self.layer.ref(x, logits, self.top_k, **kw) if self.kind == "fp8" else self.layer.ref(x, logits, **kw)

    def ws_bytes(self, tokens):
        cfg = moe.MoePrefillConfig(hidden=self.hidden, moe_intermediate=self.inter, num_experts=self.experts, top_k=self.top_k)
        return moe.moe_few_workspace_bytes(cfg, tokens, self.kind == "fp8")


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("tokens,experts", [(1, 16), (2, 33), (5, 200), (16, 64)])
def test_router(kind, tokens, experts):
    """Logits whose sums are exact in any order: the router's are the given ones'."""
    layer = Any(kind, experts, 512, 256, 3)
    g = torch.Generator(device="cuda").manual_seed(tokens)
    x = torch.randint(-4, 5, (tokens, 512), generator=g, device="cuda").to(BF16) / 4
    w = torch.randint(-8, 9, (experts, 512), generator=g, device="cuda").to(BF16) / 8
    logits, bias = (x.double() @ w.double().t()).float(), logits_of(1, experts, 7)[0]
    want = layer.run(x, logits=logits, router_bias=bias)
    assert torch.equal(layer.run(x, w_router=w, router_bias=bias), want)
    assert_near(want, *layer.ref(x, logits, bias=bias))


@pytest.mark.parametrize("tokens", [1, 3, 16])
def test_given_rows(tokens):
    """Codes and scales of any layout, x left out: the same bits as of x."""
    layer = Any("fp8", 8, 640, 384, 2, shared=128)
    x, logits = rand((tokens, 640), 3), logits_of(tokens, 8, 4)
    want = layer.run(x, logits=logits)
    q, s = moe.moe_fp8_quantize_rows(x)
    assert torch.equal(layer.run(None, rows=(q, s), logits=logits), want)
    wide = torch.zeros(tokens, 1024, dtype=torch.uint8, device="cuda").view(F8)
    wide[:, 128:768].copy_(q)
    across = torch.zeros(7, tokens + 5, device="cuda")
    across[1:6, 2:tokens + 2] = s.t()
    assert torch.equal(layer.run(None, rows=(wide[:, 128:768], across[1:6, 2:tokens + 2].t()), logits=logits), want)
    other = rand((tokens, 640), 5)  # (x is the router's alone)
    w = rand((8, 640), 6, 0.1)
    ids, wts = moe.moe_route_topk(moe.moe_router_logits(other, w), 2)
    got = layer.run(other, rows=(q, s), w_router=w)
    assert_near(got, *layer.ref(x, (other.double() @ w.double().t()).float(), rows=(q, s)))


@pytest.mark.parametrize("tokens", [1, 9])
def test_parts_of_the_experts(tokens):
    """Two parts with weights of their own strides: each against its experts, a part that no token picked gives zeros."""
    layer = Any("fp8", 12, 512, 256, 3, shared=256)
    x, logits = rand((tokens, 512), 3), logits_of(tokens, 12, 4)
    (gq, gs), (dq, ds) = layer.layer.gu, layer.layer.dn
    for first, count in ((0, 5), (5, 7)):
        out = moe.moe_fp8_few_forward(x, gq[first:first + count], gs[first:first + count], dq[first:first + count],
                                      ds[first:first + count], 3, logits=logits, num_experts=12, first=first,
                                      shared=layer.layer.shared if first == 0 else None)
        assert_near(out, *layer.ref(x, logits, held=range(first, first + count), with_shared=first == 0))
    logits[:, 9:] = -100.0
    out = torch.full((tokens, 512), 5.0, dtype=BF16, device="cuda")
    moe.moe_fp8_few_forward(x, gq[9:12], gs[9:12], dq[9:12], ds[9:12], 3, logits=logits, num_experts=12, first=9, out=out)
    assert (out == 0).all()


@pytest.mark.parametrize("tokens", [1, 9])
def test_absent_experts_and_a_shared_result(tokens):
    layer = Any("w4", 12, 512, 256, 3, absent=(0, 4, 5, 11))
    x, logits, shared = rand((tokens, 512), 3), logits_of(tokens, 12, 4), rand((tokens, 512), 5)
    assert_near(layer.run(x, logits=logits), *layer.ref(x, logits))
    assert_near(layer.run(x, logits=logits, shared_out=shared), *layer.ref(x, logits, shared_out=shared))
    assert torch.equal(layer.run(x, logits=logits, shared_out=(y := shared.clone()), out=y), layer.run(x, logits=logits, shared_out=shared))
    logits[:, [0, 4, 5]] = 100.0  # nothing that is here
    assert (layer.run(x, logits=logits) == 0).all()
    assert torch.equal(layer.run(x, logits=logits, shared_out=shared), shared)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("limit", [0.25, float("inf")])
def test_limits_and_weights(kind, limit):
    x, logits, bias = rand((4, 1024), 3, 3.0), logits_of(4, 16, 4), 3 * logits_of(1, 16, 5)[0]
    if kind == "fp8":
        layer = Any("fp8", shared=128)
        out = layer.run(x, logits=logits, router_bias=bias, limit=limit, shared_limit=0.5, renormalize=False, routed_scale=2.5)
        ref = layer.ref(x, logits, bias=bias, limit=limit, shared_limit=0.5, renormalize=False, scale=2.5)
    else:
        layer = Any("w4", limit=limit, renormalize=0, routed_scale=2.5)
        out, ref = layer.run(x, logits=logits, router_bias=bias), layer.ref(x, logits, bias=bias)
    assert_near(out, *ref)


@pytest.mark.parametrize("kind", KINDS)
def test_rows_of_very_different_columns(kind):
    """Columns a thousand times the others', groups of zeros, and magnitudes at both ends."""
    layer = Any(kind)
    x = rand((6, 1024), 3)
    x[0, ::37] *= 1000
    x[1, 128:640] = 0
    x[2] *= torch.logspace(-6, 2, 1024, device="cuda").to(BF16)
    x[3] *= 2.0 ** -60
    x[4] *= 2.0 ** 20
    x[5] = 0
    logits = logits_of(6, 16, 4)
    out = layer.run(x, logits=logits)
    assert_near(out[:5], *(v[:5] for v in layer.ref(x, logits)))
    assert (out[5] == 0).all()


@pytest.mark.parametrize("kind", KINDS)
def test_values_that_are_not_finite_stay_in_their_row(kind):
    layer = Any(kind)
    x, logits = rand((7, 1024), 3), logits_of(7, 16, 4)
    clean = layer.run(x, logits=logits)
    x[1, 5], x[3, 1000], x[4, 130] = float("nan"), float("inf"), -float("inf")
    out = layer.run(x, logits=logits)
    for t in range(7):
        assert out[t].isnan().all() if t in (1, 3, 4) else torch.equal(out[t], clean[t])


@pytest.mark.parametrize("kind", KINDS)
def test_all_tokens_pick_the_same_experts(kind):
    layer = Any(kind, 32, 512, 256, 2)
    x, logits = rand((16, 512), 3), logits_of(1, 32, 4).expand(16, -1).contiguous()
    assert_near(layer.run(x, logits=logits), *layer.ref(x, logits))
    same = rand((1, 512), 5).expand(16, -1).contiguous()
    out = layer.run(same, logits=logits)
    assert torch.equal(out, out[:1].expand(16, -1))


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("tokens", [1, 16])
def test_workspace(kind, tokens):
    """Whatever is in it, exactly as large as asked for, bytes around it stay, and calls in turn share it."""
    layer = Any(kind)
    x, logits = rand((tokens, 1024), 3), logits_of(tokens, 16, 4)
    want, n = layer.run(x, logits=logits), layer.ws_bytes(tokens)
    for fill in (0, 0xFF, 0x7F):
        whole = torch.full((n + 512,), fill, dtype=torch.uint8, device="cuda")
        ws = whole[256:256 + n]
        for _ in range(3):
            assert torch.equal(layer.run(x, logits=logits, ws=ws), want)
        assert (whole[:256] == fill).all() and (whole[256 + n:] == fill).all()
    with pytest.raises(moe.MoeError):
        layer.run(x, logits=logits, ws=ws[:-256])


@pytest.mark.parametrize("kind", KINDS)
def test_calls_of_other_sizes_in_turn_on_one_workspace(kind):
    """Nothing of an earlier call is taken for this one's: an SM's cache, a counter, a row."""
    layers = [Any(kind, 16, 1024, 512, 4), Any(kind, 40, 512, 256, 8, seed=50)]
    ws = torch.empty(max(la.ws_bytes(16) for la in layers), dtype=torch.uint8, device="cuda")
    cases = [(la, t, rand((t, la.hidden), t), logits_of(t, la.experts, t + 1)) for t in (1, 16, 3, 7) for la in layers]
    want = [la.run(x, logits=lg) for la, _, x, lg in cases]
    for _ in range(20):
        for (la, _, x, lg), w in zip(cases, want):
            assert torch.equal(la.run(x, logits=lg, ws=ws), w)


@pytest.mark.parametrize("kind", KINDS)
def test_graph(kind):
    """Captured once, replayed on other tokens and routes; a second graph replays in between."""
    layer = Any(kind)
    x, logits, w = rand((5, 1024), 3), logits_of(5, 16, 4), rand((16, 1024), 5, 0.05)
    layer.run(x, logits=logits)
    graphs = []
    for kw in (dict(logits=logits), dict(w_router=w)):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = layer.run(x, **kw)
        graphs.append((g, out, kw))
    for i in range(6):
        x.copy_(rand((5, 1024), 20 + i))
        logits.copy_(logits_of(5, 16, 30 + i))
        for g, out, kw in graphs:
            g.replay()
            got = out.clone()
            assert torch.equal(got, layer.run(x, **kw))


@pytest.mark.parametrize("kind", KINDS)
def test_stream_that_is_not_current(kind):
    layer = Any(kind)
    x, logits = rand((3, 1024), 3), logits_of(3, 16, 4)
    want = layer.run(x, logits=logits)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    outs = []
    for _ in range(10):
        outs.append(layer.run(x, logits=logits, stream=side))
        torch.full((1 << 22,), 0x7F, dtype=torch.uint8, device="cuda")  # (takes what the current stream's pool has free)
    side.synchronize()
    for out in outs:
        assert torch.equal(out, want)


def test_two_layers_at_once():
    """On two streams, with a workspace each: both finish, with the bits that they have alone."""
    layers = [Any("fp8", 32, 2048, 512, 8), Any("w4", 32, 2048, 512, 8, seed=40)]
    x, logits = rand((16, 2048), 3), logits_of(16, 32, 4)
    want = [la.run(x, logits=logits) for la in layers]
    streams = [torch.cuda.Stream() for _ in layers]
    torch.cuda.synchronize()
    outs = [[], []]
    for _ in range(100):
        for la, st, o in zip(layers, streams, outs):
            with torch.cuda.stream(st):
                o.append(la.run(x, logits=logits))
    torch.cuda.synchronize()
    for o, w in zip(outs, want):
        assert all(torch.equal(v, w) for v in o)


@pytest.mark.parametrize("kind", KINDS)
def test_no_tokens(kind):
    out = Any(kind).run(torch.zeros(0, 1024, dtype=BF16, device="cuda"), logits=torch.zeros(0, 16, device="cuda"))
    assert out.shape == (0, 1024)


@pytest.mark.parametrize("kind", KINDS)
def test_refusals(kind):
    layer = Any(kind)
    x, logits = rand((4, 1024), 3), logits_of(4, 16, 4)
    wide = torch.zeros(4, 2048, dtype=BF16, device="cuda")
    for bad in (dict(logits=logits[:, :15]), dict(logits=logits.half()), dict(logits=logits.cpu()), dict(out=wide[:, :1024]),
                dict(out=torch.zeros(4, 1024, device="cuda")), dict(router_bias=logits[0, :3]), dict(x=wide[:, :1024])):
        with pytest.raises(ValueError):
            layer.run(**{**dict(x=x, logits=logits), **bad})
    for bad in (dict(x=rand((17, 1024), 1), logits=logits_of(17, 16, 2)), dict(logits=None), dict(w_router=rand((16, 1024), 1))):
        with pytest.raises(moe.MoeError):
            layer.run(**{**dict(x=x, logits=logits), **bad})


def make(experts, hidden, inter, shared):
    (sg,), (sd,) = rand((1, 2 * shared, hidden), 20, hidden ** -0.5), rand((1, hidden, shared), 21, shared ** -0.5)
    gu, dn = rand((experts, 2 * inter, hidden), 22, hidden ** -0.5), rand((experts, hidden, inter), 23, inter ** -0.5)
    w = fp8.Fp8Weight.quantise
    return fp8.Fp8Experts(w(gu), w(dn), 4, shared=fp8.Fp8SharedExpert(w(sg), w(sd), 5.0), routed_scale=2.0)


def ref_of(experts, x, logits, rows):
    layer = Fp8Layer.__new__(Fp8Layer)
    layer.gu, layer.dn = (experts.gate_up.q, experts.gate_up.s), (experts.down.q, experts.down.s)
    sh = experts.shared
    layer.shared, layer.experts = (sh.gate_up.q, sh.gate_up.s, sh.down.q, sh.down.s), experts.num_experts
    return layer.ref(x, logits, 4, limit=7.0, shared_limit=5.0, scale=2.0, rows=rows)


@pytest.mark.parametrize("tokens", [1, 4, 16])
def test_decode_steps(tokens):
    """Two layers of a residual stream: norm with its quantiser -> router and experts -> the next norm, which adds their result.
    Captured, and each product against FP64 on what went into it."""
    layers = [make(24, 1280, 384, 256), make(24, 1280, 384, 256)]
    x, w, routers = rand((tokens, 1280), 1), 1 + rand((1280,), 2, 0.2), [rand((24, 1280), 3 + i, 0.03) for i in (0, 1)]
    stream = rand((tokens, 1280), 9, 4.0, F32)

    def steps():
        seen, y, h = [], x, stream
        for la, router in zip(layers, routers):
            q, s, h, normed = moe.moe_fp8_add_rms_norm(y, w, h, normed=True)
            y = la.forward_few(normed, router, rows=(q, s))
            seen.append((q, s, h, normed, y))
        return seen

    eager = steps()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        seen = steps()
    for _ in range(3):
        g.replay()
    torch.cuda.synchronize()
    before, h = x, stream
    for (q, s, hh, normed, y), e, la, router in zip(seen, eager, layers, routers):
        assert all(same(a, b) for a, b in zip((q, s, hh, normed, y), e))
        assert torch.equal(hh, before.float() + h)
        logits = moe.moe_router_logits(normed, router)
        # (the call's own logits are sums in another order; its picks are these, whose keys lie further apart than that)
        top = logits.sort(1, descending=True).values
        assert ((top[:, 3] - top[:, 4]) > 1e-4).all()
        out, tol = ref_of(la, normed, logits, (q, s))
        dl = 2 * 1280 * 2.0 ** -24 * (normed.double().abs() @ router.double().abs().t()).max()
        assert_near(y, out, tol + 4 * dl * magnitude(la, normed, logits, (q, s)))
        # the chunk path on the same rows: other orders of sums and other roundings of the same sums
        chunk = la.forward(normed, logits=logits, rows=(q, s))
        assert float((chunk.double() - out).norm() / out.norm()) < 2.0 ** -6
        before, h = y, hh


def magnitude(la, x, logits, rows):
    """sum_s w |y_s| of the routed experts, which a weight's error multiplies."""
    total = torch.zeros(x.shape, dtype=torch.float64, device="cuda")
    ids, _ = moe.moe_route_topk(logits, 4)
    plain = fp8.Fp8Experts(la.gate_up, la.down, 1, limit=la.limit, routed_scale=la.routed_scale)
    for s in range(4):
        alone = torch.full_like(logits, -50.0).scatter(1, ids[:, s:s + 1].long(), 50.0)
        total += plain.forward_few(None, logits=alone, rows=rows).double().abs()
    return total


def test_chunk_with_given_rows():
    la = make(24, 1280, 384, 256)
    x, logits = rand((70, 1280), 1), logits_of(70, 24, 2)
    assert torch.equal(la.forward(x, logits=logits, rows=moe.moe_fp8_quantize_rows(x)), la.forward(x, logits=logits))


@pytest.mark.parametrize("tokens", [1, 6])
def test_forward_few_on_a_stream(tokens):
    la = make(24, 1280, 384, 256)
    x, logits = rand((tokens, 1280), 1), logits_of(tokens, 24, 2)
    want, side = la.forward_few(x, logits=logits), torch.cuda.Stream()
    torch.cuda.synchronize()
    got = la.forward_few(x, logits=logits, stream=side)
    side.synchronize()
    assert torch.equal(got, want)
    assert_near(want, *ref_of(la, x, logits, moe.moe_fp8_quantize_rows(x)))


def test_norm_on_streams_and_in_graphs():
    x, r, w = rand((300, 2048), 1), rand((300, 2048), 2), rand((2048,), 3)
    want = moe.moe_fp8_add_rms_norm(x, w, r, normed=True)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = moe.moe_fp8_add_rms_norm(x, w, r, normed=True, stream=side)
    side.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        captured = moe.moe_fp8_add_rms_norm(x, w, r, normed=True)
    g.replay()
    torch.cuda.synchronize()
    for a, b, c in zip(want, got, captured):
        assert same(a, b) and same(a, c)


@pytest.mark.parametrize("k", [512, 8320, 16512, 32768])
def test_norm_codes_are_the_nearest(k):
    """Codes of h w * 448 / max |h w| in FP64, but where that lies within 2^-22 of the middle between two codes: the
    product is off by 2^-44, its one rounding by 2^-24."""
    x, r, w = rand((500, k), 1, 1.0, F32), rand((500, k), 2), 1 + rand((k,), 3, 0.3, F32)
    q, s, _, _ = moe.moe_fp8_add_rms_norm(x, w, r)
    v = ((x + r).double() * w.double()).view(500, -1, 128)
    v = (v * (448 / v.abs().amax(-1, keepdim=True))).view(500, k)
    got = dequant_rows64(q, torch.ones_like(s)).cuda()
    step = torch.ldexp(torch.ones_like(v), torch.frexp(v.abs().clamp(min=2.0 ** -6))[1] - 4)
    assert ((got - v).abs() <= step / 2 + v.abs() * 2.0 ** -22).all()


@pytest.mark.parametrize("rows,k,x_type,r_type", [(400, 32768, F32, F32), (3000, 640, BF16, BF16), (2000, 1000, F32, F32), (5000, 8, BF16, None)])
def test_norm_of_many_rows(rows, k, x_type, r_type):
    """More rows than CTAs that the GPU holds: rows too long for shared memory, several to a CTA, the shortest."""
    x, w = rand((rows, k), 1, 0.5, x_type), 1 + rand((k,), 2, 0.3, F32)
    r = None if r_type is None else rand((rows, k), 3, 2.0, r_type)
    check(x, w, r, 1e-5, *moe.moe_fp8_add_rms_norm(x, w, r, eps=1e-5, normed=True))
