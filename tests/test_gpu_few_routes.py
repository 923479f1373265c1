"""GPU tests of the few-token layers on uneven routes: the routing's warps have 64 experts each, and what any of them
finds to be the most tokens of an expert is what every product's accumulators are laid out for.  Each route is run many
times, since every CTA of every call routes by itself: equal bits, and near FP64 (bounds: few_helpers)."""

import functools

import pytest
import torch

pytestmark = pytest.mark.gpu

import moe_prefill_nvfp4_gb300 as moe  # noqa: E402

from few_helpers import Fp8Layer, W4Layer, assert_near, logits_of, rand  # noqa: E402

CALLS = 150
HIDDEN, INTER = 256, 256


@pytest.fixture(autouse=True)
def _no_device_error():
    moe.moe_get_device_error()
    yield
    assert moe.moe_get_device_error() == 0


@functools.lru_cache(maxsize=1)
def layer_of(kind, experts, top_k):
    if kind == "fp8":
        layer = Fp8Layer(experts, HIDDEN, INTER, 7)
        return (lambda x, **kw: layer.run(x, top_k, **kw)), (lambda x, logits: layer.ref(x, logits, top_k))
    layer = W4Layer(experts, HIDDEN, INTER, top_k, 7)
    return layer.run, layer.ref


def logits_for(picks, experts):
    """Logits [T, E] of which row t's largest are at picks[t]."""
    logits = logits_of(len(picks), experts, 11) - 40.0
    for t, row in enumerate(picks):
        logits[t, list(row)] += 40.0
    return logits


def together(tokens, experts, top_k, warp):
    """All tokens pick the same experts, all of one warp."""
    return [range(64 * warp + 1, 64 * warp + 1 + top_k) if experts > 65 else [64] for _ in range(tokens)]


def one_popular(tokens, experts, top_k, warp):
    """One expert of the warp has every token; their other picks are spread over the others', a token or two each."""
    popular = min(64 * warp + 37, experts - 1)
    others = [e for e in range(experts) if e // 64 != warp]
    step = 7  # (coprime to the lists' lengths)
    return [[popular] + [others[(step * (t * (top_k - 1) + i)) % len(others)] for i in range(top_k - 1)] for t in range(tokens)]


def growing(tokens, experts, top_k, warp):
    """Counts from one token up to all of them, the largest in the given warp, smaller ones in the warps before it."""
    at = [64 * w + 5 for w in range(warp + 1)] + [64 * warp + 20 + i for i in range(32)]
    rows = []
    for t in range(tokens):
        row = [64 * warp + 60 if 64 * warp + 60 < experts else experts - 1]
        row += [e for i, e in enumerate(at) if t <= i * 3 and e < experts and e not in row][: top_k - 1]
        row += [e for e in range(experts) if e not in row][: top_k - len(row)]
        rows.append(row)
    return rows


ROUTES = dict(together=together, one_popular=one_popular, growing=growing)
SIZES = [(65, 1), (160, 4), (512, 8)]


@pytest.mark.parametrize("kind,experts,top_k,warp", [(kind, e, k, w) for kind in ("w4", "fp8") for e, k in SIZES
                                                     for w in range(-(-e // 64)) if kind == "w4" or w in (1, 7)])
def test_the_most_tokens_of_an_expert_in_any_warp(kind, experts, top_k, warp):
    run, ref = layer_of(kind, experts, top_k)
    for name, route in ROUTES.items():
        if experts == 65 and warp == 0 and name == "together":
            continue
        for tokens in (1, 3, 6, 16):
            picks = route(tokens, experts, top_k, warp)
            assert all(len(set(row)) == top_k and max(row) < experts for row in picks)
            x, logits = rand((tokens, HIDDEN), 20 + tokens), logits_for(picks, experts)
            outs = [run(x, logits=logits) for _ in range(CALLS)]
            want, tol = ref(x, logits)
            assert_near(outs[0], want, tol)
            for out in outs[1:]:
                assert torch.equal(out, outs[0]), (name, tokens)


@pytest.mark.parametrize("tokens", [2, 16])
def test_shared_expert_of_all_tokens(tokens):
    """A shared expert has every token, beside routed ones of one token each in a later warp."""
    layer = Fp8Layer(160, HIDDEN, INTER, 9, shared=128)
    picks = [[70 + 4 * t + i for i in range(4)] for t in range(tokens)]
    x, logits = rand((tokens, HIDDEN), 1), logits_for(picks, 160)
    want, tol = layer.ref(x, logits, 4)
    outs = [layer.run(x, 4, logits=logits) for _ in range(CALLS)]
    assert_near(outs[0], want, tol)
    assert all(torch.equal(out, outs[0]) for out in outs)
