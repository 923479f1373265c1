"""The gate/up product's activation over the whole range of gates, in both kernels (few rows, wide tiles).

Each sum has one product of codes with power-of-two scales, so gate and up are exact in FP32 and what is seen is
silu(min(g, L)) * clamp(u, -L, L) and its quantisation: within 2^-20 of FP64 (the wide kernel's approximate power
of two 2^-22, its argument's correction 2^-21.3 at gates of -85, its reciprocal 2^-23, two products 2^-24 each:
2^-20.1 in all), the scale 2^-23 for the division by 448 and the product.  One gate to a group of 128, so that
every group's scale shows its value; the groups' largest |u| is 1.

A code stands for a value within half a step: 2^-4 of the value or 2^-10 scales."""

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

import moe_prefill_nvfp4_gb300 as moe  # noqa: E402

BLOCK = 128
FLOOR = 2.0 ** -100
REL = 2.0 ** -20 + 2.0 ** -23


@pytest.fixture(autouse=True)
def _no_device_error():
    moe.moe_get_device_error()
    yield
    assert moe.moe_get_device_error() == 0


def e4m3():
    """The positive E4M3 values."""
    return torch.arange(1, 127, dtype=torch.uint8).view(torch.float8_e4m3fn).double()


def case(rows, factors, gate_scale, up_scale=1.0):
    """Rows t (cycling through the E4M3 values a_t) and one group of 128 columns to each factor w:
    g = gate_scale a_t w, u = up_scale u_j with u_j running over E4M3 values up to 1."""
    a = e4m3()[torch.arange(rows) % 126]
    w = torch.tensor(factors, dtype=torch.float64)
    inter = BLOCK * len(factors)
    u = e4m3()[:BLOCK]
    u = torch.cat([u[u <= 1], -u[u <= 1]])
    u = u[torch.arange(inter) % len(u)]
    A = torch.zeros(rows, 256)
    A[:, 0], A[:, BLOCK] = a.float(), 1.0
    W = torch.zeros(2 * inter, 256)
    W[:inter, 0] = w.repeat_interleave(BLOCK).float()
    W[inter:, BLOCK] = u.float()
    q, wq = A.cuda().to(torch.float8_e4m3fn), W.cuda().to(torch.float8_e4m3fn)[None]
    assert torch.equal(q.float().cpu(), A) and torch.equal(wq[0].float().cpu(), W)  # E4M3 values all
    s = torch.tensor([gate_scale, up_scale], dtype=torch.float32).expand(rows, 2).contiguous().cuda()
    ws = torch.ones(1, 2 * inter // BLOCK, 2, device="cuda")
    g = gate_scale * a[:, None] * w.repeat_interleave(BLOCK)[None]
    return q, s, wq, ws, g, (up_scale * u)[None].expand(rows, inter)


def check(rows, factors, gate_scale, limit, gather, up_scale=1.0):
    q, s, wq, ws, g, u = case(rows, factors, gate_scale, up_scale)
    off = torch.tensor([0, rows], dtype=torch.int32, device="cuda")
    ids = torch.arange(rows, dtype=torch.int32, device="cuda") if gather else None
    codes, scales = moe.moe_fp8_grouped_gemm_swiglu(q, s, wq, ws, off, rows, limit=limit, gather_ids=ids)
    gm, uc = g.clamp(max=limit), u.clamp(-limit, limit)
    act = gm / (1.0 + torch.exp(-gm)) * uc
    high = act.abs().view(rows, -1, BLOCK).amax(-1).clamp_min(FLOOR)
    sc = scales.double().cpu()
    rel = (sc * 448 / high - 1).abs()
    assert (rel <= REL).all(), (float(rel.max()), g.view(rows, -1, BLOCK)[..., 0][rel > REL][:8])
    each = sc.repeat_interleave(BLOCK, -1)
    apart = (codes.double().cpu() * each - act).abs()
    assert (apart <= act.abs() * (2.0 ** -4 + REL) + each * 2.0 ** -10 * (1 + REL)).all()
    full = high > FLOOR * 2
    assert (codes.double().cpu().abs().view(rows, -1, BLOCK).amax(-1)[full] >= 440).all()  # every such group
    return codes, scales


NEGATIVE = [-0.0625, -0.15625, -0.171875, -0.1875]  # times 1/512 .. 448: gates down to -84


@pytest.mark.parametrize("gather", [False, True], ids=["sorted", "gathered"])
@pytest.mark.parametrize("rows", [7, 126, 378], ids=["few", "few-32", "wide"])
def test_negative_gates(rows, gather):
    check(rows, NEGATIVE, 1.0, 7.0, gather)


@pytest.mark.parametrize("limit", [0.5, 7.0, float("inf")])
@pytest.mark.parametrize("rows", [126, 378], ids=["few", "wide"])
def test_positive_gates_and_no_limit(rows, limit):
    """An infinite limit clamps nothing."""
    check(rows, [0.0625, 0.5, 1.0, 448.0], 1.0, limit, False)


@pytest.mark.parametrize("rows", [126, 378], ids=["few", "wide"])
def test_gates_near_the_end_of_the_range(rows):
    """Gates to -+2^127: a zero on the one side, the gate itself on the other."""
    check(rows, [-1.0, -448.0, -0.5, -2.0], 2.0 ** 100, 7.0, False)
    check(rows, [1.0, 448.0, 0.5, 288.0], 2.0 ** 110, float("inf"), False)
    check(rows, [1.0, 448.0, 0.5, 288.0], 2.0 ** 110, float("inf"), False, up_scale=2.0 ** -20)


def test_both_kernels_agree_to_the_bound():
    """The same rows in a small and in a large call: the accurate and the approximate forms."""
    a = check(126, NEGATIVE, 1.0, 7.0, False)[1]
    b = check(378, NEGATIVE, 1.0, 7.0, False)[1]
    assert float((a.double() / b[:126].double() - 1).abs().max()) <= 2 * REL


@pytest.mark.parametrize("rows", [126, 378], ids=["few", "wide"])
@pytest.mark.parametrize("where", ["gate", "up"])
@pytest.mark.parametrize("value", [float("nan"), float("inf")])
def test_not_finite_gates(rows, where, value):
    """A row whose sums are not finite (0 x inf is NaN) is NaN, no other row is."""
    q, s, wq, ws, g, u = case(rows, [0.5, -1.0], 1.0)
    s[rows - 2, 0 if where == "gate" else 1] = value
    off = torch.tensor([0, rows], dtype=torch.int32, device="cuda")
    codes, scales = moe.moe_fp8_grouped_gemm_swiglu(q, s, wq, ws, off, rows)
    bad = np.zeros(rows, bool)
    bad[rows - 2] = True
    np.testing.assert_array_equal(torch.isnan(scales).all(1).cpu().numpy(), bad)
    np.testing.assert_array_equal(torch.isnan(scales).any(1).cpu().numpy(), bad)
    np.testing.assert_array_equal(torch.isnan(codes.float()).all(1).cpu().numpy(), bad)
