"""GPU tests of the residual addition, RMS norm and row quantiser in one pass, against FP64.

h is one FP32 addition, rounded once: equal to torch's.  The sum of squares has at most 4096 terms in a chain of at
most 64 additions per thread, 5 shuffles and 16 warps: 85 * 2^-24 of itself, half of that after the square root,
and four more roundings (division, addition, root, reciprocal) and two products: y is within 2^-18 of its value.
The BF16 y: another 2^-8.  Codes stand for y to half a step, with the scale's own error (few_helpers.quantised64)."""

import pytest
import torch

pytestmark = pytest.mark.gpu

import moe_prefill_nvfp4_gb300 as moe  # noqa: E402

from few_helpers import quantised64, rand  # noqa: E402
from test_gpu_fp8 import codes, dequant_rows64, quantize_ref  # noqa: E402

BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(autouse=True)
def _no_device_error():
    moe.moe_get_device_error()
    yield
    assert moe.moe_get_device_error() == 0


def check(x, w, r, eps, q, s, h, y):
    if r is None:
        assert h is None
        h64 = x.double()
    else:
        assert torch.equal(h, (x.float() + r.float()).to(r.dtype))
        h64 = (x.float() + r.float()).double()
    n, k = x.shape
    ref = h64 / torch.sqrt((h64 * h64).mean(1, keepdim=True) + eps) * w.double()
    if y is not None:
        assert ((y.double() - ref).abs() <= ref.abs() * (2.0 ** -8 + 2.0 ** -17)).all()
    pad = -k % 128
    wide = torch.nn.functional.pad(ref, (0, pad))
    want, bound = quantised64(wide, wide.abs() * 2.0 ** -18)
    got = dequant_rows64(q, s).cuda()
    assert ((got - want[:, :k]).abs() <= bound[:, :k] + 2.0 ** -140).all()
    scale = wide.view(n, -1, 128).abs().amax(-1).clamp(min=2.0 ** -100) / 448
    assert ((s.double() - scale).abs() <= 2.0 ** -17 * scale).all()


SHAPES = [(1, 5120), (3, 128), (5, 2000), (333, 485), (7, 1), (2, 130), (9, 512), (6, 520), (2, 8200), (3, 16384), (2, 32768),
          (2, 20001), (4, 2049), (1000, 640)]


@pytest.mark.parametrize("rows,k", SHAPES)
@pytest.mark.parametrize("types", [(BF16, BF16, BF16), (BF16, F32, F32), (F32, None, BF16), (F32, BF16, F32)],
                         ids=["bbb", "bff", "f-b", "fbf"])
def test_against_fp64(rows, k, types):
    tx, tr, tw = types
    x, w = rand((rows, k), 1, 0.5, tx), 1 + rand((k,), 2, 0.3, tw)
    r = None if tr is None else rand((rows, k), 3, 2.0, tr)
    q, s, h, y = moe.moe_fp8_add_rms_norm(x, w, r, eps=1e-5, normed=True)
    check(x, w, r, 1e-5, q, s, h, y)
    again = moe.moe_fp8_add_rms_norm(x, w, r, eps=1e-5)
    assert again[3] is None and torch.equal(codes_t(again[0]), codes_t(q)) and torch.equal(again[1], s)


def codes_t(q):
    return torch.from_numpy(codes(q))


@pytest.mark.parametrize("k", [384, 1000])
def test_strides_and_given_outputs(k):
    """Rows inside wider tensors, on odd offsets, and outputs that the caller lays out."""
    rows = 37
    x, r = rand((rows, k + 9), 4)[:, 1:k + 1], rand((rows, 2 * k), 5, 1.0, F32)[:, k:]
    w = rand((k + 1,), 6)[1:]
    out = torch.zeros(rows, 1024, dtype=torch.float8_e4m3fn, device="cuda")
    scales = torch.full((rows, 16), -1.0, device="cuda")
    hs, ys = torch.zeros(rows, k + 3, device="cuda"), torch.zeros(rows, k + 5, dtype=BF16, device="cuda")
    g = -(-k // 128)
    q, s, h, y = moe.moe_fp8_add_rms_norm(x, w, r, normed=ys[:, 3:k + 3], residual_out=hs[:, 1:k + 1], out=out[:, :k],
                                          scales=scales[:, 2:2 + g])
    check(x, w, r, 1e-6, q, s, h, y)
    assert (codes(out)[:, k:] == 0).all() and (hs[:, 0] == 0).all() and (hs[:, k + 1:] == 0).all()
    assert (ys[:, :3] == 0).all() and (ys[:, k + 3:] == 0).all()
    assert (scales[:, :2] == -1).all() and (scales[:, 2 + g:] == -1).all()


@pytest.mark.parametrize("k", [512, 777])
def test_in_place(k):
    x, r, w = rand((65, k), 7), rand((65, k), 8), rand((k,), 9)
    want = moe.moe_fp8_add_rms_norm(x, w, r, normed=True)
    x2, r2 = x.clone(), r.clone()
    q, s, h, y = moe.moe_fp8_add_rms_norm(x2, w, r2, residual_out=r2, normed=x2)
    assert h is r2 and y is x2
    assert torch.equal(h, want[2]) and torch.equal(y, want[3]) and torch.equal(s, want[1])
    assert (codes(q) == codes(want[0])).all()


@pytest.mark.parametrize("k", [512, 300])
def test_values_that_are_not_finite_stay_in_their_row(k):
    x = rand((6, k), 10)
    clean = moe.moe_fp8_add_rms_norm(x, torch.ones(k, device="cuda"), normed=True)
    x[1, 5], x[2, 200], x[4] = float("nan"), float("inf"), 0.0
    q, s, _, y = moe.moe_fp8_add_rms_norm(x, torch.ones(k, device="cuda"), normed=True)
    for row in (0, 3, 5):
        assert torch.equal(y[row], clean[3][row]) and torch.equal(s[row], clean[1][row])
        assert (codes(q)[row] == codes(clean[0])[row]).all()
    assert y[1].isnan().all() and s[1].isnan().all()
    assert y[2, 200].isnan() and (y[2].nan_to_num(0.0) == 0).all() and s[2, 1].isnan() and s[2, 0] == 2.0 ** -100 / 448
    assert (y[4] == 0).all() and ((codes(q)[4] & 0x7F) == 0).all()


def test_codes_are_the_row_quantisers():
    """With w = 1 and rows of one magnitude y is exact: the quantiser's own codes and scales."""
    x = rand((8, 1024), 11).sign().float() * 2.0
    q, s, _, y = moe.moe_fp8_add_rms_norm(x, torch.ones(1024, device="cuda"), eps=0.0, normed=True)
    rq, rs = quantize_ref(y, 1)
    assert (codes(q) == rq).all() and (s.cpu().numpy() == rs).all()


def test_no_rows():
    q, s, h, y = moe.moe_fp8_add_rms_norm(torch.zeros(0, 256, device="cuda"), torch.ones(256, device="cuda"), normed=True)
    assert q.shape == (0, 256) and s.shape == (0, 2) and h is None and y.shape == (0, 256)


def test_refusals():
    x, w = rand((4, 256), 12), rand((256,), 13)
    for bad in (dict(weight=w[:255]), dict(weight=w.half()), dict(residual=rand((4, 255), 14)), dict(residual=x.half()),
                dict(residual_out=x.clone()), dict(normed=torch.zeros(4, 256, device="cuda")), dict(weight=w.cpu())):
        with pytest.raises(ValueError):
            moe.moe_fp8_add_rms_norm(**{**dict(x=x, weight=w), **bad})
    for bad in (dict(eps=-1.0), dict(eps=float("nan")), dict(eps=float("inf"))):
        with pytest.raises(moe.MoeError):
            moe.moe_fp8_add_rms_norm(x, w, **bad)
    with pytest.raises(moe.MoeError):
        moe.moe_fp8_add_rms_norm(torch.zeros(1, 32769, device="cuda"), torch.zeros(32769, device="cuda"))
