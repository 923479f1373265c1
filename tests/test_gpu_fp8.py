"""GPU tests of the FP8 (E4M3, one FP32 scale per 128 columns / 128 x 128 block) quantisers and products
against plain FP64 forms.

Quantisers: bit for bit against numpy's FP32 divisions and products and torch's CPU cast, and the codes
against the same expression in torch on the GPU.

Products: the codes' products are exact in FP32 (4-bit significands).  A k block adds 128 of them in
the MMA, each addition off by at most 2^-23 of the sum of magnitudes (truncation allowed), the product
of the two scales and the FMA into the running sum by 2^-24 each, over KB blocks:
    |got - ref| <= (128 * 2^-23 + (KB + 2) * 2^-24) * sum |a w|      (FP32 output)
    + 2^-8 |ref|                                                      (BF16 output: a unit of it)
Inputs whose sums are exact in FP32 (small integers, power-of-two scales) must come out exactly.

gate/up: |d act| <= 1.1 |u| dg + |silu(g)| du + 2^-19 |act| (silu' <= 1.1; the hardware exponential and
division), the scale follows its group's largest act, and a code stands for a value within half an
E4M3 step: 2^-4 of the value or 2^-10 scales.
"""

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

import moe_prefill_nvfp4_gb300 as moe  # noqa: E402

BLOCK = 128
FLOOR = np.float32(2.0 ** -100)


@pytest.fixture(autouse=True)
def _no_device_error():
    moe.moe_get_device_error()
    yield
    assert moe.moe_get_device_error() == 0


# ------------------------------------------------------------------------------------------ plain forms


def quantize_ref(x: torch.Tensor, rows_per_scale: int):
    """Definition on the CPU: codes (uint8) and FP32 scales."""
    a = x.float().cpu().numpy()
    n, k = a.shape
    nb, g = -(-n // rows_per_scale), -(-k // BLOCK)
    s = np.empty((nb, g), np.float32)
    q = np.empty((n, k), np.uint8)
    with np.errstate(all="ignore"):
        for i in range(nb):
            for j in range(g):
                part = a[i * rows_per_scale:(i + 1) * rows_per_scale, j * BLOCK:(j + 1) * BLOCK]
                m = np.abs(part).max()
                m = np.float32(np.nan) if not np.isfinite(m) else max(m, FLOOR)
                s[i, j] = np.float32(m) / np.float32(448)
                v = part * (np.float32(448) * (np.float32(1) / np.float32(m)))
                c = torch.from_numpy(v).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
                q[i * rows_per_scale:(i + 1) * rows_per_scale, j * BLOCK:(j + 1) * BLOCK] = c
    return q, s


def codes(t: torch.Tensor) -> np.ndarray:
    return t.contiguous().view(torch.uint8).cpu().numpy()


def assert_codes(got, ref):
    """Equal codes; a NaN code of either sign stands for NaN."""
    np.testing.assert_array_equal(np.where((got & 0x7F) == 0x7F, 0x7F, got), np.where((ref & 0x7F) == 0x7F, 0x7F, ref))


def dequant_rows64(q, s):
    k = q.shape[-1]
    return q.double().cpu() * s.double().cpu().repeat_interleave(BLOCK, -1)[..., :k]


def dequant_blocks64(q, s):
    n, k = q.shape[-2:]
    return q.double().cpu() * s.double().cpu().repeat_interleave(BLOCK, -1)[..., :k].repeat_interleave(BLOCK, -2)[..., :n, :]


def product64(a, w):
    """(a w^T, |a| |w|^T) in FP64."""
    return a @ w.t(), a.abs() @ w.abs().t()


def bound_f32(k, mags):
    kb = -(-k // BLOCK)
    return (128 * 2.0 ** -23 + (kb + 2) * 2.0 ** -24) * mags


def assert_product(got, ref, mags, k, what=""):
    tol = bound_f32(k, mags)
    if got.dtype == torch.bfloat16:
        tol = tol + ref.abs() * 2.0 ** -8
    d = (got.double().cpu() - ref).abs()
    bad = ~(d <= tol)
    assert not bad.any(), (what, int(bad.sum()), torch.nonzero(bad)[:4].tolist(), d[bad][:4], tol[bad][:4])


def rand(shape, seed, scale=1.0, dtype=torch.bfloat16):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return (torch.randn(*shape, generator=g, device="cuda") * scale).to(dtype)


def weights(e, n, k, seed):
    """[e, n, k] codes (rows whole 16 bytes apart) and [e, ...] scales from the library's quantiser."""
    ld = -(-k // 16) * 16
    q = torch.zeros(e, n, ld, dtype=torch.float8_e4m3fn, device="cuda")[..., :k]
    s = torch.empty(e, -(-n // BLOCK), -(-k // BLOCK), device="cuda")
    for i in range(e):
        moe.moe_fp8_quantize_blocks(rand((n, k), seed + i, k ** -0.5), out=q[i], scales=s[i])
    return q, s


def offsets_of(counts):
    return torch.tensor(np.concatenate([[0], np.cumsum(counts)]), dtype=torch.int32, device="cuda")


# ------------------------------------------------------------------------------------------ quantisers


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("r,k", [(1, 1), (1, 5120), (3, 127), (7, 128), (5, 129), (33, 777), (64, 1536), (130, 144), (9, 520)])
def test_quantize_rows(r, k, dtype):
    x = rand((r, k), r * 7 + k, 3.0, dtype)
    x[0, 0] = 0.0
    if r > 2:
        x[1] = 0.0  # rows of zeros
        x[2] = 1e-38  # below the floor of the scale
    q, s = moe.moe_fp8_quantize_rows(x)
    qr, sr = quantize_ref(x, 1)
    assert_codes(codes(q), qr)
    np.testing.assert_array_equal(s.cpu().numpy(), sr)
    assert q.stride(0) % 16 == 0 or r == 1


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_quantize_equals_the_torch_expression(dtype):
    """Many groups of BF16 values, whose quotients often lie on a tie between two codes."""
    x = rand((512, 2048), 77, 3.0, dtype)
    q, _ = moe.moe_fp8_quantize_rows(x)
    groups = x.float().view(512, 16, BLOCK)
    want = (groups * (448.0 / groups.abs().amax(-1, keepdim=True))).to(torch.float8_e4m3fn).view(512, 2048)
    assert torch.equal(q.view(torch.uint8), want.view(torch.uint8))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("n,k", [(1, 1), (128, 128), (127, 129), (300, 520), (256, 1000), (129, 136)])
def test_quantize_blocks(n, k, dtype):
    w = rand((n, k), n + k, 0.02, dtype)
    q, s = moe.moe_fp8_quantize_blocks(w)
    qr, sr = quantize_ref(w, BLOCK)
    assert_codes(codes(q), qr)
    np.testing.assert_array_equal(s.cpu().numpy(), sr)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_quantize_strided_rows_and_scales(dtype):
    big = rand((40, 1100), 5, 1.0, dtype)
    for x in (big[::2, 3:700], big[1:, 8:648], big[:, :1024], big[3:4, 16:272]):
        r, k = x.shape
        flat = torch.full((r * 2, -(-k // 16) * 16 + 32), 0x55, dtype=torch.uint8, device="cuda")
        out = flat.view(torch.float8_e4m3fn)[::2, 16:16 + k]
        scales = torch.full((r, 2 * -(-k // BLOCK)), -1.0, device="cuda")
        moe.moe_fp8_quantize_rows(x, out=out, scales=scales[:, ::2])
        qr, sr = quantize_ref(x, 1)
        assert_codes(codes(out), qr)
        np.testing.assert_array_equal(scales[:, ::2].cpu().numpy(), sr)
        assert (scales[:, 1::2] == -1).all()
        assert (flat[1::2] == 0x55).all() and (flat[:, :16] == 0x55).all() and (flat[:, 16 + k:] == 0x55).all()


def test_quantize_not_finite():
    x = rand((6, 300), 9)
    x[0, 5] = float("inf")
    x[1, 130] = float("-inf")
    x[2, 299] = float("nan")
    x[3, :] = 3e38
    q, s = moe.moe_fp8_quantize_rows(x)
    qr, sr = quantize_ref(x, 1)
    assert_codes(codes(q), qr)
    np.testing.assert_array_equal(s.cpu().numpy(), sr)
    assert torch.isnan(s[0, 0]) and torch.isnan(s[1, 1]) and torch.isnan(s[2, 2])
    assert int(torch.isnan(s).sum()) == 3  # no other group
    qb, sb = moe.moe_fp8_quantize_blocks(x)
    assert torch.isnan(sb).tolist() == [[True, True, True]] and torch.isnan(qb.float()).all()


def test_quantize_no_rows():
    q, s = moe.moe_fp8_quantize_rows(torch.empty(0, 256, dtype=torch.bfloat16, device="cuda"))
    assert q.shape == (0, 256) and s.shape == (0, 2)


# ------------------------------------------------------------------------------------------ dense product

# few-row tiles of 16 and 32, wide tiles of 128 and 256 weight rows; k tails, weight-row tails, one of each
DENSE = [(1, 1, 1), (1, 128, 128), (1, 5120, 1536), (2, 300, 129), (5, 130, 257), (12, 256, 2048), (13, 513, 384),
         (16, 257, 640), (32, 1000, 100), (40, 385, 1111), (41, 128, 128), (64, 200, 300), (127, 640, 256),
         (129, 255, 640), (300, 520, 200), (333, 1500, 2000), (1300, 4000, 272), (2000, 2560, 520),
         (130, 300, 3000), (257, 1013, 4100), (600, 1280, 3200),  # long and few tiles: k shared by a cluster
         (200, 1, 300), (700, 5, 130), (333, 2, 4000), (40000, 7, 33)]  # narrow outputs of wide tiles


@pytest.mark.parametrize("c_dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("r,n,k", DENSE)
def test_gemm(r, n, k, c_dtype):
    a, sa = moe.moe_fp8_quantize_rows(rand((r, k), r + n + k))
    w, sw = moe.moe_fp8_quantize_blocks(rand((n, k), r + n + k + 1, 0.05))
    ld = (n + 7) // 8 * 8 + 16
    flat = torch.full((r + 2, ld), 3.0, dtype=c_dtype, device="cuda")
    out = flat[1:r + 1, 8:8 + n]
    got = moe.moe_fp8_gemm(a, sa, w, sw, out=out, c_dtype=c_dtype)
    ref, mags = product64(dequant_rows64(a, sa), dequant_blocks64(w, sw))
    assert_product(got, ref, mags, k)
    assert (flat[0] == 3).all() and (flat[r + 1] == 3).all() and (flat[:, :8] == 3).all() and (flat[:, 8 + n:] == 3).all()
    assert torch.equal(moe.moe_fp8_gemm(a, sa, w, sw, c_dtype=c_dtype), got)  # the same sums in the same order


@pytest.mark.parametrize("gather", [False, True], ids=["sorted", "gathered"])
def test_grouped_gemm_long_k_few_tiles(gather):
    """Two experts with a long K: the wide kernel's k blocks are shared by a cluster."""
    counts, n, k = [150, 0, 131], 270, 3200
    c = grouped_case(counts, n, k, gather, 61, 2)
    for dt in (torch.bfloat16, torch.float32):
        out = torch.full((c["slots"], 272), 5.0, dtype=dt, device="cuda")[:, :n]
        moe.moe_fp8_grouped_gemm(c["a"], c["sa"], c["w"], c["sw"], c["offsets"], c["slots"], gather_ids=c["ids"], out=out,
                                 c_dtype=dt)
        ref, mags = grouped64(c)
        assert_product(out[:281], ref[:281], mags[:281], k)
        assert (out[281:] == 5).all()


@pytest.mark.parametrize("r", [1, 16, 31, 100, 1280])
def test_gemm_exact_sums(r):
    """Integers and power-of-two scales: every partial sum is exact, so any correct order gives the same."""
    n, k = 2816, 392
    g = torch.Generator().manual_seed(r)
    a = torch.randint(-4, 5, (r, k), generator=g).float()
    w = torch.randint(-4, 5, (n, k), generator=g).float()
    sa = 2.0 ** torch.randint(-3, 4, (r, 4), generator=g).float()
    sw = 2.0 ** torch.randint(-3, 4, (22, 4), generator=g).float()
    ld = 400
    qa = torch.zeros(r, ld, dtype=torch.float8_e4m3fn, device="cuda")[:, :k]
    qw = torch.zeros(n, ld, dtype=torch.float8_e4m3fn, device="cuda")[:, :k]
    qa.copy_(a)
    qw.copy_(w)
    got = moe.moe_fp8_gemm(qa, sa.cuda(), qw, sw.cuda(), c_dtype=torch.float32)
    ref = dequant_rows64(a, sa) @ dequant_blocks64(w, sw).t()
    assert torch.equal(got.double().cpu(), ref)


@pytest.mark.parametrize("r", [3, 20, 140])
def test_gemm_strided_operands(r):
    n, k = 270, 500
    big = torch.zeros(2 * r, 1024, dtype=torch.float8_e4m3fn, device="cuda")
    wbig = torch.zeros(2 * n, 1024, dtype=torch.float8_e4m3fn, device="cuda")
    a, w = big[::2, 32:32 + k], wbig[1::2, 16:16 + k]
    big.view(torch.uint8).fill_(0x7F)  # what lies between the operands' rows is NaN
    wbig.view(torch.uint8).fill_(0x7F)
    sa = torch.empty(r, 4, device="cuda")  # row-major scales
    moe.moe_fp8_quantize_rows(rand((r, k), 3), out=a, scales=sa)
    sw = torch.empty(3, 4, device="cuda")
    moe.moe_fp8_quantize_blocks(rand((n, k), 4), out=w, scales=sw)
    ref, mags = product64(dequant_rows64(a, sa), dequant_blocks64(w, sw))
    assert_product(moe.moe_fp8_gemm(a, sa, w, sw, c_dtype=torch.float32), ref, mags, k)


@pytest.mark.parametrize("r", [4, 25, 200])
def test_gemm_not_finite_stays_in_its_row(r):
    n, k = 300, 384
    x = rand((r, k), 8)
    x[1, 200] = float("nan")
    x[r - 1, 0] = float("inf")
    a, sa = moe.moe_fp8_quantize_rows(x)
    w, sw = moe.moe_fp8_quantize_blocks(rand((n, k), 9))
    got = moe.moe_fp8_gemm(a, sa, w, sw, c_dtype=torch.float32)
    nan = torch.zeros(r, dtype=torch.bool)
    nan[1] = nan[r - 1] = True
    assert torch.isnan(got[nan.cuda()]).all() and torch.isfinite(got[~nan.cuda()]).all()


def test_gemm_no_rows():
    w, sw = moe.moe_fp8_quantize_blocks(rand((128, 256), 1))
    a, sa = moe.moe_fp8_quantize_rows(torch.empty(0, 256, dtype=torch.bfloat16, device="cuda"))
    assert moe.moe_fp8_gemm(a, sa, w, sw).shape == (0, 128)


# ------------------------------------------------------------------------------------------ grouped product


COUNTS = {
    "one-token": [0, 1, 0, 1, 0, 0, 1, 0],
    "one-expert": [37],
    "empty-ends": [0, 0, 5, 17, 0, 33, 1, 0, 0],
    "skewed": [1, 200, 0, 3, 129, 64, 0, 128],
    "busy": [300, 257, 0, 128, 500],
}


def grouped_case(counts, n, k, gather, seed, extra=0):
    """Operands of one grouped call; `extra` sorted rows past the last expert's."""
    e, slots = len(counts), int(sum(counts)) + extra
    g = torch.Generator().manual_seed(seed)
    rows = max(1, slots // 2) if gather else slots
    a, sa = moe.moe_fp8_quantize_rows(rand((rows, k), seed))
    ids = torch.randint(0, rows, (slots,), generator=g, dtype=torch.int32).cuda() if gather else None
    w, sw = weights(e, n, k, seed + 100)
    return dict(a=a, sa=sa, w=w, sw=sw, ids=ids, offsets=offsets_of(counts), slots=slots, counts=counts)


def grouped64(c, first=0, count=None):
    a, w = dequant_rows64(c["a"], c["sa"]), dequant_blocks64(c["w"], c["sw"])
    if c["ids"] is not None:
        a = a[c["ids"].long().cpu()]
    n = w.shape[1]
    ref, mags = torch.zeros(c["slots"], n, dtype=torch.float64), torch.zeros(c["slots"], n, dtype=torch.float64)
    lo = 0
    for e, m in enumerate(c["counts"]):
        if first <= e < first + (len(c["counts"]) if count is None else count):
            ref[lo:lo + m], mags[lo:lo + m] = product64(a[lo:lo + m], w[e - first])
        lo += m
    return ref, mags


@pytest.mark.parametrize("gather", [False, True], ids=["sorted", "gathered"])
@pytest.mark.parametrize("n,k", [(300, 400), (512, 129), (128, 1536)])
@pytest.mark.parametrize("name", list(COUNTS))
def test_grouped_gemm(name, n, k, gather):
    counts = COUNTS[name]
    extra = 3
    c = grouped_case(counts, n, k, gather, len(name) + n, extra)
    for dt in (torch.bfloat16, torch.float32):
        out = torch.full((c["slots"], (n + 7) // 8 * 8), 5.0, dtype=dt, device="cuda")[:, :n]
        moe.moe_fp8_grouped_gemm(c["a"], c["sa"], c["w"], c["sw"], c["offsets"], c["slots"], gather_ids=c["ids"], out=out,
                                 c_dtype=dt)
        live = sum(counts)
        ref, mags = grouped64(c)
        assert_product(out[:live], ref[:live], mags[:live], k, name)
        assert (out[live:] == 5).all()  # rows past the last offset are not touched


PAIRS = [700, 300, 0, 129, 513, 1]  # 256-row tiles: whole, with an empty second half, with one row in it


@pytest.mark.parametrize("gather", [False, True], ids=["sorted", "gathered"])
@pytest.mark.parametrize("n,k", [(2300, 272), (2056, 1000)])
def test_grouped_gemm_cta_pairs(n, k, gather):
    """Enough rows per expert and tiles for the CTA-pair tiles of 256 rows."""
    c = grouped_case(PAIRS, n, k, gather, n, 3)
    for dt in (torch.bfloat16, torch.float32):
        out = torch.full((c["slots"], (n + 7) // 8 * 8), 5.0, dtype=dt, device="cuda")[:, :n]
        moe.moe_fp8_grouped_gemm(c["a"], c["sa"], c["w"], c["sw"], c["offsets"], c["slots"], gather_ids=c["ids"], out=out,
                                 c_dtype=dt)
        live = sum(PAIRS)
        ref, mags = grouped64(c)
        assert_product(out[:live], ref[:live], mags[:live], k)
        assert (out[live:] == 5).all()


@pytest.mark.parametrize("gather", [False, True], ids=["sorted", "gathered"])
@pytest.mark.parametrize("inter,k", [(1024, 400), (1152, 129)])
def test_swiglu_cta_pairs(inter, k, gather):
    c = grouped_case(PAIRS, 2 * inter, k, gather, inter + k)
    q, s = moe.moe_fp8_grouped_gemm_swiglu(c["a"], c["sa"], c["w"], c["sw"], c["offsets"], c["slots"], limit=0.75,
                                           gather_ids=c["ids"])
    ref, mags = grouped64(c)
    act, tol = swiglu64(ref, mags, k, 0.75)
    assert_quantised(q, s, act, tol)


def swiglu64(ref, mags, k, limit):
    inter = ref.shape[1] // 2
    g, u = ref[:, :inter], ref[:, inter:]
    gm, uc = g.clamp(max=limit), u.clamp(-limit, limit)
    silu = gm / (1 + torch.exp(-gm))
    act = silu * uc
    tol = bound_f32(k, mags)
    return act, 1.1 * uc.abs() * tol[:, :inter] + silu.abs() * tol[:, inter:] + 2.0 ** -19 * act.abs()


def assert_quantised(q, s, act, tol):
    """Codes and scales of act known to within tol."""
    rows, inter = act.shape
    q, s = q.double().cpu(), s.double().cpu()
    m = act.abs().view(rows, -1, BLOCK)
    t = tol.view(rows, -1, BLOCK)
    hi, lo = (m + t).amax(-1), (m - t).amax(-1)
    assert (s * 448 <= hi.clamp_min(2.0 ** -100) * (1 + 2.0 ** -22)).all()
    assert (s * 448 >= lo.clamp_min(2.0 ** -100) * (1 - 2.0 ** -22)).all()
    sc = s.repeat_interleave(BLOCK, -1)
    v = q * sc
    d = (v - act).abs()
    # half a step of the value, the value and its scale each off by their own error
    lim = tol + (act.abs() + tol) * (2.0 ** -4 + 2.0 ** -20) + sc * 2.0 ** -10 * (1 + 2.0 ** -20)
    assert (d <= lim).all(), (torch.nonzero(d > lim)[:4].tolist(), d[d > lim][:4], lim[d > lim][:4])
    # a code is the nearest one to its value: no worse than half a step from act / scale
    assert (q.abs().view(rows, -1, BLOCK).amax(-1) >= 416).all() or (m.amax(-1) < 2.0 ** -99).any()


@pytest.mark.parametrize("gather", [False, True], ids=["sorted", "gathered"])
@pytest.mark.parametrize("inter,k", [(128, 300), (384, 129), (256, 2048)])
@pytest.mark.parametrize("name", list(COUNTS))
def test_grouped_gemm_swiglu(name, inter, k, gather):
    counts = COUNTS[name]
    c = grouped_case(counts, 2 * inter, k, gather, len(name) + inter, 2)
    limit = 0.75  # clamps a good part of the sums
    out = torch.zeros(c["slots"], inter, dtype=torch.float8_e4m3fn, device="cuda")
    scales = torch.full((c["slots"], inter // BLOCK), -1.0, device="cuda")
    out.view(torch.uint8).fill_(0x55)
    q, s = moe.moe_fp8_grouped_gemm_swiglu(c["a"], c["sa"], c["w"], c["sw"], c["offsets"], c["slots"], limit=limit,
                                           gather_ids=c["ids"], out=out, scales=scales)
    live = sum(counts)
    ref, mags = grouped64(c)
    act, tol = swiglu64(ref, mags, k, limit)
    assert_quantised(q[:live], s[:live], act[:live], tol[:live])
    assert (out.view(torch.uint8)[live:] == 0x55).all() and (scales[live:] == -1).all()
    # the codes are the nearest to the values the scales stand for: a product on them is the down product's input
    wd, swd = weights(len(counts), 256, inter, 77)
    down = moe.moe_fp8_grouped_gemm(q, s, wd, swd, c["offsets"], live, c_dtype=torch.float32)
    d = dict(c, a=q[:live], sa=s[:live], w=wd, sw=swd, ids=None, slots=live)
    ref, mags = grouped64(d)
    assert_product(down, ref, mags, inter)


@pytest.mark.parametrize("name", ["empty-ends", "skewed"])
def test_swiglu_not_finite(name):
    c = grouped_case(COUNTS[name], 256, 256, False, 3)
    c["sa"][2, 1] = float("nan")
    q, s = moe.moe_fp8_grouped_gemm_swiglu(c["a"], c["sa"], c["w"], c["sw"], c["offsets"], c["slots"])
    bad = torch.isnan(s[:, 0])
    assert bad.nonzero().flatten().tolist() == [2]
    assert torch.isnan(q.float()[2]).all() and torch.isfinite(q.float()[~bad]).all()


@pytest.mark.parametrize("first,count", [(0, 2), (3, 4), (7, 1)])
@pytest.mark.parametrize("name", ["skewed", "one-token"])
def test_experts_held_elsewhere_are_zero(name, first, count):
    """Expert parallelism: W holds experts first .. first + count - 1, the others' rows are zeros."""
    c = grouped_case(COUNTS[name], 256, 300, False, 4)
    part = dict(c, w=c["w"][first:first + count], sw=c["sw"][first:first + count])
    got = moe.moe_fp8_grouped_gemm(c["a"], c["sa"], part["w"], part["sw"], c["offsets"], c["slots"], first=first,
                                   c_dtype=torch.float32)
    ref, mags = grouped64(part, first, count)
    assert_product(got, ref, mags, 300)
    assert (got.cpu()[mags.sum(1) == 0] == 0).all()
    q, s = moe.moe_fp8_grouped_gemm_swiglu(c["a"], c["sa"], part["w"], part["sw"], c["offsets"], c["slots"], first=first)
    away = (mags.sum(1) == 0).cuda()
    assert (q.float()[away] == 0).all() and (s[away] == float(FLOOR / np.float32(448))).all()


def test_bad_indices_are_recorded():
    c = grouped_case(COUNTS["skewed"], 256, 256, True, 5)
    ids = c["ids"].clone()
    ids[3], ids[100] = -1, c["a"].shape[0]
    got = moe.moe_fp8_grouped_gemm(c["a"], c["sa"], c["w"], c["sw"], c["offsets"], c["slots"], gather_ids=ids,
                                   c_dtype=torch.float32)
    assert moe.moe_get_device_error() == 5
    ids[3] = ids[100] = 0  # what was read in their place
    want = moe.moe_fp8_grouped_gemm(c["a"], c["sa"], c["w"], c["sw"], c["offsets"], c["slots"], gather_ids=ids,
                                    c_dtype=torch.float32)
    assert torch.equal(got, want)


@pytest.mark.parametrize("counts", [[1, 2, 1], [200, 100, 90]])
@pytest.mark.parametrize("fault", ["decreasing", "past-R", "not-from-zero"])
def test_bad_offsets_write_nothing(counts, fault):
    c = grouped_case(counts, 256, 256, False, 6)
    off = c["offsets"].clone()
    if fault == "decreasing":
        off[2] = off[1] - 1
    elif fault == "past-R":
        off[3] += 1
    else:
        off[0] = 1
    out = torch.full((c["slots"], 256), 2.0, dtype=torch.bfloat16, device="cuda")
    moe.moe_fp8_grouped_gemm(c["a"], c["sa"], c["w"], c["sw"], off, c["slots"], out=out)
    assert moe.moe_get_device_error() == 2
    assert (out == 2).all()


def test_no_expert_has_a_row():
    c = grouped_case([0, 0, 0], 256, 256, False, 7, extra=5)
    out = torch.full((5, 256), 2.0, dtype=torch.bfloat16, device="cuda")
    moe.moe_fp8_grouped_gemm(c["a"], c["sa"], c["w"], c["sw"], c["offsets"], 5, out=out)
    assert (out == 2).all()
    assert moe.moe_fp8_grouped_gemm(c["a"], c["sa"], c["w"], c["sw"], c["offsets"], 0).shape == (0, 256)


def test_streams_and_graph():
    """On a stream of its own, and captured: the same bits as on the current stream."""
    c = grouped_case(COUNTS["skewed"], 512, 512, True, 8)

    def chain(stream=None):
        q, s = moe.moe_fp8_grouped_gemm_swiglu(c["a"], c["sa"], c["w"], c["sw"], c["offsets"], c["slots"],
                                               gather_ids=c["ids"], stream=stream)
        return moe.moe_fp8_grouped_gemm(q, s, wd, swd, c["offsets"], c["slots"], stream=stream)

    wd, swd = weights(8, 384, 256, 50)
    want = chain()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        got = chain(side)
    side.synchronize()
    assert torch.equal(got, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = chain()
    got.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(got, want)


def test_offsets_past_32_bits():
    """Codes, scales and outputs whose last elements lie past 2^32 bytes and 2^31 elements."""
    rows, ld, k, n = 900_000, 5120, 256, 136
    flat = torch.zeros(rows * ld, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn).view(rows, ld)
    a = flat[:, ld - k:]
    x = rand((rows, k), 40)
    sa = torch.zeros(rows, 2600, device="cuda")[:, 2598:]
    moe.moe_fp8_quantize_rows(x, out=a, scales=sa)
    w, sw = weights(2, n, k, 41)
    some = [0, 1, 127, 128, 450_000, rows - 129, rows - 2, rows - 1]
    ids = torch.tensor(some, dtype=torch.int32, device="cuda")
    ref = torch.cat([product64(dequant_rows64(a[i:i + 1], sa[i:i + 1]), dequant_blocks64(w[0], sw[0]))[0] for i in some])
    mags = torch.cat([product64(dequant_rows64(a[i:i + 1], sa[i:i + 1]), dequant_blocks64(w[0], sw[0]))[1] for i in some])
    for reps in (1, 20):  # few rows (TMA gather) and many (cp.async)
        got = moe.moe_fp8_grouped_gemm(a, sa, w, sw, offsets_of([8 * reps, 0]), 8 * reps, gather_ids=ids.repeat(reps),
                                       c_dtype=torch.float32)
        assert_product(got, ref.repeat(reps, 1), mags.repeat(reps, 1), k)
    out = torch.zeros(rows, 2560, dtype=torch.bfloat16, device="cuda")[:, :n]
    got = moe.moe_fp8_gemm(a, sa, w[0], sw[0], out=out)
    assert_product(got[ids.long()], ref, mags, k)


@pytest.mark.parametrize("first_stride", [1, 0])
def test_activation_scales_of_any_layout(first_stride):
    """Row-major, group-major and one scale per group shared by all rows (stride 0)."""
    r, n, k = 150, 260, 512
    a, sa = moe.moe_fp8_quantize_rows(rand((r, k), 50))
    w, sw = moe.moe_fp8_quantize_blocks(rand((n, k), 51))
    if first_stride == 0:
        sa = sa[:1].expand(r, 4)
    else:
        sa = sa.contiguous()
    for rows in (5, r):
        ref, mags = product64(dequant_rows64(a[:rows], sa[:rows]), dequant_blocks64(w, sw))
        assert_product(moe.moe_fp8_gemm(a[:rows], sa[:rows], w, sw, c_dtype=torch.float32), ref, mags, k)


@pytest.mark.parametrize("heavy", [0, 40], ids=["few-rows", "wide-tiles"])
def test_as_many_experts_as_there_may_be(heavy):
    """512 experts, most of them without a row; the last has some."""
    e, n, k = moe.MOE_FP8_MAX_EXPERTS, 136, 144
    g = torch.Generator().manual_seed(heavy)
    counts = [int(c) + heavy for c in torch.randint(0, 3, (e,), generator=g) * torch.randint(0, 2, (e,), generator=g)]
    counts[-1] = 5
    c = grouped_case(counts, n, k, True, 70 + heavy)
    got = moe.moe_fp8_grouped_gemm(c["a"], c["sa"], c["w"], c["sw"], c["offsets"], c["slots"], gather_ids=c["ids"],
                                   c_dtype=torch.float32)
    ref, mags = grouped64(c)
    assert_product(got, ref, mags, k)


def test_bad_gather_index_in_the_few_row_kernel():
    c = grouped_case(COUNTS["empty-ends"], 256, 256, True, 80)
    ids = c["ids"].clone()
    ids[3], ids[c["slots"] - 1] = 1 << 30, -5
    got = moe.moe_fp8_grouped_gemm(c["a"], c["sa"], c["w"], c["sw"], c["offsets"], c["slots"], gather_ids=ids)
    assert moe.moe_get_device_error() == 5
    ids[3] = ids[c["slots"] - 1] = 0
    want = moe.moe_fp8_grouped_gemm(c["a"], c["sa"], c["w"], c["sw"], c["offsets"], c["slots"], gather_ids=ids)
    assert torch.equal(got, want)


def test_binding_refuses_on_the_gpu():
    """Shapes, types and strides that the binding checks before it calls the library."""
    a, sa = moe.moe_fp8_quantize_rows(rand((4, 256), 90))
    w, sw = moe.moe_fp8_quantize_blocks(rand((128, 256), 91))
    ok = moe.moe_fp8_gemm(a, sa, w, sw)
    assert ok.shape == (4, 128) and ok.dtype == torch.bfloat16
    for bad in (
        lambda: moe.moe_fp8_gemm(a[:, :128], sa, w, sw),                       # columns
        lambda: moe.moe_fp8_gemm(a, sa[:3], w, sw),                            # scales of other rows
        lambda: moe.moe_fp8_gemm(a, sa.double(), w, sw),
        lambda: moe.moe_fp8_gemm(a, sa, w, sw[:, :1]),
        lambda: moe.moe_fp8_gemm(a, sa, w.t(), sw),                            # column stride
        lambda: moe.moe_fp8_gemm(a, sa, w, sw, c_dtype=torch.float16),
        lambda: moe.moe_fp8_gemm(a, sa, w, sw, out=torch.empty(4, 127, dtype=torch.bfloat16, device="cuda")),
        lambda: moe.moe_fp8_gemm(a, sa, w, sw, out=torch.empty(4, 128, device="cuda")),
        lambda: moe.moe_fp8_gemm(a, sa, w[None], sw[None]),
        lambda: moe.moe_fp8_quantize_rows(rand((4, 256), 1).half()),
        lambda: moe.moe_fp8_quantize_rows(rand((4, 256), 1).t()),
        lambda: moe.moe_fp8_grouped_gemm(a, sa, w[None], sw[None], torch.zeros(2, device="cuda"), 4),
        lambda: moe.moe_fp8_grouped_gemm(a, sa, w[None], sw[None], offsets_of([4]), 4, gather_ids=offsets_of([4])),
        lambda: moe.moe_fp8_grouped_gemm(a, sa, w[None], sw[None], offsets_of([4]), -1),
    ):
        with pytest.raises(ValueError):
            bad()
    for bad in (
        lambda: moe.moe_fp8_grouped_gemm(a, sa, w[None], sw[None], offsets_of([4]), 5),           # rows of A
        lambda: moe.moe_fp8_grouped_gemm(a, sa, w[None], sw[None], offsets_of([4]), 4, first=1),
        lambda: moe.moe_fp8_grouped_gemm_swiglu(a, sa, w[None], sw[None], offsets_of([4]), 4),    # I = 64
        lambda: moe.moe_fp8_grouped_gemm_swiglu(a, sa, w[None], sw[None], offsets_of([4]), 4, limit=0.0),
        lambda: moe.moe_fp8_gemm(a, sa, w, sw, out=torch.empty(4, 130, dtype=torch.bfloat16, device="cuda")[:, :128]),
    ):
        with pytest.raises(moe.MoeError):
            bad()
    with pytest.raises(TypeError):
        moe.moe_fp8_grouped_gemm(a, sa, w[None], sw[None], offsets_of([4]), "four")
