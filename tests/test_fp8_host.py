"""The FP8 calls refuse bad arguments on the host, before any launch (no GPU needed)."""

import ctypes

import pytest
import torch

import moe_prefill_nvfp4_gb300 as moe
from moe_prefill_nvfp4_gb300 import _lib, build

P = 4096  # a non-NULL, aligned dummy address: never dereferenced on these paths


@pytest.fixture(scope="module")
def L():
    build.build()
    return _lib.load()


def rows(**kw):
    d = dict(q=P, ld=256, s=P, s_row=1, s_grp=8, rows=8)
    d.update(kw)
    return _lib.Fp8Rows(*[d[n] for n, _ in _lib.Fp8Rows._fields_])


def weight(**kw):
    d = dict(q=P, ld=256, expert_stride=512 * 256, s=P, first=0, count=1, N=512, K=256)
    d.update(kw)
    return _lib.Fp8Weight(*[d[n] for n, _ in _lib.Fp8Weight._fields_])


def test_quantise_rejects(L):
    f = L.moe_fp8_quantize_rows
    assert f(None, 0, 256, 4, 256, P, 256, P, 1, 4, None) == 1
    assert f(P, 2, 256, 4, 256, P, 256, P, 1, 4, None) == 1  # element type
    assert f(P, 0, 255, 4, 256, P, 256, P, 1, 4, None) == 2  # rows overlap
    assert f(P, 0, 256, -1, 256, P, 256, P, 1, 4, None) == 2
    assert f(P, 0, 256, 4, 0, P, 256, P, 1, 4, None) == 2
    assert f(P, 0, 256, 4, 250, P, 250, P, 1, 4, None) == 1  # code rows not whole 16 bytes
    assert f(P, 0, 256, 4, 256, P + 8, 256, P, 1, 4, None) == 1
    assert f(P + 1, 0, 256, 4, 256, P, 256, P, 1, 4, None) == 1
    g = L.moe_fp8_quantize_blocks
    assert g(P, 0, 256, 0, 256, P, 256, P, None) == 2
    assert g(P, 1, 256, 4, 256, P, 128, P, None) == 1
    assert g(P, 1, 256, 4, 256, P, 256, P + 2, None) == 1


@pytest.mark.parametrize("a,w,want", [
    (dict(q=None), {}, 1), (dict(s=None), {}, 1), ({}, dict(q=None), 1), ({}, dict(s=None), 1),
    (dict(ld=250), {}, 1), (dict(ld=240), {}, 1), (dict(q=P + 8), {}, 1), (dict(rows=-1), {}, 2),
    ({}, dict(ld=264), 1), ({}, dict(K=0), 2), ({}, dict(N=0), 2), ({}, dict(first=1), 2), ({}, dict(count=2), 2)])
def test_gemm_rejects(L, a, w, want):
    assert L.moe_fp8_gemm(ctypes.byref(rows(**a)), ctypes.byref(weight(**w)), P, 512, 0, None) == want


def test_gemm_rejects_output(L):
    a, w = ctypes.byref(rows()), ctypes.byref(weight())
    assert L.moe_fp8_gemm(a, w, None, 512, 0, None) == 1
    assert L.moe_fp8_gemm(a, w, P, 504, 0, None) == 2  # rows overlap
    assert L.moe_fp8_gemm(a, w, P, 514, 0, None) == 2  # rows not whole 8 elements
    assert L.moe_fp8_gemm(a, w, P + 4, 512, 0, None) == 1
    assert L.moe_fp8_gemm(a, w, P, 512, 3, None) == 1
    assert L.moe_fp8_gemm(None, w, P, 512, 0, None) == 1


def test_grouped_rejects(L):
    def call(a=None, w=None, offsets=P, E=4, R=8, ldc=512, gather=None):
        return L.moe_fp8_grouped_gemm(ctypes.byref(rows(**(a or {}))), gather,
                                      ctypes.byref(weight(**{**dict(count=4), **(w or {})})), offsets, E, R, P, ldc, 0, None)

    assert call(offsets=None) == 1
    assert call(E=0) == 2
    assert call(E=513, w=dict(count=513)) == 2
    assert call(E=3) == 2  # more experts held than there are
    assert call(w=dict(first=1)) == 2
    assert call(w=dict(first=-1)) == 2
    assert call(w=dict(expert_stride=512 * 256 - 16)) == 1  # experts overlap
    assert call(w=dict(expert_stride=512 * 256 + 8)) == 1
    assert call(R=9) == 2  # fewer rows in A than sorted rows, and no gather
    assert call(R=-1) == 2
    assert call(a=dict(rows=0), gather=P) == 2


def test_swiglu_rejects(L):
    def call(w=None, R=8, limit=7.0, act=P, ld=256, s=P):
        return L.moe_fp8_grouped_gemm_swiglu(ctypes.byref(rows()), None, ctypes.byref(weight(**{**dict(count=4), **(w or {})})),
                                             P, 4, R, limit, act, ld, s, 1, 8, None)

    assert call(limit=0.0) == 1
    assert call(limit=float("nan")) == 1
    assert call(w=dict(N=384)) == 2  # I not a multiple of 128
    assert call(act=None) == 1
    assert call(s=None) == 1
    assert call(ld=240) == 1
    assert call(R=9) == 2


def test_binding_rejects():
    cpu = torch.zeros(4, 256)
    with pytest.raises(ValueError):
        moe.moe_fp8_quantize_rows(cpu)
    with pytest.raises(ValueError):
        moe.moe_fp8_quantize_blocks(cpu)
    q = torch.zeros(4, 256).to(torch.float8_e4m3fn)
    s = torch.zeros(4, 2)
    with pytest.raises(ValueError):
        moe.moe_fp8_gemm(q, s, q, s)
    with pytest.raises(ValueError):
        moe.moe_fp8_grouped_gemm(q, s, q, s, torch.zeros(2, dtype=torch.int32), 4)
