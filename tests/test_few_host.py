"""The norm and the few-token layers refuse bad arguments on the host, before any launch (no GPU needed)."""

import ctypes

import pytest
import torch

import moe_prefill_nvfp4_gb300 as moe
from moe_prefill_nvfp4_gb300 import _lib, build

from test_fp8_device_host import Fake

P = 4096  # a non-NULL, aligned dummy address: never dereferenced on these paths
F8, F32, BF16 = torch.float8_e4m3fn, torch.float32, torch.bfloat16


@pytest.fixture(scope="module")
def L():
    build.build()
    return _lib.load()


def config(**kw):
    return _lib.MoePrefillConfig(**{**dict(hidden=512, moe_intermediate=256, num_experts=8, top_k=2, swiglu_limit=7.0, renormalize=1,
                                           routed_scale=1.0), **kw})


# ------------------------------------------------------------------------------------------------ norm

NORM = dict(x=P, x_dtype=0, ld_x=256, r=P, r_dtype=0, ld_r=256, w=P, w_dtype=0, eps=1e-6, R=4, K=256, h=P, ld_h=256, y=P, ld_y=256,
            q=P, ld_q=256, s=P, s_row=2, s_grp=1, stream=None)


@pytest.mark.parametrize("bad,want", [
    (dict(x=None), 1), (dict(w=None), 1), (dict(q=None), 1), (dict(s=None), 1), (dict(h=None), 1), (dict(x_dtype=2), 1),
    (dict(r_dtype=3), 1), (dict(w_dtype=-1), 1), (dict(eps=-1e-6), 1), (dict(eps=float("nan")), 1), (dict(eps=float("inf")), 1),
    (dict(R=-1), 2), (dict(K=0), 2), (dict(K=32769, ld_x=32769, ld_r=32769, ld_h=32769, ld_y=32769, ld_q=32784), 2),
    (dict(ld_x=255), 2), (dict(ld_r=255), 2), (dict(ld_h=255), 2), (dict(ld_y=255), 2), (dict(ld_q=250), 1),
    (dict(q=P + 8), 1), (dict(x=P + 1), 1), (dict(r=P + 1), 1), (dict(h=P + 1), 1), (dict(y=P + 1), 1), (dict(s=P + 2), 1),
    (dict(x_dtype=1, x=P + 2), 1), (dict(w_dtype=1, w=P + 2), 1)])
def test_norm_rejects(L, bad, want):
    assert len(NORM) == len(L.moe_fp8_add_rms_norm.argtypes)
    assert L.moe_fp8_add_rms_norm(*{**NORM, **bad}.values()) == want


# ------------------------------------------------------------------------------------------------ layers


def rows(**kw):
    d = dict(q=P, ld=512, s=P, s_row=4, s_grp=1, rows=3)
    d.update(kw)
    return _lib.Fp8Rows(*[d[n] for n, _ in _lib.Fp8Rows._fields_])


def weight(n, k, **kw):
    d = dict(q=P, ld=k, expert_stride=n * k, s=P, first=0, count=8, N=n, K=k)
    d.update(kw)
    return _lib.Fp8Weight(*[d[name] for name, _ in _lib.Fp8Weight._fields_])


def call_fp8(L, cfg={}, gu={}, dn={}, sgu=None, sdn=None, r=None, T=3, x=P, router=None, logits=P, bias=None, limit=7.0, ws=P,
             ws_bytes=1 << 40, out=P):
    ref = ctypes.byref
    return L.moe_fp8_few_forward(ref(config(**cfg)) if cfg is not None else None, x, ref(rows(**r)) if r is not None else None, T,
                                 router, logits, bias, ref(weight(512, 512, **gu)) if gu is not None else None,
                                 ref(weight(512, 256, **dn)) if dn is not None else None,
                                 ref(weight(768, 512, **{**dict(count=1), **sgu})) if sgu is not None else None,
                                 ref(weight(512, 384, **{**dict(count=1), **sdn})) if sdn is not None else None, limit, ws, ws_bytes,
                                 out, None)


@pytest.mark.parametrize("bad,want", [
    (dict(cfg=None), 1), (dict(x=None), 1), (dict(logits=None), 1), (dict(router=P), 1), (dict(router=P, logits=None, x=None, r={}), 1),
    (dict(ws=None), 1), (dict(out=None), 1), (dict(T=0), 2), (dict(T=17), 2), (dict(cfg=dict(hidden=520)), 2),
    (dict(cfg=dict(hidden=0)), 2), (dict(cfg=dict(moe_intermediate=192)), 2), (dict(cfg=dict(num_experts=513)), 2),
    (dict(cfg=dict(num_experts=0)), 2), (dict(cfg=dict(top_k=0)), 2), (dict(cfg=dict(top_k=9)), 2),
    (dict(cfg=dict(num_experts=64, top_k=33)), 2), (dict(cfg=dict(swiglu_limit=0.0)), 1), (dict(cfg=dict(swiglu_limit=float("nan"))), 1),
    (dict(cfg=dict(flags=1)), 1), (dict(x=P + 8), 1), (dict(logits=P + 2), 1), (dict(bias=P + 2), 1), (dict(ws=P + 128), 1),
    (dict(out=P + 1), 1), (dict(ws_bytes=1000), 3), (dict(gu=None), 1), (dict(dn=None), 1), (dict(gu=dict(q=None)), 1),
    (dict(gu=dict(s=None)), 1), (dict(gu=dict(N=256)), 2), (dict(dn=dict(K=512, ld=512)), 2), (dict(dn=dict(N=256)), 2),
    (dict(gu=dict(ld=504)), 1), (dict(gu=dict(ld=520)), 1), (dict(gu=dict(q=P + 8)), 1), (dict(gu=dict(expert_stride=1024)), 1),
    (dict(gu=dict(first=1)), 2), (dict(gu=dict(first=1), dn=dict(first=1)), 2), (dict(gu=dict(count=4)), 2),
    (dict(gu=dict(count=9), dn=dict(count=9)), 2), (dict(sgu={}), 1), (dict(sdn={}), 1), (dict(sgu={}, sdn={}, limit=0.0), 1),
    (dict(sgu=dict(N=512), sdn={}), 2), (dict(sgu={}, sdn=dict(N=256)), 2),
    (dict(sgu={}, sdn={}, gu=dict(first=4, count=4), dn=dict(first=4, count=4)), 2), (dict(r=dict(q=None)), 1), (dict(r=dict(s=None)), 1),
    (dict(r=dict(rows=4)), 2), (dict(r=dict(ld=496)), 1), (dict(r=dict(ld=520)), 1), (dict(r=dict(q=P + 4)), 1)])
def test_fp8_layer_rejects(L, bad, want):
    assert call_fp8(L, **bad) == want


def test_w4_layer_rejects(L):
    def call(cfg={}, x=P, T=3, router=None, logits=P, gu=None, dn=None, ws=P, ws_bytes=1 << 40, out=P):
        return L.moe_w4a16_few_forward(ctypes.byref(config(**cfg)), x, T, router, logits, None, gu, dn, None, ws, ws_bytes, out, None)

    assert call() == 1  # no tables
    assert call(x=None, gu=P, dn=P) == 1
    for bad in (dict(hidden=384), dict(moe_intermediate=128), dict(top_k=33), dict(num_experts=1024)):
        assert call(bad, gu=P, dn=P) == 2
    assert call(T=17, gu=P, dn=P) == 2 and call(T=0, gu=P, dn=P) == 2
    assert call(router=P, gu=P, dn=P) == 1 and call(logits=None, gu=P, dn=P) == 1
    assert call(ws_bytes=1000, gu=P, dn=P) == 3 and call(ws=P + 64, gu=P, dn=P) == 1


def test_workspace_sizes(L):
    """Grow with the tokens and hold at least every slot's activations and one slice of its sums; 0 on bad sizes."""
    for fp8, shared in ((True, 0), (True, 384), (False, 0)):
        last = 0
        for T in (1, 2, 7, 16):
            n = moe.moe_few_workspace_bytes(config(), T, fp8, shared)
            assert n > last and n >= T * 2 * (2 * 256 + 512) * 4
            last = n
        assert moe.moe_few_workspace_bytes(config(), 17, fp8, shared) == 0
        assert moe.moe_few_workspace_bytes(config(hidden=500), 4, fp8, shared) == 0
    assert moe.moe_few_workspace_bytes(config(), 4, False, 128) == 0  # (NVFP4: the shared expert's result is given)
    assert moe.moe_few_workspace_bytes(config(), 4, True, 100) == 0


# ------------------------------------------------------------------------------------------------ the binding


@pytest.fixture(scope="module")
def module(L):
    m = _lib._fp8()
    m.init(_lib.MoeError, lambda size, stride, dtype, device: Fake(dtype, *size), F8, BF16, F32, torch.int32, lambda index: 0,
           lambda: 0)
    yield m
    _lib._FP8 = None
    _lib._fp8()  # torch's functions again


def norm(m, t, residual=True):
    return m.add_rms_norm(t[0], t[1], t[2] if residual else None, 1e-6, t[5], t[6] if residual else None, t[3], t[4], None)


def few_fp8(m, t, **kw):
    d = dict(router=None, logits=t[5], bias=t[6], experts=None, first=0, shared=tuple(t[7:11]), rows=(t[11], t[12]), out=t[13], x=t[0],
             top_k=2)
    d.update(kw)
    return m.few_fp8(d["x"], t[1], t[2], t[3], t[4], d["top_k"], d["router"], d["logits"], d["bias"], 7.0, True, 1.0, d["experts"],
                     d["first"], d["shared"], 7.0, d["rows"], None, d["out"], None)


class Handle:
    value = P


def few_w4(m, t, cfg=None, **kw):
    d = dict(router=t[1], logits=None, bias=t[2], shared=t[3], out=t[4])
    d.update(kw)
    return m.few_w4(cfg or config(), t[0], Handle, Handle, d["router"], d["logits"], d["bias"], d["shared"], None, d["out"], None)


SPECS = {
    "norm": (norm, [(BF16, 4, 256), (F32, 256), (BF16, 4, 256), (F8, 4, 256), (F32, 4, 2), (BF16, 4, 256), (BF16, 4, 256)]),
    "few_fp8": (few_fp8, [(BF16, 3, 512), (F8, 8, 512, 512), (F32, 8, 4, 4), (F8, 8, 512, 256), (F32, 8, 4, 2), (F32, 3, 8), (F32, 8),
                          (F8, 768, 512), (F32, 6, 4), (F8, 512, 384), (F32, 4, 3), (F8, 3, 512), (F32, 3, 4), (BF16, 3, 512)]),
    "few_w4": (few_w4, [(BF16, 3, 512), (BF16, 8, 512), (F32, 8), (BF16, 3, 512), (BF16, 3, 512)]),
}


@pytest.mark.parametrize("name", list(SPECS))
def test_tensors_of_two_gpus_are_refused(module, name):
    call, spec = SPECS[name]
    for odd in range(len(spec)):
        with pytest.raises(ValueError, match="GPU 1"):
            call(module, [Fake(*s, gpu=int(i == odd)) for i, s in enumerate(spec)])
    with pytest.raises(ValueError, match="current"):
        call(module, [Fake(*s, gpu=1) for s in spec])


@pytest.mark.parametrize("name", list(SPECS))
def test_wrong_types_and_shapes_are_refused(module, name):
    """... one tensor at a time; with all of them right the library refuses the odd pointers."""
    call, spec = SPECS[name]
    tensors = [Fake(*s) for s in spec]
    if name != "few_w4":  # (whose tables are dummies)
        with pytest.raises(_lib.MoeError):
            call(module, tensors)
    for i, (dtype, *shape) in enumerate(spec):
        for bad in (Fake(torch.float16, *shape), Fake(dtype, *shape[:-1], shape[-1] + 128), Fake(dtype, *shape, 1)):
            with pytest.raises((ValueError, _lib.MoeError)):
                call(module, tensors[:i] + [bad] + tensors[i + 1:])


def test_binding_rejects(module):
    t = [Fake(*s) for s in SPECS["few_fp8"][1]]
    for bad in (dict(logits=None), dict(shared=(t[7],)), dict(rows=t[11]), dict(x=None, router=Fake(BF16, 8, 512), logits=None),
                dict(x=None, rows=None), dict(rows=(Fake(F8, 2, 512), Fake(F32, 2, 4)))):
        with pytest.raises((ValueError, _lib.MoeError)):
            few_fp8(module, t, **bad)
    t = [Fake(*s) for s in SPECS["few_w4"][1]]
    with pytest.raises((ValueError, TypeError)):
        few_w4(module, t, cfg=b"short")


def test_no_tokens_and_cpu_tensors():
    with pytest.raises(ValueError):
        moe.moe_fp8_add_rms_norm(torch.zeros(4, 256), torch.ones(256))
    with pytest.raises(ValueError):
        moe.moe_fp8_few_forward(torch.zeros(1, 256, dtype=BF16), torch.zeros(2, 256, 256).to(F8), torch.zeros(2, 2, 2),
                                torch.zeros(2, 256, 128).to(F8), torch.zeros(2, 2, 1), 1, logits=torch.zeros(1, 2))
