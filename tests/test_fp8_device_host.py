"""The FP8 binding takes tensors of one GPU, the current one, and refuses others before any launch.

Stand-ins for tensors of two GPUs.  Their pointers are odd, which the library refuses by itself on the host: no
call of this file can reach a launch."""

import pytest
import torch

from moe_prefill_nvfp4_gb300 import _lib, build

F8, F32, BF16, I32 = torch.float8_e4m3fn, torch.float32, torch.bfloat16, torch.int32


class Fake:
    def __init__(self, dtype, *shape, gpu=0):
        self.dtype, self.shape, self.gpu = dtype, shape, gpu
        self.is_cuda, self.device = True, f"cuda:{gpu}"

    def stride(self):
        s = [1]
        for n in self.shape[:0:-1]:
            s.insert(0, s[0] * n)
        return tuple(s)

    def data_ptr(self):
        return 4097

    def get_device(self):
        return self.gpu


def quantise(blocks):
    rows = 1 if blocks else 4
    return (lambda m, t: m.quantize(t[0], t[1], t[2], None, blocks),
            [(BF16, 4, 256), (F8, 4, 256), (F32, rows, 2)])


CALLS = {
    "quantize_rows": quantise(False),
    "quantize_blocks": quantise(True),
    "gemm": (lambda m, t: m.gemm(*t, BF16, None), [(F8, 4, 256), (F32, 4, 2), (F8, 128, 256), (F32, 1, 2), (BF16, 4, 128)]),
    "grouped": (lambda m, t: m.grouped(*t[:5], 4, t[5], 0, t[6], BF16, None),
                [(F8, 4, 256), (F32, 4, 2), (F8, 2, 128, 256), (F32, 2, 1, 2), (I32, 3), (I32, 4), (BF16, 4, 128)]),
    "grouped_swiglu": (lambda m, t: m.grouped_swiglu(*t[:5], 4, 7.0, t[5], 0, t[6], t[7], None),
                       [(F8, 4, 256), (F32, 4, 2), (F8, 2, 256, 256), (F32, 2, 2, 2), (I32, 3), (I32, 4), (F8, 4, 128),
                        (F32, 4, 1)]),
}


@pytest.fixture(scope="module")
def module():
    build.build()
    m = _lib._fp8()
    m.init(_lib.MoeError, lambda size, stride, dtype, device: Fake(dtype, *size), F8, BF16, F32, I32, lambda index: 0,
           lambda: 0)
    yield m
    _lib._FP8 = None
    _lib._fp8()  # torch's functions again


@pytest.mark.parametrize("name", list(CALLS))
def test_tensors_of_two_gpus_are_refused(module, name):
    call, spec = CALLS[name]
    for odd in range(1, len(spec)):
        with pytest.raises(ValueError, match="on GPU 1"):
            call(module, [Fake(*s, gpu=int(i == odd)) for i, s in enumerate(spec)])
    with pytest.raises(ValueError, match="GPU 1"):  # the first alone on GPU 1
        call(module, [Fake(*s, gpu=int(i == 0)) for i, s in enumerate(spec)])


@pytest.mark.parametrize("name", list(CALLS))
def test_tensors_of_another_than_the_current_gpu_are_refused(module, name):
    call, spec = CALLS[name]
    with pytest.raises(ValueError, match="current"):
        call(module, [Fake(*s, gpu=1) for s in spec])


@pytest.mark.parametrize("name", list(CALLS))
def test_the_current_gpu_passes(module, name):
    """... to the library, which refuses the odd pointers."""
    call, spec = CALLS[name]
    with pytest.raises(_lib.MoeError):
        call(module, [Fake(*s) for s in spec])
