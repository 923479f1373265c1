"""The workspace of the few-token layers is a matter of the sizes alone, not of a device: the slices of k that it holds
are also the order of the sums (no GPU needed)."""

import pytest

import moe_prefill_nvfp4_gb300 as moe
from moe_prefill_nvfp4_gb300 import build


def up(n):
    return -(-n // 256) * 256


def slices(blocks, units, least):
    """K blocks of 8 to a unit, fewer where 304 CTAs would have fewer than two units each."""
    want = 8
    while want > least and units * -(-blocks // want) < 2 * 304:
        want //= 2
    each = -(-blocks // -(-blocks // want))
    return -(-blocks // each)


def expected(T, H, I, Is, E, k, fp8):
    kb, block_bytes, least = (128, 128, 4) if fp8 else (256, 896, 2)
    entries, slots = min(E, T * k) + (Is > 0), T * k
    wide, deep = H // kb, max(I, Is) // kb
    s0, s1 = slices(wide, entries * (I // 128), least), slices(deep, entries * -(-H // 256), least)
    pitch = (lambda b: -(-b // 32) * 32) if fp8 else (lambda b: b)
    columns = -(-H // 256)
    parts = [4 * (64 + entries + entries * deep + columns), 4 * T * E, T * wide * block_bytes, 4 * T * wide, 4 * s0 * slots * 2 * I,
             slots * (I // kb) * block_bytes, 4 * slots * pitch(I // kb), 4 * s0 * T * 2 * Is, T * (Is // kb) * block_bytes,
             4 * T * pitch(Is // kb), 4 * s1 * (slots + (T if Is else 0)) * H]
    return sum(up(p) for p in parts)


@pytest.mark.parametrize("T,H,I,Is,E,k", [(1, 5120, 1536, 0, 160, 8), (16, 5120, 1536, 0, 160, 8), (4, 2048, 768, 0, 64, 8),
                                          (5, 1152, 640, 384, 33, 3), (7, 1280, 512, 0, 33, 3), (1, 256, 256, 0, 1, 1),
                                          (16, 4096, 2048, 0, 8, 8), (16, 1024, 512, 2048, 512, 32), (3, 128, 128, 128, 2, 1)])
def test_workspace_bytes_of_the_sizes(T, H, I, Is, E, k):
    build.build()
    cfg = moe.MoePrefillConfig(hidden=H, moe_intermediate=I, num_experts=E, top_k=k)
    assert moe.moe_few_workspace_bytes(cfg, T, True, Is) == expected(T, H, I, Is, E, k, True)
    if H % 256 == 0 and I % 256 == 0:
        assert moe.moe_few_workspace_bytes(cfg, T, False) == expected(T, H, I, 0, E, k, False)
    else:
        assert moe.moe_few_workspace_bytes(cfg, T, False) == 0
