"""A chunk's given rows are x's tokens, as many and as wide: others are refused before any call (no GPU needed)."""

import pytest
import torch

from moe_prefill_nvfp4_gb300 import fp8

from test_fp8_path_host import weight


def rows(tokens, hidden):
    return torch.zeros(tokens, hidden).to(torch.float8_e4m3fn), torch.ones(tokens, -(-hidden // 128))


@pytest.mark.parametrize("bad", [rows(2, 256), rows(4, 256), rows(0, 256), rows(3, 128), rows(3, 384), rows(3, 256)[:1],
                                 (rows(3, 256)[0], torch.ones(2, 2))])
@pytest.mark.parametrize("how", [dict(logits=torch.zeros(3, 4)), dict(w_router=torch.zeros(4, 256))])
def test_rows_of_another_size_are_refused(bad, how, monkeypatch):
    monkeypatch.setattr(fp8.moe, "moe_router_logits", lambda *args, **kw: torch.zeros(3, 4))
    layer = fp8.Fp8Experts(weight(4, 512, 256), weight(4, 256, 256), top_k=2)
    with pytest.raises(ValueError, match="rows: need"):
        layer.forward(torch.zeros(3, 256), rows=bad, **how)
