"""Calls of the policy's end and of the paths around the experts that are
refused on the host.  CPU only."""
from __future__ import annotations

import pytest
import torch

from precision_quantization_moe_amd import moe_layer as ml
from precision_quantization_moe_amd import policy_head as ph
from precision_quantization_moe_amd.moe_layer import b

T, H, V = 4, 64, 40


def bf16(*s):
    return torch.zeros(*s, dtype=torch.bfloat16)


def saved(**other):
    s = dict(logits=bf16(T, V), y=bf16(T, H), h=bf16(T, H), rstd=torch.ones(T), stats=torch.zeros(T, 2),
             entropy=torch.zeros(T))
    s.update(other)
    return s


@pytest.mark.parametrize("other,error", [
    (dict(logits=bf16(T, V + 1)), "logits"), (dict(logits=bf16(T - 1, V)), "logits"),
    (dict(logits=bf16(T, 2 * V)[:, :V]), "logits"), (dict(h=bf16(T + 1, H)), "h"),
    (dict(h=torch.zeros(T, H)), "h"), (dict(rstd=torch.ones(T + 1)), "rstd"),
    (dict(y=bf16(T, H + 8)), "head_w"), (dict(logits=torch.zeros(T, V)), "reuse_logits")])
def test_head_backward(other, error):
    ids, dl = torch.zeros(T, dtype=torch.int32), torch.ones(T)
    with pytest.raises((TypeError, ValueError), match=error):
        ph.policy_head_backward(saved(**other), torch.ones(H), bf16(V, H), ids, dl, reuse_logits=True)


def test_router_and_shared():
    w = [torch.zeros(8, dtype=torch.uint8)] * 6
    with pytest.raises(ValueError, match="router"):
        ml.mxfp8_moe_block_forward(bf16(T, H), None, bf16(H), bf16(8, H), *w[:4], 2, 32, router="dense")
    with pytest.raises(ValueError, match="router"):
        ml.moe_block_backward(dict(ids=torch.zeros(T, 2)), bf16(H), bf16(8, H), bf16(T, H), None, None,
                              router=None)
    with pytest.raises(ValueError, match="shared"):
        ml.nvfp4_moe_decode(bf16(T, H), None, bf16(H), bf16(8, H), *w, 2, 32, shared=True)
    assert ml.ROUTERS == ("grouped", "linear") and b is not None
