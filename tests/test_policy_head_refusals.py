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


def odd(*s):
    """Aligned to two bytes alone."""
    n = 1
    for d in s:
        n *= d
    return bf16(n + 1)[1:].view(*s)


@pytest.mark.parametrize("other,head,norm,d_h,error", [
    (dict(logits=bf16(T, V + 1)), bf16(V + 1, H), None, None, "head_w"),
    (dict(logits=bf16(T, 0)), bf16(0, H), None, None, "head_w"),
    (dict(y=bf16(T, 12), h=bf16(T, 12)), bf16(V, 12), torch.ones(12), None, "head_w"),
    (dict(y=bf16(T, 16392), h=bf16(T, 16392)), bf16(V, 16392), torch.ones(16392), None, "head_w"),
    ({}, None, None, bf16(T + 1, H), "d_h"), ({}, None, None, torch.zeros(T, H), "d_h"),
    ({}, None, None, bf16(T, 2 * H)[:, :H], "d_h"), ({}, None, None, odd(T, H), "d_h"),
    ({}, None, torch.ones(H + 1), None, "norm_w"), ({}, None, torch.ones(H, dtype=torch.float16), None, "norm_w"),
    ({}, None, odd(H), None, "norm_w"), ({}, odd(V, H), None, None, "head_w"),
    (dict(y=odd(T, H)), None, None, None, "y"), (dict(h=odd(T, H)), None, None, None, "h"),
    (dict(y=bf16(T, 2 * H)[:, :H]), None, None, None, "y"), (dict(logits=odd(T, V)), None, None, None, "logits")])
def test_head_backward_refuses_before_it_writes(other, head, norm, d_h, error):
    """What the products or the norm would refuse is refused before the gradient
    of the logits is formed, which may be over the saved ones."""
    ids, dl = torch.zeros(T, dtype=torch.int32), torch.ones(T)
    with pytest.raises((TypeError, ValueError), match=f"^{error}:"):
        ph.policy_head_backward(saved(**other), torch.ones(H) if norm is None else norm,
                                bf16(V, H) if head is None else head, ids, dl, d_h=d_h, reuse_logits=True)


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
