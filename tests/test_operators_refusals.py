"""Calls of the norm, gate, few-row products and block passes that have to be
refused before anything is launched.  CPU only."""
from __future__ import annotations

import ctypes

import pytest
import torch

import precision_quantization_moe_amd as pqm
from precision_quantization_moe_amd import moe_layer as ml

A = ctypes.c_void_p(0x10000)


@pytest.mark.parametrize("tokens,k", [((1 << 31) // 2, 1), ((1 << 31) // 16, 15), (1 << 60, 15), (1 << 62, 3),
                                      ((1 << 63) - 1, 1), ((1 << 63) - 1, 16)])
def test_gate_refuses_more_tokens_than_its_limit(tokens, k):
    """tokens (k + 1) from 2^31 on, also where the product leaves 64 bits."""
    L = pqm.lib()
    size = 1 << 40
    assert L.pqm_moe_gate(A, 1, None, tokens, 64, k, 0, 1, 1.0, A, A, 0.01, A, A, A, A, size, None) == 2
    assert L.pqm_moe_gate(A, 1, None, tokens, 64, k, 0, 1, 1.0, A, A, 0.0, None, None, None, None, 0,
                          None) == 2
    assert L.pqm_moe_gate_backward(A, 1, None, tokens, 64, k, 0, 1, 1.0, A, A, 0.01, A, A, A, 1, None) == 2


def test_workspace_queries_of_sizes_that_no_call_takes():
    L = pqm.lib()
    for n in (1 << 31, (1 << 63) - 1):
        assert L.pqm_moe_gate_workspace(n, 64) == 0
        assert L.pqm_rmsnorm_backward_workspace(n, 64) == 0
    assert L.pqm_moe_gate_workspace((1 << 30) - 1, 64) == L.pqm_moe_gate_workspace(1 << 20, 64) > 0
    assert L.pqm_rmsnorm_backward_workspace((1 << 31) - 1, 64) == \
        L.pqm_rmsnorm_backward_workspace(1 << 20, 64) > 0


# The block passes look over what they are given before any call, so that their
# refusals show on the host too: T tokens of H values, E experts of I, top-K.
T, H, E, I, K = 6, 64, 8, 32, 2


def bf16(*shape):
    return torch.zeros(*shape, dtype=torch.bfloat16)


def u8(*shape):
    return torch.zeros(*shape, dtype=torch.uint8)


def nvfp4_weights(e=E):
    return (u8(e * 2 * I, H // 2), u8(e * 2 * I, H // 16), torch.ones(e),
            u8(e * H, I // 2), u8(e * H, I // 16), torch.ones(e))


def mxfp8_weights(e=E):
    return u8(e * 2 * I, H), u8(e * 2 * I, H // 32), u8(e * H, I), u8(e * H, I // 32)


def decode(plan=None, gate_w=None, weights=None):
    return ml.nvfp4_moe_decode(bf16(T, H), bf16(T, H), bf16(H), bf16(E, H) if gate_w is None else gate_w,
                               *(weights or nvfp4_weights()), K, I, plan)


def forward(plan=None, gate_w=None, weights=None):
    return ml.mxfp8_moe_block_forward(bf16(T, H), bf16(T, H), bf16(H), bf16(E, H) if gate_w is None else gate_w,
                                      *(weights or mxfp8_weights()), K, I, plan=plan)


def saved_of(t=T, e=E, h=H):
    return dict(h=bf16(t, h), y=bf16(t, h), rstd=torch.ones(t), logits=torch.zeros(t, e),
                ids=torch.zeros(t, K, dtype=torch.int32), counts=torch.zeros(e + 1, dtype=torch.int32))


def backward(plan=None, saved=None, gate_w=None, dy=None):
    return ml.moe_block_backward(saved or saved_of(), bf16(H), bf16(E, H) if gate_w is None else gate_w,
                                 bf16(T, H) if dy is None else dy, torch.zeros(T, K), torch.ones(1), plan=plan)


PASSES = [decode, forward, backward]


@pytest.mark.parametrize("call", PASSES)
@pytest.mark.parametrize("t,k", [(T + 1, K), (T - 1, K), (4 * T, K), (0, K), (T, K + 1), (T, 1)])
def test_a_plan_for_other_sizes_is_refused(call, t, k):
    """A larger plan would send the products past their rows, a smaller one
    leave rows unwritten."""
    with pytest.raises(ValueError, match="plan"):
        call(ml.block_plan(t, k, "cpu"))


@pytest.mark.parametrize("call", PASSES)
def test_a_plan_on_another_device_or_in_parts_is_refused(call):
    with pytest.raises(ValueError, match="plan"):
        call(ml.block_plan(T, K, "meta"))
    good = ml.block_plan(T, K, "cpu")
    for name in good:
        with pytest.raises(ValueError, match="plan"):
            call({n: v for n, v in good.items() if n != name})
        with pytest.raises(ValueError, match="plan"):
            call(dict(good, **{name: good[name][:-1]}))
        with pytest.raises(ValueError, match="plan"):
            call(dict(good, **{name: good[name].float()}))
    wide = ml.block_plan(T, K + 1, "cpu")["slot"][:, :K]
    with pytest.raises(ValueError, match="plan"):
        call(dict(good, slot=wide))


@pytest.mark.parametrize("call", PASSES)
def test_the_plan_made_for_the_call_is_taken(call):
    with pytest.raises(TypeError, match="device tensor"):  # on to the first operator, which wants a GPU
        call(ml.block_plan(T, K, "cpu"))
    with pytest.raises(TypeError, match="device tensor"):
        call()


@pytest.mark.parametrize("call,weights", [(decode, nvfp4_weights), (forward, mxfp8_weights)])
@pytest.mark.parametrize("e", [E + 1, E - 1, 0, 2 * E])
def test_weights_of_other_experts_than_the_routers_are_refused(call, weights, e):
    """One group more is a shared expert, which these passes do not have: its
    product would be left out in silence."""
    with pytest.raises(ValueError, match="experts"):
        call(weights=weights(e))
    first = weights()[:len(weights()) // 2]
    with pytest.raises(ValueError, match="experts"):
        call(weights=first + weights(e)[len(first):])


@pytest.mark.parametrize("call", PASSES)
def test_a_router_weight_of_another_kind_is_refused(call):
    with pytest.raises(TypeError, match="gate_w"):
        call(gate_w=torch.zeros(E, H))
    with pytest.raises(TypeError, match="gate_w"):
        call(gate_w=bf16(E, H).to("meta"))
    with pytest.raises(ValueError, match="gate_w"):
        call(gate_w=bf16(E, H + 32))
    with pytest.raises(ValueError, match="gate_w"):
        call(gate_w=bf16(H, E).t())


def test_expert_weights_of_another_kind_are_refused():
    q1, s1, q2, s2 = mxfp8_weights()
    for bad in ((q1, s1[:-1], q2, s2), (q1, s1, q2, s2[:, :-1]), (q1.float(), s1, q2, s2),
                (u8(H, E * 2 * I).t(), s1, q2, s2), (q1, s1, q2.to("meta"), s2)):
        with pytest.raises(ValueError, match="experts"):
            forward(weights=bad)


@pytest.mark.parametrize("bad", [saved_of(t=T - 1), saved_of(t=T + 3), saved_of(e=E - 1), saved_of(e=E + 8),
                                 saved_of(h=H + 32),
                                 dict(saved_of(), y=bf16(T - 1, H)), dict(saved_of(), h=bf16(T + 1, H)),
                                 dict(saved_of(), y=torch.zeros(T, H)), dict(saved_of(), y=bf16(H, T).t()),
                                 dict(saved_of(), logits=torch.zeros(E, T).t()),
                                 dict(saved_of(), rstd=torch.ones(T - 1))],
                         ids=range(11))
def test_gradients_of_another_calls_values_are_refused(bad):
    """The weight's gradient takes as many rows of y as dy has."""
    with pytest.raises((ValueError, TypeError), match="y:|h:|rstd:|logits:|ids:|counts:"):
        backward(saved=bad)


def test_gradients_of_strided_rows_are_refused():
    wide = bf16(T, 2 * H)[:, :H]
    with pytest.raises(ValueError, match="dy:"):
        backward(dy=wide)
    with pytest.raises(TypeError, match="dy:"):
        backward(dy=torch.zeros(T, H))
