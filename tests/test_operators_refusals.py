"""Calls of the norm, gate, few-row products and block passes that have to be
refused before anything is launched.  CPU only."""
from __future__ import annotations

import ctypes

import pytest

import precision_quantization_moe_amd as pqm

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
