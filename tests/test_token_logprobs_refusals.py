"""Calls of the token log probabilities that are refused before anything is
launched, and the gradient's formula against differences.  CPU only."""
from __future__ import annotations

import ctypes
import math

import pytest
import torch

import precision_quantization_moe_amd as pqm
from test_linear_refusals import A, B1, B2, D, caller

B4 = ctypes.c_void_p(0x10004)
NAN, INF = math.nan, math.inf


def test_forward_arguments():
    # x dtype ld ids T V temp lp ent stats top_ids top_lp n ws bytes stream
    size = pqm.lib().pqm_token_logprobs_workspace
    need = size(4, 20000, 5)
    assert need > 0 and size(0, 20000, 5) == 0 and size(4, 20000, 33) == 0 and size(-1, 5, 0) == 0
    assert size(4, 4, 5) == 0 and size(1 << 40, 5, 0) == 0 and size(4096, 20000, 5) == 0
    c = caller("pqm_token_logprobs", [A, 0, 20000, A, 4, 20000, 1.0, D, D, D, D, D, 5, A, need, None])
    assert c(a1=2) == 4
    assert c(a4=-1) == 2 and c(a5=0) == 2 and c(a2=19999) == 2 and c(a12=33) == 2 and c(a12=-1) == 2
    assert c(a5=4, a2=4) == 2                                 # fewer logits than alternatives
    assert c(a4=1 << 31) == 2 and c(a4=1 << 62) == 2 and c(a2=(1 << 30) + 1) == 2
    assert c(a5=(1 << 30) + 1, a2=(1 << 30) + 1) == 2
    for t in (0.0, -1.0, NAN, INF, 1e-30, 1e30):
        assert c(a6=t) == 2, t
    assert c(a0=None) == 1 and c(a3=None) == 1 and c(a10=None) == 1 and c(a11=None) == 1
    assert c(a13=None) == 1
    assert c(a7=None, a8=None, a9=None, a10=None, a11=None, a12=0) == 1
    assert c(a14=need - 1) == 5
    for i in (3, 7, 8, 9, 10, 11):
        assert c(**{f"a{i}": B2}) == 3, i
    assert c(a0=B1) == 3 and c(a0=B2, a1=1) == 3 and c(a13=B4) == 3
    assert c(a4=0, a0=None) == 0


def test_backward_arguments():
    # x dtype ld ids T V temp stats ent d_lp d_ent dx dxdtype ldd stream
    c = caller("pqm_token_logprobs_backward", [A, 0, 64, A, 4, 64, 1.0, A, A, A, A, D, 0, 64, None])
    assert c(a1=2) == 4 and c(a12=2) == 4
    assert c(a4=-1) == 2 and c(a5=0) == 2 and c(a2=63) == 2 and c(a13=63) == 2 and c(a4=1 << 31) == 2
    assert c(a6=0.0) == 2 and c(a6=NAN) == 2 and c(a13=(1 << 30) + 1) == 2
    assert c(a11=A, a13=72) == 2 and c(a11=A, a12=1) == 2     # in place: other rows, another type
    for i in (0, 3, 7, 8, 11):
        assert c(**{f"a{i}": None}) == 1, i
    assert c(a9=None, a10=None) == 1
    for i in (3, 7, 8, 9, 10):
        assert c(**{f"a{i}": B2}) == 3, i
    assert c(a0=B1) == 3 and c(a11=B1) == 3 and c(a11=B2, a12=1) == 3
    assert c(a4=0, a0=None) == 0


def test_python_forms_refuse():
    x = torch.zeros(4, 64)
    with pytest.raises(TypeError, match="device"):
        pqm.token_logprobs(x)
    with pytest.raises(TypeError):
        pqm.token_logprobs(x.half())
    with pytest.raises(TypeError, match="device"):
        pqm.token_logprobs_backward(x, None, torch.zeros(4, 2), torch.zeros(4))


def test_gradient_against_differences():
    g = torch.Generator().manual_seed(1)
    x = torch.randn(7, generator=g, dtype=torch.float64)
    i, t, a, b = 3, 0.7, 1.3, -0.4

    def loss(x):
        lp = torch.log_softmax(x / t, 0)
        return a * lp[i] - b * (lp.exp() * lp).sum()
    lp = torch.log_softmax(x / t, 0)
    p, h = lp.exp(), -(lp.exp() * lp).sum()
    hot = torch.zeros(7, dtype=torch.float64)
    hot[i] = 1
    d = (a * (hot - p) - b * p * (lp + h)) / t
    for j in range(7):
        up, dn = x.clone(), x.clone()
        up[j] += 1e-5
        dn[j] -= 1e-5
        # h^2 / 6 of a third derivative below 50, and 2^-52 of a loss below 20 over 2e-5
        assert abs(float(loss(up) - loss(dn)) / 2e-5 - float(d[j])) < 2e-9
