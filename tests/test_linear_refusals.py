"""Calls of the dense products that are refused before anything is launched,
and the gradients' formulas against differences.  CPU only."""
from __future__ import annotations

import ctypes
import math

import pytest
import torch

import precision_quantization_moe_amd as pqm

A = ctypes.c_void_p(0x10000)
D = ctypes.c_void_p(0x20000)
B8 = ctypes.c_void_p(0x10008)
B2 = ctypes.c_void_p(0x10002)
B1 = ctypes.c_void_p(0x10001)


def caller(name, ok):
    f = getattr(pqm.lib(), name)

    def call(**kw):
        a = list(ok)
        for i, v in kw.items():
            a[int(i[1:])] = v
        return f(*a)
    return call


def test_linear_arguments():
    # x ldx w bias act res ldr M N K y ydtype z ws bytes stream
    size = pqm.lib().pqm_linear_workspace
    need = size(3000, 128, 4096)
    assert need > 0 and size(64, 128, 4096) == 0 and size(0, 128, 64) == 0 and size(300, 0, 64) == 0
    assert size(300, 128, 20) == 0 and size(-1, 128, 64) == 0 and size(1 << 40, 64, 64) == 0
    c = caller("pqm_linear", [A, 4096, A, A, 0, A, 128, 3000, 128, 4096, D, 0, D, A, need, None])
    assert c(a4=3) == 4 and c(a4=-1) == 4 and c(a11=2) == 4
    assert c(a7=-1) == 2 and c(a8=-1) == 2 and c(a9=0) == 2 and c(a9=4092) == 2
    assert c(a9=(1 << 22) + 8, a1=(1 << 22) + 8) == 2 and c(a8=(1 << 22) + 1) == 2
    assert c(a7=1 << 31) == 2 and c(a7=1 << 62) == 2 and c(a7=(1 << 31) - 1, a8=1 << 22) == 2
    assert c(a1=4088) == 2 and c(a1=(1 << 22) + 8) == 2
    assert c(a6=127) == 2 and c(a6=(1 << 22) + 1) == 2
    assert c(a5=D, a6=136) == 2 and c(a5=D, a11=1) == 2          # in place: other rows, another type
    for i in (0, 2, 10, 13):
        assert c(**{f"a{i}": None}) == 1, i
    assert c(a14=need - 1) == 5
    for i in (0, 2, 10, 12, 13):
        assert c(**{f"a{i}": B8}) == 3, i
    assert c(a1=4100) == 3 and c(a3=B2) == 3 and c(a5=B1) == 3
    assert c(a7=0, a0=None) == 0 and c(a8=0, a6=0) == 0


def test_linear_backward_arguments():
    # dy lddy x ldx w act z d_x ldd M N K dz dx dw db ws bytes stream
    size = pqm.lib().pqm_linear_backward_workspace
    need = size(4000, 128, 256)
    assert need > 0 and size(0, 128, 256) == 0 and size(10, 12, 64) == 0 and size(10, 16, 60) == 0
    c = caller("pqm_linear_backward",
               [A, 128, A, 256, A, 1, A, A, 256, 4000, 128, 256, D, D, D, D, A, need, None])
    assert c(a5=3) == 4
    assert c(a9=-1) == 2 and c(a10=0) == 2 and c(a10=132, a1=136) == 2 and c(a11=252) == 2
    assert c(a1=120) == 2 and c(a3=248) == 2 and c(a8=248) == 2
    assert c(a1=(1 << 22) + 8) == 2 and c(a3=(1 << 22) + 8) == 2 and c(a8=(1 << 22) + 8) == 2
    assert c(a7=D, a8=264) == 2                                  # d_x in place, other rows
    assert c(a13=None, a14=None, a15=None) == 1                  # nothing asked for
    for i in (0, 2, 4, 6, 12, 16):
        assert c(**{f"a{i}": None}) == 1, i
    assert c(a17=need - 1) == 5
    for i in (0, 2, 4, 6, 12, 13, 14, 15, 16):
        assert c(**{f"a{i}": B8}) == 3, i
    assert c(a1=132) == 3 and c(a3=260) == 3 and c(a7=B1) == 3


def test_python_forms_refuse():
    x, w = torch.zeros(4, 64, dtype=torch.bfloat16), torch.zeros(8, 64, dtype=torch.bfloat16)
    with pytest.raises(TypeError, match="device"):
        pqm.linear(x, w)
    with pytest.raises(TypeError):
        pqm.linear(x.float(), w)
    with pytest.raises(TypeError, match="device"):
        pqm.linear_backward(torch.zeros(4, 8, dtype=torch.bfloat16), x, w)


@pytest.mark.parametrize("gelu", [False, True])
def test_gradients_against_differences(gelu):
    """dz = dy act'(z), dx = dz W, dW = dz^T x, db = sum dz of the header against
    central differences of y in binary64."""
    g = torch.Generator().manual_seed(1)
    x, w, b, dy = (torch.randn(*s, generator=g, dtype=torch.float64)
                   for s in ((3, 5), (4, 5), (4,), (3, 4)))
    c = 2 * math.sqrt(2 / math.pi) if gelu else 1.0

    def squash(z):
        return c * (z + 0.044715 * z ** 3) if gelu else z

    def loss(x, w, b):
        z = x @ w.t() + b
        return (z * torch.sigmoid(squash(z)) * dy).sum()
    z = x @ w.t() + b
    v = torch.sigmoid(squash(z))
    ds = c * (1 + 3 * 0.044715 * z * z) if gelu else 1.0
    dz = dy * (v + z * v * (1 - v) * ds)
    for k, grad in enumerate((dz @ w, dz.t() @ x, dz.sum(0))):
        for at in range(grad.numel()):
            step = []
            for h in (1e-5, -1e-5):
                a = [x.clone(), w.clone(), b.clone()]
                a[k].view(-1)[at] += h
                step.append(loss(*a))
            # the differences' own error: h^2 / 6 of a third derivative below 100, and
            # 2^-52 of a loss below 50 over 2e-5
            assert abs(float(step[0] - step[1]) / 2e-5 - float(grad.view(-1)[at])) < 1e-8


def test_gradients_of_more_than_one_launch_holds():
    """2^24 groups of 32 rows, or 2^24 tiles of dx or of dw, are more workgroups
    of 256 threads than one launch takes: refused as sizes, with no workspace."""
    size = pqm.lib().pqm_linear_backward_workspace
    c = caller("pqm_linear_backward",
               [A, 8, A, 8, A, 1, A, None, 0, 1 << 20, 8, 8, D, D, D, D, A, 1 << 50, None])
    assert size((1 << 29) - 31, 8, 8) == 0 and size((1 << 29) - 32, 8, 8) > 0
    assert c(a9=(1 << 29) - 31) == 2 and c(a9=(1 << 29) - 1) == 2
    assert size(1 << 24, 8, 65528) == 0 and c(a9=1 << 24, a11=65528, a3=65528) == 2
    assert size(8, 1 << 22, 1 << 16) == 0 and c(a9=8, a10=1 << 22, a1=1 << 22, a11=1 << 16, a3=1 << 16) == 2
