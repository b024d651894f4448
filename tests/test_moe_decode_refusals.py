"""Calls of the whole expert layer that are refused before anything is
launched.  CPU only."""
from __future__ import annotations

import ctypes
import math

import pytest
import torch

import precision_quantization_moe_amd as pqm
from test_linear_refusals import A, B2, B8, D, caller


def test_arguments():
    # x res nw nwdtype eps gw T H I E k shared score renorm scale w1q w1s w1g w2q w2s w2g
    # h y ids prob d out ws bytes stream
    size = pqm.lib().pqm_moe_decode_nvfp4_workspace
    need = size(3, 256, 128, 16, 4, 1)
    assert need > 0 and size(0, 256, 128, 16, 4, 1) == 0 and size(65, 256, 128, 16, 4, 1) == 0
    assert size(3, 250, 128, 16, 4, 1) == 0 and size(3, 256, 128, 16, 17, 0) == 0
    ok = [A, A, A, 0, 1e-6, A, 3, 256, 128, 16, 4, 1, 0, 1, 1.0] + [A] * 6 + [D] * 6 + [A, need, None]
    c = caller("pqm_moe_decode_nvfp4", ok)
    assert c(a3=2) == 4 and c(a12=2) == 4 and c(a13=2) == 4 and c(a11=2) == 4 and c(a11=-1) == 4
    assert c(a6=-1) == 2 and c(a6=65) == 2 and c(a6=1 << 40) == 2
    for i in (7, 8):
        for bad in (0, 16, 48, 16416, 1 << 40):
            assert c(**{f"a{i}": bad}) == 2, (i, bad)
    assert c(a9=0) == 2 and c(a9=1025) == 2 and c(a10=0) == 2 and c(a10=17, a9=32) == 2 and c(a9=3) == 2
    for eps in (0.0, -1.0, math.nan, math.inf):
        assert c(a4=eps) == 2, eps
    for i in (0, 2, 5, *range(15, 28)):
        assert c(**{f"a{i}": None}) == 1, i
    assert c(a28=need - 1) == 5
    for i in (0, 1, 2, 5, 15, 18, 21, 22, 25, 26, 27):
        assert c(**{f"a{i}": B8}) == 3, i
    for i in (16, 17, 19, 20, 23, 24):
        assert c(**{f"a{i}": B2}) == 3, i
    assert c(a6=0, a0=None) == 0


T, H, E, I, K = 6, 64, 8, 32, 2


def test_python_form_refuses():
    b16 = lambda *s: torch.zeros(*s, dtype=torch.bfloat16)  # noqa: E731
    u8 = lambda *s: torch.zeros(*s, dtype=torch.uint8)  # noqa: E731
    w = [u8(E * 2 * I, H // 2), u8(E * 2 * I, H // 16), torch.ones(E), u8(E * H, I // 2), u8(E * H, I // 16),
         torch.ones(E)]
    with pytest.raises(TypeError, match="device"):
        pqm.moe_decode_nvfp4(b16(T, H), None, b16(H), b16(E, H), *w, K, I)
    with pytest.raises(TypeError):
        pqm.moe_decode_nvfp4(torch.zeros(T, H), None, b16(H), b16(E, H), *w, K, I)
