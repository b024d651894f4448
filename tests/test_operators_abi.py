"""Refusals of the norm, gate and few-row product entry points (host-side,
nothing is launched), and of their Python forms; the gradient formulas the GPU
tests use, against differences in binary64.  CPU only."""
from __future__ import annotations

import ctypes

import pytest
import torch

import operators_ref as ref
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


def test_rmsnorm_quantize_arguments():
    # x ldx residual ldr weight wdtype rows cols eps sum y q s rstd stream
    c = caller("pqm_rmsnorm_quantize_mxfp8",
               [A, 64, A, 64, A, 0, 4, 64, 1e-6, D, A, A, A, A, None])
    assert c(a5=2) == 4
    assert c(a6=-1) == 2 and c(a7=-32) == 2
    assert c(a7=48) == 2                              # quantized: cols % 32
    assert c(a7=20, a11=None, a12=None) == 2          # cols % 8
    assert c(a7=16416, a1=16416, a3=16416) == 2       # cols > 16384
    assert c(a6=1 << 31) == 2
    assert c(a1=56) == 2 and c(a3=56) == 2            # strides below cols
    assert c(a8=0.0) == 2 and c(a8=-1.0) == 2
    assert c(a8=float("nan")) == 2 and c(a8=float("inf")) == 2
    assert c(a0=None) == 1 and c(a4=None) == 1
    assert c(a11=None) == 1 and c(a12=None) == 1      # half a pair
    assert c(a10=None, a11=None, a12=None) == 1       # no output
    for i in (0, 2, 4, 9, 10):
        assert c(**{f"a{i}": B8}) == 3, i             # 16-byte
    assert c(a11=B2) == 3 and c(a13=B2) == 3
    assert c(a1=68) == 3 and c(a3=68) == 3            # stride not 16 bytes
    assert c(a1=72, a9=A, a2=D) == 2                  # sum is x, with another stride
    assert c(a0=D, a3=72, a9=A) == 2                  # sum is residual, the same
    assert c(a6=0, a0=None) == 0 and c(a7=0) == 0     # nothing to do


def test_rmsnorm_backward_arguments():
    # dy x weight wdtype rstd d_sum rows cols dx dweight ws bytes stream
    ws = pqm.lib().pqm_rmsnorm_backward_workspace
    assert ws(0, 64) == 0 and ws(4, 0) == 0 and ws(4, 16392) == 0
    need = ws(4, 64)
    assert need > 0
    c = caller("pqm_rmsnorm_backward", [A, A, A, 0, A, None, 4, 64, A, A, A, need, None])
    assert c(a3=2) == 4
    assert c(a6=-1) == 2 and c(a7=20) == 2 and c(a7=16392) == 2
    for i in (0, 1, 2, 4, 8, 9, 10):
        assert c(**{f"a{i}": None}) == 1, i
    assert c(a11=need - 1) == 5
    for i in (0, 1, 2, 5, 8, 10):
        assert c(**{f"a{i}": B8}) == 3, i
    assert c(a4=B2) == 3 and c(a9=B2) == 3
    assert c(a7=0) == 0


def test_moe_gate_arguments():
    # z dtype mask T E k score renorm scale ids prob coef counts psum loss ws bytes stream
    size = pqm.lib().pqm_moe_gate_workspace
    assert size(-1, 8) == 0 and size(4, 0) == 0 and size(4, 1025) == 0
    need = size(4, 8)
    ok = [A, 1, None, 4, 8, 2, 0, 1, 1.0, A, A, 0.01, A, A, A, A, need, None]
    c = caller("pqm_moe_gate", ok)
    assert c(a1=2) == 4 and c(a6=2) == 4 and c(a7=2) == 4
    assert c(a3=-1) == 2 and c(a4=0) == 2 and c(a4=1025) == 2
    assert c(a5=0) == 2 and c(a5=17, a4=64) == 2 and c(a5=9) == 2   # k > 16, k > E
    assert c(a3=1 << 30) == 2
    for i in (0, 9, 10, 12, 13, 14, 15):
        assert c(**{f"a{i}": None}) == 1, i
    assert c(a16=need - 1) == 5
    for i in (0, 9, 10, 12, 13, 14, 15):
        assert c(**{f"a{i}": B2}) == 3, i
    assert c(a0=B1, a1=0) == 3                        # bf16 logits: 2 bytes
    assert c(a3=0, a12=None, a13=None, a14=None) == 0  # no tokens, no loss


def test_moe_gate_backward_arguments():
    # z dtype mask T E k score renorm scale ids d_prob coef counts d_loss dz dzdtype stream
    c = caller("pqm_moe_gate_backward",
               [A, 1, None, 4, 8, 2, 0, 1, 1.0, A, A, 0.01, A, A, A, 1, None])
    assert c(a1=2) == 4 and c(a6=2) == 4 and c(a7=2) == 4 and c(a15=2) == 4
    assert c(a3=-1) == 2 and c(a4=1025) == 2 and c(a5=9) == 2
    for i in (0, 9, 12, 13, 14):
        assert c(**{f"a{i}": None}) == 1, i
    assert c(a10=None, a12=None, a13=None) == 1       # no gradient at all
    for i in (0, 9, 10, 12, 13, 14):
        assert c(**{f"a{i}": B2}) == 3, i
    assert c(a3=0) == 0


def test_moe_gemv_arguments():
    # x ids rows div wq ws wo rps G N K out dtype stream
    c = caller("pqm_moe_gemv_nvfp4", [A, A, 8, 2, A, A, A, 64, 4, 64, 64, A, 0, None])
    assert c(a12=2) == 4
    assert c(a2=-1) == 2 and c(a2=4097) == 2
    assert c(a3=0) == 2 and c(a3=4097) == 2
    assert c(a8=0) == 2 and c(a8=4097) == 2
    assert c(a9=-1) == 2 and c(a9=(1 << 20) + 1, a7=1) == 2
    assert c(a10=0) == 2 and c(a10=48) == 2 and c(a10=1 << 21) == 2
    assert c(a7=0) == 2 and c(a7=3) == 2
    assert c(a2=1 << 40) == 2 and c(a8=1 << 40) == 2  # sizes that leave 32 bits
    for i in (0, 1, 4, 5, 6, 11):
        assert c(**{f"a{i}": None}) == 1, i
    for i in (0, 4, 11):
        assert c(**{f"a{i}": B8}) == 3, i
    for i in (1, 5, 6):
        assert c(**{f"a{i}": B2}) == 3, i
    assert c(a2=0) == 0 and c(a9=0) == 0
    # x ids prob rows div wq ws wo rps G inter K d stream
    c = caller("pqm_moe_gemv_swiglu_nvfp4", [A, A, A, 8, 2, A, A, A, 64, 4, 32, 64, A, None])
    assert c(a8=3) == 2 and c(a11=48) == 2 and c(a3=4097) == 2
    for i in (0, 1, 2, 5, 6, 7, 12):
        assert c(**{f"a{i}": None}) == 1, i
    assert c(a2=B2) == 3 and c(a12=B8) == 3
    assert c(a3=0) == 0 and c(a10=0) == 0


def test_python_forms_refuse_host_and_mixed_tensors():
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    w = torch.ones(64)
    with pytest.raises(TypeError):
        pqm.rmsnorm_quantize_mxfp8(x, w)              # not on a device
    with pytest.raises(TypeError):
        pqm.rmsnorm_backward(x, x, w, torch.ones(4))
    with pytest.raises(TypeError):
        pqm.moe_gate(torch.zeros(4, 8), 2)
    with pytest.raises(TypeError):
        pqm.moe_gate(torch.zeros(4, 8, dtype=torch.float16), 2)
    with pytest.raises(TypeError):
        pqm.moe_gate_backward(torch.zeros(4, 8), torch.zeros(4, 2, dtype=torch.int32), None)
    with pytest.raises(TypeError):
        pqm.moe_gemv_nvfp4(x, torch.zeros(4, dtype=torch.int32), None, None, None, 64)


def differences(f, z, step=1e-6):
    g = torch.zeros_like(z)
    flat, out = z.view(-1), g.view(-1)
    for i in range(flat.numel()):
        keep = float(flat[i])
        flat[i] = keep + step
        up = float(f(z))
        flat[i] = keep - step
        out[i] = (up - float(f(z))) / (2 * step)
        flat[i] = keep
    return g


@pytest.mark.parametrize("softmax", [True, False])
@pytest.mark.parametrize("renorm", [True, False])
def test_gate_gradient_formula_against_differences(softmax, renorm):
    g = torch.Generator().manual_seed(3)
    z = torch.randn(5, 7, generator=g, dtype=torch.float64) * 2
    mask = torch.tensor([1, 1, 0, 1, 1])
    r = ref.gate(z, 3, softmax, renorm, 1.5, mask, 0.3)
    d_prob = torch.randn(5, 3, generator=g, dtype=torch.float64)
    args = (r["ids"], r["counts"], r["n"], softmax, renorm, 1.5, r["live"], 0.3, d_prob, 0.7)
    got, _ = ref.gate_backward(z, *args)
    want = differences(lambda v: ref.gate_objective(v, *args), z)
    # central differences: the step's square and the sum's rounding over it
    assert (got - want).abs().max() < 1e-8


def test_norm_gradient_formula_against_differences():
    g = torch.Generator().manual_seed(4)
    x = torch.randn(3, 8, generator=g, dtype=torch.float64)
    w = torch.rand(8, generator=g, dtype=torch.float64) + 0.5
    dy, ds = (torch.randn(3, 8, generator=g, dtype=torch.float64) for _ in range(2))
    eps = 1e-2
    _, rstd = ref.norm(x, w, eps)
    dx, dw, _, _ = ref.norm_backward(dy, x, w, rstd, ds)
    f = lambda v, u: (ref.norm(v, u, eps)[0] * dy).sum() + (v * ds).sum()  # noqa: E731
    assert (dx - differences(lambda v: f(v, w), x)).abs().max() < 1e-8
    assert (dw - differences(lambda u: f(x, u), w)).abs().max() < 1e-8
