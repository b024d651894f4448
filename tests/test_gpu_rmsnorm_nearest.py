"""The norm's exactness on the GPU: rstd is the binary32 value next to the
binary64 one, and y the bf16 value next to the binary64 product.

Bounds.  The kernel's binary64 sum adds at most 64 squares a thread and joins
the threads in 8 steps, the reference's no worse; with mean, root and products
both keep 2^-45 of the value.  So rstd is within half a step of binary32 and
that (subnormal: half of 2^-149), and only a product within 2^-40 of itself
from the middle of two bf16 values may go to either of them."""
from __future__ import annotations

import pytest
import torch

import operators_ref as ref
import precision_quantization_moe_amd as pqm
from gpu_util import requires_gpu

pytestmark = [pytest.mark.gpu, requires_gpu]

U = 2.0 ** -24


def nearest(v):
    """bf16 values next to binary64 v, ties to even, subnormal ones too, and
    where v lies in the middle of two."""
    step = torch.exp2((torch.frexp(v).exponent - 1).clamp(min=-126).double() - 7)
    part = v / step
    middle = ((part - part.floor() - 0.5).abs() <= 2.0 ** -40 * part.abs())
    return torch.round(part) * step, step, middle


def check(x, r, w, eps, out):
    q, s, y, total, rstd = out
    want = x if r is None else (x.float() + r.float()).to(torch.bfloat16)
    assert torch.equal(total, want)
    v = want.double()
    root = (v.square().mean(1) + eps).pow(-0.5)
    assert ((rstd.double() - root).abs() <= (1 + 2.0 ** -20) * U * root + 2.0 ** -150).all()
    n, step, middle = nearest(v * w.double() * root[:, None])
    off = (y.double() - n).abs()
    assert (off <= torch.where(middle, step, 0.0)).all(), \
        f"{int((off > 0).sum())} of {off.numel()} values are not the nearest"
    if q is not None:
        oq, os_, _, _ = pqm.quantize_mxfp8(y, colwise=False)
        assert torch.equal(q, oq) and torch.equal(s, os_)


def rows_of(kind, rows, cols, seed):
    """(x, w, eps) whose x rstd, rstd or y leave the normal numbers of binary32."""
    g = torch.Generator().manual_seed(seed)
    u = torch.randn(rows, cols, generator=g)
    w = 1 + 0.3 * torch.randn(cols, generator=g)
    if kind == "small values of a large row":      # x rstd about 2^-140, lifted by w
        x, w, eps = u * 2.0 ** -80, w * 2.0 ** 20, 1e-6
        x[:, ::cols // 8] = 2.0 ** 60
    elif kind == "values that vanish before w":    # x rstd about 2^-160
        x, w, eps = u * 2.0 ** -100, w * 2.0 ** 100, 1e-6
        x[:, 5] = 2.0 ** 60
        w[5] = 1
    elif kind == "rows of the largest values":     # rstd below 2^-126
        x, eps = torch.sign(u) * (1 + torch.rand(rows, cols, generator=g)) * 2.0 ** 127, 1e-6
        x = x.clamp(-3.3e38, 3.3e38)
    elif kind == "subnormal output":
        x, w, eps = u, w * 2.0 ** -131, 1e-6
    elif kind == "subnormal input":                # x rstd about 2^-126
        x, w, eps = u * 2.0 ** -131, w * 2.0 ** 20, 2.0 ** -10
    else:                                          # every size in one row
        x = torch.sign(u) * torch.exp2(torch.rand(rows, cols, generator=g) * 250 - 130)
        w, eps = torch.exp2(torch.rand(cols, generator=g) * 100), 2.0 ** -100
    return x.to(torch.bfloat16).cuda(), w.cuda(), eps


KINDS = ["small values of a large row", "values that vanish before w", "rows of the largest values",
         "subnormal output", "subnormal input", "every size"]


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("rows,cols", [(64, 512), (40, 2048), (1100, 2048), (33, 4096), (9, 7168)])
@pytest.mark.parametrize("wf32", [False, True])
def test_y_is_the_nearest_value_beyond_the_normal_numbers(kind, rows, cols, wf32):
    x, w, eps = rows_of(kind, rows, cols, rows + cols)
    w = w if wf32 else w.to(torch.bfloat16)
    check(x, None, w, eps, pqm.rmsnorm_quantize_mxfp8(x, w, eps, keep_y=True))


@pytest.mark.parametrize("cols", [96, 2048, 5024])
@pytest.mark.parametrize("wf32", [False, True])
def test_infinities_and_nan_in_a_row(cols, wf32):
    """An infinity makes rstd 0: zeros beside it, no value in its own place.  A
    NaN takes its whole row; the other rows are as without them."""
    g = torch.Generator().manual_seed(cols)
    x = torch.randn(12, cols, generator=g).to(torch.bfloat16).cuda()
    w = (1 + 0.3 * torch.randn(cols, generator=g)).cuda()
    w = w if wf32 else w.to(torch.bfloat16)
    clean = pqm.rmsnorm_quantize_mxfp8(x, w, 1e-6, keep_y=True)
    x[1, 7] = float("inf")
    x[3, cols - 1] = -float("inf")
    x[5, ::3] = float("inf")
    x[7, 9] = float("nan")
    x[9, 2], x[9, 70] = float("nan"), float("inf")
    q, s, y, total, rstd = pqm.rmsnorm_quantize_mxfp8(x, w, 1e-6, keep_y=True)
    keep = [0, 2, 4, 6, 8, 10, 11]
    for a, b in zip(clean, (q, s, y, total, rstd)):
        assert torch.equal(a[keep], b[keep])
    assert not rstd[[1, 3, 5]].any() and rstd[[7, 9]].isnan().all()
    for row in (1, 3, 5):
        there = torch.isinf(x[row])
        assert y[row][there].isnan().all() and not y[row][~there].any()
    assert y[[7, 9]].isnan().all()
    oq, os_, _, _ = pqm.quantize_mxfp8(y, colwise=False)
    assert torch.equal(q, oq) and torch.equal(s, os_)
    # finite values whose sum leaves bf16: the sum is an infinity
    a = torch.full((1, cols), 3e38).to(torch.bfloat16).cuda()
    _, _, y, total, rstd = pqm.rmsnorm_quantize_mxfp8(a, w, 1e-6, residual=a, keep_y=True)
    assert torch.isinf(total).all() and not rstd.any() and y.isnan().all()


def usual(rows, cols, wf32, residual, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = (torch.randn(rows, cols, generator=g, device="cuda")
         * torch.exp(torch.randn(rows, 1, generator=g, device="cuda"))).to(torch.bfloat16)
    r = torch.randn(rows, cols, generator=g, device="cuda").to(torch.bfloat16) if residual else None
    w = 1 + 0.3 * torch.randn(cols, generator=g, device="cuda")
    return x, r, w if wf32 else w.to(torch.bfloat16)


# every width's kernel, with and without streaming (from 2^21 values on)
@pytest.mark.parametrize("rows,cols", [(1, 32), (5, 96), (9, 1024), (33, 1056), (300, 2048), (3, 4128),
                                       (131, 7168), (2, 8224), (3, 16384),
                                       (4200, 512), (2100, 1024), (1030, 2048), (515, 4096), (300, 7168),
                                       (260, 8192), (130, 16384)])
@pytest.mark.parametrize("wf32", [False, True])
@pytest.mark.parametrize("residual", [False, True])
def test_y_and_rstd_are_the_nearest_values(rows, cols, wf32, residual):
    x, r, w = usual(rows, cols, wf32, residual, rows + cols)
    out = pqm.rmsnorm_quantize_mxfp8(x, w, 1e-6, residual=r, keep_y=True)
    check(x, r, w, 1e-6, out)
    again = pqm.rmsnorm_quantize_mxfp8(x, w, 1e-6, residual=r)
    for i in (0, 1, 3, 4):
        assert torch.equal(out[i], again[i]), i
    if residual:
        mine = r.clone()
        again = pqm.rmsnorm_quantize_mxfp8(x, w, 1e-6, residual=mine, keep_y=True, inplace=True)
        assert again[3] is mine and all(torch.equal(a, b) for a, b in zip(out, again))


# every width's gradients with streaming loads (from 2^25 values on)
@pytest.mark.parametrize("rows,cols", [(65540, 512), (32771, 1024), (16385, 2048), (8193, 4096), (4700, 7168),
                                       (2050, 16384)])
@pytest.mark.parametrize("wf32", [False, True])
def test_gradients_of_large_calls(rows, cols, wf32):
    x, ds, w = usual(rows, cols, wf32, True, rows + cols)
    g = torch.Generator(device="cuda").manual_seed(1)
    dy = torch.randn(rows, cols, generator=g, device="cuda").to(torch.bfloat16)
    rstd = (x.double().square().mean(1) + 1e-6).pow(-0.5).float()
    for d_sum in (ds, None):
        dx, dw = pqm.rmsnorm_backward(dy, x, w, rstd, d_sum=d_sum)
        want, want_dw, bound, size = ref.norm_backward(
            dy.double(), x.double(), w.double(), rstd.double(), None if d_sum is None else d_sum.double())
        assert ((dx.double() - want).abs() <= ref.HALF_BF16 * want.abs() + bound).all()
        assert ((dw.double() - want_dw).abs() <= (rows + 3) * ref.U * size).all()


@pytest.mark.parametrize("wf32", [False, True])
def test_y_beyond_bf16_is_an_infinity(wf32):
    """From the middle between the largest value, 2^128 - 2^120, and 2^128 on."""
    x, _, _ = usual(64, 1024, True, False, 3)
    w = torch.full((1024,), 1.5 * 2.0 ** 127, device="cuda")
    w = w if wf32 else w.to(torch.bfloat16)
    q, s, y, _, _ = pqm.rmsnorm_quantize_mxfp8(x, w, 1e-6, keep_y=True)
    v = x.double()
    v = v * w.double() * (v.square().mean(1, keepdim=True) + 1e-6).pow(-0.5)
    beyond = v.abs() >= 2.0 ** 128 - 2.0 ** 119
    assert 0.1 < beyond.float().mean() < 0.9
    assert torch.equal(torch.isinf(y), beyond) and not y.isnan().any()
    assert torch.equal(torch.sign(y.float()), torch.sign(v).float())
    oq, os_, _, _ = pqm.quantize_mxfp8(y, colwise=False)
    assert torch.equal(q, oq) and torch.equal(s, os_)
