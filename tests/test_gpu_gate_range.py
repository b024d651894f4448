"""Sigmoid scores of logits far below zero, where e^-z leaves binary32.

Bounds.  A score keeps the exponential's and the quotient's few roundings,
which (2 |z| + 32) U covers (U = 2^-24), and a score below the normal numbers
(2^-126) may vanish.  So a probability may be off by that share of itself and,
renormalized, by (k + 1) 2^-126 over the sum it is divided by; a row's share
likewise by (E + 1) 2^-126 over the row's sum."""
from __future__ import annotations

import pytest
import torch

import operators_ref as ref
import precision_quantization_moe_amd as pqm
from gpu_util import requires_gpu

pytestmark = [pytest.mark.gpu, requires_gpu]

GONE = 2.0 ** -126
TOL = (2 * 210 + 32) * ref.U


def values(bf16):
    """Logits from -210 to -80: 2000 of binary32, or every bf16 value."""
    z = torch.linspace(-210, -80, 2000)
    return z.to(torch.bfloat16).unique() if bf16 else z


def low_rows(E, bf16, seed, ordinary):
    """Rows of E such values, each value in several places; `ordinary` of each
    row's logits are of the usual size instead."""
    g = torch.Generator().manual_seed(seed)
    v = values(bf16)
    T = max(8, -(-4 * v.numel() // E))
    pick = torch.arange(T * E) % v.numel()
    z = v[pick[torch.randperm(T * E, generator=g)]].view(T, E).clone()
    if ordinary:
        at = torch.rand(T, E, generator=g).argsort(1)[:, :ordinary]
        z.scatter_(1, at, torch.randn(T, ordinary, generator=g).to(z.dtype))
    return z


SIZES = [(16, 16), (13, 13), (40, 8), (100, 16), (300, 6), (700, 16)]


@pytest.mark.parametrize("E,k", SIZES)
@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("renorm", [False, True])
def test_scores_far_below_zero(E, k, bf16, renorm):
    z = low_rows(E, bf16, E + k, 2)
    T = z.shape[0]
    ids, prob, counts, prob_sum, loss = pqm.moe_gate(z.cuda(), k, pqm.SCORE_SIGMOID, renorm, 2.5,
                                                     loss_coef=0.1)
    want = ref.gate(ref.f64(z), k, False, renorm, 2.5, None, 0.1)
    assert torch.equal(ids.cpu().long(), want["ids"])
    for t in (prob, prob_sum, loss):
        assert torch.isfinite(t).all()
    total = want["v"].gather(1, want["ids"]).sum(1, keepdim=True)
    lost = 2.5 * GONE * ((k + 1) / total if renorm else 1)
    assert ((ref.f64(prob) - want["prob"]).abs() <= TOL * want["prob"] + lost).all()
    assert torch.equal(counts.cpu()[:E].double(), want["counts"])
    lost = ((E + 1) * GONE / want["v"].sum(1)).sum()
    tol = TOL + (T + E) * ref.U
    assert ((ref.f64(prob_sum) - want["prob_sum"]).abs() <= tol * want["prob_sum"] + lost).all()
    # counts sum to k T, so that coef E sum counts / (k T) lost / T is coef E lost / T
    assert abs(float(loss) - float(want["loss"])) <= \
        (tol + 8 * ref.U) * float(want["loss"]) + 0.1 * E * float(lost) / T


@pytest.mark.parametrize("E,k", SIZES)
@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("renorm", [False, True])
def test_gradients_far_below_zero(E, k, bf16, renorm):
    z = low_rows(E, bf16, E + k + 1, 2)
    T = z.shape[0]
    want = ref.gate(ref.f64(z), k, False, renorm, 2.5, None, 0.1)
    counts = torch.cat([want["counts"], torch.tensor([T]).double()]).to(torch.int32)
    d = torch.randn(T, k, generator=torch.Generator().manual_seed(k))
    dz = pqm.moe_gate_backward(z.cuda(), want["ids"].to(torch.int32).cuda(), d.cuda(), pqm.SCORE_SIGMOID,
                               renorm, 2.5, None, 0.1, counts.cuda(), torch.ones(1).cuda(),
                               out_dtype=pqm.OUT_FP32)
    g, size = ref.gate_backward(ref.f64(z), want["ids"], want["counts"], T, False, renorm, 2.5,
                                want["live"], 0.1, ref.f64(d), 1.0)
    # a score that vanished takes its part of the gradient with it; the sums it
    # is divided by are above 0.02, so that part is below 2^-126 2.5 |d| / 0.02^2
    total = want["v"].gather(1, want["ids"]).sum(1, keepdim=True)
    assert float(total.min()) > 0.02
    lost = 4 * (k + 1) * GONE * 2.5 * float(d.abs().max()) / 0.02 ** 2
    assert ((ref.f64(dz) - g).abs() <= 3 * (2 * 210 + 48) * ref.U * size + lost).all()


@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("E,k", [(16, 16), (40, 8), (300, 6)])
def test_rows_whose_scores_all_vanish(E, k, renorm):
    """Below -88 every score is under 2^-126: no weight, no share, no gradient."""
    z = torch.linspace(-1e5, -88, 64 * E).view(64, E)
    ids, prob, counts, prob_sum, loss = pqm.moe_gate(z.cuda(), k, pqm.SCORE_SIGMOID, renorm, 1.0,
                                                     loss_coef=0.1)
    assert torch.equal(ids.cpu().long(), ref.gate(ref.f64(z), k, False, renorm, 1.0)["ids"])
    assert not prob.any() and not prob_sum.any() and float(loss) == 0.0
    dz = pqm.moe_gate_backward(z.cuda(), ids, torch.ones(64, k).cuda(), pqm.SCORE_SIGMOID, renorm, 1.0,
                               None, 0.1, counts, torch.ones(1).cuda())
    assert not dz.any()


@pytest.mark.parametrize("E,k", SIZES + [(20, 1)])
@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("size", [1e-5, 1.0, 1e4])
def test_gradients_of_rows_that_almost_vanish(E, k, renorm, size):
    """Scores of 2^-125 to 2^-115 alone in a row: their quotients are ordinary
    numbers, and so are the gradients, whatever the products on the way."""
    z = torch.linspace(-86.5, -80, 48 * E)[torch.randperm(48 * E, generator=torch.Generator().manual_seed(E))]
    z = z.view(48, E)
    want = ref.gate(ref.f64(z), k, False, renorm, 2.5, None, 0.1)
    counts = torch.cat([want["counts"], torch.tensor([48]).double()]).to(torch.int32)
    d = size * torch.randn(48, k, generator=torch.Generator().manual_seed(k))
    args = (want["ids"], want["counts"], 48, False, renorm, 2.5, want["live"], 0.1)
    for d_loss in (None, 1.0):
        dz = pqm.moe_gate_backward(z.cuda(), want["ids"].to(torch.int32).cuda(), d.cuda(), pqm.SCORE_SIGMOID,
                                   renorm, 2.5, None, 0.1, None if d_loss is None else counts.cuda(),
                                   None if d_loss is None else torch.ones(1).cuda())
        g, terms = ref.gate_backward(ref.f64(z), *args, ref.f64(d), d_loss or 0.0)
        # without renormalization the gradient is of the scores' own size, where
        # binary32 keeps 2^-149 and a product may vanish below 2^-126
        assert ((ref.f64(dz) - g).abs() <= 3 * (2 * 87 + 48) * ref.U * terms + 4 * GONE).all()
