"""Logits of a run that has diverged: a NaN reaches what is computed from it,
whatever the order of its place, and nothing else.  (Ids stay experts and counts
whole numbers, since they are indexes and sizes further on.)"""
from __future__ import annotations

import pytest
import torch

import precision_quantization_moe_amd as pqm
from gpu_util import requires_gpu

pytestmark = [pytest.mark.gpu, requires_gpu]

INF, NAN = float("inf"), float("nan")
BOTH = [pqm.SCORE_SOFTMAX, pqm.SCORE_SIGMOID]


def logits(E, bf16):
    z = 2 * torch.randn(30, E, generator=torch.Generator().manual_seed(E))
    return z.to(torch.bfloat16) if bf16 else z


def both(z, k, score, renorm, mask=None, counts=None, loss=True):
    z = z.cuda()
    f = pqm.moe_gate(z, k, score, renorm, 2.5, mask, 0.1 if loss else None)
    d = torch.randn(z.shape[0], k, generator=torch.Generator().manual_seed(k)).cuda()
    g = pqm.moe_gate_backward(z, f[0], d, score, renorm, 2.5, mask, 0.1, counts if loss else None,
                              torch.ones(1).cuda() if loss else None)
    return f + (g,)


@pytest.mark.parametrize("E,k", [(40, 4), (100, 8), (256, 8), (300, 8), (700, 2)])
@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("score", BOTH)
@pytest.mark.parametrize("renorm", [False, True])
def test_a_nan_takes_its_token(E, k, bf16, score, renorm):
    z = logits(E, bf16)
    counts = pqm.moe_gate(z.cuda(), k, score, renorm, 2.5, None, 0.1)[2]
    want = both(z, k, score, renorm, counts=counts)
    bad = z.clone()
    bad[3, 0] = NAN
    bad[8, E - 1] = NAN
    bad[11] = NAN
    bad[17, int(z[17].float().argmax())] = NAN
    bad[29, E // 2], bad[29, 1] = -NAN, -INF
    rows = [3, 8, 11, 17, 29]
    keep = [i for i in range(30) if i not in rows]
    ids, prob, c, prob_sum, loss, dz = both(bad, k, score, renorm, counts=counts)
    assert prob[rows].isnan().all() and torch.equal(prob[keep], want[1][keep])
    assert dz[rows].isnan().all() and torch.equal(dz[keep], want[5][keep])
    assert prob_sum.isnan().all() and loss.isnan().all()
    assert torch.equal(ids[keep], want[0][keep])
    assert int(ids.min()) >= 0 and int(ids.max()) < E
    assert all(row.unique().numel() == k for row in ids.cpu())
    assert int(c[:E].sum()) == 30 * k and int(c[E]) == 30
    # without a loss
    _, prob, _, _, _, dz = both(bad, k, score, renorm, loss=False)
    assert prob[rows].isnan().all() and torch.equal(prob[keep], want[1][keep])
    assert dz[rows].isnan().all() and torch.isfinite(dz[keep]).all()
    # and behind a mask
    mask = torch.ones(30, dtype=torch.bool)
    mask[rows] = False
    a, b = (both(t, k, score, renorm, mask.cuda(), counts) for t in (z, bad))
    assert all(torch.equal(u, v) for u, v in zip(a, b))
    assert all(torch.isfinite(t).all() for t in b)


@pytest.mark.parametrize("E,k", [(40, 4), (300, 8)])
@pytest.mark.parametrize("renorm", [False, True])
def test_an_infinite_logit(E, k, renorm):
    """Softmax: inf / inf.  Sigmoid: the score 1, as of any large logit."""
    z = logits(E, False)
    z[2, 5], z[7, E - 1], z[7, 0] = INF, INF, INF
    large = torch.where(z == INF, torch.full_like(z, 1e30), z)
    counts = pqm.moe_gate(large.cuda(), k, pqm.SCORE_SIGMOID, renorm, 2.5, None, 0.1)[2]
    a, b = (both(t, k, pqm.SCORE_SIGMOID, renorm, counts=counts) for t in (z, large))
    assert all(torch.equal(u, v) for u, v in zip(a, b)) and all(torch.isfinite(t).all() for t in a)
    ids, prob, _, prob_sum, loss, dz = both(z, k, pqm.SCORE_SOFTMAX, renorm, counts=counts)
    rows, keep = [2, 7], [i for i in range(30) if i not in (2, 7)]
    assert prob[rows].isnan().all() and dz[rows].isnan().all()
    assert torch.isfinite(prob[keep]).all() and torch.isfinite(dz[keep]).all()
    assert prob_sum.isnan().all() and loss.isnan().all()
    assert int(ids[2, 0]) == 5 and ids[7, :2].tolist() == [0, E - 1]
