"""The one-call expert layer in both of its forms, one kernel of tickets up to
eight tokens and the separate products, where they differ: what is not a number
in the scaled binary16 of y, more than 256 experts, the down projection in
parts.  Stages are held to test_gpu_moe_decode's bounds."""
from __future__ import annotations

import math

import pytest
import torch

import operators_ref as ref
import precision_quantization_moe_amd as pqm
from precision_quantization_moe_amd import moe_layer as ml
from gpu_util import kernels, requires_gpu
from operators_ref import HALF_BF16, U, f64
from test_gpu_moe_decode import check, tokens, weights

pytestmark = [pytest.mark.gpu, requires_gpu]

# T, E, k, H, I, shared, one kernel
SIZES = [(5, 16, 4, 256, 128, True, True), (5, 16, 4, 256, 1024, True, True), (8, 128, 8, 2048, 192, False, True),
         (2, 700, 16, 64, 32, True, True), (20, 16, 4, 256, 128, True, False), (7, 20, 4, 2048, 1536, True, False)]


@pytest.mark.parametrize("T,E,k,H,I,shared,one", SIZES)
@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
def test_what_is_not_finite_stays_in_its_token(T, E, k, H, I, shared, one, bad):
    q, norm_w, gate_w, g = weights(E, H, I, 20 + T, shared)
    x, r = tokens(g, T, H)

    def call():
        return pqm.moe_decode_nvfp4(x, r, norm_w, gate_w, *q, k, I, shared)
    assert any("k_decode_experts" in n for n in kernels(call)) == one
    clean = call()
    at = T // 2
    x[at, H - 7] = bad
    for _ in range(3):
        out, h, y, ids, prob, d = call()
        torch.cuda.synchronize()
        assert out[at].isnan().all() and prob[at].isnan().all() and ((ids[at] >= 0) & (ids[at] < E)).all()
        assert len(set(ids[at].tolist())) == k and d.view(T, -1)[at].isnan().any()
        rest = [t for t in range(T) if t != at]
        for a, b in ((h, clean[1]), (y, clean[2]), (ids, clean[3]), (prob, clean[4])):
            assert torch.equal(a[rest], b[rest])
        # another choice of that token may change the order of a sum: last bits
        for a, b in ((out, clean[0]), (d.view(T, -1), clean[5].view(T, -1))):
            assert a[rest].isfinite().all()
            assert (f64(a[rest]) - f64(b[rest])).abs().max() <= 4 * HALF_BF16 * f64(b).abs().max()


@pytest.mark.parametrize("T,E,k,H,I,shared", [(1, 257, 1, 64, 32, False), (1, 512, 8, 256, 96, True),
                                              (3, 1024, 16, 64, 32, False), (8, 300, 8, 128, 64, True),
                                              (8, 1024, 16, 544, 160, True), (5, 16, 4, 256, 1024, True)])
@pytest.mark.parametrize("softmax,renorm", [(True, True), (True, False), (False, True)])
def test_one_kernel_of_many_experts(T, E, k, H, I, shared, softmax, renorm):
    q, norm_w, gate_w, g = weights(E, H, I, T + E, shared)
    x, r = tokens(g, T, H)
    score = pqm.SCORE_SOFTMAX if softmax else pqm.SCORE_SIGMOID

    def call():
        return pqm.moe_decode_nvfp4(x, r, norm_w, gate_w, *q, k, I, shared, score, renorm, 1.5)
    assert any("k_decode_experts" in n for n in kernels(call))
    o = call()
    torch.cuda.synchronize()
    check(o, x, r, norm_w, gate_w, q, k, I, shared, softmax, renorm, 1.5)
    for _ in range(20):
        assert all(torch.equal(a, b) for a, b in zip(call(), o))


def test_the_last_experts_are_met():
    """Tokens whose logits choose the highest numbers of 1024, and all the same ones."""
    E, k, H, I, T = 1024, 8, 64, 32, 8
    q, norm_w, gate_w, g = weights(E, H, I, 9, True)
    x = torch.rand(T, H, generator=g).add_(0.5).to(torch.bfloat16).cuda()
    gate_w.zero_()
    gate_w[E - k:] = torch.arange(1, k + 1)[:, None].to(torch.bfloat16).cuda() / 16
    o = pqm.moe_decode_nvfp4(x, None, norm_w.abs(), gate_w, *q, k, I, True)
    torch.cuda.synchronize()
    assert (o[3].cpu() == torch.arange(E - 1, E - 1 - k, -1)).all()
    check(o, x, None, norm_w.abs(), gate_w, q, k, I, True, True, True, 1.0)


@pytest.mark.parametrize("T", [1, 6, 20])
@pytest.mark.parametrize("power", [30, 40, 60])
def test_one_value_far_above_its_row(T, power):
    """y's first value 2^power times the others, with weights of 0 for it: the others
    are exact down to 2^-31 of it, and off by less than 2^-38 of it below."""
    E, k, H, I = 16, 4, 256, 128
    g = torch.Generator().manual_seed(T + power)
    w1 = (torch.randn(E * 2 * I, H, generator=g) * 0.05).to(torch.bfloat16)
    w1[:, 0] = 0
    w2 = (torch.randn(E * H, I, generator=g) * 0.05).to(torch.bfloat16).cuda()
    q = ml.quantize_expert_weights_nvfp4(w1.cuda(), w2, I, H)
    gate_w = (torch.randn(E, H, generator=g) / H ** 0.5).to(torch.bfloat16)
    gate_w[:, 0] = 0
    # the others between 1 and 2 of a power of two, so that all are 2^-31 of the first at 30
    x = (1 + torch.rand(T, H, generator=g)) * (1 - 2.0 * torch.randint(0, 2, (T, H), generator=g))
    norm_w = torch.ones(H)
    norm_w[0] = 2.0 ** power
    x, gate_w, norm_w = x.to(torch.bfloat16).cuda(), gate_w.cuda(), norm_w.cuda()
    o = pqm.moe_decode_nvfp4(x, None, norm_w, gate_w, *q, k, I)
    torch.cuda.synchronize()
    y, ids, prob, d = o[2].cpu(), o[3].cpu(), f64(o[4]).reshape(-1, 1), f64(o[5])
    s, size = ref.gemv(y, ids, *q[:3], 2 * I, 2 * I, k)
    e = (H / 32 + 64) * 2 * U * size
    if power > 30:
        _, ones = ref.gemv(torch.ones_like(y), ids, *q[:3], 2 * I, 2 * I, k)
        e = e + 2.0 ** -38 * f64(y).abs().amax(1).repeat_interleave(k)[:, None] * ones
    gate, up, eg, eu = s[:, :I], s[:, I:], e[:, :I], e[:, I:]
    want = gate * torch.sigmoid(gate) * up * prob
    bound = prob * (1.1 * eg * (up.abs() + eu) + (gate * torch.sigmoid(gate)).abs() * eu) + \
        (gate.abs() + 9) * 2 * U * want.abs()
    assert ((d - want).abs() <= HALF_BF16 * (want.abs() + bound) + bound).all()
