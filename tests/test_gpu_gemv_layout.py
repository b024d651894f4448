"""The few-row NVFP4 products against the library's own reading of the same
weights: its dequantizer, and the NVFP4 grouped GEMM that takes over for many
rows.

Scales are powers of two and activations values that NVFP4 holds, so both read
exactly the same operands, and only the binary32 sums differ, each within
operators_ref.gemv_bound (the grouped GEMM adds 128 products a step: no more
steps than that bound counts)."""
from __future__ import annotations

import pytest
import torch

import operators_ref as ref
import precision_quantization_moe_amd as pqm
from gpu_util import requires_gpu

pytestmark = [pytest.mark.gpu, requires_gpu]


def nvfp4(rows, K, seed, rows_per_scale):
    """Codes and scales whose every product is a bf16 value: outer scales are
    powers of two."""
    g = torch.Generator().manual_seed(seed)
    q, sb = ref.random_nvfp4(g, rows, K)
    sg = torch.exp2(torch.randint(-12, -6, (rows // rows_per_scale,), generator=g).float())
    return q.cuda(), sb.cuda(), sg.cuda()


# direct and staged kernels, ends inside a chunk, experts above and below the rows
SIZES = [(12, 4, 64, 256), (37, 8, 256, 512), (5, 40, 96, 160), (45, 40, 640, 1088), (300, 3, 1280, 768),
         (64, 16, 2048, 1536)]


@pytest.mark.parametrize("rows,G,N,K", SIZES)
def test_weights_are_the_dequantizers(rows, G, N, K):
    q, sb, sg = nvfp4(G * N, K, N + K, N)
    w = pqm.dequantize(pqm.FMT_NVFP4, q, sb, sg, rows_per_scale=N).double().view(G, N, K)
    g = torch.Generator().manual_seed(rows)
    x = torch.randn(rows, K, generator=g).to(torch.bfloat16).cuda()
    ids = torch.randint(0, G, (rows,), generator=g, dtype=torch.int32).cuda()
    got = pqm.moe_gemv_nvfp4(x, ids, q, sb, sg, N, out_dtype=pqm.OUT_FP32).double()
    want, size = torch.zeros_like(got), torch.zeros_like(got)
    for e in range(G):
        mine = ids == e
        want[mine] = x[mine].double() @ w[e].t().contiguous()
        size[mine] = x[mine].double().abs() @ w[e].abs().t().contiguous()
    assert ((got - want).abs() <= ref.gemv_bound(size, K)).all()
    # gate rows, then up rows
    I = N // 2
    prob = torch.rand(rows, generator=g).cuda()
    d = pqm.moe_gemv_swiglu_nvfp4(x, ids, prob, q, sb, sg, I).double()
    e = ref.gemv_bound(size, K)
    gate, up = want[:, :I], want[:, I:]
    act, p = gate * torch.sigmoid(gate), prob.double()[:, None]
    value = act * up * p
    # silu's slope is at most 1.1; its own arithmetic keeps (|g| + 8) U
    bound = p * (1.1 * e[:, :I] * (up.abs() + e[:, I:]) + act.abs() * e[:, I:]) + \
        (gate.abs() + e[:, :I] + 8) * 2 * ref.U * value.abs()
    assert ((d - value).abs() <= bound + ref.HALF_BF16 * (value.abs() + bound) + 2.0 ** -133).all()


@pytest.mark.parametrize("rows,G,N,K", SIZES)
def test_the_grouped_gemm_gives_the_same_products(rows, G, N, K):
    q, sb, sg = nvfp4(G * N, K, N + K, N)
    xq, xb, xg = nvfp4(rows, K, rows + K, 1)
    x = pqm.dequantize(pqm.FMT_NVFP4, xq, xb, xg)
    ids = torch.randint(0, G, (rows, 1), generator=torch.Generator().manual_seed(rows), dtype=torch.int32).cuda()
    got = pqm.moe_gemv_nvfp4(x, ids, q, sb, sg, N, out_dtype=pqm.OUT_FP32).double()
    off, _, tok, slot = pqm.moe_route(ids, G)
    y = pqm.moe_grouped_gemm(pqm.FMT_NVFP4, pqm.GEMM_FPROP, pqm.moe_gather_rows(xq, tok), q, off, N, K,
                             a_scale=pqm.moe_gather_rows(xb, tok),
                             a_outer=pqm.moe_gather_rows(xg.view(-1, 1), tok).view(-1), b_scale=sb, b_outer=sg,
                             b_rows_per_scale=N, out_dtype=pqm.OUT_FP32)
    want = y[slot.view(-1).long()].double()
    _, size = ref.gemv(x, ids, q, sb, sg, N, N, 1)
    assert ((got - want).abs() <= 2 * ref.gemv_bound(size.cuda(), K)).all()


@pytest.mark.parametrize("G,N", [(3, 20), (40, 640)])
def test_subnormal_activations(G, N):
    """bf16 values below 2^-126, in both kernels, with an outer scale that lifts
    the sums back."""
    K, rows = 512, 41
    q, sb, _ = nvfp4(G * N, K, 5, N)
    sg = torch.full((G,), 2.0 ** 40, device="cuda")
    x = (torch.randn(rows, K, generator=torch.Generator().manual_seed(3)) * 2.0 ** -129).to(torch.bfloat16)
    assert (x.float().abs() < 2.0 ** -126).all() and x.float().abs().gt(0).float().mean() > 0.9
    ids = torch.arange(rows, dtype=torch.int32) % G
    want, size = ref.gemv(x, ids, q, sb, sg, N, N, 1)
    got = pqm.moe_gemv_nvfp4(x.cuda(), ids.cuda(), q, sb, sg, N, out_dtype=pqm.OUT_FP32)
    # a sum before the outer scale may be subnormal: half of 2^-149 each step
    bound = ref.gemv_bound(size, K) + (K // 128 + 8) * 2.0 ** -149 * 2.0 ** 40
    assert ((ref.f64(got) - want).abs() <= bound).all()
