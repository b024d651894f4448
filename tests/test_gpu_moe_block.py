"""The norm, the gate and the experts together, as a layer uses them: one
decode step with NVFP4 weights, and a training step's forward pass and the
gradients of its gate and norm.

Each stage is compared with the one that the same values give through the
entry points that were there before, or with binary64 on the stage's own
inputs."""
from __future__ import annotations

import pytest
import torch

import operators_ref as ref
import precision_quantization_moe_amd as pqm
from precision_quantization_moe_amd import moe_layer as ml
from gpu_util import gpu_normal_bf16, requires_gpu

pytestmark = [pytest.mark.gpu, requires_gpu]

E, H, I, K = 16, 256, 128, 4


def layer(nvfp4):
    w1 = gpu_normal_bf16(E * 2 * I, H, 0.05, 1)
    w2 = gpu_normal_bf16(E * H, I, 0.05, 2)
    q = ml.quantize_expert_weights_nvfp4(w1, w2, I, H) if nvfp4 else \
        ml.quantize_expert_weights_mxfp8(w1, w2)
    g = torch.Generator().manual_seed(3)
    norm_w = (1 + 0.1 * torch.randn(H, generator=g)).to(torch.bfloat16).cuda()
    gate_w = (torch.randn(E, H, generator=g) * 0.1).to(torch.bfloat16).cuda()
    return q, norm_w, gate_w


def tokens(T, seed):
    return gpu_normal_bf16(T, H, 1.0, seed), gpu_normal_bf16(T, H, 1.0, seed + 1)


@pytest.mark.parametrize("T", [1, 3, 40])
def test_decode_step(T):
    q, norm_w, gate_w = layer(True)
    x, r = tokens(T, 10)
    o = ml.nvfp4_moe_decode(x, r, norm_w, gate_w, *q, K, I, ml.block_plan(T, K, x.device))
    assert torch.equal(o["h"], (x.float() + r.float()).to(torch.bfloat16))
    # the router on the layer's own y
    z = ref.f64(o["y"]) @ ref.f64(gate_w).t()
    near = torch.sort(z, 1, descending=True).values
    clear = (near[:, K - 1] - near[:, K]) > 1e-3
    want = ref.gate(z, K, True, True, 1.0)
    got = torch.sort(o["ids"].cpu().long(), 1).values
    assert torch.equal(got[clear], torch.sort(want["ids"], 1).values[clear])
    # both products on the layer's own inputs to them
    ids, prob = o["ids"].cpu(), ref.f64(o["prob"]).view(-1, 1)
    c, size = ref.gemv(o["y"].cpu(), ids, *q[:3], 2 * I, 2 * I, K)
    e = ref.gemv_bound(size, H)
    g, u = c[:, :I], c[:, I:]
    act = g * torch.sigmoid(g)
    d = act * u * prob
    bound = prob * (1.1 * e[:, :I] * (u.abs() + e[:, I:]) + act.abs() * e[:, I:]) + \
        (g.abs() + 9) * 2 * ref.U * d.abs()
    assert ((ref.f64(o["d"]) - d).abs() <= ref.HALF_BF16 * (d.abs() + bound) + bound).all()
    y, size = ref.gemv(o["d"].cpu(), ids, *q[3:], H, H, 1)
    bound = ref.gemv_bound(size, I)
    bound = bound + ref.HALF_BF16 * (y.abs() + bound)
    y, bound = y.view(T, K, H).sum(1), bound.view(T, K, H).sum(1)
    bound = bound * (1 + K * ref.U) + K * ref.U * y.abs()
    assert ((ref.f64(o["out"]) - y).abs() <= bound + ref.HALF_BF16 * (y.abs() + bound)).all()


def test_no_tokens():
    q, norm_w, gate_w = layer(True)
    x, r = tokens(1, 15)
    o = ml.nvfp4_moe_decode(x[:0], r[:0], norm_w, gate_w, *q, K, I)
    assert o["out"].shape == (0, H) and o["h"].shape == (0, H) and o["ids"].shape == (0, K)
    q, norm_w, gate_w = layer(False)
    f = ml.mxfp8_moe_block_forward(x[:0], r[:0], norm_w, gate_w, *q, K, I)
    assert f["out"].shape == (0, H) and float(f["loss"]) == 0 and not f["counts"].any()
    one = torch.ones(1, device="cuda")
    b = ml.moe_block_backward(f, norm_w, gate_w, x[:0], f["prob"], one, r[:0])
    assert b["dx"].shape == (0, H) and not b["d_norm_w"].any() and not b["d_gate_w"].any()


def test_decode_step_captured():
    q, norm_w, gate_w = layer(True)
    x, r = tokens(2, 20)
    plan = ml.block_plan(2, K, x.device)
    step = lambda: ml.nvfp4_moe_decode(x, r, norm_w, gate_w, *q, K, I, plan)  # noqa: E731
    step()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for i in range(3):
        a, b = tokens(2, 30 + i)
        x.copy_(a)
        r.copy_(b)
        for t in out.values():
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        want = step()
        torch.cuda.synchronize()
        assert all(torch.equal(want[n], out[n]) for n in want), i


def test_training_step():
    q, norm_w, gate_w = layer(False)
    T = 70
    x, r = tokens(T, 40)
    mask = torch.ones(T, dtype=torch.uint8, device="cuda")
    mask[60:] = 0
    plan = ml.block_plan(T, K, x.device)
    f = ml.mxfp8_moe_block_forward(x, r, norm_w, gate_w, *q, K, I, 0.05, mask, plan)
    # the experts on the fused encoding: the bytes of the separate passes
    old = ml.mxfp8_moe_forward(f["y"], f["ids"], f["prob"].view(-1), *q, E, I)
    for n in ("off", "qa", "sa", "qd", "sd", "out"):
        assert torch.equal(f[n], old[n]), n
    assert not f["out"][60:].any()            # padding has no weight
    dy, dh = tokens(T, 50)
    d_prob = torch.randn(T, K, generator=torch.Generator().manual_seed(5)).cuda()
    one = torch.ones(1, device="cuda")
    b = ml.moe_block_backward(f, norm_w, gate_w, dy, d_prob, one, dh, 0.05, mask, plan)
    # binary64 on the saved values, the gate's gradient rounded to bf16 where
    # the products take it
    z = ref.f64(f["logits"])
    live = mask.cpu() != 0
    dz, size = ref.gate_backward(z, f["ids"].cpu().long(), f["counts"].cpu()[:E].double(), 60, True,
                                 True, 1.0, live, 0.05, ref.f64(d_prob), 1.0)
    tol = 3 * (2 * float(z.abs().max()) + 48) * ref.U
    assert ((ref.f64(b["d_logits"]) - dz).abs() <= ref.HALF_BF16 * dz.abs() + 1.01 * tol * size).all()
    dz = ref.f64(b["d_logits"])
    want = dz.t() @ ref.f64(f["y"])
    # binary32 sums over T rows
    assert ((ref.f64(b["d_gate_w"]) - want).abs()
            <= 2 * (T + 32) * ref.U * (dz.abs().t() @ ref.f64(f["y"]).abs())).all()
    through = dz @ ref.f64(gate_w)
    slack = 2 * (E + 32) * ref.U * (dz.abs() @ ref.f64(gate_w).abs()) + ref.HALF_BF16 * through.abs()
    d64 = through + ref.f64(dy)
    slack = 1.01 * (slack + ref.HALF_BF16 * d64.abs())   # the sum is rounded to bf16 too
    dx, dw, bound, dw_size = ref.norm_backward(d64, ref.f64(f["h"]), ref.f64(norm_w),
                                               ref.f64(f["rstd"]), ref.f64(dh))
    rs, w = ref.f64(f["rstd"])[:, None], ref.f64(norm_w)
    h = ref.f64(f["h"]) * rs
    moved = rs * (slack * w.abs() + h.abs() * (slack * w.abs() * h.abs()).mean(1, keepdim=True))
    bound = bound * 1.01 + moved
    assert ((ref.f64(b["dx"]) - dx).abs() <= ref.HALF_BF16 * (dx.abs() + bound) + bound).all()
    assert ((ref.f64(b["d_norm_w"]) - dw).abs()
            <= (slack * h.abs()).sum(0) + 1.01 * (T + 3) * ref.U * dw_size).all()


def test_training_step_captured():
    """Forward pass and gradients in one graph, the choice of experts, the
    counts and the mask different at every replay."""
    q, norm_w, gate_w = layer(False)
    T = 33
    x, r = tokens(T, 60)
    mask = torch.ones(T, dtype=torch.uint8, device="cuda")
    dy, dh = tokens(T, 61)
    d_prob = torch.randn(T, K, generator=torch.Generator().manual_seed(6)).cuda()
    one = torch.ones(1, device="cuda")
    plan = ml.block_plan(T, K, x.device)

    def step():
        f = ml.mxfp8_moe_block_forward(x, r, norm_w, gate_w, *q, K, I, 0.05, mask, plan)
        b = ml.moe_block_backward(f, norm_w, gate_w, dy, d_prob, one, dh, 0.05, mask, plan)
        return dict({n: f[n] for n in ("out", "h", "ids", "prob", "counts", "prob_sum", "loss")}, **b)

    step()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for i in range(4):
        a, b = tokens(T, 70 + i)
        x.copy_(a)
        r.copy_(b)
        mask.fill_(1)
        mask[T - 5 * i:] = 0
        for t in out.values():
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        want = step()
        torch.cuda.synchronize()
        for n in want:
            assert torch.equal(want[n], out[n]), (i, n)
