"""The policy's end and the paths that use the dense products and the one-call
expert layer: each stage against binary64 on the stage's own inputs, then
rollout and training together, captured and replayed.

The bounds of each operator are those of its own tests: a binary32 sum of n
exact products is off by at most n + 96 whole steps (2 U) of its magnitudes."""
from __future__ import annotations

import pytest
import torch

import operators_ref as ref
import precision_quantization_moe_amd as pqm
from precision_quantization_moe_amd import moe_layer as ml
from precision_quantization_moe_amd import policy_head as ph
from gpu_util import gpu_normal_bf16, requires_gpu
from operators_ref import HALF_BF16, U, f64
from test_gpu_moe_block import E, H, I, K, layer, tokens
from test_gpu_token_logprobs import check as check_logprobs

pytestmark = [pytest.mark.gpu, requires_gpu]


def product_bound(a, b):
    """Of a [M, n] times b [n, N]'s binary32 sums."""
    return 1.01 * (a.shape[1] + 96) * 2 * U * (a.abs() @ b.abs())


def head(V):
    g = torch.Generator().manual_seed(V)
    norm_w = (1 + 0.1 * torch.randn(H, generator=g)).cuda()
    return norm_w, (torch.randn(V, H, generator=g) * (3 / H ** 0.5)).to(torch.bfloat16).cuda(), g


@pytest.mark.parametrize("T,V", [(1, 1000), (5, 8), (33, 1003), (130, 4096), (700, 520)])
@pytest.mark.parametrize("f32", [False, True])
def test_head_forward(T, V, f32):
    norm_w, head_w, g = head(V)
    x, r = tokens(T, T)
    ids = torch.randint(0, V, (T,), generator=g).to(torch.int32)
    if T > 4:
        ids[2] = -1
    o = ph.policy_head_forward(x, r, norm_w, head_w, ids.cuda(), 0.8, 7,
                               logits_dtype=pqm.OUT_FP32 if f32 else pqm.OUT_BF16)
    _, _, y, h, rstd = pqm.rmsnorm_quantize_mxfp8(x, norm_w, residual=r, quantize=False)
    assert torch.equal(o["y"], y) and torch.equal(o["h"], h) and torch.equal(o["rstd"], rstd)
    z, slack = f64(y) @ f64(head_w).t(), product_bound(f64(y), f64(head_w).t())
    if not f32:
        slack = slack + HALF_BF16 * (z.abs() + slack)
    assert o["logits"].dtype is (torch.float32 if f32 else torch.bfloat16)
    assert ((f64(o["logits"]) - z).abs() <= slack).all()
    check_logprobs(o["logits"].cpu(), ids, 0.8, 7,
                   tuple(o[n] for n in ("logprob", "entropy", "stats", "top_ids", "top_logprob")))


@pytest.mark.parametrize("T,V", [(1, 1000), (5, 8), (33, 1008), (130, 4096)])
@pytest.mark.parametrize("entropy,past", [(False, False), (True, True)])
def test_head_backward(T, V, entropy, past):
    norm_w, head_w, g = head(V)
    x, r = tokens(T, T + 1)
    ids = torch.randint(0, V, (T,), generator=g).to(torch.int32)
    if T > 4:
        ids[3] = -1
    ids = ids.cuda()
    dl = torch.randn(T, generator=g).cuda()
    de = torch.randn(T, generator=g).cuda() if entropy else None
    dh = gpu_normal_bf16(T, H, 1.0, T + 9) if past else None
    f = ph.policy_head_forward(x, r, norm_w, head_w, ids, 1.3)
    b = ph.policy_head_backward(f, norm_w, head_w, ids, dl, de, dh, 1.3)
    # of the logits: the operator's own call, whose tests hold it to binary64
    dz = pqm.token_logprobs_backward(f["logits"], ids, f["stats"], dl, 1.3, f["entropy"], de)
    assert torch.equal(b["d_logits"], dz)
    z, y = f64(dz), f64(f["y"])
    want, slack = z.t() @ y, product_bound(z.t(), y)
    assert ((f64(b["d_head_w"]) - want).abs() <= slack).all()
    # back through the head, rounded to bf16, then through the norm
    d64 = z @ f64(head_w)
    slack = product_bound(z, f64(head_w))
    slack = 1.01 * (slack + HALF_BF16 * (d64.abs() + slack))
    dx, dw, bound, dw_size = ref.norm_backward(d64, f64(f["h"]), f64(norm_w), f64(f["rstd"]),
                                               f64(dh) if past else None)
    rs, w = f64(f["rstd"])[:, None], f64(norm_w)
    h = f64(f["h"]) * rs
    moved = rs * (slack * w.abs() + h.abs() * (slack * w.abs() * h.abs()).mean(1, keepdim=True))
    bound = bound * 1.01 + moved
    assert ((f64(b["dx"]) - dx).abs() <= HALF_BF16 * (dx.abs() + bound) + bound).all()
    assert ((f64(b["d_norm_w"]) - dw).abs()
            <= (slack * h.abs()).sum(0) + 1.01 * (T + 3) * U * dw_size).all()
    # over the saved logits: the same bits
    again = ph.policy_head_backward(f, norm_w, head_w, ids, dl, de, dh, 1.3, reuse_logits=True)
    assert again["d_logits"] is f["logits"] and all(torch.equal(again[n], b[n]) for n in b)


def test_head_gradient_against_differences():
    """Differences in binary64 along a random direction and along the
    gradient: of the log probabilities
    and entropies from the saved y on (logits in binary32, so nothing is rounded
    to bf16 but d_logits: half a step of it), then of the norm under the gradient
    that d_logits gives its output (dy rounded to bf16, then dx).  The binary32
    sums and the differences themselves stay within 2^-14 of the magnitudes."""
    T, V = 9, 64
    norm_w, head_w, g = head(V)
    x, _ = tokens(T, 77)
    ids = torch.randint(0, V, (T,), generator=g).to(torch.int32)
    dl, de = torch.randn(T, generator=g), torch.randn(T, generator=g)
    f = ph.policy_head_forward(x, None, norm_w, head_w, ids.cuda(), logits_dtype=pqm.OUT_FP32)
    b = ph.policy_head_backward(f, norm_w, head_w, ids.cuda(), dl.cuda(), de.cuda())
    y, hw, dz = f64(f["y"]), f64(head_w), f64(b["d_logits"])

    def value(z):
        lp = torch.log_softmax(z, 1)
        return (f64(dl) * lp.gather(1, ids.long()[:, None])[:, 0] - f64(de) * (lp.exp() * lp).sum(1)).sum()

    def norm(xx, nw):
        return ((dz @ hw) * xx * torch.rsqrt((xx * xx).mean(1, keepdim=True) + 1e-6) * nw).sum()

    def close(fn, at, got, size, what):
        v = torch.randn(at.shape, generator=g).double()
        for v in (v, v.abs() * f64(got).sign()):
            want = float(fn(at + 1e-6 * v) - fn(at - 1e-6 * v)) / 2e-6
            bound = float((size * v.abs()).sum()) + 1e-6 * (1 + abs(want))
            assert abs(float((f64(got) * v).sum()) - want) <= bound, what
        assert abs(want) > 3 * bound, what   # along the gradient the comparison says something

    small = 2.0 ** -14
    size = dz.abs() * HALF_BF16 * 1.01
    each = f64(dl).abs()[:, None] + f64(de).abs()[:, None] * 8     # of the logits' gradient, in units of p
    close(lambda z: value(z), y @ hw.t(), b["d_logits"], size + small * (dz.abs() + each * torch.softmax(y @ hw.t(), 1)),
          "d_logits")
    size = size + small * (dz.abs() + each * torch.softmax(y @ hw.t(), 1))
    close(lambda w: value(y @ w.t()), hw, b["d_head_w"], size.t() @ y.abs() + small * (dz.t().abs() @ y.abs()),
          "d_head_w")
    dy, rs, w = (dz @ hw).abs(), f64(f["rstd"])[:, None], f64(norm_w).abs()
    off = HALF_BF16 * 1.01 * dy + small * (dz.abs() @ hw.abs())
    xs = (f64(x) * rs).abs()
    close(lambda nw: norm(f64(x), nw), f64(norm_w), b["d_norm_w"], (off * xs).sum(0) + small * (dy * xs).sum(0),
          "d_norm_w")
    through = rs * (off * w + xs * (off * w * xs).mean(1, keepdim=True))
    close(lambda xx: norm(xx, f64(norm_w)), f64(x), b["dx"],
          through + (HALF_BF16 + small) * f64(b["dx"]).abs() + small * rs * dy * w, "dx")


def test_decode_in_one_call():
    q, norm_w, gate_w = layer(True)
    for T in (0, 1, 5, 64):
        x, r = tokens(max(T, 1), 90 + T)
        x, r = x[:T], r[:T]
        o = ml.nvfp4_moe_decode(x, r, norm_w, gate_w, *q, K, I, fused=True)
        want = pqm.moe_decode_nvfp4(x, r, norm_w, gate_w, *q, K, I)
        assert all(torch.equal(a, b) for a, b in zip(o.values(), want)) and o["out"].shape == (T, H)
    # the last expert's weights as a shared one
    x, r = tokens(3, 95)
    o = ml.nvfp4_moe_decode(x, r, norm_w, gate_w[:E - 1], *q, K, I, fused=True, shared=True)
    assert o["d"].shape == (3 * (K + 1), I) and int(o["ids"].max()) < E - 1


@pytest.mark.parametrize("T", [0, 1, 70])
def test_training_step_with_the_dense_router(T):
    q, norm_w, gate_w = layer(False)
    x, r = tokens(max(T, 1), 40)
    x, r = x[:T], r[:T]
    f = ml.mxfp8_moe_block_forward(x, r, norm_w, gate_w, *q, K, I, 0.05, router="linear")
    z, slack = f64(f["y"]) @ f64(gate_w).t(), product_bound(f64(f["y"]), f64(gate_w).t())
    assert ((f64(f["logits"]) - z).abs() <= slack).all()
    dy, dh = tokens(max(T, 1), 50)
    dy, dh = dy[:T], dh[:T]
    d_prob = torch.randn(T, K, generator=torch.Generator().manual_seed(5)).cuda()
    one = torch.ones(1, device="cuda")
    b = ml.moe_block_backward(f, norm_w, gate_w, dy, d_prob, one, dh, 0.05, router="linear")
    old = ml.moe_block_backward(f, norm_w, gate_w, dy, d_prob, one, dh, 0.05)
    assert torch.equal(b["d_logits"], old["d_logits"])
    dz = f64(b["d_logits"])
    want = dz.t() @ f64(f["y"])
    assert ((f64(b["d_gate_w"]) - want).abs() <= product_bound(dz.t(), f64(f["y"]))).all()
    d64 = dz @ f64(gate_w) + f64(dy)
    slack = product_bound(dz, f64(gate_w))
    slack = 1.01 * (slack + (HALF_BF16 + U) * (d64.abs() + slack))   # one rounding to bf16
    dx, dw, bound, dw_size = ref.norm_backward(d64, f64(f["h"]), f64(norm_w), f64(f["rstd"]), f64(dh))
    rs, w = f64(f["rstd"])[:, None], f64(norm_w)
    h = f64(f["h"]) * rs
    moved = rs * (slack * w.abs() + h.abs() * (slack * w.abs() * h.abs()).mean(1, keepdim=True))
    bound = bound * 1.01 + moved
    assert ((f64(b["dx"]) - dx).abs() <= HALF_BF16 * (dx.abs() + bound) + bound).all()
    assert ((f64(b["d_norm_w"]) - dw).abs()
            <= (slack * h.abs()).sum(0) + 1.01 * (T + 3) * U * dw_size).all()


def test_rollout_and_training_captured():
    """Two expert layers of a rollout's step and its head, then a training block,
    its head and all their gradients, in one graph; tokens, ids and gradients
    change between replays, and eager calls of the same run beside them."""
    qn, norm_w, gate_w = layer(True)
    qm, _, _ = layer(False)
    V, T = 1000, 40
    norm_h, head_w, g = head(V)
    x1, r1 = tokens(2, 100)
    x, r = tokens(T, 101)
    ids1 = torch.zeros(2, dtype=torch.int32, device="cuda")
    ids = torch.zeros(T, dtype=torch.int32, device="cuda")
    dl, de = torch.ones(T, device="cuda"), torch.ones(T, device="cuda")
    one = torch.ones(1, device="cuda")
    plan = ml.block_plan(T, K, x.device)

    def step():
        a = ml.nvfp4_moe_decode(x1, r1, norm_w, gate_w, *qn, K, I, fused=True)
        a = ml.nvfp4_moe_decode(a["out"], a["h"], norm_w, gate_w, *qn, K, I, fused=True)
        o = ph.policy_head_forward(a["out"], a["h"], norm_h, head_w, ids1, 0.9, 8)
        f = ml.mxfp8_moe_block_forward(x, r, norm_w, gate_w, *qm, K, I, 0.05, None, plan, router="linear")
        t = ph.policy_head_forward(f["out"], f["h"], norm_h, head_w, ids, 0.9)
        b = ph.policy_head_backward(t, norm_h, head_w, ids, dl, de, None, 0.9)
        # the experts' own backward pass is another entry point's: its place is taken by dx
        c = ml.moe_block_backward(f, norm_w, gate_w, b["dx"], f["prob"], one, b["dx"], 0.05, None, plan,
                                  router="linear")
        got = {}
        for n, d in (("rollout", a), ("sample", o), ("forward", f), ("head", t), ("back", b), ("block", c)):
            got.update({(n, k): v for k, v in d.items() if v is not None})
        return got

    step()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for i in range(4):
        for t, s in ((x1, 0), (r1, 1)):
            t.copy_(tokens(2, 110 + 10 * i + s)[0])
        for t, s in ((x, 2), (r, 3)):
            t.copy_(tokens(T, 110 + 10 * i + s)[0])
        ids1.copy_(torch.randint(-1, V, (2,), generator=g))
        ids.copy_(torch.randint(-1, V, (T,), generator=g))
        dl.copy_(torch.randn(T, generator=g))
        de.copy_(torch.randn(T, generator=g))
        for t in out.values():
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        want = step()
        torch.cuda.synchronize()
        for n in want:
            assert torch.equal(want[n], out[n]), (i, n)


def test_two_streams_at_once():
    """Calls that run at the same time, each with its own workspace, give the bits
    that they give alone."""
    q, norm_w, gate_w = layer(True)
    norm_h, head_w, g = head(5000)
    sets = [tokens(4, 200 + 2 * i) for i in range(2)]

    def step(i):
        a = ml.nvfp4_moe_decode(*sets[i], norm_w, gate_w, *q, K, I, fused=True)
        o = ph.policy_head_forward(a["out"], a["h"], norm_h, head_w, None, 1.0, 4)
        return [a["out"], a["d"], a["ids"], o["logits"], o["entropy"], o["top_ids"], o["top_logprob"]]

    want = [step(i) for i in range(2)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [[], []]
    for _ in range(20):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(step(i))
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(a, b) for o in got[i] for a, b in zip(o, want[i])), i


@pytest.mark.parametrize("V,bad", [(1003, None), (1000, "d_h"), (1000, "norm_w"), (1000, "y")])
def test_a_refused_gradient_leaves_the_logits(V, bad):
    """A call over the saved logits that is refused has not written them."""
    T = 6
    norm_w, head_w, g = head(V)
    x, r = tokens(T, 300)
    ids = torch.randint(0, V, (T,), generator=g).to(torch.int32).cuda()
    f = ph.policy_head_forward(x, r, norm_w, head_w, ids)
    before = f["logits"].clone()
    d_h = torch.zeros(T, H + 8, dtype=torch.bfloat16, device="cuda") if bad == "d_h" else None
    if bad == "norm_w":
        norm_w = norm_w[:-1]
    if bad == "y":
        f["y"] = torch.zeros(T * H + 1, dtype=torch.bfloat16, device="cuda")[1:].view(T, H)
    with pytest.raises((ValueError, TypeError)):
        ph.policy_head_backward(f, norm_w, head_w, ids, torch.ones(T, device="cuda"), d_h=d_h, reuse_logits=True)
    torch.cuda.synchronize()
    assert torch.equal(f["logits"], before)


def test_no_tokens():
    V = 1000
    norm_w, head_w, _ = head(V)
    x = torch.zeros(0, H, dtype=torch.bfloat16, device="cuda")
    ids = torch.zeros(0, dtype=torch.int32, device="cuda")
    f = ph.policy_head_forward(x, x, norm_w, head_w, ids, 0.9, 4)
    assert f["logits"].shape == (0, V) and f["top_ids"].shape == (0, 4) and f["logprob"].shape == (0,)
    none = torch.zeros(0, device="cuda")
    b = ph.policy_head_backward(f, norm_w, head_w, ids, none, none, x, 0.9, reuse_logits=True)
    torch.cuda.synchronize()
    assert b["dx"].shape == (0, H) and not b["d_head_w"].any() and not b["d_norm_w"].any()
    assert b["d_head_w"].shape == (V, H) and b["d_norm_w"].shape == (H,)
