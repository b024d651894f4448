"""A whole expert layer for a few tokens in one call, stage by stage: its norm
against the norm's entry point, its choice against binary64 logits of its own y,
d against binary64 products of its own y and choice, out against those of its
own d.

Bounds, from the arithmetic (U half a step of binary32): a matrix instruction's
sum of 32 exact products and the addition to the running sum are each off by at
most 33 whole steps (2 U) of the magnitudes; a wave adds K / 32 of them, up to 16
waves or parts are joined, one product with the outer scale: (K / 32 + 64) 2 U of
the sum of magnitudes covers both.  The logits' partial sums are joined in
binary64: 34 2 U of the magnitudes, and one rounding."""
from __future__ import annotations

import pytest
import torch

import operators_ref as ref
import precision_quantization_moe_amd as pqm
from precision_quantization_moe_amd import moe_layer as ml
from gpu_util import requires_gpu
from operators_ref import HALF_BF16, U, f64

pytestmark = [pytest.mark.gpu, requires_gpu]


def weights(E, H, I, seed, shared=False):
    g = torch.Generator().manual_seed(seed)
    G = E + 1 if shared else E
    w1 = (torch.randn(G * 2 * I, H, generator=g) * 0.05).to(torch.bfloat16).cuda()
    w2 = (torch.randn(G * H, I, generator=g) * 0.05).to(torch.bfloat16).cuda()
    q = ml.quantize_expert_weights_nvfp4(w1, w2, I, H)
    norm_w = (1 + 0.1 * torch.randn(H, generator=g)).to(torch.bfloat16).cuda()
    gate_w = (torch.randn(E, H, generator=g) / H ** 0.5).to(torch.bfloat16).cuda()
    return q, norm_w, gate_w, g


def tokens(g, T, H):
    x = torch.randn(T, H, generator=g) * torch.exp(torch.randn(T, 1, generator=g))
    return x.to(torch.bfloat16).cuda(), torch.randn(T, H, generator=g).to(torch.bfloat16).cuda()


def check(o, x, r, norm_w, gate_w, q, k, I, shared, softmax, renorm, scale, eps=1e-6):
    out, h, y, ids, prob, d = o
    T, H = x.shape
    E = gate_w.shape[0]
    c = k + (1 if shared else 0)
    _, _, wy, wh, _ = pqm.rmsnorm_quantize_mxfp8(x, norm_w, eps, residual=r, quantize=False)
    assert torch.equal(y, wy) and torch.equal(h, wh)
    # the choice: equal wherever neighbours in the order are further apart than the
    # logits can be off
    yd, gd = f64(y), f64(gate_w)
    z, zs = yd @ gd.t(), yd.abs() @ gd.abs().t()
    e_z = 34 * 2 * U * zs + U * z.abs()
    got = ids.cpu().long()
    assert ((got >= 0) & (got < E)).all() and all(len(set(t)) == k for t in got.tolist())
    zi, ei = z.gather(1, got), e_z.gather(1, got)
    if k > 1:
        assert (zi[:, 1:] - zi[:, :-1] <= ei[:, 1:] + ei[:, :-1]).all()
    left = z.clone().scatter_(1, got, -float("inf"))
    if E > k:
        best, at = left.max(1)
        assert (best - zi[:, -1] <= ei[:, -1] + e_z.gather(1, at[:, None])[:, 0]).all()
    # probabilities of the chosen, from its own choice: a relative error of the scores of
    # the logits' own (twice, against the largest) and 24 roundings, a few of them the sum's
    v, _ = ref.shares(z, softmax)
    p = v.gather(1, got)
    rel = 2 * e_z.max(1, keepdim=True).values + (24 + E) * U + 4 * U * z.abs().max(1, keepdim=True).values
    if renorm:
        p = p / p.sum(1, keepdim=True)
        rel = 2 * rel
    p = p * scale
    assert ((f64(prob) - p).abs() <= 1.05 * rel * p).all()
    # d on its own y and probabilities
    all_ids = ids.cpu()
    all_p = f64(prob)
    if shared:
        all_ids = torch.cat([all_ids, torch.full((T, 1), E, dtype=torch.int32)], 1)
        all_p = torch.cat([all_p, torch.ones(T, 1).double()], 1)
    w1, w2 = q[:3], q[3:]
    s, size = ref.gemv(y.cpu(), all_ids, *w1, 2 * I, 2 * I, c)
    e = (H / 32 + 64) * 2 * U * size
    gate, up, eg, eu = s[:, :I], s[:, I:], e[:, :I], e[:, I:]
    all_p = all_p.reshape(-1, 1)
    act = gate * torch.sigmoid(gate)
    want = act * up * all_p
    bound = all_p * (1.1 * eg * (up.abs() + eu) + act.abs() * eu) + (gate.abs() + 9) * 2 * U * want.abs()
    err = (f64(d) - want).abs()
    assert (err <= HALF_BF16 * (want.abs() + bound) + bound).all()
    # out on its own d
    rows, size = ref.gemv(d.cpu(), all_ids, *w2, H, H, 1)
    bound = ((I / 32 + 64) * 2 * U * size + (c + 16) * 2 * U * size).view(T, c, H).sum(1)
    want = rows.view(T, c, H).sum(1)
    assert ((f64(out) - want).abs() <= HALF_BF16 * (want.abs() + bound) + bound).all()


CASES = [
    # T, E, k, H, I, shared, softmax, renorm
    (1, 1, 1, 32, 32, False, True, True),
    (1, 16, 4, 256, 128, False, True, True),
    (1, 130, 8, 2048, 768, False, True, True),
    (2, 9, 2, 96, 160, True, False, True),
    (3, 20, 16, 544, 96, True, True, False),
    (5, 64, 8, 1056, 352, False, False, False),
    (7, 128, 8, 2048, 192, False, True, True),
    (16, 17, 3, 288, 64, True, False, True),
    (17, 33, 4, 512, 288, False, True, True),
    (33, 8, 2, 320, 256, True, True, True),
    (37, 65, 8, 640, 160, True, False, True),
    (64, 4, 4, 256, 96, False, True, False),
    (64, 300, 16, 128, 32, True, True, True),
    (9, 1024, 16, 64, 32, False, False, True),
    (4, 12, 2, 7168, 64, False, True, True),
    (3, 5, 2, 64, 16384, False, True, True),
    (2, 40, 2, 16384, 32, True, True, True),
    (64, 2, 1, 4128, 64, True, True, True),
]


@pytest.mark.parametrize("T,E,k,H,I,shared,softmax,renorm", CASES)
def test_stages(T, E, k, H, I, shared, softmax, renorm):
    q, norm_w, gate_w, g = weights(E, H, I, T + E, shared)
    x, r = tokens(g, T, H)
    score = pqm.SCORE_SOFTMAX if softmax else pqm.SCORE_SIGMOID
    for res, scale, w in ((r, 1.0, norm_w), (None, 2.5, norm_w.float())):
        o = pqm.moe_decode_nvfp4(x, res, w, gate_w, *q, k, I, shared, score, renorm, scale)
        torch.cuda.synchronize()
        check(o, x, res, w, gate_w, q, k, I, shared, softmax, renorm, scale)


@pytest.mark.parametrize("T,E,k,H,I,shared", [(4, 64, 8, 2048, 1024, True), (1, 12, 8, 4096, 2080, False),
                                              (8, 40, 8, 1056, 1536, True), (20, 16, 4, 4128, 544, True)])
def test_large_experts(T, E, k, H, I, shared):
    """Few tokens whose experts' weights are too many for one kernel, and odd widths."""
    q, norm_w, gate_w, g = weights(E, H, I, T + E, shared)
    x, r = tokens(g, T, H)
    o = pqm.moe_decode_nvfp4(x, r, norm_w, gate_w, *q, k, I, shared, pqm.SCORE_SIGMOID, True, 1.5)
    torch.cuda.synchronize()
    check(o, x, r, norm_w, gate_w, q, k, I, shared, False, True, 1.5)


def test_like_the_separate_calls():
    """Against nvfp4_moe_decode, which makes the six calls: the same norm and
    choice, and out within its roundings."""
    E, k, H, I, T = 32, 4, 512, 256, 12
    q, norm_w, gate_w, g = weights(E, H, I, 1)
    x, r = tokens(g, T, H)
    a = ml.nvfp4_moe_decode(x, r, norm_w, gate_w, *q, k, I)
    out, h, y, ids, prob, d = pqm.moe_decode_nvfp4(x, r, norm_w, gate_w, *q, k, I)
    assert torch.equal(a["h"], h) and torch.equal(a["y"], y) and torch.equal(a["ids"], ids)
    assert (a["prob"] - prob).abs().max() < 1e-5
    # the separate calls round each expert's row to bf16 before the sum
    scale = f64(a["out"]).abs().max()
    assert (f64(a["out"]) - f64(out)).abs().max() < 8 * HALF_BF16 * scale


def test_a_nan_stays_in_its_token():
    E, k, H, I, T, = 16, 4, 256, 128, 20
    q, norm_w, gate_w, g = weights(E, H, I, 2, True)
    x, r = tokens(g, T, H)
    clean = pqm.moe_decode_nvfp4(x, r, norm_w, gate_w, *q, k, I, True)
    x[7, 100] = float("nan")
    out, h, y, ids, prob, d = pqm.moe_decode_nvfp4(x, r, norm_w, gate_w, *q, k, I, True)
    torch.cuda.synchronize()
    assert out[7].isnan().all() and prob[7].isnan().all() and ((ids[7] >= 0) & (ids[7] < E)).all()
    rest = [t for t in range(T) if t != 7]
    assert torch.equal(ids[rest], clean[3][rest]) and torch.equal(prob[rest], clean[4][rest])
    assert out[rest].isfinite().all()
    # another choice of token 7 may change which wave adds what: a few last bits
    assert (f64(out[rest]) - f64(clean[0][rest])).abs().max() <= \
        4 * HALF_BF16 * f64(clean[0]).abs().max()


def test_no_tokens():
    q, norm_w, gate_w, g = weights(8, 64, 32, 3)
    x, r = tokens(g, 1, 64)
    out, h, y, ids, prob, d = pqm.moe_decode_nvfp4(x[:0], r[:0], norm_w, gate_w, *q, 2, 32)
    assert out.shape == h.shape == y.shape == (0, 64) and ids.shape == prob.shape == (0, 2)
    assert d.shape == (0, 32)


@pytest.mark.parametrize("T", [1, 6, 40])
def test_captured_and_same_bits(T):
    """Captured and replayed over changing tokens, with eager calls between the
    replays: the same bits every time."""
    E, k, H, I = 24, 4, 384, 160
    q, norm_w, gate_w, g = weights(E, H, I, 4, True)
    x, r = tokens(g, T, H)

    def step():
        return pqm.moe_decode_nvfp4(x, r, norm_w, gate_w, *q, k, I, True)
    step()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for i in range(4):
        a, b = tokens(g, T, H)
        x.copy_(a)
        r.copy_(b)
        for t in out:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        want, again = step(), step()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, want)), i
        assert all(torch.equal(a, b) for a, b in zip(again, want)), i


def test_calls_at_the_same_time():
    """Many calls on three streams at once, each with its own outputs and
    workspace, between other work."""
    E, k, H, I = 64, 8, 1024, 256
    q, norm_w, gate_w, g = weights(E, H, I, 5, True)
    inputs = [tokens(g, T, H) for T in (1, 24, 9)]
    want = [pqm.moe_decode_nvfp4(x, r, norm_w, gate_w, *q, k, I, True) for x, r in inputs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in inputs]
    got = []
    big = torch.zeros(64 << 20, device="cuda")
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    for turn in range(20):
        big.add_(1.0)
        for s, (x, r) in zip(streams, inputs):
            with torch.cuda.stream(s):
                got.append(pqm.moe_decode_nvfp4(x, r, norm_w, gate_w, *q, k, I, True))
    torch.cuda.synchronize()
    for i, o in enumerate(got):
        assert all(torch.equal(a, b) for a, b in zip(o, want[i % 3])), i


def test_nothing_else_is_written():
    """The bytes behind every output and the workspace stay as they were."""
    E, k, H, I, T = 20, 3, 160, 96, 5
    q, norm_w, gate_w, g = weights(E, H, I, 6, True)
    x, r = tokens(g, T, H)
    want = pqm.moe_decode_nvfp4(x, r, norm_w, gate_w, *q, k, I, True)
    L = pqm.lib()
    size = L.pqm_moe_decode_nvfp4_workspace(T, H, I, E, k, 1)
    buffers = [torch.full((t.numel() * t.element_size() + 4096,), 0xA5, dtype=torch.uint8, device="cuda")
               for t in want] + [torch.full((size + 4096,), 0xA5, dtype=torch.uint8, device="cuda")]
    out, h, y, ids, prob, d, ws = (b.data_ptr() for b in buffers)
    code = L.pqm_moe_decode_nvfp4(x.data_ptr(), r.data_ptr(), norm_w.data_ptr(), 0, 1e-6, gate_w.data_ptr(),
                                  T, H, I, E, k, 1, 0, 1, 1.0, *(t.data_ptr() for t in q), h, y, ids, prob, d,
                                  out, ws, size, torch.cuda.current_stream().cuda_stream)
    torch.cuda.synchronize()
    assert code == 0
    for b, t in zip(buffers, want):
        n = t.numel() * t.element_size()
        assert torch.equal(b[:n], t.contiguous().view(torch.uint8).view(-1)) and (b[n:] == 0xA5).all()
    assert (buffers[-1][size:] == 0xA5).all()
