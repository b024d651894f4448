"""Dense products in each of their forms: rows straight from memory, 128 x 128
tiles with eight and with four steps in flight, a split contraction and its
join, 256 x 256 tiles, outputs and residuals past the caches.  The bounds are
those of test_gpu_linear.

A form is taken by size; FORMS names it by the kernels that the call launches,
so that a later change of the rule cannot leave one untested."""
from __future__ import annotations

import math

import pytest
import torch

import precision_quantization_moe_amd as pqm
from gpu_util import kernels, requires_gpu
from operators_ref import HALF_BF16, U
from test_gpu_linear import TINY, activation, forward, rand

pytestmark = [pytest.mark.gpu, requires_gpu]

FEW, DEEP, TILES, LARGE, JOIN = ("k_linear_few<", "k_linear<0, 128, 128, 8>", "k_linear<0, 128, 128, 4>",
                                 "k_linear<0, 256, 256, 4>", "k_linear_join")
FORMS = [((48, 136, 264), (FEW,)), ((300, 61, 256), (FEW,)), ((1500, 520, 512), (DEEP,)),
         ((1501, 517, 520), (DEEP,)), ((4100, 1160, 264), (TILES,)), ((4100, 1157, 264), (TILES,)),
         ((3000, 128, 4096), (DEEP, JOIN)), ((2999, 125, 4104), (DEEP, JOIN)), ((3600, 4104, 264), (LARGE,)),
         ((3601, 4101, 296), (LARGE,))]
SIZES = [s for s, _ in FORMS]


@pytest.mark.parametrize("size,names", FORMS)
def test_the_form_is_taken(size, names):
    M, N, K = size
    x = torch.zeros(M, K, dtype=torch.bfloat16, device="cuda")
    w = torch.zeros(N, K, dtype=torch.bfloat16, device="cuda")
    assert (pqm.lib().pqm_linear_workspace(M, N, K) > 0) == (JOIN in names)
    got = kernels(lambda: pqm.linear(x, w))
    assert len(got) == len(names) and all(n in g for n, g in zip(names, got)), got


@pytest.mark.parametrize("M,N,K", SIZES)
@pytest.mark.parametrize("act", [pqm.ACT_NONE, pqm.ACT_SILU, pqm.ACT_GELU])
def test_epilogues(M, N, K, act):
    for bias, residual, f32, keep_z in ((False, False, True, False), (True, True, False, True),
                                        (True, False, True, True), (False, True, True, False)):
        forward(M, N, K, act, bias, residual, f32, keep_z)


@pytest.mark.parametrize("M,N,K", SIZES)
def test_strides(M, N, K):
    forward(M, N, K, pqm.ACT_SILU, True, True, False, True, ldx=8, ldr=8)
    forward(M, N, K, pqm.ACT_GELU, False, True, False, False, ldx=40, ldr=3)


def operands(M, N, K, seed=0):
    g = torch.Generator().manual_seed(M + N + K + seed)
    return (rand(g, M, K).cuda(), rand(g, N, K, scale=1 / math.sqrt(K)).cuda(),
            torch.randn(N, generator=g).cuda(), rand(g, M, N).cuda(), g)


def guarded(n):
    """n bytes and 4096 on either side, all of one value: (the whole, address)."""
    t = torch.full((n + 8192,), 0xA5, dtype=torch.uint8, device="cuda")
    return t, t.data_ptr() + 4096


def untouched(t):
    return bool((t[:4096] == 0xA5).all() and (t[-4096:] == 0xA5).all())


def inside(t, like):
    return t[4096:-4096].view(like.dtype).view(like.shape)


@pytest.mark.parametrize("M,N,K", SIZES)
@pytest.mark.parametrize("f32", [False, True])
def test_in_place_and_nothing_beside(M, N, K, f32):
    """y (bf16) in the residual's memory gives the bits of a y of its own, and the
    bytes around y, z and the workspace stay as they were."""
    x, w, b, r, _ = operands(M, N, K)
    out = pqm.OUT_FP32 if f32 else pqm.OUT_BF16
    want, wz = pqm.linear(x, w, b, pqm.ACT_SILU, r, True, out)
    size = pqm.lib().pqm_linear_workspace(M, N, K)
    y, yp = guarded(want.numel() * want.element_size())
    z, zp = guarded(wz.numel() * 2)
    ws, wp = guarded(size)
    if not f32:
        inside(y, want).copy_(r)
    code = pqm.lib().pqm_linear(x.data_ptr(), K, w.data_ptr(), b.data_ptr(), pqm.ACT_SILU,
                                r.data_ptr() if f32 else yp, N, M, N, K, yp, out, zp, wp, size,
                                torch.cuda.current_stream().cuda_stream)
    torch.cuda.synchronize()
    assert code == 0 and torch.equal(inside(y, want), want) and torch.equal(inside(z, wz), wz)
    assert untouched(y) and untouched(z) and untouched(ws)


@pytest.mark.parametrize("M,N,K", SIZES)
def test_nothing_leaves_its_row_or_column(M, N, K):
    x, w, b, r, _ = operands(M, N, K)
    clean, cz = pqm.linear(x, w, b, pqm.ACT_NONE, r, True)
    x[M // 2, K - 1] = math.nan
    x[M - 1, 0] = math.inf
    w[N - 3, 1] = math.nan
    r[3, 5] = math.nan
    y, z = pqm.linear(x, w, b, pqm.ACT_NONE, r, True)
    torch.cuda.synchronize()
    rows, cols = torch.ones(M, dtype=torch.bool), torch.ones(N, dtype=torch.bool)
    rows[[M // 2, M - 1]], cols[N - 3] = False, False
    clean[3, 5] = y[3, 5]
    assert y[3, 5].isnan() and z[3, 5].isfinite()
    for a, c in ((y, clean), (z, cz)):
        assert torch.equal(a[rows][:, cols].view(torch.int16), c[rows][:, cols].view(torch.int16))
        assert a[M // 2].isnan().all() and a[:, N - 3].isnan().all() and not a[M - 1].isfinite().any()


@pytest.mark.parametrize("M,N,K", SIZES)
def test_rows_do_not_depend_on_their_place(M, N, K):
    x, w, b, r, g = operands(M, N, K)
    p = torch.randperm(M, generator=g).cuda()
    y, z = pqm.linear(x, w, b, pqm.ACT_GELU, r, True)
    py, pz = pqm.linear(x[p].contiguous(), w, b, pqm.ACT_GELU, r[p].contiguous(), True)
    assert torch.equal(py, y[p]) and torch.equal(pz, z[p])


@pytest.mark.parametrize("M,N,K", SIZES)
def test_captured(M, N, K):
    x, w, b, r, g = operands(M, N, K)

    def step():
        return pqm.linear(x, w, b, pqm.ACT_SILU, r, True) + pqm.linear(x, w, out_dtype=pqm.OUT_FP32)[:1]
    step()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for i in range(3):
        x.copy_(rand(g, M, K))
        for t in out:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        want = step()
        torch.cuda.synchronize()
        assert all(torch.equal(a, c) for a, c in zip(out, want)), i


def test_split_calls_at_the_same_time():
    """Split contractions on two streams, each with a workspace of its own."""
    sets = [operands(3000, 128, 4096, i) for i in range(2)]
    want = [pqm.linear(x, w, b, pqm.ACT_SILU, r, True) for x, w, b, r, _ in sets]
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream() for _ in sets], []
    for _ in range(10):
        for s, (x, w, b, r, _) in zip(streams, sets):
            with torch.cuda.stream(s):
                got.append(pqm.linear(x, w, b, pqm.ACT_SILU, r, True))
    torch.cuda.synchronize()
    for i, o in enumerate(got):
        assert all(torch.equal(a, c) for a, c in zip(o, want[i % 2])), i


def on_device(y, want, slack, what):
    """check() of a bf16 result, on the device: 2^26 values."""
    err = (y.double() - want).abs()
    assert (err <= slack + HALF_BF16 * (want.abs() + slack) + TINY).all(), (what, float(err.max()))


@pytest.mark.parametrize("M,N,K", [(8200, 8200, 264), (8192, 8192, 72), (5000, 5040, 264), (6240, 4048, 40)])
def test_past_the_caches(M, N, K):
    """From 3 * 2^23 outputs on y and z go past the caches, from 2^26 on the
    residual's reads too: all values, in tiles of both sizes, and y in the
    residual's memory."""
    assert M * N >= 3 << 23
    x, w, b, r, _ = operands(M, N, K)
    xd, wd = x.double(), w.double()
    zd = xd @ wd.t() + b.double()
    slack = 1.01 * ((K + 96) * 2 * U * (xd.abs() @ wd.abs().t()) + U * zd.abs())
    for act in (pqm.ACT_NONE, pqm.ACT_SILU):
        y, z = pqm.linear(x, w, b, act, r, True)
        on_device(z, zd, slack, "z")
        a, _, steps = activation(zd, act)
        s = 1.2 * slack + steps * U * a.abs()
        a = a + r.double()
        on_device(y, a, s + 2 * U * a.abs(), "y")
    del zd, slack, a, s, steps
    alone, _ = pqm.linear(x, w, b, pqm.ACT_SILU)
    apart = r.clone()
    code = pqm.lib().pqm_linear(x.data_ptr(), K, w.data_ptr(), b.data_ptr(), pqm.ACT_SILU, apart.data_ptr(),
                                N, M, N, K, apart.data_ptr(), pqm.OUT_BF16, None,
                                torch.empty(16, dtype=torch.uint8, device="cuda").data_ptr(), 16,
                                torch.cuda.current_stream().cuda_stream)
    torch.cuda.synchronize()
    assert pqm.lib().pqm_linear_workspace(M, N, K) == 0
    assert code == 0 and torch.equal(apart, y) and not torch.equal(alone, y)


BACKWARD = [(40, 72, 264), (1000, 264, 8), (500, 512, 520), (4100, 1160, 264), (3600, 264, 4104), (300, 3592, 3848)]


@pytest.mark.parametrize("M,N,K", BACKWARD)
@pytest.mark.parametrize("act", [pqm.ACT_NONE, pqm.ACT_GELU])
def test_gradients_write_nothing_beside(M, N, K, act):
    """dx in d_x's memory and dz in z's, the bits of a call with outputs of its own,
    and the bytes around dx, dw, dbias, dz and the workspace as they were."""
    x, w, _, dy, g = operands(M, N, K)
    z = rand(g, M, N).cuda() if act != pqm.ACT_NONE else None
    d_x = rand(g, M, K).cuda()
    want = pqm.linear_backward(dy, x, w, act, z, d_x, need_dbias=True)
    size = pqm.lib().pqm_linear_backward_workspace(M, N, K)
    buf = [guarded(t.numel() * t.element_size()) if t is not None else (None, None) for t in want]
    ws, wp = guarded(size)
    inside(buf[0][0], d_x).copy_(d_x)
    if z is not None:
        inside(buf[3][0], z).copy_(z)
    dx, dw, db, dz = (p for _, p in buf)
    code = pqm.lib().pqm_linear_backward(dy.data_ptr(), N, x.data_ptr(), K, w.data_ptr(), act, dz, dx, K, M, N, K,
                                         dz, dx, dw, db, wp, size, torch.cuda.current_stream().cuda_stream)
    torch.cuda.synchronize()
    assert code == 0 and untouched(ws)
    for t, (b, _) in zip(want, buf):
        assert t is None or torch.equal(inside(b, t), t) and untouched(b)


@pytest.mark.parametrize("M,N,K", [(16400, 136, 2056), (5000, 320, 5040)])
def test_dx_past_the_caches(M, N, K):
    """dx of 3 * 2^23 values and more, alone, joined with d_x, and in its memory."""
    assert M * K >= 3 << 23
    x, w, _, dy, g = operands(M, N, K)
    d_x = rand(g, M, K + 8).cuda()[:, :K]
    d, wd = dy.double(), w.double()
    want, slack = d @ wd, 1.01 * (N + 96) * 2 * U * (d.abs() @ wd.abs())
    on_device(pqm.linear_backward(dy, x, w, need_dw=False)[0], want, slack, "dx")
    dx = pqm.linear_backward(dy, x, w, d_x=d_x, need_dw=False)[0]
    want = want + d_x.double()
    on_device(dx, want, slack + 2 * U * want.abs(), "dx")
    own = d_x.contiguous()
    size = pqm.lib().pqm_linear_backward_workspace(M, N, K)
    ws = torch.empty(max(size, 16), dtype=torch.uint8, device="cuda")
    code = pqm.lib().pqm_linear_backward(dy.data_ptr(), N, None, K, w.data_ptr(), pqm.ACT_NONE, None, own.data_ptr(),
                                         K, M, N, K, None, own.data_ptr(), None, None, ws.data_ptr(), size,
                                         torch.cuda.current_stream().cuda_stream)
    torch.cuda.synchronize()
    assert code == 0 and torch.equal(own, dx)


@pytest.mark.parametrize("M", [40, 300])
def test_the_widest_row_strides(M):
    """Rows 2^22 values apart, the most that is taken: a tile's offsets come close to
    2^31 bytes."""
    N, K, wide = 4096, 512, 1 << 22
    x, w, b, r, g = operands(M, N, K)
    dy = rand(g, M, N).cuda()
    far = [torch.empty(M * wide, dtype=torch.bfloat16, device="cuda").view(M, wide) for _ in range(2)]
    fx, fr = far[0][:, 64:64 + K], far[1][:, wide - N:]
    fx.copy_(x)
    fr.copy_(r)
    want = pqm.linear(x, w, b, pqm.ACT_SILU, r, True)
    got = pqm.linear(fx, w, b, pqm.ACT_SILU, fr, True)
    assert all(torch.equal(a, c) for a, c in zip(got, want))
    want = pqm.linear_backward(dy, x, w, d_x=x, need_dbias=True)
    fr.copy_(dy)
    got = pqm.linear_backward(fr, fx, w, d_x=fx, need_dbias=True)
    assert all(torch.equal(a, c) for a, c in zip(got[:3], want[:3]))


def test_binary32_outputs_beside_streamed_ones():
    """y in binary32 with a streamed z and residual gives z the same bits as y in bf16,
    whose values are y's rounded."""
    x, w, b, r, _ = operands(8200, 8200, 264)
    y, z = pqm.linear(x, w, b, pqm.ACT_GELU, r, True, pqm.OUT_FP32)
    y16, z16 = pqm.linear(x, w, b, pqm.ACT_GELU, r, True)
    assert torch.equal(z, z16) and torch.equal(y.to(torch.bfloat16), y16)
