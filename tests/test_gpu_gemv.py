"""A few routed rows times NVFP4 expert weights on the GPU against binary64;
the bounds are operators_ref.gemv_bound's, plus the output's own rounding."""
from __future__ import annotations

import pytest
import torch

import operators_ref as ref
import precision_quantization_moe_amd as pqm
from gpu_util import requires_gpu

pytestmark = [pytest.mark.gpu, requires_gpu]


def weights(G, N, K, seed, rps=None):
    g = torch.Generator().manual_seed(seed)
    q, sb = ref.random_nvfp4(g, G * N, K)
    rps = rps or N
    sg = torch.rand(G * N // rps, generator=g) * 1e-3 + 1e-4
    return q, sb, sg, rps


def acts(rows, K, seed):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(rows, K, generator=g) * torch.exp(torch.randn(rows, 1, generator=g))
            ).to(torch.bfloat16)


def run_plain(x, ids, w, N, div=1, f32=True):
    q, sb, sg, rps = w
    return pqm.moe_gemv_nvfp4(x.cuda(), ids.cuda(), q.cuda(), sb.cuda(), sg.cuda(), N, rps, div,
                              pqm.OUT_FP32 if f32 else pqm.OUT_BF16)


def check_plain(x, ids, w, N, div=1):
    K = x.shape[1]
    want, size = ref.gemv(x, ids, w[0], w[1], w[2], N, w[3], div)
    bound = ref.gemv_bound(size, K)
    got = run_plain(x, ids, w, N, div)
    assert ((ref.f64(got) - want).abs() <= bound).all()
    low = run_plain(x, ids, w, N, div, f32=False)
    assert ((ref.f64(low) - want).abs() <= bound + ref.HALF_BF16 * (want.abs() + bound)).all()
    assert torch.equal(low, got.to(torch.bfloat16))


def check_act(x, ids, prob, w, inter, div=1):
    K = x.shape[1]
    c, size = ref.gemv(x, ids, w[0], w[1], w[2], 2 * inter, w[3], div)
    e = ref.gemv_bound(size, K)
    g, u, eg, eu = c[:, :inter], c[:, inter:], e[:, :inter], e[:, inter:]
    p = ref.f64(prob).view(-1, 1)
    act = g * torch.sigmoid(g)
    want = act * u * p
    # silu's slope is at most 1.1; its own arithmetic keeps (|g| + 8) U
    bound = p.abs() * (1.1 * eg * (u.abs() + eu) + act.abs() * eu) + \
        (g.abs() + eg + 8) * 2 * ref.U * want.abs()
    q, sb, sg, rps = w
    got = pqm.moe_gemv_swiglu_nvfp4(x.cuda(), ids.cuda(), prob.cuda(), q.cuda(), sb.cuda(),
                                    sg.cuda(), inter, rps, div)
    d = (ref.f64(got) - want).abs()
    assert (d <= bound + ref.HALF_BF16 * (want.abs() + bound) + 2.0 ** -133).all()


@pytest.mark.parametrize("T,k,G,N,K", [(1, 1, 1, 1, 32), (1, 2, 3, 17, 64), (1, 8, 16, 33, 160),
                                       (3, 4, 40, 64, 512), (5, 3, 4, 100, 544), (2, 8, 128, 48, 2048),
                                       (37, 4, 8, 70, 288), (1, 8, 9, 256, 768), (64, 2, 3, 40, 96),
                                       (1, 1, 2, 5, 5120)])
@pytest.mark.parametrize("first", [True, False])
def test_plain(T, k, G, N, K, first):
    """Both projections' row layouts: one x row per token, or per assignment."""
    g = torch.Generator().manual_seed(T + N)
    ids = torch.randint(0, G, (T, k), generator=g, dtype=torch.int32)
    x = acts(T if first else T * k, K, N + K)
    check_plain(x, ids, weights(G, N, K, K), N, k if first else 1)


@pytest.mark.parametrize("T,k,G,I,K", [(1, 1, 1, 1, 32), (1, 8, 16, 33, 160), (3, 4, 40, 64, 512),
                                       (2, 8, 128, 24, 2048), (37, 4, 8, 35, 288), (9, 3, 5, 130, 1056)])
def test_swiglu(T, k, G, I, K):
    g = torch.Generator().manual_seed(T + I)
    ids = torch.randint(0, G, (T, k), generator=g, dtype=torch.int32)
    prob = torch.rand(T, k, generator=g)
    check_act(acts(T, K, I + K), ids, prob, weights(G, 2 * I, K, K), I, k)


# N / 128 (swiglu: / 64) tiles times min(rows, G) reach 160 workgroups here: the
# kernel that stages x, with one to four rows a wave, blocks and turns of
# scales cut short (K % 512, K % 1024) and ragged tiles
@pytest.mark.parametrize("T,k,G,N,K", [(40, 1, 40, 520, 64), (41, 4, 41, 500, 448), (24, 8, 8, 2600, 576),
                                       (400, 1, 40, 513, 1088), (1, 8, 9, 2561, 2304),
                                       (170, 3, 160, 20, 1024)])
def test_many_workgroups(T, k, G, N, K):
    g = torch.Generator().manual_seed(T + N)
    ids = torch.randint(-1, G, (T, k), generator=g, dtype=torch.int32)
    w = weights(G, N, K, K)
    check_plain(acts(T, K, N + K), ids, w, N, k)
    check_plain(acts(T * k, K, N + K), ids, w, N, 1)


@pytest.mark.parametrize("T,k,G,I,K", [(40, 1, 40, 260, 64), (41, 4, 41, 250, 448), (60, 8, 16, 700, 1600)])
def test_many_workgroups_swiglu(T, k, G, I, K):
    g = torch.Generator().manual_seed(T + I)
    ids = torch.randint(0, G, (T, k), generator=g, dtype=torch.int32)
    check_act(acts(T, K, I + K), ids, torch.rand(T, k, generator=g), weights(G, 2 * I, K, K), I, k)


@pytest.mark.parametrize("order", ["rising", "falling", "spikes", "tiny", "zero"])
def test_rows_of_wide_range(order):
    """x whose magnitude changes by 2^60 along the row, in both kernels: what a
    scaled binary16 loses is bounded by 2^-38 of the row's largest value."""
    for G, N in ((3, 20), (40, 640)):
        K, rows = 2048, 45
        ids = torch.arange(rows, dtype=torch.int32) % G
        g = torch.Generator().manual_seed(7)
        x = torch.randn(rows, K, generator=g)
        step = torch.linspace(-30, 30, K)
        if order == "rising":
            x = x * torch.exp2(step)
        elif order == "falling":
            x = x * torch.exp2(-step)
        elif order == "spikes":
            x[:, 1000::700] *= 2.0 ** 40
        elif order == "tiny":
            x = x * 2.0 ** -120
        else:
            x[::2] = 0
        x = x.to(torch.bfloat16)
        q, sb, sg, rps = weights(G, N, K, 7)
        want, size = ref.gemv(x, ids, q, sb, sg, N, rps, 1)
        top = ref.f64(x).abs().amax(1, keepdim=True)
        ones = torch.ones(rows, K, dtype=torch.bfloat16)
        # sum of |w|: the size of a product with ones
        weight = ref.gemv(ones, ids, q, sb, sg, N, rps, 1)[1]
        got = run_plain(x, ids, (q, sb, sg, rps), N)
        bound = ref.gemv_bound(size, K) + 2.0 ** -38 * top * weight + 2.0 ** -149
        assert ((ref.f64(got) - want).abs() <= bound).all()


def test_large_gates_do_not_overflow():
    q, sb, sg, rps = weights(2, 64, 256, 3)
    x = acts(4, 256, 4) * 3000
    prob = torch.tensor([0.5, 0.0, 1.0, 0.25])
    check_act(x, torch.tensor([0, 1, 1, 0], dtype=torch.int32), prob, (q, sb, sg, rps), 32)


@pytest.mark.parametrize("rps", [1, 8, 24, 48])
def test_outer_scales_of_any_scope(rps):
    ids = torch.tensor([2, 0, 1, 2], dtype=torch.int32)
    w = weights(3, 48, 128, rps, rps)
    check_plain(acts(4, 128, rps), ids, w, 48)
    check_act(acts(4, 128, rps), ids, torch.rand(4), w, 24)


@pytest.mark.parametrize("G", [4, 100])
def test_rows_without_an_expert_give_zero(G):
    """Both ways of finding an expert's rows (G above and below the rows)."""
    ids = torch.tensor([1, -1, 3, G, 1, -7, 2 ** 31 - 1, 0, 3], dtype=torch.int32)
    w = weights(G, 36, 96, G)
    check_plain(acts(9, 96, 1), ids, w, 36)
    got = run_plain(acts(9, 96, 1), ids, w, 36)
    assert not got[[1, 3, 5, 6]].any()
    check_act(acts(9, 96, 1), ids, torch.rand(9), weights(G, 36, 96, G), 18)
    none = torch.full((5,), -1, dtype=torch.int32)
    assert not run_plain(acts(5, 96, 1), none, w, 36).any()


@pytest.mark.parametrize("rows,G", [(15, 64), (16, 64), (17, 64), (33, 2), (100, 1), (700, 3)])
def test_many_rows_of_one_expert(rows, G):
    ids = torch.full((rows,), G - 1, dtype=torch.int32)
    ids[::7] = 0
    check_plain(acts(rows, 192, rows), ids, weights(G, 40, 192, rows), 40)
    check_act(acts(rows, 192, rows), ids, torch.rand(rows), weights(G, 40, 192, rows), 20)


def test_most_rows_that_are_taken():
    ids = torch.randint(0, 6, (4096,), generator=torch.Generator().manual_seed(1),
                        dtype=torch.int32)
    check_plain(acts(4096, 64, 1), ids, weights(6, 16, 64, 1), 16)


@pytest.mark.parametrize("N", [32, 7000])
def test_a_row_depends_on_its_own_values_alone(N):
    """NaN and infinities in one row of x stay in the rows computed from it."""
    ids = torch.tensor([2, 2, 2, 1, 2], dtype=torch.int32)
    x = acts(5, 128, 2)
    w = weights(3, N, 128, 2)
    want = run_plain(x, ids, w, N)
    bad = x.clone()
    bad[1] = float("nan")
    bad[3, 7] = float("inf")
    got = run_plain(bad, ids, w, N)
    keep = [0, 2, 4]
    assert torch.equal(got[keep], want[keep])
    assert not torch.isfinite(got[1]).any()


@pytest.mark.parametrize("N,K", [(40, 96), (40, 64), (40, 320), (40, 800), (640, 64), (640, 320), (640, 832),
                                 (640, 1088)])
def test_a_weight_row_of_nan_scales_stays_alone(N, K):
    """Rows end inside a chunk of 256: what is read past the end belongs to the
    next row, whose NaN must not meet the zeros that x has there."""
    rows = G = 41
    ids = torch.arange(rows, dtype=torch.int32)
    x = acts(rows, K, K)
    q, sb, sg, rps = weights(G, N, K, K)
    clean = run_plain(x, ids, (q, sb, sg, rps), N)
    bad = sb.clone()
    bad.view(G, N, -1)[:, 1::2] = 0x7F
    got = run_plain(x, ids, (q, bad, sg, rps), N)
    assert torch.equal(got[:, 0::2], clean[:, 0::2])
    assert got[:, 1::2].isnan().all()
    prob = torch.ones(rows, 1)
    act = [pqm.moe_gemv_swiglu_nvfp4(x.cuda(), ids.view(-1, 1).cuda(), prob.cuda(), q.cuda(), s.cuda(), sg.cuda(),
                                     N // 2, rps, 1) for s in (sb, bad)]
    assert torch.equal(act[0][:, 0::2], act[1][:, 0::2])


@pytest.mark.parametrize("N", [96, 2050])
def test_same_result_whatever_else_is_in_the_batch(N):
    """The same number of rows, the others' experts and values changed."""
    w = weights(20, N, 256, 5)
    x = acts(30, 256, 5)
    g = torch.Generator().manual_seed(5)
    ids = torch.randint(0, 20, (30,), generator=g, dtype=torch.int32)
    whole = run_plain(x, ids, w, N)
    for r in (0, 7, 29):
        other, elsewhere = acts(30, 256, r + 50) * 1000, torch.randint(-1, 20, (30,), generator=g,
                                                                        dtype=torch.int32)
        other[r], elsewhere[r] = x[r], ids[r]
        assert torch.equal(run_plain(other, elsewhere, w, N)[r], whole[r])


def test_nothing_behind_the_rows_is_written():
    w = weights(4, 50, 64, 6)
    q, sb, sg, rps = (t.cuda() if torch.is_tensor(t) else t for t in w)
    x, ids = acts(3, 64, 6).cuda(), torch.tensor([3, 0, 3], dtype=torch.int32).cuda()
    out = torch.full((5, 50), 7.0, device="cuda")
    f = pqm.lib().pqm_moe_gemv_nvfp4
    st = torch.cuda.current_stream().cuda_stream
    assert f(x.data_ptr(), ids.data_ptr(), 3, 1, q.data_ptr(), sb.data_ptr(), sg.data_ptr(), rps, 4,
             50, 64, out.data_ptr(), pqm.OUT_FP32, st) == 0
    torch.cuda.synchronize()
    assert (out[3:] == 7.0).all() and torch.equal(out[:3].cpu(), run_plain(x.cpu(), ids.cpu(), w, 50).cpu())


def test_no_rows_and_refusals():
    w = weights(4, 32, 64, 6)
    e = torch.zeros(0, dtype=torch.int32)
    assert run_plain(acts(0, 64, 1), e, w, 32).shape == (0, 32)
    x, ids = acts(4, 64, 1), torch.zeros(4, dtype=torch.int32)
    with pytest.raises(ValueError):
        run_plain(x, ids[:3], w, 32)               # x has one row too many
    with pytest.raises(TypeError):
        run_plain(x, ids.long(), w, 32)
    with pytest.raises(ValueError):
        run_plain(x, ids, (w[0], w[1][:-1], w[2], w[3]), 32)
    with pytest.raises(ValueError):
        run_plain(x, ids, (w[0], w[1], w[2][:-1], w[3]), 32)
    with pytest.raises(pqm.PqmError):
        run_plain(acts(4, 48, 1), ids, weights(4, 32, 48, 6), 32)   # K % 32
    with pytest.raises(pqm.PqmError):
        run_plain(acts(4097, 64, 1), torch.zeros(4097, dtype=torch.int32), w, 32)


def test_offsets_beyond_32_bits():
    """The last expert of a weight array of more than 2^32 bytes."""
    G, N, K = 520, 2048, 8192
    q = torch.zeros(G * N, K // 2, dtype=torch.uint8, device="cuda")
    sb = torch.zeros(G * N, K // 16, dtype=torch.uint8, device="cuda")
    sg = torch.zeros(G, device="cuda")
    assert q.numel() > 2 ** 32
    few = weights(1, N, K, 7)
    for dst, src in zip((q, sb), few[:2]):
        dst[(G - 1) * N:] = src.cuda()
    sg[G - 1] = few[2].item()
    x = acts(2, K, 7)
    a = pqm.moe_gemv_nvfp4(x.cuda(), torch.tensor([G - 1, 3], dtype=torch.int32).cuda(), q, sb, sg,
                           N, out_dtype=pqm.OUT_FP32)
    b = run_plain(x[:1], torch.zeros(1, dtype=torch.int32), few, N)
    assert torch.equal(a[0], b[0]) and not a[1].any()


def test_quantizer_weights_other_stream_and_graph_replay():
    """Weights from the quantizer; the same bits on another stream and from a
    captured graph whose ids change between replays."""
    g = torch.Generator().manual_seed(8)
    w = (torch.randn(16 * 96, 256, generator=g) * 0.02).to(torch.bfloat16).cuda()
    q, sb, sg = pqm.quantize_nvfp4_per_token(w, rows_per_scale=96)
    x = acts(24, 256, 8).cuda()
    ids = torch.randint(0, 16, (24,), generator=g, dtype=torch.int32).cuda()
    prob = torch.rand(24, generator=g).cuda()

    def both():
        return (pqm.moe_gemv_nvfp4(x, ids, q, sb, sg, 96),
                pqm.moe_gemv_swiglu_nvfp4(x, ids, prob, q, sb, sg, 48))
    check_plain(x.cpu(), ids.cpu(), (q.cpu(), sb.cpu(), sg.cpu(), 96), 96)
    want = both()
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        got = both()
    st.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = both()
    for i in range(4):
        ids.copy_(torch.randint(-1, 16, (24,), generator=g, dtype=torch.int32))
        for t in out:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(both(), out)), i
        torch.cuda.synchronize()
