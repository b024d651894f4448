"""Log probabilities, entropies, alternatives and their gradient against
binary64 on the same logits.

Bounds, from the arithmetic (U half a step of binary32): an exponent u is off by
4 U |u| (the difference, the constant and its product, the division); the
hardware's exponential by 2 U; a thread adds at most n values, its own maxima
move the sum at most n times by a factor off by 4 U 200 where it matters not, so
a sum of S positive terms is off by (n + 16) 2 U + 4 U sum p |u|.  With n from
the plan of 256 threads a part that is the relative error of S, and the absolute
one of log S.  log itself and the final difference add 4 U of their values."""
from __future__ import annotations

import math

import pytest
import torch

import precision_quantization_moe_amd as pqm
from gpu_util import requires_gpu
from operators_ref import HALF_BF16, U, f64

pytestmark = [pytest.mark.gpu, requires_gpu]

INF = math.inf


def reference(x, t):
    """(M, u, log S, p, H) of rows in binary64; rows of -inf alone have p = 0."""
    z = f64(x)
    m = z.amax(1, keepdim=True)
    none = m == -INF
    u = (z - torch.where(none, torch.zeros_like(m), m)) / t
    e = torch.exp(u)
    s = e.sum(1, keepdim=True)
    ls = torch.where(none, torch.zeros_like(s), torch.log(s))
    p = torch.where(none, torch.zeros_like(e), e / s)
    uu = torch.where(p > 0, u, torch.zeros_like(u))
    h = torch.where(none, torch.zeros_like(s), ls - (p * uu).sum(1, keepdim=True))
    return m[:, 0], u, ls[:, 0], p, h[:, 0], (p * uu.abs()).sum(1)


def logits(T, V, dtype, seed, masked=True):
    g = torch.Generator().manual_seed(seed)
    x = 2.5 * torch.randn(T, V, generator=g)
    x.scatter_(1, torch.randint(0, V, (T, 4), generator=g), 9.0)
    if masked and V > 8:
        x[:, V - V // 8:] = -INF
    ids = torch.randint(0, max(V - V // 8, 1), (T,), generator=g).to(torch.int32)
    return x.to(dtype), ids, g


def order(x, n):
    """The n best, ties to the lowest index."""
    z = x.float().cpu()
    return torch.sort(z, dim=1, descending=True, stable=True).indices[:, :n]


def check(x, ids, t, n, out):
    lp, ent, stats, top_ids, top_lp = out
    T, V = x.shape
    m, u, ls, p, h, mean_u = reference(x, t)
    live = (ids >= 0) & (ids < V)
    terms = V / 256 + 16  # of a thread at most, and the joining
    e_s = 1.05 * ((terms + 16) * 2 * U + 4 * U * mean_u)  # of log S
    got = f64(stats)
    zero = torch.zeros(T).double()
    assert torch.equal(got[:, 0], torch.where(live, m, zero))
    assert ((got[:, 1] - torch.where(live, ls, zero)).abs() <= e_s + 4 * U * ls.abs()).all()
    if lp is not None:
        i = ids.long().clamp(0, V - 1)[:, None]
        ui = u.gather(1, i)[:, 0]
        want = torch.where(live, ui - ls, zero)
        inf = want == -INF
        assert torch.equal(f64(lp) == -INF, inf)
        bound = e_s + 4 * U * (ls.abs() + ui.abs()) + 4 * U * want.abs()
        assert ((f64(lp) - want).abs() <= bound)[~inf].all(), float(((f64(lp) - want).abs() / bound)[~inf].max())
    # sum p |u| is off by itself times the error of S twice, and each term's own
    bound = e_s + mean_u * (2 * e_s + 16 * U) + 8 * U * (ls.abs() + mean_u) + (p * u.clamp(min=-200) ** 2).sum(1) * 4 * U
    want = torch.where(live, h, zero)
    assert ((f64(ent) - want).abs() <= bound).all(), float(((f64(ent) - want).abs() / bound).max())
    if n:
        best = order(x, n)
        assert torch.equal(top_ids.cpu().long(), torch.where(live[:, None], best, torch.full_like(best, -1)))
        ub = u.gather(1, best)
        want = torch.where(live[:, None], ub - ls[:, None], torch.zeros_like(ub))
        inf = want == -INF
        assert torch.equal(f64(top_lp) == -INF, inf)
        bound = (e_s + 4 * U * ls.abs())[:, None] + 4 * U * ub.abs() + 4 * U * want.abs()
        assert ((f64(top_lp) - want).abs() <= bound)[~inf].all()


SHAPES = [(1, 1), (1, 7), (3, 8), (2, 33), (5, 255), (1, 2047), (2, 2048), (3, 2049), (4, 8191),
          (70, 1000), (1, 50257), (3, 32000), (1, 151936), (1100, 4099), (1030, 513)]


@pytest.mark.parametrize("T,V", SHAPES)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("n", [0, 1, 20, 32])
def test_forward(T, V, dtype, n):
    x, ids, _ = logits(T, V, dtype, 7 * T + V)
    if T > 2:
        ids[1], ids[T - 1] = -1, V
    n = min(n, V)
    for t in (1.0, 0.7):
        check(x, ids, t, n, pqm.token_logprobs(x.cuda(), ids.cuda(), t, n))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_rows_of_a_wider_tensor(dtype):
    """Rows that start at any element, with something else between them."""
    for T, V, a, b in ((5, 1001, 3, 4), (3, 5000, 1, 0), (2, 20011, 0, 7)):
        x, ids, _ = logits(T, V + a + b, dtype, V, False)
        x[:, :a], x[:, a + V:] = math.nan, math.nan
        d, ids = x.cuda()[:, a:a + V], (ids % V).to(torch.int32)
        check(x[:, a:a + V], ids, 1.3, 5, pqm.token_logprobs(d, ids.cuda(), 1.3, 5))


@pytest.mark.parametrize("n", [1, 8, 32])
@pytest.mark.parametrize("T", [1, 40, 1200])
def test_alternatives_in_any_order(n, T):
    """Ascending, descending, equal, few different and hidden maxima: the choice
    and its order do not depend on where the largest stand."""
    V = 9000
    g = torch.Generator().manual_seed(n)
    rows = [torch.linspace(-5, 5, V), torch.linspace(5, -5, V), torch.full((V,), 1.5), torch.full((V,), -INF),
            torch.randint(0, 3, (V,), generator=g).float(), -torch.zeros(V)]
    last = torch.full((V,), -3.0)
    last[V - n:] = torch.arange(n).float()
    rows.append(last)
    alternate = torch.zeros(V)
    alternate[1::2] = -0.0
    rows.append(alternate)
    x = torch.stack([rows[i % len(rows)] for i in range(T)]).to(torch.bfloat16)
    ids = torch.zeros(T, dtype=torch.int32)
    out = pqm.token_logprobs(x.cuda(), ids.cuda(), 1.0, n)
    best = order(x + 0.0, n)
    assert torch.equal(out[3].cpu().long(), best)
    no_ids = pqm.token_logprobs(x.cuda(), None, 1.0, n)
    assert no_ids[0] is None and all(torch.equal(a, b) for a, b in zip(no_ids[1:], out[1:]))


@pytest.mark.parametrize("T", [1, 1200])
@pytest.mark.parametrize("n", [0, 4])
def test_infinities_and_nan(T, n):
    V = 3000
    x = torch.randn(T, V, generator=torch.Generator().manual_seed(1))
    ids = torch.full((T,), 11, dtype=torch.int32)

    def run(row, i=11):
        a = x.clone()
        a[0] = row
        ids[0] = i
        d = a.cuda()
        o = pqm.token_logprobs(d, ids.cuda(), 1.0, n)
        lp, ent, st = (t[0].cpu() for t in o[:3])
        one = torch.ones(T).cuda()
        g = pqm.token_logprobs_backward(d, ids.cuda(), o[2], one, 1.0, o[1], one)[0].cpu()
        return lp, ent, st, g, o
    # nothing left
    lp, ent, st, g, o = run(torch.full((V,), -INF))
    assert lp == -INF and ent == 0 and st[0] == -INF and st[1] == 0 and not g.any()
    if n:
        assert o[3][0].cpu().tolist() == list(range(n)) and (o[4][0] == -INF).all()
    # one left: certain
    r = torch.full((V,), -INF)
    r[2999] = -5.0
    lp, ent, st, g, _ = run(r, 2999)
    assert lp == 0 and ent == 0 and st[0] == -5 and st[1] == 0 and not g.any()
    lp, ent, st, g, _ = run(r)
    assert lp == -INF and ent == 0 and g[11] == 1 and g[2999] == -1
    # the lowest value as the mask: alone it masks nothing
    low = torch.finfo(torch.float32).min
    r = torch.full((V,), low)
    lp, ent, st, g, _ = run(r)
    assert abs(float(lp) + math.log(V)) < 1e-5 and abs(float(ent) - math.log(V)) < 1e-5 and st[0] == low
    r[5:9] = 3.0
    lp, ent, st, g, _ = run(r, 7)
    assert abs(float(lp) + math.log(4)) < 1e-6 and abs(float(ent) - math.log(4)) < 1e-6
    assert not g[9:].any()
    # the same logits far from zero
    r = x[0] + 0
    a = run(r)
    r2 = (r * 1024).round() / 1024 + 4096.0  # exact in binary32
    b = run(r2)
    c = run((r * 1024).round() / 1024)
    assert b[0] == c[0] and b[1] == c[1] and torch.equal(b[3], c[3]) and abs(float(a[0] - c[0])) < 1e-2
    # what is not a number shows
    for bad in (math.nan, INF):
        r = x[0] + 0
        r[17] = bad
        lp, ent, st, g, o = run(r)
        assert lp.isnan() and ent.isnan() and st[1].isnan() and g.isnan().all()
        if n:
            assert int(o[3][0, 0]) == 17 and o[4][0].isnan().all()
        if T > 1:
            assert o[0][1:].isfinite().all()
    r = torch.full((V,), -INF)
    r[3] = math.nan
    lp, ent, st, g, _ = run(r)
    assert lp.isnan() and ent.isnan() and g.isnan().all()
    # a row that is left out is not read
    lp, ent, st, g, o = run(torch.full((V,), math.nan), -1)
    assert lp == 0 and ent == 0 and not st.any() and not g.any()
    if n:
        assert (o[3][0] == -1).all() and not o[4][0].any()


@pytest.mark.parametrize("T,V", [(1, 1), (2, 9), (3, 255), (2, 8192), (3, 8193), (5, 20001), (1, 151936),
                                 (300, 1023)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("which", ["logprob", "entropy", "both"])
def test_backward(T, V, dtype, which):
    x, ids, g = logits(T, V, dtype, T + V)
    if T > 2:
        ids[1], ids[2] = -1, V + 5
    t = 0.8
    d, i = x.cuda(), ids.cuda()
    lp, ent, stats, _, _ = pqm.token_logprobs(d, i, t)
    gl = torch.randn(T, generator=g) if which != "entropy" else None
    gh = torch.randn(T, generator=g) if which != "logprob" else None
    args = (d, i, stats, gl.cuda() if gl is not None else None, t, ent, gh.cuda() if gh is not None else None)
    for out_dtype in (pqm.OUT_FP32, pqm.OUT_BF16):
        got = pqm.token_logprobs_backward(*args, out_dtype=out_dtype)
        torch.cuda.synchronize()
        m, u, ls, p, h, mean_u = reference(x, t)
        live = ((ids >= 0) & (ids < V))[:, None]
        a = f64(gl)[:, None] if gl is not None else torch.zeros(T, 1).double()
        b = f64(gh)[:, None] if gh is not None else torch.zeros(T, 1).double()
        logp = torch.where(p > 0, u - ls[:, None], torch.zeros_like(u))
        hot = torch.zeros_like(p).scatter_(1, ids.long().clamp(0, V - 1)[:, None], 1.0)
        want = (a * (hot - p) - b * p * (logp + h[:, None])) / t
        # the exponent: as the forward's, and stats' own error; the entropy's too
        e_s = 1.05 * ((V / 256 + 32) * 2 * U + 4 * U * mean_u)[:, None] + 4 * U * ls.abs()[:, None]
        e_u = e_s + 6 * U * (u.clamp(min=-200).abs() + ls.abs()[:, None])
        e_h = e_s * (3 + 2 * mean_u[:, None]) + 16 * U * (ls + mean_u)[:, None] + \
            (p * u.clamp(min=-200) ** 2).sum(1, keepdim=True) * 4 * U
        size = a.abs() + b.abs() * (logp.abs() + h.abs()[:, None])
        bound = 1.05 * (p * (size * (e_u + 12 * U) + b.abs() * (e_u + e_h)) + hot * a.abs() * 4 * U) / t
        want, bound = torch.where(live, want, 0 * want), torch.where(live, bound, 0 * bound)
        if out_dtype == pqm.OUT_BF16:
            bound = bound + HALF_BF16 * (want.abs() + bound)
        err = (f64(got) - want).abs()
        assert (err <= bound + 2.0 ** -125).all(), (which, out_dtype, float((err / (bound + 1e-30)).max()))
    # in the logits' own memory, and into a wider tensor
    same = pqm.token_logprobs_backward(*args)
    wide = torch.full((T, V + 3), 7.0, dtype=dtype).cuda()
    pqm.token_logprobs_backward(*args, out=wide[:, 2:2 + V])
    assert torch.equal(wide[:, 2:2 + V], same) and (wide[:, :2] == 7).all() and (wide[:, 2 + V:] == 7).all()
    assert pqm.token_logprobs_backward(*args, out=d) is d
    assert torch.equal(d, same)


def test_no_rows():
    x = torch.zeros(0, 100).cuda()
    ids = torch.zeros(0, dtype=torch.int32).cuda()
    lp, ent, st, ti, tl = pqm.token_logprobs(x, ids, 1.0, 4)
    assert lp.shape == ent.shape == (0,) and st.shape == (0, 2) and ti.shape == tl.shape == (0, 4)
    assert pqm.token_logprobs_backward(x, ids, st, lp).shape == (0, 100)


def test_same_bits_and_captured():
    """Every call gives the same bits, also captured and replayed beside eager
    calls, in parts (one row) and whole (many)."""
    for T in (2, 1500):
        x, ids, g = logits(T, 5001, torch.bfloat16, T)
        x, ids = x.cuda(), ids.cuda()
        one = torch.ones(T).cuda()

        def step():
            o = pqm.token_logprobs(x, ids, 0.9, 6)
            return o + (pqm.token_logprobs_backward(x, ids, o[2], one, 0.9, o[1], one),)
        step()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = step()
        for i in range(3):
            n, _, _ = logits(T, 5001, torch.bfloat16, 100 + i)
            x.copy_(n)
            for t in out:
                t.zero_()
            graph.replay()
            torch.cuda.synchronize()
            want = step()
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(out, want)), (T, i)


def test_rows_beyond_32_bits():
    """More than 2^31 logits, and a row stride that takes offsets there alone."""
    T, V = 70000, 32000
    g = torch.Generator(device="cuda").manual_seed(2)
    x = torch.randn(T, V, generator=g, device="cuda", dtype=torch.bfloat16)
    ids = torch.full((T,), -1, dtype=torch.int32)
    rows = torch.tensor([0, 67108, 67109, 69999])
    ids[rows] = torch.tensor([5, 31999, 0, 77], dtype=torch.int32)
    o = pqm.token_logprobs(x, ids.cuda(), 1.0)
    pick = rows.cuda()
    check(x[pick].cpu(), ids[rows], 1.0, 0, tuple(t[pick] if t is not None else None for t in o))
    one = torch.ones(T).cuda()
    d = pqm.token_logprobs_backward(x, ids.cuda(), o[2], one)
    alone = pqm.token_logprobs_backward(x[pick].contiguous(), ids[rows].cuda(), o[2][pick].contiguous(),
                                        one[:4].contiguous())
    assert torch.equal(d[pick], alone) and not d[69990:69999].any()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("n", [0, 4])
def test_more_logits_than_the_caches_hold(dtype, n):
    """From 200 MB on logits and gradients go past the caches: the same results, at
    odd lengths and offsets too, and nothing beside the rows is written."""
    T, V = 1100, 100003 if dtype is torch.bfloat16 else 50001
    g = torch.Generator(device="cuda").manual_seed(V)
    x = torch.randn(T, V + 3, generator=g, device="cuda").mul_(3).to(dtype)[:, 1:V + 1]
    ids = torch.full((T,), -1, dtype=torch.int32)
    rows = torch.tensor([0, 1, 700, 1098, 1099])
    ids[rows] = torch.tensor([5, V - 1, 0, 77, V - 2], dtype=torch.int32)
    o = pqm.token_logprobs(x, ids.cuda(), 0.9, n)
    pick = rows.cuda()
    few = x[pick].contiguous()
    check(few.cpu(), ids[rows], 0.9, n, tuple(t[pick] if t is not None else None for t in o))
    one = torch.ones(T).cuda()
    for out_dtype in (torch.bfloat16, torch.float32):
        wide = torch.full((T, V + 3), 7.0, dtype=out_dtype, device="cuda")
        d = pqm.token_logprobs_backward(x, ids.cuda(), o[2], one, 0.9, o[1], one, out=wide[:, 2:V + 2])
        alone = pqm.token_logprobs_backward(few, ids[rows].cuda(), o[2][pick].contiguous(), one[:5].contiguous(), 0.9,
                                            o[1][pick].contiguous(), one[:5].contiguous(),
                                            out_dtype=pqm.OUT_BF16 if out_dtype is torch.bfloat16 else pqm.OUT_FP32)
        assert torch.equal(d[pick], alone) and not d[2:700].any()
        assert (wide[:, :2] == 7).all() and (wide[:, V + 2:] == 7).all()
    same = x.contiguous()
    want = pqm.token_logprobs_backward(x, ids.cuda(), o[2], one, 0.9, o[1], one)
    assert pqm.token_logprobs_backward(same, ids.cuda(), o[2], one, 0.9, o[1], one, out=same) is same
    assert torch.equal(same, want)


@pytest.mark.parametrize("T,V", [(1, 151936), (2, 9), (40, 5000), (1200, 3001)])
@pytest.mark.parametrize("n", [0, 3])
def test_nearly_certain_rows(T, V, n):
    """Rows whose largest logit holds all but 2^-10 to 2^-60 of the probability: the
    entropy and that token's log probability, as small as what is left, keep their
    relative precision.  r = S - 1 is a sum of positive terms of a relative error of
    4 U |u| + 2 U each, V / 256 + 32 additions; log(1 + r) and the quotient add 8 U;
    both parts of the entropy are positive."""
    g = torch.Generator().manual_seed(T + V)
    x = torch.rand(T, V, generator=g)
    top = torch.randint(0, V, (T,), generator=g)
    x.scatter_(1, top[:, None], (7 + 30 * torch.rand(T, 1, generator=g)) + math.log(V))
    lp, ent, stats, _, _ = pqm.token_logprobs(x.cuda(), top.to(torch.int32).cuda(), 1.0, n)
    z = f64(x)
    u = z - z.gather(1, top[:, None])
    e = torch.exp(u).scatter_(1, top[:, None], 0.0)
    r = e.sum(1)
    ls, h = torch.log1p(r), torch.log1p(r) - (e * u).sum(1) / (1 + r)
    rel = 1.05 * (2 * (V / 256 + 32) + 4 * float(u.abs().max()) + 16) * U
    assert ((f64(ent) - h).abs() <= rel * h).all(), float(((f64(ent) - h).abs() / h / rel).max())
    assert ((f64(lp) + ls).abs() <= rel * ls).all() and ((f64(stats)[:, 1] - ls).abs() <= rel * ls).all()


@pytest.mark.parametrize("T,V", [(1, 151936), (2, 9), (40, 5000), (1200, 3001)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("which", ["logprob", "entropy", "both"])
def test_gradients_of_nearly_certain_rows(T, V, dtype, which):
    """The taken token's gradient of such rows, g (1 - p) - h p (log p + H), is as
    small as what is left and keeps its relative precision: 1 - p is that of log S
    (rel above) and expm1's 4 U, and both terms of log p + H are off by rel of
    themselves and 16 U for the factors."""
    g = torch.Generator().manual_seed(T + V + 1)
    x = torch.rand(T, V, generator=g)
    top = torch.randint(0, V, (T,), generator=g)
    x.scatter_(1, top[:, None], (7 + 30 * torch.rand(T, 1, generator=g)) + math.log(V))
    x = x.to(dtype)
    ids = top.to(torch.int32).cuda()
    o = pqm.token_logprobs(x.cuda(), ids)
    a = torch.randn(T, generator=g) if which != "entropy" else torch.zeros(T)
    b = torch.randn(T, generator=g) if which != "logprob" else torch.zeros(T)
    d = pqm.token_logprobs_backward(x.cuda(), ids, o[2], a.cuda() if which != "entropy" else None, 1.0,
                                    o[1], b.cuda() if which != "logprob" else None, out_dtype=pqm.OUT_FP32)
    got = f64(d).gather(1, top[:, None])[:, 0]
    z = f64(x)
    u = z - z.gather(1, top[:, None])
    e = torch.exp(u).scatter_(1, top[:, None], 0.0)
    r, ls = e.sum(1), torch.log1p(e.sum(1))
    h = ls - (e * u).sum(1) / (1 + r)
    p, left = 1 / (1 + r), r / (1 + r)
    want = f64(a) * left - f64(b) * p * (h - ls)
    rel = 1.05 * (2 * (V / 256 + 32) + 4 * float(u.abs().max()) + 32) * U
    bound = rel * (f64(a).abs() * left + f64(b).abs() * (h + ls))
    assert ((got - want).abs() <= bound).all(), float(((got - want).abs() / bound).max())


@pytest.mark.parametrize("n", [0, 5])
def test_rows_do_not_depend_on_their_place(n):
    """In calls of the same sizes a row has the same bits wherever it stands; in calls
    of other sizes they are within the bounds of both."""
    T, V = 1500, 9001
    x, ids, g = logits(T, V, torch.bfloat16, 5)
    p = torch.randperm(T, generator=g)
    a = pqm.token_logprobs(x.cuda(), ids.cuda(), 0.7, n)
    b = pqm.token_logprobs(x[p].cuda(), ids[p].cuda(), 0.7, n)
    one = torch.ones(T).cuda()
    da = pqm.token_logprobs_backward(x.cuda(), ids.cuda(), a[2], one, 0.7, a[1], one)
    db = pqm.token_logprobs_backward(x[p].cuda(), ids[p].cuda(), b[2], one, 0.7, b[1], one)
    for u, v in zip(a + (da,), b + (db,)):
        assert u is None and v is None or torch.equal(u[p.cuda()], v)
    for few in (1, 3, 300):
        check(x[:few], ids[:few], 0.7, n, pqm.token_logprobs(x[:few].cuda(), ids[:few].cuda(), 0.7, n))


def test_a_row_of_many_logits():
    """2^28 + 5 logits in one row: places beyond 2^24, parts of many turns, the best
    ones near the end.  A thread adds 2^28 / 128 / 256 = 8192 values and the joining 140
    more; |u| is below 12."""
    V = (1 << 28) + 5
    g = torch.Generator(device="cuda").manual_seed(3)
    x = torch.rand(1, V, generator=g, device="cuda", dtype=torch.float32).to(torch.bfloat16)
    best = [V - 1, V - 7, 5, V // 2 + 1]
    for i, at in enumerate(best):
        x[0, at] = 9.0 - i
    id_ = torch.tensor([V - 7], dtype=torch.int32).cuda()
    lp, ent, stats, ids, top = pqm.token_logprobs(x, id_, 1.0, 4)
    u = x[0].double() - 9.0
    s = torch.exp(u).sum()
    h = torch.log(s) - (torch.exp(u) * u).sum() / s
    rel = 1.05 * ((8192 + 156) * 2 + 4 * 12) * U
    assert ids[0].tolist() == best and float(stats[0, 0]) == 9.0
    assert abs(float(stats[0, 1]) - float(torch.log(s))) <= rel + 4 * U * 20
    assert abs(float(lp) - float(-1.0 - torch.log(s))) <= rel + 8 * U * 20
    assert abs(float(ent) - float(h)) <= rel + 12 * (2 * rel + 16 * U) + 8 * U * 32 + 144 * 4 * U
    d = pqm.token_logprobs_backward(x, id_, stats, torch.ones(1, device="cuda"), out_dtype=pqm.OUT_FP32)
    p = torch.exp(u[best] - torch.log(s))
    want = -p + torch.tensor([0.0, 1.0, 0.0, 0.0], dtype=torch.float64, device="cuda")
    assert ((d[0, best].double() - want).abs() <= p * (rel + 200 * U) + 4 * U * want.abs()).all()
