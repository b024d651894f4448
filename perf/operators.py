"""Measured cases of the operators around the MoE experts' products.

Three operators and their two backward passes, each as the library's entry
points (`own` true) and as a plain form in elementary torch operations:

* norm      RMS norm with the residual's addition, output in MXFP8
* norm_bwd  its gradients
* gate      top-k router gate, per-expert counts and balance loss
* gate_bwd  its gradient
* gemv      a few routed rows times NVFP4 expert weights, plain or with the
            gate/up SwiGLU

`exact` computes the same from the definitions in binary64.
"""
import math

import torch

own = False

DEV = "cuda"
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# ------------------------------------------------------------------- cases

def listed():
    return [
        # one decode step of eight sequences: latency
        dict(name="norm_8x2048", op="norm", rows=8, cols=2048, residual=True, keep_y=True, w="bf16"),
        # a training micro-batch of the quantizers' benchmark shape
        dict(name="norm_16384x2048", op="norm", rows=16384, cols=2048, residual=True, keep_y=False,
             w="bf16"),
        # its backward pass, with the gradient that comes down the residual stream
        dict(name="norm_bwd_16384x2048", op="norm_bwd", rows=16384, cols=2048, residual=True, w="bf16"),
        # a ragged batch of wide rows, first norm of a network (nothing behind it)
        dict(name="norm_bwd_1021x7168", op="norm_bwd", rows=1021, cols=7168, residual=False, w="f32"),
        # decode: the gate of a small batch, no loss
        dict(name="gate_16x256", op="gate", tokens=16, experts=256, k=8, dtype="bf16",
             score="sigmoid", renorm=True, loss=False, masked=False),
        # training: two packed sequences of 8192 with padding behind each
        dict(name="gate_16384x128", op="gate", tokens=16384, experts=128, k=8, dtype="f32",
             score="softmax", renorm=True, loss=True, masked=True),
        dict(name="gate_bwd_16384x128", op="gate_bwd", tokens=16384, experts=128, k=8, dtype="f32",
             score="softmax", renorm=True, loss=True, masked=True),
        # a ragged batch, logits in bf16
        dict(name="gate_bwd_4093x256", op="gate_bwd", tokens=4093, experts=256, k=8, dtype="bf16",
             score="sigmoid", renorm=True, loss=True, masked=False),
        # decode of one sequence: gate/up and down of the top-8 of 128 experts
        dict(name="gemv_up_1tok", op="gemv", act=True, tokens=1, experts=128, k=8, hidden=2048,
             inter=768, out="bf16"),
        dict(name="gemv_down_1tok", op="gemv", act=False, tokens=1, experts=128, k=8, hidden=2048,
             inter=768, out="bf16"),
        # a decode batch in which every expert is met several times
        dict(name="gemv_up_37tok", op="gemv", act=True, tokens=37, experts=64, k=8, hidden=5120,
             inter=1280, out="bf16"),
        dict(name="gemv_down_29tok", op="gemv", act=False, tokens=29, experts=64, k=8, hidden=5120,
             inter=1280, out="f32"),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "norm_bwd", "gate", "gate_bwd", "gemv"])
    if op in ("norm", "norm_bwd"):
        cols = 32 * _log_int(rng, 4, 256)
        rows = min(_log_int(rng, 1, 16384), (16384 * 2048) // cols)
        c = dict(op=op, rows=rows, cols=cols, residual=rng.random() < 0.7,
                 w=rng.choice(["bf16", "f32"]))
        if op == "norm":
            c["keep_y"] = rng.random() < 0.5
        return c
    if op in ("gate", "gate_bwd"):
        experts = _log_int(rng, 8, 512)
        tokens = min(_log_int(rng, 1, 16384), (16384 * 128) // experts)
        return dict(op=op, tokens=tokens, experts=experts, k=rng.randint(1, 8),
                    dtype=rng.choice(["bf16", "f32"]), score=rng.choice(["softmax", "sigmoid"]),
                    renorm=rng.random() < 0.7, loss=True if op == "gate_bwd" else rng.random() < 0.7,
                    masked=rng.random() < 0.4)
    return dict(op="gemv", act=rng.random() < 0.5, tokens=_log_int(rng, 1, 28),
                experts=rng.randint(8, 64), k=rng.randint(1, 8), hidden=32 * rng.randint(16, 160),
                inter=32 * rng.randint(4, 40), out=rng.choice(["bf16", "f32"]))


# ------------------------------------------------------------------ inputs

def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(int(seed))


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device=DEV)


def _activations(g, rows, cols):
    """Log-normal magnitude per row, a few outlier channels."""
    x = _randn(g, rows, cols) * torch.exp(_randn(g, rows, 1))
    ch = torch.randint(0, cols, (8,), generator=g, device=DEV)
    x[:, ch] *= 1.0 + 20.0 * torch.rand(rows, 1, generator=g, device=DEV)
    return x


def _nvfp4_weights(g, groups, n, k):
    """NVFP4 weights of N(0, 0.02^2) with one outer scale per expert: packed
    codes [groups n, k/2], block scales [groups n, k/16], outer [groups]."""
    q = torch.empty(groups * n, k // 2, dtype=torch.uint8, device=DEV)
    sb = torch.empty(groups * n, k // 16, dtype=torch.uint8, device=DEV)
    sg = torch.empty(groups, device=DEV)
    mids = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device=DEV)
    for e in range(groups):
        w = _randn(g, n, k // 16, 16) * 0.02
        outer = w.abs().amax() / 2688.0
        s8 = (w.abs().amax(-1) / (6.0 * outer)).clamp(max=448.0).to(torch.float8_e4m3fn)
        v = w / (s8.float() * outer).clamp(min=1e-30)[..., None]
        code = torch.bucketize(v.abs(), mids, out_int32=True).to(torch.uint8)
        code = (code | (v < 0).to(torch.uint8) << 3).reshape(n, k)
        q[e * n:(e + 1) * n] = code[:, 0::2] | code[:, 1::2] << 4
        sb[e * n:(e + 1) * n] = s8.view(torch.uint8)
        sg[e] = outer
    return q, sb, sg


def _router_choice(z, mask, k):
    """The k largest logits of each row, ties to the lowest index; rows that
    the mask leaves out take experts in turn."""
    t, e = z.shape
    ids = torch.sort(z.float(), dim=1, descending=True, stable=True).indices[:, :k]
    if mask is not None:
        turn = torch.arange(t * k, device=z.device).view(t, k) % e
        ids = torch.where(mask[:, None] != 0, ids, turn)
    return ids


def _padding_mask(tokens):
    """Two sequences of half the tokens, the first with a fifth of padding
    behind it, the second with a seventh."""
    half = (tokens + 1) // 2
    m = torch.ones(tokens, dtype=torch.uint8, device=DEV)
    m[half - half // 5:half] = 0
    if tokens > half:
        m[tokens - (tokens - half) // 7:] = 0
    return m


def prepare(case, seed):
    g = _gen(seed)
    op = case["op"]
    s = dict(case)
    if op in ("norm", "norm_bwd"):
        rows, cols = case["rows"], case["cols"]
        x = _activations(g, rows, cols)
        w = 1.0 + 0.2 * _randn(g, cols)
        s["weight"] = w.to(torch.bfloat16) if case["w"] == "bf16" else w
        s["eps"] = 1e-6
        s["x"] = x.to(torch.bfloat16)
        r = _randn(g, rows, cols).to(torch.bfloat16) if case["residual"] else None
        if op == "norm":
            s["residual"] = r
        else:
            # x stands for the sum that the forward pass kept
            s["dsum"] = r
            s["dy"] = _randn(g, rows, cols).to(torch.bfloat16)
            ms = s["x"].double().square().mean(1)
            s["rstd"] = (1.0 / torch.sqrt(ms + s["eps"])).float()
        return s
    if op in ("gate", "gate_bwd"):
        t, e, k = case["tokens"], case["experts"], case["k"]
        z = 1.5 * _randn(g, t, e) + 0.7 * _randn(g, e)
        s["logits"] = z.to(torch.bfloat16) if case["dtype"] == "bf16" else z
        s["mask"] = _padding_mask(t) if case["masked"] else None
        s["scale"] = 2.5 if case["score"] == "sigmoid" else 1.0
        s["coef"] = 0.01
        if op == "gate_bwd":
            ids = _router_choice(s["logits"], s["mask"], k)
            valid = torch.ones(t, device=DEV) if s["mask"] is None else s["mask"].float()
            counts = torch.zeros(e + 1, dtype=torch.int64, device=DEV)
            counts.scatter_add_(0, ids.reshape(-1), valid.repeat_interleave(k).long())
            counts[e] = valid.sum().long()
            s["ids"] = ids.to(torch.int32)
            s["counts"] = counts.to(torch.int32)
            s["d_prob"] = _randn(g, t, k) * 0.01
            s["d_loss"] = torch.ones(1, device=DEV)
        return s
    t, e, k, h, i = (case[n] for n in ("tokens", "experts", "k", "hidden", "inter"))
    k = min(k, e)
    s["ids"] = torch.argsort(torch.rand(t, e, generator=g, device=DEV), dim=1)[:, :k].to(
        torch.int32).contiguous().view(-1)
    if case["act"]:
        s["x"] = _activations(g, t, h).to(torch.bfloat16)
        s["q"], s["sb"], s["sg"] = _nvfp4_weights(g, e, 2 * i, h)
        p = torch.rand(t, k, generator=g, device=DEV) + 0.1
        s["prob"] = (p / p.sum(1, keepdim=True)).view(-1)
        s["n"], s["div"] = 2 * i, k
    else:
        s["x"] = (_randn(g, t * k, i) * 0.3).to(torch.bfloat16)
        s["q"], s["sb"], s["sg"] = _nvfp4_weights(g, e, h, i)
        s["n"], s["div"] = h, 1
    return s


# ------------------------------------------------------- the library's calls

def _run_own(s):
    import precision_quantization_moe_amd as pqm
    op = s["op"]
    if op == "norm":
        q, sc, y, total, rstd = pqm.rmsnorm_quantize_mxfp8(
            s["x"], s["weight"], s["eps"], residual=s["residual"], keep_y=s["keep_y"])
        out = dict(q=q.view(torch.float8_e4m3fn), scale=sc.view(torch.float8_e8m0fnu), rstd=rstd)
        if s["keep_y"]:
            out["y"] = y
        if s["residual"] is not None:
            out["sum"] = total
        return out
    if op == "norm_bwd":
        dx, dw = pqm.rmsnorm_backward(s["dy"], s["x"], s["weight"], s["rstd"], d_sum=s["dsum"])
        return dict(dx=dx, dw=dw)
    score = pqm.SCORE_SOFTMAX if s.get("score") == "softmax" else pqm.SCORE_SIGMOID
    if op == "gate":
        ids, prob, counts, prob_sum, loss = pqm.moe_gate(
            s["logits"], s["k"], score=score, renormalize=s["renorm"], scale=s["scale"],
            mask=s["mask"], loss_coef=s["coef"] if s["loss"] else None)
        out = dict(ids=ids, prob=prob)
        if s["loss"]:
            out.update(counts=counts, prob_sum=prob_sum, loss=loss)
        return out
    if op == "gate_bwd":
        return pqm.moe_gate_backward(
            s["logits"], s["ids"], s["d_prob"], score=score, renormalize=s["renorm"],
            scale=s["scale"], mask=s["mask"], loss_coef=s["coef"], counts=s["counts"],
            d_loss=s["d_loss"])
    if s["act"]:
        return pqm.moe_gemv_swiglu_nvfp4(s["x"], s["ids"], s["prob"], s["q"], s["sb"], s["sg"],
                                         s["n"] // 2, divisor=s["div"])
    return pqm.moe_gemv_nvfp4(s["x"], s["ids"], s["q"], s["sb"], s["sg"], s["n"],
                              divisor=s["div"],
                              out_dtype=pqm.OUT_BF16 if s["out"] == "bf16" else pqm.OUT_FP32)


# ------------------------------------------------------------- plain forms

def _plain_norm(s):
    x = s["x"]
    if s["residual"] is not None:
        x = (x.float() + s["residual"].float()).to(torch.bfloat16)
    f = x.float()
    rstd = 1.0 / torch.sqrt((f * f).mean(1) + s["eps"])
    y = (f * rstd[:, None] * s["weight"].float()).to(torch.bfloat16)
    # MXFP8 rows: the smallest power of two that keeps 32 values within 448
    b = y.float().view(y.shape[0], -1, 32)
    m, ex = torch.frexp(b.abs().amax(-1))
    e = torch.where(m > 0.875, ex - 8, ex - 9)
    e = torch.where(m == 0, torch.full_like(e, -127), e.clamp(min=-127))
    down = ((127 - e) << 23).view(torch.float32)  # 2^-e by its bits: exact
    q = (b * down[..., None]).to(torch.float8_e4m3fn).view(y.shape)
    out = dict(q=q, scale=(e + 127).to(torch.uint8).view(torch.float8_e8m0fnu), rstd=rstd)
    if s["keep_y"]:
        out["y"] = y
    if s["residual"] is not None:
        out["sum"] = x
    return out


def _plain_norm_bwd(s):
    dy, rstd = s["dy"].float(), s["rstd"][:, None]
    xhat = s["x"].float() * rstd
    g = dy * s["weight"].float()
    dx = rstd * (g - xhat * (g * xhat).mean(1, keepdim=True))
    if s["dsum"] is not None:
        dx = dx + s["dsum"].float()
    return dict(dx=dx.to(torch.bfloat16), dw=(dy * xhat).sum(0))


def _plain_scores(z, score):
    """Per expert: the score that weighs it and its share of the row."""
    if score == "softmax":
        p = torch.exp(z - z.amax(1, keepdim=True))
        p = p / p.sum(1, keepdim=True)
        return p, p
    v = 1.0 / (1.0 + torch.exp(-z))
    return v, v / v.sum(1, keepdim=True)


def _plain_gate(s):
    z, k = s["logits"].float(), s["k"]
    t, e = z.shape
    valid = torch.ones(t, device=z.device) if s["mask"] is None else s["mask"].float()
    v, p = _plain_scores(z, s["score"])
    ids = _router_choice(s["logits"], s["mask"], k)
    sel = v.gather(1, ids)
    if s["renorm"]:
        sel = sel / sel.sum(1, keepdim=True)
    out = dict(ids=ids.to(torch.int32), prob=sel * s["scale"] * valid[:, None])
    if s["loss"]:
        tv = valid.sum()
        counts = torch.zeros(e, device=z.device).index_add_(
            0, ids.reshape(-1), valid.repeat_interleave(k))
        prob_sum = (p * valid[:, None]).sum(0)
        loss = s["coef"] * e / (k * tv * tv) * (counts * prob_sum).sum()
        out.update(counts=torch.cat([counts, tv[None]]).to(torch.int32), prob_sum=prob_sum,
                   loss=loss[None])
    return out


def _plain_gate_bwd(s):
    z, ids, k = s["logits"].float(), s["ids"].long(), s["k"]
    e = z.shape[1]
    counts = s["counts"].float()
    valid = torch.ones(z.shape[0], device=z.device) if s["mask"] is None else s["mask"].float()
    v, p = _plain_scores(z, s["score"])
    sel, d = v.gather(1, ids), s["d_prob"] * s["scale"]
    if s["renorm"]:
        total = sel.sum(1, keepdim=True)
        d = (d - (d * sel).sum(1, keepdim=True) / total) / total
    dv = torch.zeros_like(z).scatter_add_(1, ids, d)
    h = s["d_loss"] * s["coef"] * e / (k * counts[e] * counts[e]) * counts[:e]
    if s["score"] == "softmax":
        dv = dv + h
        dz = p * (dv - (p * dv).sum(1, keepdim=True))
    else:
        dv = dv + (h - (p * h).sum(1, keepdim=True)) / v.sum(1, keepdim=True)
        dz = v * (1.0 - v) * dv
    return (dz * valid[:, None]).to(s["logits"].dtype)


def _decode(q, sb):
    """q s_b in binary32 (exact): [..., k/2] codes, [..., k/16] scales."""
    v = torch.tensor(E2M1, device=q.device)
    v = torch.cat([v, -v])
    byte = torch.arange(256, device=q.device)
    pair = torch.stack([v[byte & 15], v[byte >> 4]], 1)
    w = pair[q.long()].view(*q.shape[:-1], -1, 16)
    return (w * sb.view(torch.float8_e4m3fn).float()[..., None]).flatten(-2)


def _plain_gemv(s):
    n, ids = s["n"], s["ids"].long()
    rows, e = ids.numel(), s["sg"].numel()
    x = s["x"].float()
    x = x[torch.arange(rows, device=x.device) // s["div"]]
    q, sb = s["q"].view(e, n, -1), s["sb"].view(e, n, -1)
    if rows <= e:  # few rows: the weights of each row's expert
        y = torch.matmul(_decode(q[ids], sb[ids]), x[:, :, None])[:, :, 0]
    else:          # many: every expert's product, then each row's own
        y = (x @ _decode(q, sb).view(e * n, -1).t()).view(rows, e, n)
        y = y[torch.arange(rows, device=x.device), ids]
    y = y * s["sg"][ids][:, None]
    if s["act"]:
        gate, up = y[:, :n // 2], y[:, n // 2:]
        y = gate / (1.0 + torch.exp(-gate)) * up * s["prob"][:, None]
        return y.to(torch.bfloat16)
    return y.to(torch.bfloat16) if s["out"] == "bf16" else y


def run(s):
    if own:
        return _run_own(s)
    return dict(norm=_plain_norm, norm_bwd=_plain_norm_bwd, gate=_plain_gate,
                gate_bwd=_plain_gate_bwd, gemv=_plain_gemv)[s["op"]](s)


# -------------------------------------------------------------------- work

def work(case):
    op = case["op"]
    if op in ("norm", "norm_bwd"):
        r, c = case["rows"], case["cols"]
        w = c * (2 if case["w"] == "bf16" else 4)
        if op == "norm":
            per = 2 + 1 + 1 / 32 + (4 if case["residual"] else 0) + (2 if case["keep_y"] else 0)
            return dict(bytes=r * c * per + w + 4 * r, flops=6 * r * c)
        per = 6 + (2 if case["residual"] else 0)
        return dict(bytes=r * c * per + w + 4 * c + 4 * r, flops=10 * r * c)
    if op in ("gate", "gate_bwd"):
        t, e, k = case["tokens"], case["experts"], case["k"]
        b = 2 if case["dtype"] == "bf16" else 4
        m = t if case["masked"] else 0
        if op == "gate":
            return dict(bytes=t * e * b + t * k * 8 + m + (8 * e if case["loss"] else 0),
                        flops=6 * t * e)
        return dict(bytes=2 * t * e * b + t * k * 8 + m + 4 * e, flops=10 * t * e)
    t, e, h, i = (case[n] for n in ("tokens", "experts", "hidden", "inter"))
    k = min(case["k"], e)
    rows = t * k
    n, kk = (2 * i, h) if case["act"] else (h, i)
    met = e * (1.0 - (1.0 - k / e) ** t)  # experts that any token chose, on average
    x = (t if case["act"] else rows) * kk * 2
    out = rows * (i * 2 if case["act"] else h * (2 if case["out"] == "bf16" else 4))
    return dict(bytes=met * n * kk * (1 / 2 + 1 / 16) + x + out + 8 * rows,
                flops=2.0 * rows * n * kk)


# ------------------------------------------------ the definitions, 64 bits

def _bf16_of(v):
    """Nearest bf16 of binary64 values, ties to even (normal range)."""
    u = v.contiguous().view(torch.int64)
    u = u + (2 ** 44 - 1) + ((u >> 45) & 1)
    return (u & ~(2 ** 45 - 1)).view(torch.float64)


def _pow2(e):
    """2^e of whole numbers, by its bits."""
    return ((e.to(torch.int64) + 1023) << 52).view(torch.float64)


def _exponent(v):
    """floor(log2 v) of positive binary64 values, by their bits."""
    return (v.contiguous().view(torch.int64) >> 52) - 1023


def _exact_norm(s):
    x = s["x"].double()
    out = {}
    if s["residual"] is not None:
        x = _bf16_of(x + s["residual"].double())
        out["sum"] = x
    rstd = (x.square().sum(1) / x.shape[1] + s["eps"]).pow(-0.5)
    y = _bf16_of(x * s["weight"].double() * rstd[:, None])
    out["rstd"] = rstd
    if s["keep_y"]:
        out["y"] = y
    blocks = y.unflatten(1, (-1, 32))
    top = blocks.abs().amax(2)
    # the smallest e with top <= 448 2^e: 448 = 1.75 2^8
    e = (_exponent(top.clamp(min=2.0 ** -140)) - 8).clamp(min=-127)
    e = torch.where(448.0 * _pow2(e) < top, e + 1, e)
    v = blocks * _pow2(-e)[..., None]
    step = _pow2(_exponent(v.abs().clamp(min=2.0 ** -6)) - 3)
    out["q"] = (torch.round(v / step) * step).flatten(1)
    out["scale"] = _pow2(e)
    return out


def _exact_norm_bwd(s):
    dy, x, w, r = (s[n].double() for n in ("dy", "x", "weight", "rstd"))
    c = x.shape[1]
    dot = torch.einsum("tc,tc,c->t", dy, x, w)
    dx = r[:, None] * dy * w - (r ** 3 * dot / c)[:, None] * x
    if s["dsum"] is not None:
        dx = dx + s["dsum"].double()
    return dict(dx=dx, dw=torch.einsum("tc,tc,t->c", dy, x, r))


def _exact_gate(s, z=None):
    z = s["logits"].double() if z is None else z
    t, e = z.shape
    k = s["k"]
    live = torch.ones(t, dtype=torch.float64, device=z.device)
    if s["mask"] is not None:
        live = (s["mask"] != 0).double()
    # an expert's place in its row: how many are larger, or equal and before it
    keys = s["logits"].double()
    place = torch.empty(t, e, dtype=torch.int64, device=z.device)
    for a in range(0, t, 256):
        u = keys[a:a + 256]
        before = torch.ones(e, e, dtype=torch.bool, device=z.device).tril(-1)
        more = (u[:, None, :] > u[:, :, None]) | ((u[:, None, :] == u[:, :, None]) & before)
        place[a:a + 256] = more.sum(2)
    ids = torch.argsort(place, dim=1)[:, :k]
    turn = torch.arange(t * k, device=z.device).view(t, k) % e
    ids = torch.where(live[:, None] > 0, ids, turn)
    if s["score"] == "softmax":
        v = share = torch.softmax(z, 1)
    else:
        v = torch.sigmoid(z)
        share = v / v.sum(1, keepdim=True)
    prob = torch.gather(v, 1, ids)
    if s["renorm"]:
        prob = prob / prob.sum(1, keepdim=True)
    prob = s["scale"] * prob * live[:, None]
    hits = torch.zeros(t, e, dtype=torch.float64, device=z.device).scatter_(1, ids, 1.0)
    counts = (hits * live[:, None]).sum(0)
    prob_sum = (share * live[:, None]).sum(0)
    tv = live.sum()
    loss = s["coef"] * e * ((counts / (k * tv)) * (prob_sum / tv)).sum()
    out = dict(ids=ids.to(torch.int32), prob=prob)
    if s["loss"]:
        out.update(counts=torch.cat([counts, tv[None]]).to(torch.int32), prob_sum=prob_sum,
                   loss=loss[None])
    return out


def _exact_gate_bwd(s):
    # through autograd in binary64: the counts are held fixed
    z = s["logits"].double().requires_grad_(True)
    e, k = z.shape[1], s["k"]
    counts = s["counts"].double()
    live = torch.ones(z.shape[0], dtype=torch.float64, device=z.device)
    if s["mask"] is not None:
        live = (s["mask"] != 0).double()
    if s["score"] == "softmax":
        v = share = torch.softmax(z, 1)
    else:
        v = torch.sigmoid(z)
        share = v / v.sum(1, keepdim=True)
    prob = torch.gather(v, 1, s["ids"].long())
    if s["renorm"]:
        prob = prob / prob.sum(1, keepdim=True)
    prob = s["scale"] * prob * live[:, None]
    mean = (share * live[:, None]).sum(0) / counts[e]
    loss = s["coef"] * e * (counts[:e] / (k * counts[e]) * mean).sum()
    total = (prob * s["d_prob"].double()).sum() + loss * s["d_loss"].double().sum()
    return torch.autograd.grad(total, z)[0]


def _exact_gemv(s):
    n, ids = s["n"], s["ids"].tolist()
    e = s["sg"].numel()
    q, sb = s["q"].view(e, n, -1), s["sb"].view(e, n, -1)
    y = torch.zeros(len(ids), n, dtype=torch.float64, device=q.device)
    for g in sorted(set(ids)):
        low, high = (q[g] & 15).int(), (q[g] >> 4).int()
        code = torch.stack([low, high], 2).flatten(1)
        mag = code & 7
        # E2M1: 0, 1/2, then (1 + bit / 2) 2^(exponent - 1)
        val = torch.where(mag < 2, mag * 0.5,
                          (1.0 + (mag & 1) * 0.5) * torch.exp2((mag >> 1).double() - 1.0))
        val = torch.where(code >= 8, -val, val)
        w = val.unflatten(1, (-1, 16)) * sb[g].view(torch.float8_e4m3fn).double()[..., None]
        mine = [r for r, i in enumerate(ids) if i == g]
        x = s["x"][[r // s["div"] for r in mine]].double()
        y[mine] = (x @ w.flatten(1).t()) * s["sg"][g].double()
    if s["act"]:
        gate, up = y[:, :n // 2], y[:, n // 2:]
        return gate * torch.sigmoid(gate) * up * s["prob"].double()[:, None]
    return y


def exact(case, seed):
    s = prepare(case, seed)
    return dict(norm=_exact_norm, norm_bwd=_exact_norm_bwd, gate=_exact_gate,
                gate_bwd=_exact_gate_bwd, gemv=_exact_gemv)[case["op"]](s)
