"""Measured cases of the operators between an expert layer and its policy
loss: dense products with their epilogues, an expert layer for a few tokens,
and the log probabilities of given tokens.

Three operators and two backward passes, each as the library's entry points
(`own` true) and as a plain form in elementary torch operations:

* linear      y = act(x W^T + bias) + residual
* linear_bwd  its gradients: of x (joined with another gradient of x), of W
              and of the bias
* decode      a whole expert layer with NVFP4 weights for a few tokens:
              residual, norm, router, gate, experts, sum
* logprob     log probabilities of given tokens, entropy, top alternatives
* logprob_bwd the gradient of the log probabilities and of the entropy

`exact` computes the same from the definitions in binary64.
"""
import math

import torch

own = False

DEV = "cuda"
NONE, SILU, GELU = "none", "silu", "gelu"


# ------------------------------------------------------------------- cases

def listed():
    return [
        # decode: the output head for eight sequences, logits in binary32
        dict(name="linear_head_8tok", op="linear", m=8, n=32768, k=2048, act=NONE, bias=False,
             residual=False, out="f32", keep_z=False),
        # training: the router's logits of a micro-batch
        dict(name="linear_router_16384", op="linear", m=16384, n=128, k=2048, act=NONE, bias=True,
             residual=False, out="f32", keep_z=False),
        # training: a dense layer of a ragged batch, everything in its epilogue
        dict(name="linear_dense_8190", op="linear", m=8190, n=4096, k=2048, act=GELU, bias=True,
             residual=True, out="bf16", keep_z=True),
        # the router's gradients; dx joins the gradient through the experts
        dict(name="linear_bwd_router_16384", op="linear_bwd", m=16384, n=128, k=2048, act=NONE,
             bias=True, add=True),
        # the dense layer's gradients
        dict(name="linear_bwd_dense_8190", op="linear_bwd", m=8190, n=4096, k=2048, act=SILU,
             bias=True, add=False),
        # one decode step of one sequence: latency
        dict(name="decode_1tok", op="decode", tokens=1, experts=128, k=8, hidden=2048, inter=768,
             score="softmax", renorm=True, shared=False),
        # a small batch, a third of the experts met
        dict(name="decode_7tok", op="decode", tokens=7, experts=128, k=8, hidden=2048, inter=768,
             score="softmax", renorm=True, shared=False),
        # a batch that meets every expert several times, with a shared expert
        dict(name="decode_37tok", op="decode", tokens=37, experts=64, k=8, hidden=5120, inter=1280,
             score="sigmoid", renorm=True, shared=True),
        # decode: the sampled token's log probability and the 20 best, one row
        dict(name="logprob_1x151936", op="logprob", tokens=1, vocab=151936, dtype="f32", top=20,
             temperature=0.7, ignored=False),
        # the policy's log probabilities and entropies over packed rollouts
        dict(name="logprob_4093x32768", op="logprob", tokens=4093, vocab=32768, dtype="bf16",
             top=0, temperature=1.0, ignored=True),
        # their gradient, over a larger vocabulary
        dict(name="logprob_bwd_2048x151936", op="logprob_bwd", tokens=2048, vocab=151936,
             dtype="bf16", temperature=1.0, ignored=True, entropy=True),
        # an odd vocabulary, logits in binary32
        dict(name="logprob_bwd_509x50257", op="logprob_bwd", tokens=509, vocab=50257, dtype="f32",
             temperature=0.8, ignored=False, entropy=False),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["linear", "linear_bwd", "decode", "logprob", "logprob_bwd"])
    if op == "linear":
        k = 8 * _log_int(rng, 8, 640)
        n = _log_int(rng, 8, 32768)
        m = _log_int(rng, 1, 16384)
        n = max(1, min(n, 2048 * 32768 // k))
        m = max(1, min(m, 8190 * 4096 * 2048 // (n * k), 8190 * 4096 // n))
        out = rng.choice(["bf16", "f32"])
        return dict(op=op, m=m, n=n, k=k, act=rng.choice([NONE, SILU, GELU]),
                    bias=rng.random() < 0.5, residual=rng.random() < 0.5, out=out,
                    keep_z=rng.random() < 0.3)
    if op == "linear_bwd":
        k = 8 * _log_int(rng, 8, 640)
        n = 8 * _log_int(rng, 1, 1024)
        m = _log_int(rng, 1, 16384)
        m = max(1, min(m, 8190 * 4096 * 2048 // (n * k), 8190 * 4096 // n))
        return dict(op=op, m=m, n=n, k=k, act=rng.choice([NONE, SILU, GELU]),
                    bias=rng.random() < 0.5, add=rng.random() < 0.5)
    if op == "decode":
        experts = rng.randint(8, 64)
        return dict(op=op, tokens=_log_int(rng, 1, 37), experts=experts, k=rng.randint(1, 8),
                    hidden=32 * rng.randint(16, 160), inter=32 * rng.randint(4, 40),
                    score=rng.choice(["softmax", "sigmoid"]), renorm=rng.random() < 0.7,
                    shared=rng.random() < 0.4)
    vocab = _log_int(rng, 1000, 160000)
    c = dict(op=op, vocab=vocab, dtype=rng.choice(["bf16", "f32"]),
             temperature=rng.choice([1.0, 0.6, 0.85, 1.3]), ignored=rng.random() < 0.4)
    size = 2048 * 151936 if c["dtype"] == "bf16" else 1024 * 151936
    if op == "logprob":
        c["top"] = rng.choice([0, 0, 1, 5, 20, 32])
        # alternatives are asked for while decoding
        most = 64 if c["top"] else min(4096, 4093 * 32768 // vocab)
        c["tokens"] = _log_int(rng, 1, most)
    else:
        c["tokens"] = _log_int(rng, 1, min(4096, size // vocab))
        c["entropy"] = rng.random() < 0.5
    return c


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


def _bf16(t):
    return t.to(torch.bfloat16)


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


def _prepare_linear(s, g):
    m, n, k = s["m"], s["n"], s["k"]
    x = _randn(g, m, k)
    x *= torch.exp(0.5 * _randn(g, m, 1))
    s["x"] = _bf16(x)
    s["w"] = _bf16(_randn(g, n, k) / math.sqrt(k))
    if s["op"] == "linear":
        s["b"] = 0.3 * _randn(g, n) if s["bias"] else None
        s["r"] = _bf16(_randn(g, m, n)) if s["residual"] else None
        return
    s["dy"] = _bf16(_randn(g, m, n) * 0.1)
    s["z"] = None if s["act"] == NONE else _bf16(1.5 * _randn(g, m, n))
    s["add"] = _bf16(_randn(g, m, k) * 0.1) if s["add"] else None


def _prepare_decode(s, g):
    t, e, h, i = s["tokens"], s["experts"], s["hidden"], s["inter"]
    s["k"] = min(s["k"], e)
    s["x"] = _bf16(_activations(g, t, h))
    s["residual"] = _bf16(_randn(g, t, h))
    s["norm_w"] = _bf16(1.0 + 0.2 * _randn(g, h))
    s["gate_w"] = _bf16(_randn(g, e, h) * (1.5 / math.sqrt(h)))
    groups = e + 1 if s["shared"] else e
    s["w1"] = _nvfp4_weights(g, groups, 2 * i, h)
    s["w2"] = _nvfp4_weights(g, groups, h, i)
    s["scale"] = 2.5 if s["score"] == "sigmoid" else 1.0
    s["eps"] = 1e-6


def _prepare_logprob(s, g):
    t, v = s["tokens"], s["vocab"]
    x = torch.empty(t, v, device=DEV)
    for a in range(0, t, 256):  # by rows: the largest cases are large
        x[a:a + 256] = 2.0 * _randn(g, min(256, t - a), v) - 4.0
    # a few candidates stand out, as a trained model's do
    few = torch.randint(0, v, (t, 16), generator=g, device=DEV)
    x.scatter_(1, few, 9.0 + 3.0 * _randn(g, t, 16))
    x[:, v - v // 300:] = -math.inf  # columns that only pad the vocabulary
    ids = few[:, 0].clone()
    other = torch.rand(t, generator=g, device=DEV) < 0.2
    ids = torch.where(other, torch.randint(0, v - v // 300, (t,), generator=g, device=DEV), ids)
    if s["ignored"]:  # prompts and padding between the answers
        ids[torch.rand(t, generator=g, device=DEV) < 0.2] = -1
    s["logits"] = _bf16(x) if s["dtype"] == "bf16" else x
    s["ids"] = ids.to(torch.int32)
    if s["op"] == "logprob":
        return
    s["d_logprob"] = 0.01 * _randn(g, t)
    s["d_entropy"] = -0.001 * torch.rand(t, generator=g, device=DEV) if s["entropy"] else None
    # what the forward pass kept: each row's largest logit and the logarithm of
    # its sum, and the entropy
    stats = torch.zeros(t, 2, device=DEV)
    ent = torch.zeros(t, device=DEV)
    for a in range(0, t, 256):
        z = s["logits"][a:a + 256].double()
        m = z.amax(1, keepdim=True)
        u = (z - m) / s["temperature"]
        p = torch.exp(u)
        total = p.sum(1, keepdim=True)
        stats[a:a + 256, 0] = m[:, 0]
        stats[a:a + 256, 1] = torch.log(total)[:, 0]
        u = torch.where(p > 0, u, torch.zeros_like(u))
        ent[a:a + 256] = torch.log(total)[:, 0] - (p * u).sum(1) / total[:, 0]
    live = s["ids"] >= 0
    s["stats"] = torch.where(live[:, None], stats, torch.zeros_like(stats))
    s["entropy_value"] = torch.where(live, ent, torch.zeros_like(ent))


def prepare(case, seed):
    g = _gen(seed)
    s = dict(case)
    if case["op"] in ("linear", "linear_bwd"):
        _prepare_linear(s, g)
    elif case["op"] == "decode":
        _prepare_decode(s, g)
    else:
        _prepare_logprob(s, g)
    return s


# ------------------------------------------------------- the library's calls

def _run_own(s):
    import precision_quantization_moe_amd as pqm
    op = s["op"]
    if op in ("linear", "linear_bwd"):
        act = {NONE: pqm.ACT_NONE, SILU: pqm.ACT_SILU, GELU: pqm.ACT_GELU}[s["act"]]
        if op == "linear":
            y, z = pqm.linear(s["x"], s["w"], s["b"], act, s["r"], keep_z=s["keep_z"],
                              out_dtype=pqm.OUT_BF16 if s["out"] == "bf16" else pqm.OUT_FP32)
            return dict(y=y, z=z) if s["keep_z"] else dict(y=y)
        dx, dw, db, dz = pqm.linear_backward(s["dy"], s["x"], s["w"], act, s["z"], d_x=s["add"],
                                             need_dbias=s["bias"])
        out = dict(dx=dx, dw=dw)
        if s["bias"]:
            out["db"] = db
        if act != pqm.ACT_NONE:
            out["dz"] = dz
        return out
    if op == "decode":
        out, h, y, ids, prob, d = pqm.moe_decode_nvfp4(
            s["x"], s["residual"], s["norm_w"], s["gate_w"], *s["w1"], *s["w2"], s["k"],
            s["inter"], shared=s["shared"],
            score=pqm.SCORE_SOFTMAX if s["score"] == "softmax" else pqm.SCORE_SIGMOID,
            renormalize=s["renorm"], scale=s["scale"], eps=s["eps"])
        return dict(out=out, h=h, y=y, ids=ids, prob=prob, d=d)
    if op == "logprob":
        lp, ent, stats, top_ids, top_lp = pqm.token_logprobs(
            s["logits"], s["ids"], temperature=s["temperature"], top_n=s["top"])
        out = dict(logprob=lp, entropy=ent, stats=stats)
        if s["top"]:
            out.update(top_ids=top_ids, top_logprob=top_lp)
        return out
    return pqm.token_logprobs_backward(
        s["logits"], s["ids"], s["stats"], s["d_logprob"], temperature=s["temperature"],
        entropy=s["entropy_value"] if s["entropy"] else None, d_entropy=s["d_entropy"])


# ------------------------------------------------------------- plain forms

def _squash(z, act):
    """The sigmoid's argument: act(z) = z sigmoid(squash)."""
    if act == SILU:
        return z
    return 2.0 * math.sqrt(2.0 / math.pi) * (z + 0.044715 * z * z * z)


def _plain_linear(s):
    z = s["x"].float() @ s["w"].float().t()
    if s["b"] is not None:
        z = z + s["b"]
    out = dict(z=_bf16(z)) if s["keep_z"] else {}
    if s["act"] != NONE:
        z = z / (1.0 + torch.exp(-_squash(z, s["act"])))
    if s["r"] is not None:
        z = z + s["r"].float()
    out["y"] = _bf16(z) if s["out"] == "bf16" else z
    return out


def _plain_linear_bwd(s):
    d = s["dy"].float()
    out = {}
    if s["act"] != NONE:
        z = s["z"].float()
        slope = 1.0 if s["act"] == SILU else \
            2.0 * math.sqrt(2.0 / math.pi) * (1.0 + 3.0 * 0.044715 * z * z)
        v = 1.0 / (1.0 + torch.exp(-_squash(z, s["act"])))
        out["dz"] = _bf16(d * (v + z * v * (1.0 - v) * slope))
        d = out["dz"].float()
    dx = d @ s["w"].float()
    if s["add"] is not None:
        dx = dx + s["add"].float()
    out["dx"] = _bf16(dx)
    out["dw"] = d.t() @ s["x"].float()
    if s["bias"]:
        out["db"] = d.sum(0)
    return out


E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def _decode(q, sb):
    """q s_b in binary32 (exact): [..., k/2] codes, [..., k/16] scales."""
    v = torch.tensor(E2M1, device=q.device)
    v = torch.cat([v, -v])
    byte = torch.arange(256, device=q.device)
    pair = torch.stack([v[byte & 15], v[byte >> 4]], 1)
    w = pair[q.long()].view(*q.shape[:-1], -1, 16)
    return (w * sb.view(torch.float8_e4m3fn).float()[..., None]).flatten(-2)


def _plain_products(x, ids, w, n):
    """x [rows, k] times the weights of each row's expert."""
    q, sb, sg = w
    e = sg.numel()
    q, sb = q.view(e, n, -1), sb.view(e, n, -1)
    if ids.numel() <= e:
        y = torch.matmul(_decode(q[ids], sb[ids]), x[:, :, None])[:, :, 0]
    else:
        y = (x @ _decode(q, sb).view(e * n, -1).t()).view(-1, e, n)
        y = y[torch.arange(ids.numel(), device=x.device), ids]
    return y * sg[ids][:, None]


def _nearest_bf16(v):
    """bf16 of binary64 values in one rounding (a cast goes through binary32)."""
    m, ex = torch.frexp(v)
    return _bf16(torch.ldexp(torch.round(m * 256.0), ex - 8))


def _plain_decode(s):
    t, h = s["x"].shape
    e, k, i = s["experts"], s["k"], s["inter"]
    stream = _bf16(s["x"].float() + s["residual"].float())
    # y's rounding and the order of the logits stand at borders: 64 bits
    f = stream.double()
    y = _nearest_bf16(f * s["norm_w"].double() / torch.sqrt((f * f).mean(1, keepdim=True) + s["eps"]))
    z = y.double() @ s["gate_w"].double().t()
    ids = torch.sort(z, dim=1, descending=True, stable=True).indices[:, :k]
    z = z.float()
    if s["score"] == "softmax":
        v = torch.exp(z - z.amax(1, keepdim=True))
        v = v / v.sum(1, keepdim=True)
    else:
        v = 1.0 / (1.0 + torch.exp(-z))
    prob = v.gather(1, ids)
    if s["renorm"]:
        prob = prob / prob.sum(1, keepdim=True)
    prob = prob * s["scale"]
    rows, weight = ids, prob
    if s["shared"]:
        rows = torch.cat([ids, torch.full_like(ids[:, :1], e)], 1)
        weight = torch.cat([prob, torch.ones_like(prob[:, :1])], 1)
    c = rows.shape[1]
    u = _plain_products(y.float().repeat_interleave(c, 0), rows.reshape(-1), s["w1"], 2 * i)
    gate, up = u[:, :i], u[:, i:]
    d = _bf16(gate / (1.0 + torch.exp(-gate)) * up * weight.reshape(-1, 1))
    o = _plain_products(d.float(), rows.reshape(-1), s["w2"], h)
    return dict(out=_bf16(o.view(t, c, h).sum(1)), h=stream, y=y, ids=ids.to(torch.int32),
                prob=prob, d=d)


def _plain_logprob(s):
    z = s["logits"].float()
    ids, n = s["ids"].long(), s["top"]
    live = ids >= 0
    zero = torch.zeros(z.shape[0], device=z.device)
    top = z.amax(1, keepdim=True)
    u = (z - top) / s["temperature"]
    p = torch.exp(u)
    total = p.sum(1, keepdim=True)
    log_total = torch.log(total)
    lp = u.gather(1, ids.clamp(min=0)[:, None]) - log_total
    ent = log_total[:, 0] - (p * torch.where(p > 0, u, torch.zeros_like(u))).sum(1) / total[:, 0]
    out = dict(logprob=torch.where(live, lp[:, 0], zero), entropy=torch.where(live, ent, zero),
               stats=torch.where(live[:, None], torch.cat([top, log_total], 1), zero[:, None]))
    if n:
        best = torch.sort(z, dim=1, descending=True, stable=True).indices[:, :n]
        lp = u.gather(1, best) - log_total
        out["top_ids"] = torch.where(live[:, None], best, torch.full_like(best, -1)).to(torch.int32)
        out["top_logprob"] = torch.where(live[:, None], lp, zero[:, None])
    return out


def _plain_logprob_bwd(s):
    z = s["logits"].float()
    ids = s["ids"].long()
    live = (ids >= 0)[:, None]
    lp = (z - s["stats"][:, :1]) / s["temperature"] - s["stats"][:, 1:]
    p = torch.exp(lp)
    d = -s["d_logprob"][:, None] * p
    d = d.scatter_add(1, ids.clamp(min=0)[:, None], s["d_logprob"][:, None])
    if s["entropy"]:
        lp = torch.where(p > 0, lp, torch.zeros_like(lp))
        d = d - s["d_entropy"][:, None] * p * (lp + s["entropy_value"][:, None])
    d = torch.where(live, d / s["temperature"], torch.zeros_like(d))
    return d.to(s["logits"].dtype)


def run(s):
    if own:
        return _run_own(s)
    return dict(linear=_plain_linear, linear_bwd=_plain_linear_bwd, decode=_plain_decode,
                logprob=_plain_logprob, logprob_bwd=_plain_logprob_bwd)[s["op"]](s)


# -------------------------------------------------------------------- work

def work(case):
    op = case["op"]
    if op in ("linear", "linear_bwd"):
        m, n, k = case["m"], case["n"], case["k"]
        if op == "linear":
            out = 2 if case["out"] == "bf16" else 4
            per = out + (2 if case["residual"] else 0) + (2 if case["keep_z"] else 0)
            return dict(bytes=2 * (m * k + n * k) + per * m * n + (4 * n if case["bias"] else 0),
                        flops=2.0 * m * n * k)
        per = 2 if case["act"] == NONE else 6
        return dict(bytes=2 * (m * k + n * k) + per * m * n + (4 if case["add"] else 2) * m * k +
                    4 * n * k + (4 * n if case["bias"] else 0), flops=4.0 * m * n * k)
    if op == "decode":
        t, e, h, i = (case[x] for x in ("tokens", "experts", "hidden", "inter"))
        k = min(case["k"], e)
        met = e * (1.0 - (1.0 - k / e) ** t) + (1 if case["shared"] else 0)
        rows = t * (k + (1 if case["shared"] else 0))
        return dict(bytes=met * 3 * h * i * (1 / 2 + 1 / 16) + 2 * e * h + 10 * t * h + 2 * h +
                    8 * t * k + 2 * rows * i, flops=2.0 * rows * 3 * h * i + 2.0 * t * e * h)
    t, v = case["tokens"], case["vocab"]
    b = 2 if case["dtype"] == "bf16" else 4
    if op == "logprob":
        return dict(bytes=t * v * b + 20 * t + 8 * t * case["top"], flops=6.0 * t * v)
    return dict(bytes=2 * t * v * b + 20 * t, flops=6.0 * t * v)


# ------------------------------------------------ the definitions, 64 bits

def _bf16_of(v):
    """Nearest bf16 of binary64 values, ties to even (normal range)."""
    u = v.contiguous().view(torch.int64)
    u = u + (2 ** 44 - 1) + ((u >> 45) & 1)
    return (u & ~(2 ** 45 - 1)).view(torch.float64)


def _act64(z, act):
    if act == NONE:
        return z
    if act == SILU:
        return z * torch.sigmoid(z)
    return 0.5 * z * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (z + 0.044715 * z.pow(3))))


def _exact_linear(s):
    z = torch.matmul(s["x"].double(), s["w"].double().t())
    if s["b"] is not None:
        z += s["b"].double()
    y = _act64(z, s["act"])
    if s["r"] is not None:
        y = y + s["r"].double()
    return dict(y=y, z=z) if s["keep_z"] else dict(y=y)


def _exact_linear_bwd(s):
    g = s["dy"].double()
    out = {}
    if s["act"] != NONE:
        z = s["z"].double().requires_grad_(True)
        (slope,) = torch.autograd.grad(_act64(z, s["act"]).sum(), z)
        out["dz"] = g * slope
        g = _bf16_of(out["dz"])  # the products' operand
    out["dx"] = torch.matmul(g, s["w"].double())
    if s["add"] is not None:
        out["dx"] += s["add"].double()
    out["dw"] = torch.matmul(g.t(), s["x"].double())
    if s["bias"]:
        out["db"] = g.sum(0)
    return out


def _expert64(w, e, n):
    """Expert e's weights [n, k] in binary64."""
    q, sb, sg = w
    q, sb = q.view(sg.numel(), n, -1)[e], sb.view(sg.numel(), n, -1)[e]
    code = torch.stack([(q & 15).int(), (q >> 4).int()], 2).flatten(1)
    mag = code & 7
    # E2M1: 0, 1/2, then (1 + bit / 2) 2^(exponent - 1)
    val = torch.where(mag < 2, mag * 0.5,
                      (1.0 + (mag & 1) * 0.5) * torch.exp2((mag >> 1).double() - 1.0))
    val = torch.where(code >= 8, -val, val)
    val = val.unflatten(1, (-1, 16)) * sb.view(torch.float8_e4m3fn).double()[..., None]
    return val.flatten(1) * sg[e].double()


def _exact_decode(s):
    t, e, k, i, h = s["tokens"], s["experts"], s["k"], s["inter"], s["hidden"]
    stream = _bf16_of(s["x"].double() + s["residual"].double())
    y = _bf16_of(stream * s["norm_w"].double() *
                 (stream.square().sum(1, keepdim=True) / h + s["eps"]).pow(-0.5))
    z = torch.einsum("th,eh->te", y, s["gate_w"].double())
    # an expert's place: how many logits are larger, or equal and before it
    before = torch.ones(e, e, dtype=torch.bool, device=z.device).tril(-1)
    more = (z[:, None, :] > z[:, :, None]) | ((z[:, None, :] == z[:, :, None]) & before)
    ids = torch.argsort(more.sum(2), dim=1)[:, :k]
    v = torch.softmax(z, 1) if s["score"] == "softmax" else torch.sigmoid(z)
    prob = torch.gather(v, 1, ids)
    if s["renorm"]:
        prob = prob / prob.sum(1, keepdim=True)
    prob = prob * s["scale"]
    c = k + 1 if s["shared"] else k
    d = torch.zeros(t, c, i, dtype=torch.float64, device=z.device)
    out = torch.zeros(t, h, dtype=torch.float64, device=z.device)
    chosen = ids.tolist()
    for g in range(e + 1 if s["shared"] else e):
        at = [(r, j) for r in range(t) for j in range(k) if chosen[r][j] == g]
        if g == e:
            at = [(r, k) for r in range(t)]
        if not at:
            continue
        r = torch.tensor([a[0] for a in at], device=z.device)
        j = torch.tensor([a[1] for a in at], device=z.device)
        p = prob[r, j] if g < e else torch.ones(t, dtype=torch.float64, device=z.device)
        u = y[r] @ _expert64(s["w1"], g, 2 * i).t()
        d[r, j] = u[:, :i] * torch.sigmoid(u[:, :i]) * u[:, i:] * p[:, None]
        out.index_add_(0, r, _bf16_of(d[r, j]) @ _expert64(s["w2"], g, h).t())
    return dict(out=out, h=stream, y=y, ids=ids.to(torch.int32), prob=prob,
                d=d.view(t * c, i))


def _exact_logprob(s):
    t, n = s["tokens"], s["top"]
    f64 = dict(dtype=torch.float64, device=s["logits"].device)
    out = dict(logprob=torch.zeros(t, **f64), entropy=torch.zeros(t, **f64),
               stats=torch.zeros(t, 2, **f64))
    if n:
        out["top_ids"] = torch.full((t, n), -1, dtype=torch.int32, device=f64["device"])
        out["top_logprob"] = torch.zeros(t, n, **f64)
    for r in range(t):
        i = int(s["ids"][r])
        if i < 0:
            continue
        z = s["logits"][r].double()
        full = torch.log_softmax(z / s["temperature"], 0)
        out["logprob"][r] = full[i]
        out["entropy"][r] = torch.special.entr(torch.exp(full)).sum()
        out["stats"][r, 0] = z.max()
        out["stats"][r, 1] = torch.logsumexp((z - z.max()) / s["temperature"], 0)
        if n:
            # whole numbers in the order of the logits, the lower index above
            bits = s["logits"][r].float().view(torch.int32).long()
            order = torch.where(bits < 0, -(bits & 0x7FFFFFFF), bits)
            key = order * 2 ** 20 + (2 ** 20 - 1 - torch.arange(z.numel(), device=z.device))
            best = torch.topk(key, n).indices
            out["top_ids"][r] = best.to(torch.int32)
            out["top_logprob"][r] = full[best]
    return out


def _exact_logprob_bwd(s):
    t = s["tokens"]
    out = torch.zeros(t, s["vocab"], dtype=torch.float64, device=s["logits"].device)
    for r in range(t):
        i = int(s["ids"][r])
        if i < 0:
            continue
        z = s["logits"][r].double()
        p = torch.softmax(z / s["temperature"], 0)
        g = -s["d_logprob"][r].double() * p
        g[i] += s["d_logprob"][r].double()
        if s["entropy"]:
            # dH / du = -p (log p + H)
            h = torch.special.entr(p).sum()
            g += s["d_entropy"][r].double() * (torch.special.entr(p) - p * h)
        out[r] = g / s["temperature"]
    return out


def exact(case, seed):
    s = prepare(case, seed)
    return dict(linear=_exact_linear, linear_bwd=_exact_linear_bwd, decode=_exact_decode,
                logprob=_exact_logprob, logprob_bwd=_exact_logprob_bwd)[case["op"]](s)
