"""MoE expert-layer forward passes composed from the library's entry points.

Each function only sequences calls into libpqmoe (routing, quantization,
gather, grouped GEMM, weighted SwiGLU, combine) on torch's current stream;
all arithmetic happens in the HIP kernels.  The structure follows the
pages: the routed experts run through one grouped GEMM per projection over a
contiguous, offset-delimited buffer ("miniTE technical report", 5.2); the
weighted SwiGLU feeds the FC2 quantizer (5.3/5.4); routed outputs are
reduced in high precision ("Towards Blackwell-Native 8-bit and 4-bit RL",
fine-grained precision control).  Weights are quantized once per update and
passed in quantized form.
"""
from __future__ import annotations

import torch

from . import _binding as b


def quantize_expert_weights_mxfp8(w1: torch.Tensor, w2: torch.Tensor):
    """w1 [E*2I, H] (gate rows then up rows per expert), w2 [E*H, I] bf16 ->
    row-wise MXFP8 (q, s) of each (blocks along the GEMM reduction axis)."""
    w1q, w1s, _, _ = b.quantize_mxfp8(w1, colwise=False)
    w2q, w2s, _, _ = b.quantize_mxfp8(w2, colwise=False)
    return w1q, w1s, w2q, w2s


def column_copies_mxfp8(w1: torch.Tensor, w2: torch.Tensor):
    """Column-wise MXFP8 copies (32 x 1 blocks, stored transposed) of the
    stacked expert weights, the data-gradient operands of the low-precision
    backward: w1 [E*2I, H] -> ([H, E*2I], [H, E*2I/32]); w2 [E*H, I] ->
    ([I, E*H], [I, E*H/32])."""
    _, _, w1T, w1sT = b.quantize_mxfp8(w1, rowwise=False)
    _, _, w2T, w2sT = b.quantize_mxfp8(w2, rowwise=False)
    return w1T, w1sT, w2T, w2sT


def saved_activation_mxfp8(rows: torch.Tensor, off: torch.Tensor):
    """The forward-side column-wise MXFP8 copy of an expert-sorted
    activation (FC1 input X or FC2 input D) for the weight gradient: each
    expert's rows padded to whole 32-row blocks, then quantized down the
    columns.  Returns (qT [C, Mp], sT [C, Mp/32], padded offsets)."""
    xp, poff = b.moe_pad_rows(rows, off)
    _, _, qT, sT = b.quantize_mxfp8(xp, rowwise=False)
    return qT, sT, poff


def mxfp8_expert_backward(dy, dc, saved_x, saved_d, w_col, off, inter: int):
    """MXFP8 low-precision backward of the two expert GEMMs ([BW] MXFP8
    training: the data- and weight-gradient GEMMs run in MXFP8 on the
    column-wise copies).
      dy [M, H] bf16   gradient of the down-projection output rows
      dc [M, 2I] bf16  gradient of the gate_up output rows
      saved_x, saved_d (qT, sT, padded offsets) from saved_activation_mxfp8
      w_col            column_copies_mxfp8(W1, W2)
    Both gradients are padded per expert (pqm_moe_pad_rows) and quantized
    once into their row-wise (data gradient) and column-wise (weight
    gradient) copies.  Returns dict(dd [Mp, I] bf16, dx [Mp, H] bf16,
    dw2 [E, H, I] fp32, dw1 [E, 2I, H] fp32, poff): dd and dx are in the
    padded row order (row poff[e] + j of expert e is routed row off[e] + j)."""
    H = dy.shape[1]
    w1T, w1sT, w2T, w2sT = w_col
    xT, xsT, _ = saved_x
    dT, dsT, _ = saved_d
    dyp, poff = b.moe_pad_rows(dy, off)
    dcp, _ = b.moe_pad_rows(dc, off)
    qy, sy, qyT, syT = b.quantize_mxfp8(dyp)
    qc, sc, qcT, scT = b.quantize_mxfp8(dcp)
    dd = b.moe_grouped_gemm(b.FMT_MXFP8, b.GEMM_DGRAD, qy, w2T, poff, inter, H,
                            a_scale=sy, b_scale=w2sT, out_dtype=b.OUT_BF16)
    dw2 = b.moe_grouped_gemm(b.FMT_MXFP8, b.GEMM_WGRAD, qyT, dT, poff, H, inter,
                             a_scale=syT, b_scale=dsT, out_dtype=b.OUT_FP32)
    dx = b.moe_grouped_gemm(b.FMT_MXFP8, b.GEMM_DGRAD, qc, w1T, poff, H, 2 * inter,
                            a_scale=sc, b_scale=w1sT, out_dtype=b.OUT_BF16)
    dw1 = b.moe_grouped_gemm(b.FMT_MXFP8, b.GEMM_WGRAD, qcT, xT, poff, 2 * inter, H,
                             a_scale=scT, b_scale=xsT, out_dtype=b.OUT_FP32)
    return dict(dd=dd, dx=dx, dw2=dw2, dw1=dw1, poff=poff)


def quantize_expert_weights_nvfp4(w1: torch.Tensor, w2: torch.Tensor, inter: int, hidden: int):
    """NVFP4 weights with one FP32 outer scale per expert tensor; gate and up
    of an expert share one scale (joint)."""
    w1q, w1b, w1g = b.quantize_nvfp4_per_token(w1, rows_per_scale=2 * inter)
    w2q, w2b, w2g = b.quantize_nvfp4_per_token(w2, rows_per_scale=hidden)
    return w1q, w1b, w1g, w2q, w2b, w2g


def mxfp8_moe_forward(x, topk_ids, prob_flat, w1q, w1s, w2q, w2s, num_experts: int,
                      inter: int, keep_intermediates: bool = True):
    """x [T, H] bf16; topk_ids [T, k] int32; prob_flat [T*k] float32.
    Returns a dict of every stage's output (out = [T, H] bf16).  With
    keep_intermediates the gate_up output c and d = SwiGLU(c) x prob are
    materialised (bf16; d and its MXFP8 encoding in one fused pass);
    without, the gate_up GEMM's epilogue produces the MXFP8 encoding of d
    directly and c, d are None (same bytes)."""
    qx, sx, _, _ = b.quantize_mxfp8(x, colwise=False)
    return _mxfp8_experts(qx, sx, topk_ids, prob_flat, w1q, w1s, w2q, w2s, num_experts, inter,
                          keep_intermediates)


def _mxfp8_experts(qx, sx, topk_ids, prob_flat, w1q, w1s, w2q, w2s, num_experts: int, inter: int,
                   keep_intermediates: bool):
    """The routed experts on tokens already in row-wise MXFP8 (qx, sx)."""
    H = qx.shape[1]
    off, src, tok, slot = b.moe_route(topk_ids, num_experts)
    qa = b.moe_gather_rows(qx, tok)
    sa = b.moe_gather_rows(sx, tok)
    if keep_intermediates or inter % 128 or H % 128 or H > 2048:
        c = b.moe_grouped_gemm(b.FMT_MXFP8, b.GEMM_FPROP, qa, w1q, off, 2 * inter, H,
                               a_scale=sa, b_scale=w1s, out_dtype=b.OUT_BF16)
        qd, sd, d = b.swiglu_prob_quantize_mxfp8(c, prob_flat, src, keep_d=keep_intermediates)
    else:
        c = d = None
        qd, sd = b.moe_gemm_swiglu_quantize_mxfp8(qa, sa, w1q, w1s, off, inter, prob_flat, src)
    y = b.moe_grouped_gemm(b.FMT_MXFP8, b.GEMM_FPROP, qd, w2q, off, H, inter,
                           a_scale=sd, b_scale=w2s, out_dtype=b.OUT_BF16)
    out = b.moe_combine(y, slot)
    return dict(off=off, src=src, tok=tok, slot=slot, qa=qa, sa=sa, c=c, d=d, qd=qd, sd=sd,
                y=y, out=out)


def nvfp4_moe_forward(x, topk_ids, prob_all, w1q, w1b, w1g, w2q, w2b, w2g, num_experts: int,
                      inter: int, keep_intermediates: bool = True):
    """Routed experts plus one shared expert (group num_experts, every token)
    with per-token NVFP4 activations.  prob_all [T*k + T] float32: router
    probabilities, then 1.0 for each token's shared-expert row.  The weighted
    SwiGLU and the per-token NVFP4 quantization of its output D run as one
    fused pass; D is materialised (bf16) only with keep_intermediates (same
    bytes either way)."""
    T, H = x.shape
    k = topk_ids.shape[1]
    off, src, tok, slot = b.moe_route(topk_ids, num_experts, shared_expert=True)
    qx, sbx, sgx = b.quantize_nvfp4_per_token(x)
    qa = b.moe_gather_rows(qx, tok)
    sba = b.moe_gather_rows(sbx, tok)
    sga = b.moe_gather_rows(sgx.view(T, 1), tok).view(-1)
    c = b.moe_grouped_gemm(b.FMT_NVFP4, b.GEMM_FPROP, qa, w1q, off, 2 * inter, H,
                           a_scale=sba, a_outer=sga, b_scale=w1b, b_outer=w1g,
                           b_rows_per_scale=2 * inter, out_dtype=b.OUT_BF16)
    qd, sbd, sgd, d = b.swiglu_prob_quantize_nvfp4(c, prob_all, src, keep_d=keep_intermediates)
    y = b.moe_grouped_gemm(b.FMT_NVFP4, b.GEMM_FPROP, qd, w2q, off, H, inter,
                           a_scale=sbd, a_outer=sgd, b_scale=w2b, b_outer=w2g,
                           b_rows_per_scale=H, out_dtype=b.OUT_BF16)
    out = b.moe_combine(y[:T * k], slot, shared=y[T * k:])
    return dict(off=off, src=src, tok=tok, slot=slot, qa=qa, sba=sba, sga=sga, c=c, d=d,
                qd=qd, sbd=sbd, sgd=sgd, y=y, out=out)


def block_plan(tokens: int, k: int, device):
    """The index tensors that the block passes below need for `tokens` tokens,
    made once: off [2] the one group of all tokens, slot [tokens, k] each
    assignment's own row, row [tokens, 1] each token's own row."""
    i32 = dict(dtype=torch.int32, device=device)
    return dict(off=torch.tensor([0, tokens], dtype=torch.int64, device=device),
                slot=torch.arange(tokens * k, **i32).view(tokens, k),
                row=torch.arange(tokens, **i32).view(tokens, 1))


def _plan(plan, tokens: int, k: int, device):
    """plan, or a new one without it.  A plan for other sizes would send the
    products past their rows or leave some unwritten, so its shapes are
    compared on the host (what it holds is on the device and not read)."""
    if not plan:
        return block_plan(tokens, k, device)
    i32 = torch.int32
    for name, shape, dtype in (("off", (2,), torch.int64), ("slot", (tokens, k), i32),
                               ("row", (tokens, 1), i32)):
        t = plan.get(name)
        if (t is None or t.shape != shape or t.dtype is not dtype or t.device != device
                or not t.is_contiguous()):
            raise ValueError(f"plan: {name} is not of block_plan({tokens}, {k}, {device})")
    return plan


def _router(gate_w, hidden: int, device) -> int:
    """The experts, E, of the router's weight gate_w [E, hidden] bf16."""
    E = gate_w.shape[0]
    b._want(gate_w, "gate_w", torch.bfloat16, (E, hidden), device)
    return E


def _of_experts(E: int, name: str, w, size: int):
    """Refuses weights that are not of E experts with `size` bytes each: the
    products would read past the end of fewer and leave more out."""
    if w.numel() != E * size:
        raise ValueError(f"{name}: expected {size} bytes for each of the router's {E} experts, got "
                         f"{w.numel()} (no shared expert here)")


def _router_logits(y, gate_w, off):
    """y [T, H] times the router's weight [E, H], both bf16, in binary32."""
    E, H = gate_w.shape
    return b.moe_grouped_gemm(b.FMT_BF16, b.GEMM_FPROP, y, gate_w, off, E, H,
                              out_dtype=b.OUT_FP32)


def nvfp4_moe_decode(x, residual, norm_w, gate_w, w1q, w1b, w1g, w2q, w2b, w2g, k: int,
                     inter: int, plan=None, score: int = b.SCORE_SOFTMAX,
                     renormalize: bool = True, scale: float = 1.0, eps: float = 1e-6):
    """One decode step of an expert layer with NVFP4 weights for a few tokens
    (T * k <= 4096; up to about 16 assignments an expert, beyond which the
    grouped GEMM of nvfp4_moe_forward is faster): residual addition and RMS
    norm, router gate, gate_up with SwiGLU, down projection, combine.
    Activations stay in bf16, and nothing is sorted or gathered.  x, residual
    [T, H] bf16 (residual may be None);
    gate_w [E, H] bf16, E % 8 == 0; the weights of those E experts as
    quantize_expert_weights_nvfp4 returns them (routed experts alone: weights
    with a shared expert's group, as nvfp4_moe_forward takes them, are refused);
    plan from block_plan(T, k, device).  Returns dict(out [T, H] bf16, h (the new
    residual stream), y, ids, prob, d)."""
    T, H = x.shape
    plan = _plan(plan, T, k, x.device)
    E = _router(gate_w, H, x.device)
    _of_experts(E, "w1q", w1q, inter * H)  # the few-row products check the rest
    _of_experts(E, "w2q", w2q, H * inter // 2)
    _, _, y, h, _ = b.rmsnorm_quantize_mxfp8(x, norm_w, eps, residual=residual, quantize=False)
    logits = _router_logits(y, gate_w, plan["off"])
    ids, prob, _, _, _ = b.moe_gate(logits, k, score, renormalize, scale)
    d = b.moe_gemv_swiglu_nvfp4(y, ids, prob, w1q, w1b, w1g, inter, divisor=k)
    rows = b.moe_gemv_nvfp4(d, ids, w2q, w2b, w2g, H)
    out = b.moe_combine(rows, plan["slot"])
    return dict(out=out, h=h, y=y, ids=ids, prob=prob, d=d)


def mxfp8_moe_block_forward(x, residual, norm_w, gate_w, w1q, w1s, w2q, w2s, k: int, inter: int,
                            loss_coef: float = 0.01, mask=None, plan=None,
                            score: int = b.SCORE_SOFTMAX, renormalize: bool = True,
                            scale: float = 1.0, eps: float = 1e-6):
    """An expert layer's training forward pass from the residual stream on:
    residual addition, RMS norm and MXFP8 encoding in one pass, router gate
    with its balance loss, then the experts of mxfp8_moe_forward.  mask [T]
    marks padding with 0: no part in the loss, no weight, no gradient to the
    gate; its x must be finite, since its rows still pass through the products.
    The weights are those of gate_w's E experts, as quantize_expert_weights_mxfp8
    returns them.  Returns the experts' dict and h, y, rstd, logits, ids, prob,
    counts, prob_sum, loss."""
    T, H = x.shape
    plan = _plan(plan, T, k, x.device)
    E = _router(gate_w, H, x.device)
    for name, w, size in (("w1q", w1q, 2 * inter * H), ("w1s", w1s, inter * H // 16),
                          ("w2q", w2q, H * inter), ("w2s", w2s, H * inter // 32)):
        _of_experts(E, name, w, size)
        if w.element_size() != 1 or w.device != x.device or not w.is_contiguous():
            raise ValueError(f"{name}: expected the experts' contiguous bytes on {x.device}")
    qx, sx, y, h, rstd = b.rmsnorm_quantize_mxfp8(x, norm_w, eps, residual=residual, keep_y=True)
    logits = _router_logits(y, gate_w, plan["off"])
    ids, prob, counts, prob_sum, loss = b.moe_gate(logits, k, score, renormalize, scale, mask,
                                                   loss_coef)
    r = _mxfp8_experts(qx, sx, ids, prob.view(-1), w1q, w1s, w2q, w2s, E, inter, True)
    r.update(h=h, y=y, rstd=rstd, logits=logits, ids=ids, prob=prob, counts=counts,
             prob_sum=prob_sum, loss=loss)
    return r


def moe_block_backward(saved, norm_w, gate_w, dy, d_prob, d_loss, d_h=None,
                       loss_coef: float = 0.01, mask=None, plan=None,
                       score: int = b.SCORE_SOFTMAX, renormalize: bool = True,
                       scale: float = 1.0):
    """The gradients of a block's gate and norm, behind the experts' own
    backward pass.  saved: what mxfp8_moe_block_forward returned; a tensor of
    other sizes or with strides is refused.
      dy [T, H] bf16     gradient of y through the experts
      d_prob [T, k] f32  gradient of the routing probabilities
      d_loss [1] f32     gradient of the balance loss
      d_h [T, H] bf16    gradient of h past the norm (may be None)
    d_logits enters its two products in bf16, their operand type, and what comes
    back through the gate is rounded to bf16 before and after it joins dy, the
    type that rmsnorm_backward takes; all sums are binary32.
    Returns dict(dx [T, H] bf16, the gradient of x and of residual; d_norm_w
    [H] f32, d_gate_w [E, H] f32, d_logits [T, E] bf16)."""
    T, H = dy.shape
    dev, bf16, k = dy.device, torch.bfloat16, saved["ids"].shape[1]
    E = _router(gate_w, H, dev)
    plan = _plan(plan, T, k, dev)
    # the products and the combine take their sizes from here (ids and counts are
    # the gate's to check)
    b._want(dy, "dy", bf16, (T, H), dev)
    b._want(saved["y"], "y", bf16, (T, H), dev)
    b._want(saved["h"], "h", bf16, (T, H), dev)
    b._want(saved["rstd"], "rstd", torch.float32, (T,), dev)
    b._want(saved["logits"], "logits", saved["logits"].dtype, (T, E), dev)
    off = plan["off"]
    dz = b.moe_gate_backward(saved["logits"], saved["ids"], d_prob, score, renormalize, scale,
                             mask, loss_coef, saved["counts"], d_loss, out_dtype=b.OUT_BF16)
    d_gate_w = b.moe_grouped_gemm(b.FMT_BF16, b.GEMM_WGRAD, dz, saved["y"], off, E, H,
                                  out_dtype=b.OUT_FP32)[0]
    through_gate = b.moe_grouped_gemm(b.FMT_BF16, b.GEMM_DGRAD, dz, gate_w, off, H, E,
                                      out_dtype=b.OUT_BF16)
    dy = b.moe_combine(through_gate, plan["row"], shared=dy)
    dx, d_norm_w = b.rmsnorm_backward(dy, saved["h"], norm_w, saved["rstd"], d_sum=d_h)
    return dict(dx=dx, d_norm_w=d_norm_w, d_gate_w=d_gate_w, d_logits=dz)
