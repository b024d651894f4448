"""The end of a policy: from the residual stream to log probabilities of the
tokens that were taken, and back.

Reinforcement learning compares the log probabilities that the rollout engine
gave its tokens with the ones that training gives them; both sides run these
passes, so that what differs between them is the layers below ("Towards
Blackwell-Native 8-bit and 4-bit RL"), and last bits: the order of the sums goes
by the number of rows, so a call of 8 rows and one of 2048 give the same row's
logits off by roundings of binary32, which now and then is a step of bf16
(logits_dtype OUT_FP32 keeps it at binary32's).  Each function only sequences
calls into libpqmoe on torch's current stream.
"""
from __future__ import annotations

import torch

from . import _binding as b


def policy_head_forward(x, residual, norm_w, head_w, ids=None, temperature: float = 1.0,
                        top_n: int = 0, eps: float = 1e-6, logits_dtype: int = b.OUT_BF16):
    """Residual addition and RMS norm, the head's product, log probabilities.
      x, residual [T, H] bf16  residual may be None
      norm_w [H]               bf16 or f32
      head_w [V, H] bf16       V % 8 == 0 if the backward pass is to follow
      ids [T] int32            the tokens taken, negative for rows to leave out
                               (their x must be finite, since they still pass
                               through the products); None for entropy and
                               alternatives alone
    Returns dict(logprob [T] f32 or None, entropy [T] f32, top_ids [T, top_n]
    int32 and top_logprob f32 or None, stats, logits [T, V], h, y, rstd): entropy
    and the last five are what policy_head_backward reads.  logits_dtype OUT_FP32 keeps the
    logits' sums as they are, at twice the bytes."""
    _, _, y, h, rstd = b.rmsnorm_quantize_mxfp8(x, norm_w, eps, residual=residual, quantize=False)
    logits, _ = b.linear(y, head_w, out_dtype=logits_dtype)
    logprob, entropy, stats, top_ids, top_logprob = b.token_logprobs(logits, ids, temperature,
                                                                     top_n)
    return dict(logprob=logprob, entropy=entropy, top_ids=top_ids, top_logprob=top_logprob,
                stats=stats, logits=logits, h=h, y=y, rstd=rstd)


def policy_head_backward(saved, norm_w, head_w, ids, d_logprob=None, d_entropy=None, d_h=None,
                         temperature: float = 1.0, reuse_logits: bool = False):
    """The gradients of policy_head_forward.  saved: what it returned, of which
    logits, stats, h, y, rstd and, with d_entropy, entropy are read; a tensor of
    other sizes or with strides is refused, and so is V % 8 != 0.
      d_logprob, d_entropy [T] f32  either may be None
      d_h [T, H] bf16               gradient of h past the norm (may be None)
    d_logits is bf16, the products' operand type; reuse_logits writes it over the
    saved logits (bf16 alone), for vocabularies whose second copy is too much; a
    call that is refused leaves them as they were.
    Returns dict(dx [T, H] bf16, the gradient of x and of residual; d_norm_w [H]
    f32, d_head_w [V, H] f32, d_logits [T, V] bf16)."""
    logits = saved["logits"]
    T, H = saved["y"].shape
    V, dev = head_w.shape[0], saved["y"].device
    b._want(head_w, "head_w", torch.bfloat16, (V, H), dev)
    b._want(logits, "logits", logits.dtype, (T, V), dev)
    b._want(saved["h"], "h", torch.bfloat16, (T, H), dev)
    b._want(saved["rstd"], "rstd", torch.float32, (T,), dev)
    if reuse_logits and logits.dtype is not torch.bfloat16:
        raise TypeError("reuse_logits: the logits have to be bf16")
    # what the calls behind the first one refuse, before it writes
    b._want(saved["y"], "y", torch.bfloat16, (T, H), dev)
    b._bf16_or_f32(norm_w, "norm_w")
    b._want(norm_w, "norm_w", norm_w.dtype, (H,), dev)
    if d_h is not None:
        b._want(d_h, "d_h", torch.bfloat16, (T, H), dev)
    if V % 8 or H % 8 or not 8 <= V <= 1 << 22 or not 8 <= H <= 16384:
        raise ValueError(f"head_w: no gradient of {V} outputs of {H} values (whole groups of eight, "
                         "up to 2^22 and 16384)")
    for name, t in (("y", saved["y"]), ("h", saved["h"]), ("head_w", head_w), ("norm_w", norm_w),
                    ("d_h", d_h), ("logits", logits if reuse_logits else None)):
        if t is not None and t.data_ptr() % 16:
            raise ValueError(f"{name}: must be aligned to 16 bytes")
    dz = b.token_logprobs_backward(logits, ids, saved["stats"], d_logprob, temperature,
                                   saved["entropy"] if d_entropy is not None else None, d_entropy,
                                   out_dtype=b.OUT_BF16, out=logits if reuse_logits else None)
    dy, d_head_w, _, _ = b.linear_backward(dz, saved["y"], head_w)
    dx, d_norm_w = b.rmsnorm_backward(dy, saved["h"], norm_w, saved["rstd"], d_sum=d_h)
    return dict(dx=dx, d_norm_w=d_norm_w, d_head_w=d_head_w, d_logits=dz)
