"""Gradient of the log probabilities of rows whose largest logit times the
scale leaves float32, so that their lse is infinite."""

import math

import pytest
import torch

import rotated_codebook_bit_amd as cq

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16
TYPES = pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
DEV, U = "cuda", 2.0 ** -24
HALF = {F32: 2.0 ** -24, BF16: 2.0 ** -8}


@TYPES
@pytest.mark.parametrize("vocab", [6, 5000, 40000])
@pytest.mark.parametrize("in_place", [False, True], ids=["apart", "in_place"])
def test_gradient_where_the_largest_logit_leaves_float32(vocab, in_place, dtype):
    """Rows of the type's lowest value (every token masked) under a scale above
    one, and rows with its largest: lse is infinite, the probabilities are not.

    Tolerance: p = 1 / n for the n values at the maximum; its exponent is
    log2 n, off by half a step of at most 2^4 2^-24 and the sum's (vocab / 256 + 40)
    2^-24, the exponential by 2^-22: ep of p.  g p and h p (log p + H), in which
    log p + H of equal values is the difference of two numbers off by (vocab / 256 +
    80) 2^-24 log n; then half a step of the result."""
    lowest, largest = torch.finfo(dtype).min, torch.finfo(dtype).max
    logits = torch.full((5, vocab), lowest, dtype=dtype, device=DEV)
    logits[1, 2] = -math.inf
    logits[2, 3] = largest
    logits[3] = largest
    logits[4] = -math.inf
    tokens = torch.tensor([1, 1, 3, -1, 2], device=DEV)
    scale = 1.25
    r = cq.token_logprobs(logits, tokens, scale)
    count = torch.tensor([vocab, vocab - 1, 1, vocab, 0], dtype=torch.float64, device=DEV)
    log_n = torch.where(count > 0, count, 1.0).log()
    assert r.lse.tolist() == [-math.inf, -math.inf, math.inf, math.inf, -math.inf]
    ep = (vocab / 256 + 40) * U + 16 * U + 2.0 ** -22
    assert ((r.logprob.double() + log_n)[:3].abs() <= ep + 4 * U * log_n[:3]).all() and r.logprob[4] == -math.inf
    g, h = torch.tensor([1.0, -2.0, 3.0, 1.0, 1.0], device=DEV), torch.tensor([0.5, 0.0, 1.0, -1.0, 1.0], device=DEV)
    own = logits.clone()
    got = cq.token_logprobs_grad(own, tokens, r.lse, g, h, r.entropy, scale, dlogits=own if in_place else None)
    at_top = logits == logits.max(1, keepdim=True).values
    at_top[4] = False
    p = at_top.double() / torch.where(count > 0, count, 1.0)[:, None]
    g64 = torch.where((tokens >= 0) & (count > 0), g.double(), 0.0)[:, None]
    want = -g64 * p
    want.scatter_add_(1, tokens.clamp(min=0)[:, None], g64)  # log p + H = 0 where p is not
    want *= scale
    tol = scale * (p * (g64.abs() * (ep + 8 * U) + h.double().abs()[:, None] * ((vocab / 256 + 80) * U * (1 + log_n) + ep)[:, None]) + 2 * U * g64.abs())
    tol = tol + HALF[dtype] * want.abs()
    err = (got.double() - want).abs()
    assert (err <= tol).all(), (err / tol).amax(1).tolist()
