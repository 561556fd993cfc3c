"""Trains a small language model with quantized weights and serves it from CQ
storage, on one GPU: the embedding lookup and its gradient, the residual norm
and its gradient, and the 8-bit norm with the product that reads it, as they
are used together.

The model is an embedding, one residual block of two matrices and a tied
output: logits = norm(h + down(relu(up(norm(h))))) . E^T with h = sqrt(dim) *
E[token].  Training runs every weight through fake quantization with a
straight-through gradient ("Cactus Quants CQ2-bit Quantization: Extreme
Compression for Edge LLMs", section Training with Quantization).  Serving
quantizes the trained weights once and decodes from the packed form: the
lookup, the up projection and the logits read nothing but packed weights and
8-bit activations; the down projection's input has no norm in front of it and
takes the float32 product.

The data are synthetic: the next token is (5 * token + 7) mod vocab.

    python examples/small_lm.py [steps]
"""

import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import rotated_codebook_bit_amd as cq  # noqa: E402

VOCAB, DIM, HIDDEN, BITS = 512, 256, 512, 4
SCALE = math.sqrt(DIM)


class Quantized(torch.autograd.Function):
    """A weight as quantization would leave it; the gradient passes through."""

    @staticmethod
    def forward(ctx, w):
        return cq.fake_quant(w, BITS, None)

    @staticmethod
    def backward(ctx, d):
        return d


class Embed(torch.autograd.Function):
    @staticmethod
    def forward(ctx, tokens, table):
        ctx.save_for_backward(tokens)
        ctx.vocab = table.shape[0]
        return cq.embed(tokens, table, SCALE)

    @staticmethod
    def backward(ctx, d):
        (tokens,) = ctx.saved_tensors
        return None, cq.embed_grad(tokens, d.contiguous(), ctx.vocab, SCALE)


class AddNorm(torch.autograd.Function):
    """(norm(x + residual) * weight, x + residual); residual may be None."""

    @staticmethod
    def forward(ctx, x, residual, weight):
        out, total = cq.add_rms_norm(x, residual, weight)
        if residual is None:
            total = x.clone()
        ctx.has_residual = residual is not None
        ctx.save_for_backward(total, weight)
        return out, total

    @staticmethod
    def backward(ctx, dout, dtotal):
        total, weight = ctx.saved_tensors
        dx, dweight = cq.rms_norm_grad(dout.contiguous(), total, weight, dsum=dtotal.contiguous())
        return dx, dx if ctx.has_residual else None, dweight


def init(seed=0, device="cuda"):
    gen = torch.Generator(device=device)
    gen.manual_seed(seed)

    def matrix(rows, cols):
        return (torch.randn(rows, cols, generator=gen, device=device) / math.sqrt(cols)).requires_grad_()

    return {"embed": matrix(VOCAB, DIM), "up": matrix(HIDDEN, DIM), "down": matrix(DIM, HIDDEN),
            "norm1": torch.ones(DIM, device=device, requires_grad=True),
            "norm2": torch.ones(DIM, device=device, requires_grad=True)}


def logits_of(p, tokens):
    """The training forward, with fake-quantized weights."""
    table = Quantized.apply(p["embed"])
    n1, h = AddNorm.apply(Embed.apply(tokens, table), None, p["norm1"])
    block = torch.relu(n1 @ Quantized.apply(p["up"]).t()) @ Quantized.apply(p["down"]).t()
    n2, _ = AddNorm.apply(block, h, p["norm2"])
    return n2 @ table.t()


def train(p, steps, batch=256, seed=1):
    opt = torch.optim.Adam(p.values(), lr=3e-3)
    gen = torch.Generator(device=p["embed"].device)
    gen.manual_seed(seed)
    losses = []
    for _ in range(steps):
        tokens = torch.randint(0, VOCAB, (batch,), generator=gen, device=p["embed"].device)
        loss = torch.nn.functional.cross_entropy(logits_of(p, tokens), (5 * tokens + 7) % VOCAB)
        opt.zero_grad()
        loss.backward()
        opt.step()
        losses.append(loss.detach())
    return torch.stack(losses).tolist()


class Served:
    """The trained model in CQ storage."""

    def __init__(self, p):
        self.q = {k: cq.quantize(p[k].detach(), BITS, None) for k in ("embed", "up", "down")}
        self.norm1, self.norm2 = p["norm1"].detach(), p["norm2"].detach()
        self.levels = cq.q8_levels(BITS)

    def logits(self, tokens):
        h = cq.embed_packed(tokens, *self.q["embed"], VOCAB, DIM, BITS, None, SCALE)
        a, s, _ = cq.add_rms_norm_q8(h, None, self.norm1)
        up = torch.relu(cq.dequant_gemm_q8(*self.q["up"], HIDDEN, DIM, BITS, self.levels, a, s))
        block = cq.dequant_gemm(*self.q["down"], DIM, HIDDEN, BITS, None, up)
        a, s, _ = cq.add_rms_norm_q8(block, h, self.norm2)
        return cq.dequant_gemm_q8(*self.q["embed"], VOCAB, DIM, BITS, self.levels, a, s)


def main(steps=400):
    p = init()
    losses = train(p, steps)
    tokens = torch.arange(VOCAB, device="cuda")
    target = (5 * tokens + 7) % VOCAB
    with torch.no_grad():
        trained = logits_of(p, tokens)
    served = Served(p)
    out = served.logits(tokens)
    one = served.logits(tokens[3:4])  # a decode step
    far = ((out - trained).norm() / trained.norm()).item()
    accuracy = (out.argmax(1) == target).float().mean().item()
    print(f"loss {losses[0]:.3f} -> {losses[-1]:.3f}; served next-token accuracy {accuracy:.3f}; "
          f"served logits {far:.4f} off the training forward; one token alone {(one - out[3:4]).abs().max().item():.2e} off")
    return losses, accuracy, far, (one - out[3:4]).abs().max().item() / out.abs().max().item()


if __name__ == "__main__":
    main(int(sys.argv[1]) if len(sys.argv) > 1 else 400)
