"""The example model end to end on the GPU: it trains through the operators'
gradients, and its served form (packed weights, 8-bit activations) predicts
what the training forward does."""

import os
import sys

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover - CPU container
    pytest.skip("no GPU", allow_module_level=True)

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
import small_lm as E  # noqa: E402


def test_gradients_match_plain_autograd():
    """One step's gradients against the same model in plain float64 torch
    (the quantized weights taken as given, gradients passed through)."""
    print("[gpu] small_lm gradients", flush=True)
    p = E.init()
    tokens = torch.arange(0, E.VOCAB, 3, device="cuda").repeat(2)
    loss = torch.nn.functional.cross_entropy(E.logits_of(p, tokens), (5 * tokens + 7) % E.VOCAB)
    loss.backward()
    q = {k: E.cq.fake_quant(p[k].detach(), E.BITS, None).double() if p[k].dim() == 2 else p[k].detach().double() for k in p}
    for v in q.values():
        v.requires_grad_()

    def norm(h, w):
        return h * torch.rsqrt((h * h).mean(1, keepdim=True) + 1e-6) * w

    h = q["embed"][tokens] * E.SCALE
    block = torch.relu(norm(h, q["norm1"]) @ q["up"].t()) @ q["down"].t()
    ref = torch.nn.functional.cross_entropy(norm(h + block, q["norm2"]) @ q["embed"].t(), (5 * tokens + 7) % E.VOCAB)
    ref.backward()
    assert abs(loss.item() - ref.item()) <= 1e-4 * ref.item()
    for k in p:  # float32 through five products: 1e-4 of the gradient's norm
        assert (p[k].grad.double() - q[k].grad).norm() <= 1e-4 * q[k].grad.norm(), k


def test_trains_and_serves():
    print("[gpu] small_lm train and serve", flush=True)
    losses, accuracy, far, alone = E.main(300)
    assert losses[-1] < 0.5 * losses[0]
    assert accuracy > 0.95
    # 8-bit activations: half a step of 1/127 of the row's largest, about 1% of a typical value, twice
    assert far < 0.05
    # a token's activations do not depend on its batch; sums may be ordered otherwise
    assert alone < 1e-3
