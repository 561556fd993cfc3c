"""An attention block as a model runs it: the fused projection's output through
the norm and rotation, attention, and at the end the tokens' log probabilities;
its training step against autograd in float64, and serving token by token from
a cache against the whole prompt at once."""

import math

import pytest
import torch

import rotated_codebook_bit_amd as cq

pytestmark = pytest.mark.gpu
DEV, D, HEADS, KV, VOCAB = "cuda", 32, 4, 2, 200
DIM = HEADS * D


def randn(*shape, seed=0, scale=1.0):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed + sum(shape))
    return torch.randn(shape, generator=gen, device=DEV) * scale


class Rotate(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, qw, kw, positions, freqs):
        ctx.save_for_backward(q, k, qw, kw, positions, freqs)
        return cq.qk_norm_rope(q, k, positions, freqs, qw, kw)

    @staticmethod
    def backward(ctx, dq, dk):
        q, k, qw, kw, positions, freqs = ctx.saved_tensors
        return *cq.qk_norm_rope_grad(dq, dk, q, k, positions, freqs, qw, kw), None, None


class Attend(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, v, starts):
        out, lse = cq.attention(q, k, v, q_starts=starts, k_starts=starts)
        ctx.save_for_backward(q, k, v, out, lse, starts)
        return out

    @staticmethod
    def backward(ctx, dout):
        q, k, v, out, lse, starts = ctx.saved_tensors
        return *cq.attention_grad(dout, q, k, v, out, lse, q_starts=starts, k_starts=starts), None


class Score(torch.autograd.Function):
    @staticmethod
    def forward(ctx, logits, tokens):
        r = cq.token_logprobs(logits, tokens)
        ctx.save_for_backward(logits, tokens, r.lse, r.entropy)
        return r.logprob, r.entropy

    @staticmethod
    def backward(ctx, dlogprob, dentropy):
        logits, tokens, lse, entropy = ctx.saved_tensors
        return cq.token_logprobs_grad(logits, tokens, lse, dlogprob.contiguous(), dentropy.contiguous(), entropy), None


def weights():
    return {"qkv": randn((HEADS + 2 * KV) * D, DIM, scale=DIM ** -0.5), "o": randn(DIM, DIM, seed=1, scale=DIM ** -0.5),
            "out": randn(VOCAB, DIM, seed=2, scale=DIM ** -0.5), "qw": 1 + randn(D, scale=0.1), "kw": 1 + randn(D, seed=1, scale=0.1)}


FREQS = (10000.0 ** (-torch.arange(D // 2, dtype=torch.float64) / (D // 2))).float()


def loss_own(w, x, tokens, positions, starts):
    qkv = (x @ w["qkv"].t()).view(-1, HEADS + 2 * KV, D)
    q, k, v = qkv.split([HEADS, KV, KV], 1)
    q, k = Rotate.apply(q, k, w["qw"], w["kw"], positions, FREQS.to(DEV))
    h = x + Attend.apply(q, k, v, starts).flatten(1) @ w["o"].t()
    logprob, entropy = Score.apply(h @ w["out"].t(), tokens)
    return -logprob.sum() - 0.1 * entropy.sum()


def loss_64(w, x, tokens, positions, lens):
    n = x.shape[0]
    qkv = (x @ w["qkv"].t()).view(n, HEADS + 2 * KV, D)
    angle = positions.double()[:, None] * FREQS.to(DEV).double()
    cos, sin = angle.cos()[:, None], angle.sin()[:, None]

    def rotate(t, weight):
        t = t / torch.sqrt((t * t).mean(-1, keepdim=True) + 1e-6) * weight
        a, b = t[..., :D // 2], t[..., D // 2:]
        return torch.cat([a * cos - b * sin, b * cos + a * sin], -1)

    q, k, v = qkv.split([HEADS, KV, KV], 1)
    q, k = rotate(q, w["qw"]), rotate(k, w["kw"])
    outs, at = [], 0
    for m in lens:
        a, b, c = (t[at:at + m].transpose(0, 1) for t in (q, k.repeat_interleave(HEADS // KV, 1), v.repeat_interleave(HEADS // KV, 1)))
        s = torch.matmul(a, b.transpose(1, 2).contiguous()) / math.sqrt(D)
        s = s.masked_fill(torch.ones(m, m, dtype=torch.bool, device=DEV).triu(1), -math.inf)
        outs.append(torch.matmul(torch.softmax(s, -1), c.contiguous()).transpose(0, 1))
        at += m
    h = x + torch.cat(outs).flatten(1) @ w["o"].t()
    logp = torch.log_softmax(h @ w["out"].t(), 1)
    inside = tokens >= 0
    logprob = logp.gather(1, tokens.clamp(min=0)[:, None])[:, 0] * inside
    return -logprob.sum() + 0.1 * (logp.exp() * logp).sum()


def test_training_step():
    lens = [37, 1, 60]
    n = sum(lens)
    starts = torch.tensor([0, 37, 38, 98], dtype=torch.int32, device=DEV)
    positions = torch.cat([torch.arange(m, device=DEV) for m in lens])
    gen = torch.Generator(device=DEV)
    gen.manual_seed(0)
    tokens = torch.randint(0, VOCAB, (n,), generator=gen, device=DEV)
    tokens[::9] = -1
    x = randn(n, DIM, seed=5)
    w = {name: t.requires_grad_() for name, t in weights().items()}
    x.requires_grad_()
    got = loss_own(w, x, tokens, positions, starts)
    got.backward()
    w64 = {name: t.detach().double().requires_grad_() for name, t in w.items()}
    x64 = x.detach().double().requires_grad_()
    want = loss_64(w64, x64, tokens, positions, lens)
    want.backward()
    # Sums of some hundred terms in float32 one after another in five stages: 1e-5 of the largest value.
    assert (got.double() - want).abs() <= 1e-5 * want.abs()
    for name, t in (*w.items(), ("x", x)):
        g64 = (w64[name] if name != "x" else x64).grad
        assert (t.grad.double() - g64).abs().max() <= 1e-5 * g64.abs().max(), name


def test_a_captured_backward_beside_an_eager_graph():
    """A captured training step while an eager graph of the same leaves is alive."""
    starts = torch.tensor([0, 20, 50], dtype=torch.int32, device=DEV)
    positions = torch.arange(50, device=DEV)
    tokens = torch.arange(50, device=DEV)
    q, k, v, dout = randn(50, HEADS, D), randn(50, KV, D), randn(50, KV, D), randn(50, HEADS, D, seed=4)
    freqs = FREQS.to(DEV)

    def step():
        a, b = cq.qk_norm_rope(q, k, positions, freqs)
        out, lse = cq.attention(a, b, v, q_starts=starts, k_starts=starts)
        da, db, dv = cq.attention_grad(dout, a, b, v, out, lse, q_starts=starts, k_starts=starts)
        logits = out.flatten(1)
        r = cq.token_logprobs(logits, tokens, top=3)
        return (*cq.qk_norm_rope_grad(da, db, q, k, positions, freqs)[:2], dv, r.logprob, r.top,
                cq.token_logprobs_grad(logits, tokens, r.lse, r.logprob))

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for turn in range(3):
        q.copy_(randn(50, HEADS, D, seed=10 + turn))
        want = step()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_serving_from_a_cache():
    """Prompts of two conversations into a cache, then token by token; the
    outputs against the whole conversations at once."""
    w = weights()
    lens, new, cap = [13, 40], 6, 64
    x = [randn(m + new, DIM, seed=20 + i) for i, m in enumerate(lens)]
    k_cache = torch.full((2 * cap, KV, D), math.nan, device=DEV)
    v_cache = k_cache.clone()
    freqs = FREQS.to(DEV)

    def block(rows, positions, slots):
        q, k, v = (rows @ w["qkv"].t()).view(-1, HEADS + 2 * KV, D).split([HEADS, KV, KV], 1)
        return cq.qk_norm_rope(q, k, positions, freqs, w["qw"], w["kw"], v=v, slots=slots, k_out=k_cache, v_out=v_cache)[0]

    def finish(rows, out):
        return cq.token_logprobs((rows + out.flatten(1) @ w["o"].t()) @ w["out"].t(), torch.zeros(len(rows), dtype=torch.int64, device=DEV), top=4)

    # the whole conversations, packed
    rows = torch.cat(x)
    positions = torch.cat([torch.arange(len(t), device=DEV) for t in x])
    q, k, v = (rows @ w["qkv"].t()).view(-1, HEADS + 2 * KV, D).split([HEADS, KV, KV], 1)
    q, k = cq.qk_norm_rope(q, k, positions, freqs, w["qw"], w["kw"])
    starts = torch.tensor([0, lens[0] + new, sum(lens) + 2 * new], device=DEV)
    out, _ = cq.attention(q, k, v, q_starts=starts, k_starts=starts)
    whole = finish(rows, out)
    # prompts, packed, into the cache
    rows = torch.cat([t[:m] for t, m in zip(x, lens)])
    slots = torch.cat([i * cap + torch.arange(m, device=DEV) for i, m in enumerate(lens)])
    starts = torch.tensor([0, lens[0], sum(lens)], device=DEV)
    at = torch.tensor([0, cap], device=DEV)
    q = block(rows, slots % cap, slots)
    out, _ = cq.attention(q, k_cache, v_cache, q_starts=starts, k_starts=at, k_lens=torch.tensor(lens, device=DEV))
    got = [finish(rows, out).logprob]
    for step in range(new):
        rows = torch.stack([t[m + step] for t, m in zip(x, lens)])
        positions = torch.tensor([m + step for m in lens], device=DEV)
        q = block(rows, positions, at + positions)
        out, _ = cq.attention(q, k_cache, v_cache, sequences=2, k_lens=positions + 1)
        r = finish(rows, out)
        got.append(r.logprob)
        for i, m in enumerate(lens):
            j = (lens[0] + new) * i + m + step
            assert torch.equal(r.top[i], whole.top[j]) or (r.top_logprob[i] - whole.top_logprob[j]).abs().max() < 1e-4
    # float32 sums of the same terms in another order: 1e-5 of log probabilities of about 5
    want0 = torch.cat([whole.logprob[:lens[0]], whole.logprob[lens[0] + new:lens[0] + new + lens[1]]])
    assert (got[0] - want0).abs().max() <= 5e-5
    for step in range(new):
        want = whole.logprob[[lens[0] + step, lens[0] + new + lens[1] + step]]
        assert (got[1 + step] - want).abs().max() <= 5e-5
