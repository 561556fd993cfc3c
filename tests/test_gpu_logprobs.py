"""Log probabilities of tokens, entropy, top tokens and the gradient, against
float64.

Bounds: the row's sum of V exponentials is off by (V / 256 + 40) 2^-24 (a
thread's terms one after the other, then a tree), by the exponential's 2^-22 and
by what the rounding of its argument x - m does, 4 |x - m| 2^-24 of each term.
"""

import math

import pytest
import torch

import rotated_codebook_bit_amd as cq

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16
TYPES = pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
DEV, U = "cuda", 2.0 ** -24
HALF = {F32: 2.0 ** -24, BF16: 2.0 ** -8}
TINY = 2.0 ** -126


def logits_of(rows, vocab, dtype, seed=0, scale=3.0):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed + rows + vocab)
    return (torch.randn((rows, vocab), generator=gen, device=DEV) * scale).to(dtype)


def tokens_of(rows, vocab, dtype=torch.int64, seed=0):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed + 77)
    t = torch.randint(0, vocab, (rows,), generator=gen, device=DEV)
    t[::5] = -1
    if rows > 3:
        t[3] = vocab
    return t.to(dtype)


def reference(logits, tokens, scale):
    vocab = logits.shape[1]
    x = logits.double() * scale
    m = x.max(1).values
    d = x - m[:, None]
    log_sum = d.exp().sum(1).log()  # apart from m: next to the type's lowest value it would be lost in 64 bits, too
    lse, logp = m + log_sum, d - log_sum[:, None]
    p = logp.exp()
    plogp = torch.where(p == 0, 0.0, p * logp)
    pd = torch.where(p == 0, 0.0, p * d.abs())
    pdd = torch.where(p == 0, 0.0, p * d * d)
    inside = (tokens >= 0) & (tokens < vocab)
    t = torch.where(inside, tokens, 0).long()
    logprob = torch.where(inside, logp.gather(1, t[:, None])[:, 0], 0.0)
    adds = (vocab / 256 + 40) * U
    es = adds + 2.0 ** -22 + 4 * U * pd.sum(1)
    tol = {"lse": es + 4 * U * (lse.abs() + m.abs()), "logprob": es + 4 * U * (logprob.abs() + log_sum + 1),
           "entropy": es * (2 + pd.sum(1)) + (adds + 2.0 ** -22) * pd.sum(1) + 4 * U * (pdd.sum(1) + pd.sum(1) + 1)}
    tol["log_sum"] = es + 4 * U * (log_sum + 1)
    return {"lse": lse, "logprob": logprob, "entropy": -plogp.sum(1), "log_sum": log_sum}, tol, logp, es


def close(got, want, tol, what):
    same = got.double() == want
    err = torch.where(same, 0.0, (got.double() - want).abs())
    bad = ~(err <= tol)
    assert not bad.any(), (what, int(bad.sum()), err[bad][:4].tolist())


def top_of(logits, k):
    # descending, equal ones by index
    return torch.sort(logits.float(), dim=1, descending=True, stable=True).indices[:, :k]


def check(logits, tokens, scale, top):
    r = cq.token_logprobs(logits, tokens, scale, top)
    want, tol, logp, es = reference(logits, tokens, scale)
    for name in ("lse", "logprob", "entropy"):
        close(getattr(r, name), want[name], tol[name], name)
    if top:
        order = top_of(logits, top)
        assert torch.equal(r.top, order)
        lp = logp.gather(1, order)
        close(r.top_logprob, lp, es[:, None] + 4 * U * (2 * lp.abs() + 1), "top_logprob")
    else:
        assert r.top.shape == r.top_logprob.shape == (*r.lse.shape, 0)
    return r, want, tol, logp


def check_grad(logits, tokens, scale, r, want, tol, logp, entropy=True, **out):
    rows, vocab = logits.shape
    kept = logits.double()
    gen = torch.Generator(device=DEV)
    gen.manual_seed(3)
    g = torch.randn(rows, generator=gen, device=DEV)
    h = torch.randn(rows, generator=gen, device=DEV) if entropy else None
    got = cq.token_logprobs_grad(logits, tokens, r.lse, g, h, r.entropy if entropy else None, scale, **out)
    inside = (tokens >= 0) & (tokens < vocab)
    g64 = torch.where(inside, g.double(), 0.0)[:, None]
    h64 = (h.double() if entropy else torch.zeros(rows, dtype=torch.float64, device=DEV))[:, None]
    p = logp.exp()
    dead = torch.isinf(logp)
    rest = torch.where(dead, 0.0, g64 + h64 * (logp + want["entropy"][:, None]))
    d = -p * rest
    hit = torch.zeros_like(logp)
    hit.scatter_(1, torch.where(inside, tokens, 0).long()[:, None], g64)
    x = torch.where(dead, 0.0, kept * scale)
    # Rows with lse past 1024 are summed again, against their own maximum: the exponent is off by what x - max is.
    far = (want["lse"].abs() > 1023)[:, None]
    el = torch.where(far, tol["log_sum"][:, None] + 4 * U * logp.abs() + 4 * U, tol["lse"][:, None] + 3 * U * (x.abs() + want["lse"].abs()[:, None]))
    el = torch.where(dead, 0.0, el)
    et = torch.where(dead, 0.0, p * (h64.abs() * (el + tol["entropy"][:, None]) + (2 * el + 2.0 ** -21) * rest.abs()
                                     + 4 * U * (g64.abs() + h64.abs() * (torch.where(dead, 0.0, logp).abs() + want["entropy"][:, None]))))
    value = scale * (d + hit)
    close(got, value, scale * (et + 2 * U * (d.abs() + hit.abs()) + 8 * TINY * (1 + g64.abs() + 200 * h64.abs())) + HALF[logits.dtype] * value.abs(), "dlogits")
    return got


@TYPES
@pytest.mark.parametrize("rows,vocab,top", [(1, 1, 1), (1, 2, 2), (3, 7, 5), (5, 300, 20), (2, 512, 64), (4, 1000, 5), (6, 8191, 20), (6, 8193, 8),
                                            (3, 16001, 3), (5, 32000, 20), (2, 50257, 64), (2, 65537, 5), (2, 128256, 20), (1, 262145, 64)])
def test_sizes(rows, vocab, top, dtype):
    logits, tokens = logits_of(rows, vocab, dtype), tokens_of(rows, vocab)
    r, want, tol, logp = check(logits, tokens, 0.7, top)
    check_grad(logits, tokens, 0.7, r, want, tol, logp)


@TYPES
def test_many_rows(dtype):
    logits, tokens = logits_of(700, 1003, dtype), tokens_of(700, 1003, torch.int32)
    r, want, tol, logp = check(logits, tokens, 1.0, 7)
    check_grad(logits, tokens, 1.0, r, want, tol, logp, entropy=False)


@TYPES
@pytest.mark.parametrize("vocab", [1003, 40000])
def test_strided_rows_and_in_place(vocab, dtype):
    wide = torch.full((9, vocab + 13), 1e4, dtype=F32, device=DEV).to(dtype)
    wide[:, :vocab] = logits_of(9, vocab, dtype)
    logits, tokens = wide[:, :vocab], tokens_of(9, vocab)
    r, want, tol, logp = check(logits, tokens, 1.3, 10)
    apart = check_grad(logits, tokens, 1.3, r, want, tol, logp)
    assert apart.is_contiguous()
    inner = wide.clone()
    got = check_grad(inner[:, :vocab], tokens, 1.3, r, want, tol, logp, dlogits=inner[:, :vocab])
    assert got.data_ptr() == inner.data_ptr() and torch.equal(got, apart)
    assert torch.equal(inner[:, vocab:], wide[:, vocab:])  # what lies between the rows stays


@TYPES
def test_masked_logits(dtype):
    """Tokens not allowed: -inf, or the type's lowest value."""
    vocab = 5000
    lowest = torch.finfo(dtype).min
    logits, tokens = logits_of(6, vocab, dtype), torch.tensor([10, 10, 11, 4999, 0, 0], device=DEV)
    logits[0, 11:] = -math.inf          # few left, the token among them
    logits[1, :20] = -math.inf          # the token is not allowed
    logits[2, :11] = lowest
    logits[3, :-1] = -math.inf          # one token left
    logits[4] = lowest                  # all alike
    logits[5, 1:] = lowest
    r, want, tol, logp = check(logits, tokens, 1.0, 20)
    assert r.logprob[1] == -math.inf and r.logprob[3] == 0 and r.entropy[3] == 0
    check_grad(logits, tokens, 1.0, r, want, tol, logp)


@TYPES
@pytest.mark.parametrize("vocab", [9, 5000, 300000])
def test_a_row_with_nothing_left(vocab, dtype):
    logits = torch.full((2, vocab), -math.inf, dtype=dtype, device=DEV)
    logits[1, 5] = 2.0
    tokens = torch.tensor([3, 5], device=DEV)
    r = cq.token_logprobs(logits, tokens, 1.0, 4)
    assert r.lse[0] == -math.inf and r.entropy[0] == 0 and r.logprob[0] == -math.inf
    assert r.top[0].tolist() == [0, 1, 2, 3] and (r.top_logprob[0] == -math.inf).all()
    assert r.lse[1] == 2 and r.logprob[1] == 0 and r.top[1].tolist() == [5, 0, 1, 2] and r.top_logprob[1, 0] == 0
    d = cq.token_logprobs_grad(logits, tokens, r.lse, torch.ones(2, device=DEV), torch.ones(2, device=DEV), r.entropy)
    assert (d == 0).all()


@TYPES
def test_values_that_are_not_finite(dtype):
    logits = logits_of(4, 9000, dtype)
    clean = cq.token_logprobs(logits, tokens_of(4, 9000), 1.0, 3)
    logits[1, 77], logits[1, 8000], logits[2, 40] = math.nan, math.inf, math.inf
    r = cq.token_logprobs(logits, torch.tensor([0, 1, 2, -1], device=DEV), 1.0, 3)
    for name in ("lse", "entropy", "logprob"):
        assert torch.isnan(getattr(r, name)[1:3]).all()
    assert r.top[1, :2].tolist() == [77, 8000] and r.top[2, 0] == 40
    assert torch.equal(r.lse[[0, 3]], clean.lse[[0, 3]]) and torch.equal(r.top[[0, 3]], clean.top[[0, 3]])


@TYPES
@pytest.mark.parametrize("vocab,top", [(300, 64), (5000, 33), (32000, 64), (140000, 10), (270000, 5)])
def test_ties(vocab, top, dtype):
    """Equal logits, in numbers that overflow any list of candidates, and the
    largest values all in one thread's pieces."""
    logits = torch.zeros((4, vocab), dtype=dtype, device=DEV)
    logits[1] = logits_of(1, vocab, dtype)[0].round()
    logits[2, vocab // 2:] = 1.0
    step = (8 if dtype == BF16 else 4) * 1024
    logits[3, ::step] = 5.0
    logits[3, 1::step] = 4.0
    logits[3, 2::step] = 6.0
    logits[0, ::2] = -0.0  # equal to 0
    tokens = tokens_of(4, vocab)
    check(logits, tokens, 1.0, top)


@TYPES
def test_large_logits(dtype):
    logits, tokens = logits_of(5, 40000, dtype, scale=1e4), tokens_of(5, 40000)
    r, want, tol, logp = check(logits, tokens, 2.0, 5)
    apart = check_grad(logits, tokens, 2.0, r, want, tol, logp)
    own = logits.clone()
    check_grad(own, tokens, 2.0, r, want, tol, logp, dlogits=own)
    assert torch.equal(own, apart)


@TYPES
def test_leading_shapes_and_empty_calls(dtype):
    logits, tokens = logits_of(6, 100, dtype), tokens_of(6, 100)
    flat = cq.token_logprobs(logits, tokens, 1.0, 2)
    shaped = cq.token_logprobs(logits.view(2, 3, 100), tokens.view(2, 3), 1.0, 2)
    assert torch.equal(shaped.logprob.flatten(), flat.logprob) and shaped.top.shape == (2, 3, 2)
    none = cq.token_logprobs(logits[:0], tokens[:0], 1.0, 2)
    assert none.logprob.shape == (0,) and none.top.shape == (0, 2)
    assert cq.token_logprobs_grad(logits[:0], tokens[:0], none.lse, none.lse).shape == (0, 100)
    empty = cq.token_logprobs(logits[:, :0].contiguous(), tokens)
    assert (empty.lse == -math.inf).all() and (empty.entropy == 0).all() and (empty.logprob == 0).all()


def test_differences():
    logits, tokens = logits_of(3, 50, F32), torch.tensor([4, 49, -1], device=DEV)
    r = cq.token_logprobs(logits, tokens, 0.9)
    gen = torch.Generator(device=DEV)
    gen.manual_seed(3)
    g, h, dirs = (torch.randn(s, generator=gen, device=DEV) for s in ((3,), (3,), (3, 50)))
    d = cq.token_logprobs_grad(logits, tokens, r.lse, g, h, r.entropy, 0.9)

    def loss(step):
        want, _, _, _ = reference(logits.double() + step * dirs.double(), tokens, 0.9)
        return (want["logprob"] * g.double()).sum() + (want["entropy"] * h.double()).sum()

    slope = (loss(1e-4) - loss(-1e-4)) / 2e-4
    got = (d.double() * dirs.double()).sum()
    assert (got - slope).abs() <= 1e-5 * (d.double() * dirs.double()).abs().sum()


@TYPES
def test_same_bits_streams_and_graphs(dtype):
    logits, tokens = logits_of(20, 12001, dtype), tokens_of(20, 12001)
    g = torch.linspace(-1, 1, 20, device=DEV)

    def step(stream=None):
        r = cq.token_logprobs(logits, tokens, 0.8, 6, stream=stream)
        return (*r, cq.token_logprobs_grad(logits, tokens, r.lse, g, g, r.entropy, 0.8, stream=stream))

    want = step()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = step(side)
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for turn in range(3):
        logits.copy_(logits_of(20, 12001, dtype, seed=9 + turn))
        want = step()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_refusals():
    logits, tokens = logits_of(4, 100, F32), tokens_of(4, 100)
    r = cq.token_logprobs(logits, tokens)
    for bad in (lambda: cq.token_logprobs(logits.half(), tokens), lambda: cq.token_logprobs(logits, tokens.float())):
        with pytest.raises(TypeError):
            bad()
    for bad in (lambda: cq.token_logprobs(logits, tokens[:2]), lambda: cq.token_logprobs(logits.cpu(), tokens),
                lambda: cq.token_logprobs(logits.t(), tokens_of(100, 4)), lambda: cq.token_logprobs(logits, tokens.cpu()),
                lambda: cq.token_logprobs_grad(logits, tokens, r.lse[:2], r.lse), lambda: cq.token_logprobs_grad(logits, tokens, r.lse, r.lse, r.lse),
                lambda: cq.token_logprobs_grad(logits, tokens, r.lse.double(), r.lse),
                lambda: cq.token_logprobs_grad(logits, tokens, r.lse, r.lse, dlogits=logits[:2])):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: cq.token_logprobs(logits, tokens, 0.0), lambda: cq.token_logprobs(logits, tokens, -1.0),
                lambda: cq.token_logprobs(logits, tokens, math.inf), lambda: cq.token_logprobs(logits, tokens, 1.0, 65),
                lambda: cq.token_logprobs(logits[:, :3].contiguous(), tokens, 1.0, 4), lambda: cq.token_logprobs(logits[:, 1:], tokens),
                lambda: cq.token_logprobs_grad(logits, tokens, r.lse, r.lse, dlogits=logits[:1].expand(4, 100))):
        with pytest.raises((cq.CQError, ValueError)):
            bad()
