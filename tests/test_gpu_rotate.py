"""The norm of queries and keys per head with the position rotation, and its
gradient, against float64.

Bounds: the mean square of D values is off by a relative D 2^-24, its root by
half of that, each product by 2^-24, sine and cosine by 2^-24; a sum of n terms
by n 2^-24 of their magnitudes.  Results are rounded once, half a step.
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


def randn(*shape, dtype=F32, seed=0, scale=1.0):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed + sum(shape))
    return (torch.randn(shape, generator=gen, device=DEV) * scale).to(dtype)


def turn(y, cos, sin, interleaved):
    """(turned y, magnitudes of what was added)."""
    half = cos.shape[-1]
    c, s = cos[:, None], sin[:, None]
    idx = torch.arange(2 * half, device=y.device)
    first, second = (idx[0::2], idx[1::2]) if interleaved else (idx[:half], idx[half:])
    out, mag = y.clone(), y.abs()
    a, b = y[..., first], y[..., second]
    out[..., first], out[..., second] = a * c - b * s, b * c + a * s
    mag[..., first], mag[..., second] = (a * c).abs() + (b * s).abs(), (b * c).abs() + (a * s).abs()
    return out, mag


def forward64(x, w, eps, norm, cos, sin, interleaved):
    x = x.double()
    d = x.shape[-1]
    if norm:
        x = x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps) * (1.0 if w is None else w.double())
    out, mag = turn(x, cos, sin, interleaved)
    return out, ((d / 2 if norm else 0) + 12) * U * mag


def backward64(g, x, w, eps, norm, cos, sin, interleaved):
    u, mag = turn(g.double(), cos, -sin, interleaved)
    eu = 4 * U * mag
    if not norm:
        return u, eu, None, None
    x = x.double()
    d = x.shape[-1]
    w = torch.ones(d, dtype=torch.float64, device=x.device) if w is None else w.double()
    r = 1 / torch.sqrt((x * x).mean(-1, keepdim=True) + eps)
    z = u * w
    k = (z * x).mean(-1, keepdim=True)
    dx = r * (z - x * r * r * k)
    tol = r * (eu * w.abs() + x.abs() * r * r * (eu * w.abs() * x.abs()).mean(-1, keepdim=True)
               + (2 * d + 20) * U * (z.abs() + x.abs() * r * r * (z * x).abs().mean(-1, keepdim=True)))
    n = x.shape[0] * x.shape[1]
    dw = (u * x * r).sum((0, 1))
    wtol = (eu * (x * r).abs() + (d / 2 + 12 + n) * U * (u * x * r).abs()).sum((0, 1))
    return dx, tol, dw, wtol


def close(got, want, tol, what):
    err = (got.double() - want).abs()
    tol = tol + HALF[got.dtype] * want.abs() + TINY
    bad = ~(err <= tol)
    assert not bad.any(), (what, int(bad.sum()), float((err / tol)[bad].max()))


def angles(positions, freqs):
    t = positions.double()[:, None] * freqs.double()
    return t.cos(), t.sin()


def inputs(n, qh, kvh, d, rot, dtype, pos=torch.int64, far=100000):
    qkv = randn(n, qh + 2 * kvh, d, dtype=dtype)
    q, k, v = qkv.split([qh, kvh, kvh], 1)
    positions = (far + torch.arange(n, device=DEV) * 7 - 3).to(pos)
    freqs = (10000.0 ** (-torch.arange(rot // 2, device=DEV, dtype=torch.float64) / max(rot // 2, 1))).float()
    return q, k, v, positions, freqs


def check(n, qh, kvh, d, rot, dtype, interleaved=False, norm=True, wtype=F32, weights=True, eps=1e-6, pos=torch.int64):
    q, k, v, positions, freqs = inputs(n, qh, kvh, d, rot, dtype, pos)
    qw = (1 + randn(d, scale=0.2)).to(wtype) if norm and weights else None
    kw = (1 + randn(d, scale=0.2, seed=1)).to(wtype) if norm and weights else None
    cos, sin = angles(positions, freqs)
    where = dict(eps=eps, norm=norm, interleaved=interleaved)
    args = (positions, freqs, qw, kw) if rot else (None, None, qw, kw)
    qo, ko, vo = cq.qk_norm_rope(q, k, *args, v=v, **where)
    for got, x, w in ((qo, q, qw), (ko, k, kw)):
        want, tol = forward64(x, w, eps, norm, cos, sin, interleaved)
        close(got, want, tol, "out")
    assert torch.equal(vo, v)
    gq, gk = randn(n, qh, d, dtype=dtype, seed=5), randn(n, kvh, d, dtype=dtype, seed=6)
    dq, dk, dqw, dkw = cq.qk_norm_rope_grad(gq, gk, q, k, *args, **where)
    for got, dw, g, x, w in ((dq, dqw, gq, q, qw), (dk, dkw, gk, k, kw)):
        want, tol, wwant, wtol = backward64(g, x, w, eps, norm, cos, sin, interleaved)
        close(got, want, tol, "dx")
        if norm:
            close(dw, wwant, wtol, "dw")
        else:
            assert dw is None


@TYPES
@pytest.mark.parametrize("interleaved", [False, True], ids=["halves", "neighbours"])
@pytest.mark.parametrize("n,qh,kvh,d,rot", [
    (1, 1, 1, 8, 8), (1, 32, 32, 128, 128), (3, 4, 2, 64, 32), (17, 8, 2, 64, 64), (5, 3, 1, 96, 48), (33, 5, 5, 80, 40), (2, 2, 1, 256, 256),
    (100, 2, 2, 40, 20), (7, 6, 3, 24, 6), (300, 8, 2, 128, 2), (4, 1, 1, 200, 198), (1200, 2, 1, 32, 32), (64, 40, 8, 128, 128)])
def test_shapes(n, qh, kvh, d, rot, interleaved, dtype):
    check(n, qh, kvh, d, rot, dtype, interleaved)


@TYPES
@pytest.mark.parametrize("case", [dict(norm=False), dict(rot=0), dict(rot=0, norm=False), dict(weights=False), dict(wtype=BF16), dict(eps=0.0),
                                  dict(eps=0.5), dict(pos=torch.int32)], ids=str)
def test_variants(case, dtype):
    check(**{**dict(n=50, qh=4, kvh=2, d=64, rot=64, dtype=dtype), **case})


@TYPES
@pytest.mark.parametrize("n,qh,kvh,d,rot", [(3, 300, 30, 32, 32), (700, 257, 1, 16, 16), (1, 600, 200, 64, 32)])
def test_many_heads(n, qh, kvh, d, rot, dtype):
    check(n, qh, kvh, d, rot, dtype)


@TYPES
@pytest.mark.parametrize("rot,interleaved", [(16, False), (20, False), (24, True)])
def test_values_only_move_and_what_does_not_turn_stays_apart(rot, interleaved, dtype):
    n, d = 9, 64
    q, k, v, positions, freqs = inputs(n, 4, 2, d, rot, dtype)
    q, k, v = q.clone(), k.clone(), v.clone()
    odd = torch.tensor([math.inf, -math.inf, math.nan, -0.0], device=DEV).to(dtype)
    v[:4, 0, 3], v[4:8, 1, 50] = odd, odd
    q[2, 1, rot + 1], q[2, 1, 63], k[5, 0, 40] = -math.inf, math.nan, math.inf
    qo, ko, vo = cq.qk_norm_rope(q, k, positions, freqs, norm=False, interleaved=interleaved, v=v)
    bits = torch.int16 if dtype == BF16 else torch.int32
    assert torch.equal(vo.view(bits), v.view(bits))
    assert torch.isfinite(qo[..., :rot]).all() and torch.isfinite(ko[..., :rot]).all()
    for out, x in ((qo, q), (ko, k)):
        assert torch.equal(out[..., rot:].nan_to_num(7.0), x[..., rot:].nan_to_num(7.0))
    dq, dk, _, _ = cq.qk_norm_rope_grad(q, k, q, k, positions, freqs, norm=False, interleaved=interleaved)
    for out, x in ((dq, q), (dk, k)):
        assert torch.isfinite(out[..., :rot]).all()
        assert torch.equal(out[..., rot:].nan_to_num(7.0), x[..., rot:].nan_to_num(7.0))


@TYPES
def test_offsets_past_32_bits(dtype):
    # a cache with rows 2^22 values apart, 5 to 10 GB
    rows, stride = 1200, 1 << 22
    q, k, v, positions, freqs = inputs(5, 2, 2, 64, 64, dtype)
    buf = torch.zeros(rows * stride, dtype=dtype, device=DEV)
    cache_k, cache_v = buf.as_strided((rows, 2, 64), (stride, 64, 1)), buf.as_strided((rows, 2, 64), (stride, 64, 1), 128)
    slots = torch.tensor([1199, 3, 700, -1, 1150], device=DEV)
    cq.qk_norm_rope(q, k, positions, freqs, v=v, slots=slots, k_out=cache_k, v_out=cache_v)
    _, want, _ = cq.qk_norm_rope(q, k, positions, freqs, v=v)
    for i, slot in enumerate(slots.tolist()):
        if slot >= 0:
            assert torch.equal(cache_k[slot], want[i]) and torch.equal(cache_v[slot], v[i])
    # the same rows as inputs of the gradient
    at = slots[slots >= 0].sort().values
    g = buf.as_strided((rows, 2, 64), (stride, 64, 1))
    x = torch.zeros_like(cache_k.contiguous()) + 1
    dq, dk, _, _ = cq.qk_norm_rope_grad(g, g, x, x, torch.arange(rows, device=DEV), freqs, norm=False)
    small, _, _, _ = cq.qk_norm_rope_grad(g[at], g[at], x[at], x[at], at, freqs, norm=False)
    assert torch.equal(dq[at], small) and torch.equal(dk[at], small) and torch.count_nonzero(dq) == torch.count_nonzero(small)
    del buf


@TYPES
def test_many_tokens(dtype):
    check(20000, 4, 1, 64, 64, dtype)


@TYPES
def test_far_and_negative_positions(dtype):
    q, k, _, _, freqs = inputs(6, 2, 1, 64, 64, dtype)
    positions = torch.tensor([0, -1, 1 << 20, -(1 << 30), (1 << 31) - 1, 1 << 40], device=DEV)
    qo, ko = cq.qk_norm_rope(q, k, positions, freqs)
    cos, sin = angles(positions, freqs)
    # the angle itself is off by a few steps of float64
    off = 4 * 2.0 ** -53 * (positions.double().abs()[:, None] * freqs.double()).max(-1).values[:, None, None]
    for got, x in ((qo, q), (ko, k)):
        want, tol = forward64(x, None, 1e-6, True, cos, sin, False)
        close(got, want, tol + off * 2 * want.abs().amax(-1, keepdim=True), "out")


@TYPES
@pytest.mark.parametrize("slot", [torch.int32, torch.int64])
def test_cache(slot, dtype):
    n, kvh, d, rows = 40, 2, 64, 100
    q, k, v, positions, freqs = inputs(n, 4, kvh, d, d, dtype)
    gen = torch.Generator(device=DEV)
    gen.manual_seed(1)
    slots = torch.randperm(rows, generator=gen, device=DEV)[:n]
    slots[3], slots[5], slots[7] = -1, rows, 1 << 30  # padding: not written
    slots = slots.to(slot)
    cache = torch.full((2, rows, kvh, d), 9.0, dtype=dtype, device=DEV)
    qo, ko, vo = cq.qk_norm_rope(q, k, positions, freqs, v=v, slots=slots, k_out=cache[0], v_out=cache[1])
    want_q, want_k = cq.qk_norm_rope(q, k, positions, freqs)
    assert ko.data_ptr() == cache[0].data_ptr() and vo.data_ptr() == cache[1].data_ptr()
    want = torch.full_like(cache, 9.0)
    keep = (slots >= 0) & (slots < rows)
    want[0, slots[keep].long()], want[1, slots[keep].long()] = want_k[keep], v[keep]
    assert torch.equal(qo, want_q) and torch.equal(cache, want)


@TYPES
@pytest.mark.parametrize("rot,interleaved", [(64, False), (40, False), (64, True)])
def test_in_place_and_strided(rot, interleaved, dtype):
    q, k, v, positions, freqs = inputs(70, 4, 2, 64, rot, dtype)
    w = 1 + randn(64, scale=0.2)
    want = cq.qk_norm_rope(q, k, positions, freqs, w, w, interleaved=interleaved)
    hf = [t.transpose(0, 1).contiguous().transpose(0, 1) for t in (q, k)]  # heads first
    for a, b in zip(cq.qk_norm_rope(*hf, positions, freqs, w, w, interleaved=interleaved), want):
        assert torch.equal(a, b)
    g = [randn(70, 4, 64, dtype=dtype, seed=8), randn(70, 2, 64, dtype=dtype, seed=9)]
    grads = cq.qk_norm_rope_grad(*g, q, k, positions, freqs, w, w, interleaved=interleaved)
    again = cq.qk_norm_rope_grad(*g, q, k, positions, freqs, w, w, interleaved=interleaved, dq=g[0], dk=g[1])
    assert again[0].data_ptr() == g[0].data_ptr()
    for a, b in zip(again, grads):
        assert torch.equal(a, b)
    kept = v.clone()
    out = cq.qk_norm_rope(q, k, positions, freqs, w, w, interleaved=interleaved, v=v, q_out=q, k_out=k, v_out=v)
    assert out[0].data_ptr() == q.data_ptr() and torch.equal(q, want[0]) and torch.equal(k, want[1]) and torch.equal(v, kept)


@TYPES
def test_zero_rows_and_empty_calls(dtype):
    q, k, _, positions, freqs = inputs(4, 2, 1, 64, 64, dtype)
    z = torch.zeros_like(q)
    qo, ko = cq.qk_norm_rope(z, k, positions, freqs, eps=1e-6)
    assert (qo == 0).all()
    dq, _, dqw, _ = cq.qk_norm_rope_grad(q.contiguous(), k.contiguous(), z, k, positions, freqs)
    assert torch.isfinite(dq).all() and (dqw == 0).all()
    out = cq.qk_norm_rope(q[:0], k[:0], positions[:0], freqs)
    assert out[0].shape == (0, 2, 64) and out[1].shape == (0, 1, 64)
    grads = cq.qk_norm_rope_grad(q[:0], k[:0], q[:0], k[:0], positions[:0], freqs)
    assert (grads[2] == 0).all() and (grads[3] == 0).all()


def test_differences():
    n, d = 9, 24
    q, k, _, positions, freqs = inputs(n, 3, 1, d, 12, F32)
    qw, kw = 1 + randn(d, scale=0.2), 1 + randn(d, scale=0.2, seed=1)
    g = randn(n, 3, d, seed=2), randn(n, 1, d, seed=3)
    dq, dk, dqw, dkw = cq.qk_norm_rope_grad(*g, q, k, positions, freqs, qw, kw)
    cos, sin = angles(positions, freqs)
    h = 1e-4  # differences: off by h^2 of a third derivative, some 1e-7 of the gradient
    for dx, dw, x, w, gg in ((dq, dqw, q, qw, g[0]), (dk, dkw, k, kw, g[1])):
        tx, tw = randn(*x.shape, seed=7).double(), randn(d, seed=8).double()

        def loss(step):
            out, _ = forward64(x.double() + step * tx, w.double() + step * tw, 1e-6, True, cos, sin, False)
            return (out * gg.double()).sum()

        slope = (loss(h) - loss(-h)) / (2 * h)
        got = (dx.double() * tx).sum() + (dw.double() * tw).sum()
        size = (dx.double() * tx).abs().sum() + (dw.double() * tw).abs().sum()
        assert (got - slope).abs() <= 1e-5 * size


@TYPES
def test_same_bits_streams_and_graphs(dtype):
    q, k, v, positions, freqs = inputs(900, 8, 2, 64, 64, dtype)
    w = 1 + randn(64, scale=0.2)
    g = randn(900, 8, 64, dtype=dtype, seed=8), randn(900, 2, 64, dtype=dtype, seed=9)

    def step(**kw):
        return (*cq.qk_norm_rope(q, k, positions, freqs, w, w, v=v, **kw), *cq.qk_norm_rope_grad(*g, q, k, positions, freqs, w, w, **kw))

    want = step()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = step(stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for turn_ in range(3):
        q.copy_(randn(900, 8, 64, dtype=dtype, seed=50 + turn_))
        positions += 11
        want = step()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_refusals():
    q, k, v, positions, freqs = inputs(10, 4, 2, 64, 64, F32)
    g = q.contiguous(), k.contiguous()
    for bad in (lambda: cq.qk_norm_rope(q.half(), k.half(), positions, freqs), lambda: cq.qk_norm_rope(q, k, positions.float(), freqs),
                lambda: cq.qk_norm_rope(q, k, positions, freqs.double())):
        with pytest.raises(TypeError):
            bad()
    cache = torch.empty(20, 2, 64, device=DEV)
    for bad in (lambda: cq.qk_norm_rope(q, k[:5], positions, freqs), lambda: cq.qk_norm_rope(q, k, positions[:5], freqs),
                lambda: cq.qk_norm_rope(q, k, None, freqs), lambda: cq.qk_norm_rope(q, k, positions, freqs, freqs),
                lambda: cq.qk_norm_rope(q, k, positions, freqs, q_weight=q[0, 0], norm=False),
                lambda: cq.qk_norm_rope(q, k, positions, freqs, slots=positions), lambda: cq.qk_norm_rope(q, k, positions, freqs, v=v, slots=positions, k_out=cache),
                lambda: cq.qk_norm_rope(q, k, positions, freqs, slots=positions[:3], k_out=cache), lambda: cq.qk_norm_rope(q.cpu(), k, positions, freqs),
                lambda: cq.qk_norm_rope(q, k, positions, freqs, v_out=cache), lambda: cq.qk_norm_rope_grad(q, k, q, k[:, :1], positions, freqs)):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: cq.qk_norm_rope(q[..., :32], k[..., :32], positions, freqs), lambda: cq.qk_norm_rope(q, k, positions, freqs, eps=-1.0),
                lambda: cq.qk_norm_rope(q, k, positions, freqs, q_out=k.expand(10, 2, 64).repeat(1, 2, 1)[:1].expand(10, 4, 64)),
                lambda: cq.qk_norm_rope(q[..., :60], k[..., :60]), lambda: cq.qk_norm_rope(q, k, positions, freqs, k_out=k, slots=positions),
                lambda: cq.qk_norm_rope(randn(2, 1, 264), randn(2, 1, 264)),
                lambda: cq.qk_norm_rope_grad(*g, q, k, positions, freqs, dq=q),
                lambda: cq.qk_norm_rope_grad(*g, q, k, positions, freqs, workspace=torch.empty(8, dtype=torch.uint8, device=DEV))):
        with pytest.raises(cq.CQError):
            bad()
