"""Attention over packed sequences and caches, and its gradient, against
float64 (attention_reference.py: the bounds)."""

import math

import pytest
import torch

import rotated_codebook_bit_amd as cq
from attention_reference import attend, close

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16
TYPES = pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
DEV = "cuda"


def randn(*shape, dtype=F32, seed=0, scale=1.0):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed + 1000 * len(shape) + sum(shape))
    return (torch.randn(shape, generator=gen, device=DEV) * scale).to(dtype)


def starts(lens, dtype=torch.int32, at=0):
    out = [at]
    for n in lens:
        out.append(out[-1] + n)
    return torch.tensor(out, dtype=dtype, device=DEV)


def check_packed(lens, heads, kv_heads, d, dtype, causal=True, scale=None, grad=True, index=torch.int32, spread=1.0):
    """lens: (queries, keys) per sequence; q, k, v are parts of one tensor each."""
    m, n = sum(a for a, _ in lens), sum(b for _, b in lens)
    q = randn(m, heads + 1, d, dtype=dtype, seed=1, scale=spread)[:, 1:]
    kv = randn(n, 2 * kv_heads, d, dtype=dtype, seed=2)
    k, v = kv[:, :kv_heads], kv[:, kv_heads:]
    dout = randn(m, heads, d, dtype=dtype, seed=3)
    scale = 1 / math.sqrt(d) if scale is None else scale
    where = dict(q_starts=starts([a for a, _ in lens], index), k_starts=starts([b for _, b in lens], index), causal=causal, scale=scale)
    out, lse = cq.attention(q, k, v, **where)
    got = {"out": out, "lse": lse}
    if grad:
        got.update(zip(("dq", "dk", "dv"), cq.attention_grad(dout, q, k, v, out, lse, **where)))
    i = j = 0
    for a, b in lens:
        want, tol = attend(q[i:i + a], k[j:j + b], v[j:j + b], scale, causal, dout[i:i + a])
        for name, t in got.items():
            rows = slice(j, j + b) if name in ("dk", "dv") else slice(i, i + a)
            close(t[rows], want[name], tol[name], (name, a, b))
        i, j = i + a, j + b


LENS = {
    "one": [(1, 1)],
    "square": [(64, 64)],
    "ragged": [(5, 5), (1, 1), (0, 0), (33, 33), (130, 130), (127, 127), (129, 129)],
    "longer_keys": [(3, 70), (64, 200), (40, 41), (1, 129)],
    "empty_rows": [(5, 2), (130, 3), (4, 0), (0, 7), (70, 66)],
    "many": [(k % 7, k % 7) for k in range(150)],
}


@TYPES
@pytest.mark.parametrize("lens", LENS.values(), ids=LENS.keys())
@pytest.mark.parametrize("heads,kv_heads,d", [(8, 2, 64), (4, 4, 128)])
def test_packed(lens, heads, kv_heads, d, dtype):
    check_packed(lens, heads, kv_heads, d, dtype)


@TYPES
@pytest.mark.parametrize("heads,kv_heads", [(1, 1), (6, 2), (5, 1), (3, 3), (16, 1)])
@pytest.mark.parametrize("d", [8, 40, 72, 96, 120])
def test_head_layouts(heads, kv_heads, d, dtype):
    check_packed([(37, 37), (2, 2), (100, 101)], heads, kv_heads, d, dtype)


@TYPES
@pytest.mark.parametrize("lens", [LENS["ragged"], LENS["longer_keys"], LENS["empty_rows"]], ids=["ragged", "longer_keys", "empty_rows"])
def test_not_causal(lens, dtype):
    check_packed(lens, 4, 2, 64, dtype, causal=False)


@TYPES
def test_long_sequence_and_int64_starts(dtype):
    check_packed([(700, 1300), (257, 257)], 4, 1, 128, dtype, index=torch.int64)


@pytest.mark.parametrize("causal", [True, False], ids=["causal", "full"])
@pytest.mark.parametrize("heads,kv_heads,d", [(8, 2, 64), (5, 1, 40), (3, 3, 64), (4, 2, 128), (3, 1, 72)])
@pytest.mark.parametrize("lens", [[(700, 700), (1, 1), (300, 300)], [(513, 600), (0, 500), (200, 900)], [(1037, 1037)], [(600, 300), (64, 700)]],
                         ids=["prompts", "continued", "one", "empty_rows"])
def test_float_prompts_of_long_sequences(lens, heads, kv_heads, d, causal):
    check_packed(lens, heads, kv_heads, d, F32, causal=causal)


@TYPES
@pytest.mark.parametrize("count", [64, 65, 130])
def test_many_sequences_of_several_tiles(count, dtype):
    # around the 64 sequences that one wave orders at once
    check_packed([(k * 53 % 170, k * 53 % 170 + k % 3) for k in range(count)], 4, 2, 64, dtype)


@TYPES
def test_no_sequences(dtype):
    q, k, v = randn(6, 4, 64, dtype=dtype), randn(9, 2, 64, dtype=dtype), randn(9, 2, 64, dtype=dtype)
    torch.full((1 << 20,), 7.0, device=DEV)  # what new tensors would hold otherwise
    out, lse = cq.attention(q, k, v, sequences=0)
    grads = cq.attention_grad(q.clone(), q, k, v, out, lse, sequences=0)
    for t in (out, lse, *grads):
        assert (t == 0).all()


@TYPES
def test_large_scores(dtype):
    # scores of up to some hundred: one key takes nearly all of a row, the reference moves often
    check_packed([(150, 150), (20, 300)], 2, 1, 64, dtype, spread=30.0, scale=0.25)


@TYPES
def test_equal_parts_need_no_starts(dtype):
    q, k, v, dout = (randn(3 * n, h, 64, dtype=dtype, seed=s) for n, h, s in ((50, 4, 1), (60, 2, 2), (60, 2, 3), (50, 4, 4)))
    out, lse = cq.attention(q, k, v, sequences=3)
    grads = cq.attention_grad(dout, q, k, v, out, lse, sequences=3)
    same, lse2 = cq.attention(q, k, v, q_starts=starts([50] * 3), k_starts=starts([60] * 3))
    assert torch.equal(out, same) and torch.equal(lse, lse2)
    for a, b in zip(grads, cq.attention_grad(dout, q, k, v, out, lse, q_starts=starts([50] * 3), k_starts=starts([60] * 3))):
        assert torch.equal(a, b)


@TYPES
@pytest.mark.parametrize("new", [1, 2, 5])
@pytest.mark.parametrize("heads,kv_heads,d", [(8, 2, 64), (32, 8, 128), (6, 6, 80), (5, 1, 96)])
def test_cache(heads, kv_heads, d, new, dtype):
    cap, lens = 1400, [1400, new, 0, 1399, 700, 33, 1, 64, 129]
    b = len(lens)
    q = randn(b * new, heads, d, dtype=dtype)
    k, v = randn(b * cap, kv_heads, d, dtype=dtype, seed=1), randn(b * cap, kv_heads, d, dtype=dtype, seed=2)
    for i, n in enumerate(lens):  # what lies behind the length is never read
        k[i * cap + n:(i + 1) * cap] = math.nan
        v[i * cap + n:(i + 1) * cap] = math.nan
    out, lse = cq.attention(q, k, v, sequences=b, k_lens=torch.tensor(lens, device=DEV))
    for i, n in enumerate(lens):
        rows, keys = slice(i * new, (i + 1) * new), slice(i * cap, i * cap + n)
        want, tol = attend(q[rows], k[keys], v[keys], 1 / math.sqrt(d), True)
        close(out[rows], want["out"], tol["out"], ("out", n))
        close(lse[rows], want["lse"], tol["lse"], ("lse", n))


@TYPES
@pytest.mark.parametrize("new,lens", [(20, [3000, 1000, 20]), (64, [2900]), (200, [4000]), (37, [3000] * 4)])
def test_new_tokens_over_a_long_cache(new, lens, dtype):
    cap, heads, kv_heads, d, b = max(lens), 8, 2, 128, len(lens)
    q = randn(b * new, heads, d, dtype=dtype)
    k, v = randn(b * cap, kv_heads, d, dtype=dtype, seed=1), randn(b * cap, kv_heads, d, dtype=dtype, seed=2)
    out, lse = cq.attention(q, k, v, sequences=b, k_lens=torch.tensor(lens, device=DEV))
    for i, n in enumerate(lens):
        rows, keys = slice(i * new, (i + 1) * new), slice(i * cap, i * cap + n)
        want, tol = attend(q[rows], k[keys], v[keys], 1 / math.sqrt(d), True)
        close(out[rows], want["out"], tol["out"], ("out", n))
        close(lse[rows], want["lse"], tol["lse"], ("lse", n))


@TYPES
def test_one_long_cache_of_one_token(dtype):
    n, heads, d = 40000, 4, 128
    q, k, v = randn(1, heads, d, dtype=dtype), randn(n, 1, d, dtype=dtype, seed=1), randn(n, 1, d, dtype=dtype, seed=2)
    out, lse = cq.attention(q, k, v)
    want, tol = attend(q, k, v, 1 / math.sqrt(d), True)
    close(out, want["out"], tol["out"], "out")
    close(lse, want["lse"], tol["lse"], "lse")


@TYPES
def test_shared_prefix(dtype):
    # Two sequences whose keys overlap: a prompt's rows, then each one's view of them.
    q, k, v = randn(2, 4, 64, dtype=dtype), randn(300, 2, 64, dtype=dtype, seed=1), randn(300, 2, 64, dtype=dtype, seed=2)
    out, _ = cq.attention(q, k, v, q_starts=starts([1, 1]), k_starts=torch.tensor([0, 100], dtype=torch.int32, device=DEV),
                          k_lens=torch.tensor([250, 200], dtype=torch.int32, device=DEV))
    for i, (a, n) in enumerate([(0, 250), (100, 200)]):
        want, tol = attend(q[i:i + 1], k[a:a + n], v[a:a + n], 1 / 8, True)
        close(out[i:i + 1], want["out"], tol["out"], i)


@TYPES
@pytest.mark.parametrize("m", [3, 200])
def test_offsets_past_32_bits(m, dtype):
    # Rows of a cache more than 2^32 bytes in, by a row stride and by a start.
    rows = 900
    stride = 1 << 22
    big = torch.empty((rows - 1) * stride + 128, dtype=dtype, device=DEV)
    k = torch.as_strided(big, (rows, 1, 64), (stride, 64, 1))
    v = torch.as_strided(big, (rows, 1, 64), (stride, 64, 1), 64)
    k.copy_(randn(rows, 1, 64, dtype=dtype, seed=1))
    v.copy_(randn(rows, 1, 64, dtype=dtype, seed=2))
    assert (rows - 210) * stride * big.element_size() > 1 << 32
    q = randn(m, 2, 64, dtype=dtype)
    at, n = rows - 205, 203
    out, lse = cq.attention(q, k, v, k_starts=torch.tensor([at], device=DEV), k_lens=torch.tensor([n], device=DEV))
    want, tol = attend(q, k[at:at + n], v[at:at + n], 1 / 8, True)
    close(out, want["out"], tol["out"], "out")
    close(lse, want["lse"], tol["lse"], "lse")


@TYPES
@pytest.mark.parametrize("new", [1, 90])
def test_rows_of_no_sequence_are_left(new, dtype):
    lens = [new, 0, new + 2]
    total = sum(lens) + 4
    q, k, v, dout = (randn(total, h, 64, dtype=dtype, seed=h) for h in (4, 2, 2, 4))
    at = starts(lens, at=3)
    outs = [torch.full_like(q, 7), torch.full((total, 4), 7.0, device=DEV), torch.full_like(q, 7), torch.full_like(k, 7), torch.full_like(v, 7)]
    k[:3] = math.nan
    v[-1:] = math.nan
    where = dict(q_starts=at, k_starts=at)
    out, lse = cq.attention(q, k, v, out=outs[0], lse=outs[1], **where)
    cq.attention_grad(dout, q, k, v, out, lse, dq=outs[2], dk=outs[3], dv=outs[4], **where)
    for t in outs:
        assert (t[:3] == 7).all() and (t[-1:] == 7).all()
        assert torch.isfinite(t[3:-1]).all() and (t[3:-1] != 7).any()
    # Allocated by the call: zeros.
    out2, lse2 = cq.attention(q, k, v, **where)
    grads = cq.attention_grad(dout, q, k, v, out, lse, **where)
    for t, u in zip((out2, lse2, *grads), outs):
        assert (t[:3] == 0).all() and (t[-1:] == 0).all() and torch.equal(t[3:-1], u[3:-1])


@TYPES
@pytest.mark.parametrize("rows", [2, 200])
def test_starts_outside_the_tensors(rows, dtype):
    """Whatever the arrays hold, no access leaves the tensors: cut starts and
    lengths give what they would give if they were in range."""
    q, k, v = randn(rows, 2, 64, dtype=dtype), randn(50, 1, 64, dtype=dtype, seed=1), randn(50, 1, 64, dtype=dtype, seed=2)
    bad = torch.tensor([-5, 10 ** 6], device=DEV)
    out, _ = cq.attention(q, k, v, q_starts=bad, k_starts=torch.tensor([-3], device=DEV), k_lens=torch.tensor([10 ** 9], device=DEV))
    same, _ = cq.attention(q, k, v)
    assert torch.equal(out, same)
    out, lse = cq.attention(q, k, v, k_starts=torch.tensor([10 ** 6], device=DEV), k_lens=torch.tensor([5], device=DEV))
    assert (out == 0).all() and (lse == -math.inf).all()
    out, lse = cq.attention(q, k, v, k_lens=torch.tensor([-4], device=DEV))
    assert (out == 0).all() and (lse == -math.inf).all()


@TYPES
def test_values_that_are_not_finite_stay_in_their_sequence(dtype):
    lens = [70, 65, 90]
    q, k, v = randn(225, 4, 64, dtype=dtype), randn(225, 2, 64, dtype=dtype, seed=1), randn(225, 2, 64, dtype=dtype, seed=2)
    clean, _ = cq.attention(q, k, v, q_starts=starts(lens), k_starts=starts(lens))
    k[80], v[100], q[75] = math.nan, math.inf, math.nan
    out, _ = cq.attention(q, k, v, q_starts=starts(lens), k_starts=starts(lens))
    assert torch.equal(out[:70], clean[:70]) and torch.equal(out[135:], clean[135:])
    assert not torch.isfinite(out[134]).all()


@TYPES
def test_empty_calls(dtype):
    for m, n in ((0, 0), (0, 5), (6, 0)):
        q, k, v = randn(m, 4, 64, dtype=dtype), randn(n, 2, 64, dtype=dtype), randn(n, 2, 64, dtype=dtype)
        out, lse = cq.attention(q, k, v)
        dq, dk, dv = cq.attention_grad(q.clone(), q, k, v, out, lse)
        torch.cuda.synchronize()
        assert (out == 0).all() and (lse == -math.inf).all()
        assert (dq == 0).all() and (dk == 0).all() and (dv == 0).all()


@TYPES
def test_heads_first_layout_and_gradients_into_one_tensor(dtype):
    m, heads, kvh, d = 150, 4, 2, 64
    q, k, v, dout = (randn(h, m, d, dtype=dtype, seed=s).transpose(0, 1) for s, h in enumerate((heads, kvh, kvh, heads)))
    out, lse = cq.attention(q, k, v, out=torch.empty_like(q))
    assert out.stride() == q.stride()
    plain, lse2 = cq.attention(q.contiguous(), k.contiguous(), v.contiguous())
    assert torch.equal(out, plain) and torch.equal(lse, lse2)
    dqkv = torch.empty((m, heads + 2 * kvh, d), dtype=dtype, device=DEV)
    parts = dqkv.split([heads, kvh, kvh], 1)
    cq.attention_grad(dout, q, k, v, out, lse, dq=parts[0], dk=parts[1], dv=parts[2])
    for a, b in zip(parts, cq.attention_grad(dout.contiguous(), q.contiguous(), k.contiguous(), v.contiguous(), plain, lse)):
        assert torch.equal(a, b)
    # [q, k, v] of each head side by side
    mixed = torch.empty((m, heads, 3, d), dtype=dtype, device=DEV)
    k4, v4 = k.repeat_interleave(2, 1), v.repeat_interleave(2, 1)
    cq.attention_grad(dout, q, k4, v4, out, lse, dq=mixed[:, :, 0], dk=mixed[:, :, 1], dv=mixed[:, :, 2])
    for a, b in zip(mixed.unbind(2), cq.attention_grad(dout, q, k4, v4, out, lse)):
        assert torch.equal(a, b)


@TYPES
def test_broadcast_keys(dtype):
    # One head's keys for all heads, by a stride of 0, against the same keys copied.
    q, one = randn(70, 4, 64, dtype=dtype), randn(70, 1, 64, dtype=dtype, seed=1)
    k = one.expand(70, 4, 64)
    a, _ = cq.attention(q, k, k)
    b, _ = cq.attention(q, k.contiguous(), k.contiguous())
    assert torch.equal(a, b)


@TYPES
def test_differences(dtype):
    """The gradient along a direction against differences of the definition."""
    lens = [(40, 45), (70, 70)]
    m, n = 110, 115
    q, k, v = randn(m, 4, 40, dtype=dtype), randn(n, 2, 40, dtype=dtype, seed=1), randn(n, 2, 40, dtype=dtype, seed=2)
    dout = randn(m, 4, 40, dtype=dtype, seed=3)
    where = dict(q_starts=starts([40, 70]), k_starts=starts([45, 70]), scale=0.2)
    out, lse = cq.attention(q, k, v, **where)
    grads = cq.attention_grad(dout, q, k, v, out, lse, **where)
    dirs = [randn(*t.shape, seed=5 + i).double() for i, t in enumerate((q, k, v))]

    def loss(step):
        total, i, j = 0.0, 0, 0
        for a, b in lens:
            # float64 inputs: attend() takes them as float32's bounds, which are not used here
            w = attend64(q[i:i + a].double() + step * dirs[0][i:i + a], k[j:j + b].double() + step * dirs[1][j:j + b],
                         v[j:j + b].double() + step * dirs[2][j:j + b], 0.2)
            total = total + (w * dout[i:i + a].double()).sum()
            i, j = i + a, j + b
        return total

    h = 1e-4  # the differences' own error is about h^2 of the loss's third derivative, 1e-8 of the gradient
    slope = (loss(h) - loss(-h)) / (2 * h)
    got = sum((g.double() * d).sum() for g, d in zip(grads, dirs))
    tol, i, j = 1e-6 * slope.abs(), 0, 0
    for a, b in lens:
        _, t = attend(q[i:i + a], k[j:j + b], v[j:j + b], 0.2, True, dout[i:i + a])
        tol = tol + (t["dq"] * dirs[0][i:i + a].abs()).sum() + (t["dk"] * dirs[1][j:j + b].abs()).sum() + (t["dv"] * dirs[2][j:j + b].abs()).sum()
        i, j = i + a, j + b
    assert (got - slope).abs() <= tol, (float(got), float(slope), float(tol))


def attend64(q, k, v, scale):
    m, n, g = q.shape[0], k.shape[0], q.shape[1] // k.shape[1]
    q, k, v = q.transpose(0, 1), k.transpose(0, 1).repeat_interleave(g, 0), v.transpose(0, 1).repeat_interleave(g, 0)
    x = scale * torch.matmul(q, k.transpose(1, 2).contiguous())
    seen = torch.arange(n, device=q.device)[None] <= torch.arange(m, device=q.device)[:, None] + n - m
    return torch.matmul(torch.softmax(x.masked_fill(~seen, -math.inf), -1), v).transpose(0, 1)


@TYPES
def test_same_bits_on_every_run(dtype):
    q, k, v, dout = (randn(500, h, 128, dtype=dtype, seed=h) for h in (8, 2, 2, 8))
    at = starts([300, 200])
    runs = []
    for _ in range(3):
        out, lse = cq.attention(q, k, v, q_starts=at, k_starts=at)
        one, _ = cq.attention(q[:2], k, v, sequences=2)
        runs.append((out, lse, one, *cq.attention_grad(dout, q, k, v, out, lse, q_starts=at, k_starts=at)))
    for r in runs[1:]:
        assert all(torch.equal(a, b) for a, b in zip(r, runs[0]))


@TYPES
def test_another_stream_and_graphs(dtype):
    q, k, v, dout = (randn(260, h, 64, dtype=dtype, seed=h) for h in (8, 2, 2, 8))
    new = randn(2, 8, 64, dtype=dtype, seed=20)
    lens = torch.tensor([130, 90], dtype=torch.int32, device=DEV)

    def step():
        out, lse = cq.attention(q, k, v, sequences=2)
        one, _ = cq.attention(new, k, v, sequences=2, k_lens=lens)
        return (out, lse, one, *cq.attention_grad(dout, q, k, v, out, lse, sequences=2))

    want = step()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    out, lse = cq.attention(q, k, v, sequences=2, stream=side)
    grads = cq.attention_grad(dout, q, k, v, out, lse, sequences=2, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    for a, b in zip((out, lse, *grads), (want[0], want[1], *want[3:])):
        assert torch.equal(a, b)
    with torch.cuda.stream(side):
        step()
        graph, other = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            got = step()
        with torch.cuda.graph(other, stream=side):
            got2 = step()
    torch.cuda.current_stream().wait_stream(side)
    for turn in range(3):
        q.copy_(randn(260, 8, 64, dtype=dtype, seed=30 + turn))
        lens.copy_(torch.tensor([40 + turn, 129], dtype=torch.int32))
        want = step()
        graph.replay()
        other.replay()
        torch.cuda.synchronize()
        for a, b, c in zip(got, got2, want):
            assert torch.equal(a, c) and torch.equal(b, c)


def test_refusals():
    q, k, v = randn(10, 4, 64), randn(10, 2, 64), randn(10, 2, 64)
    out, lse = cq.attention(q, k, v)
    at = starts([4, 6])
    for bad in (lambda: cq.attention(q.half(), k.half(), v.half()), lambda: cq.attention(q, k, v, q_starts=at.float(), k_starts=at),
                lambda: cq.attention(q, k, v, q_starts=at, k_starts=at.long())):
        with pytest.raises(TypeError):
            bad()
    for bad in (lambda: cq.attention(q, k[:5], v), lambda: cq.attention(q, k.bfloat16(), v), lambda: cq.attention(q.cpu(), k, v),
                lambda: cq.attention(q[0], k, v), lambda: cq.attention(q, k, v, sequences=3, q_starts=at),
                lambda: cq.attention(q, k, v, q_starts=at, k_starts=at[:2]), lambda: cq.attention(q, k, v, out=out[:5]),
                lambda: cq.attention(q, k, v, lse=lse[:, :2]), lambda: cq.attention(q.transpose(1, 2), k, v),
                lambda: cq.attention_grad(out, q, k, v, out, lse[:5])):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: cq.attention(q, k, v, sequences=3), lambda: cq.attention(q, k, v, scale=0.0), lambda: cq.attention(q, k, v, scale=-1.0),
                lambda: cq.attention(q, k, v, scale=math.nan), lambda: cq.attention(q[:, :3], k, v), lambda: cq.attention(q, k, v, out=q),
                lambda: cq.attention(q[..., :60], k[..., :60], v[..., :60]), lambda: cq.attention(q[..., 2:58], k[..., :56], v[..., :56]),
                lambda: cq.attention(randn(4, 2, 136), randn(4, 2, 136), randn(4, 2, 136)),
                lambda: cq.attention(q, k, v, out=q[:1].expand(10, 4, 64)),
                lambda: cq.attention_grad(out, q, k, v, out, lse, dq=q), lambda: cq.attention_grad(out, q, k, v, out, lse, dk=k, dv=k),
                lambda: cq.attention_grad(out, q, k, v, out, lse, workspace=torch.empty(16, dtype=torch.uint8, device=DEV))):
        with pytest.raises(cq.CQError):
            bad()
