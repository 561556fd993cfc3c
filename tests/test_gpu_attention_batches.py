"""Attention over batches of many sequences and of very different lengths,
against float64 (attention_reference.py: the bounds)."""

import math

import pytest
import torch

import rotated_codebook_bit_amd as cq
from attention_reference import attend, close

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16
TYPES = pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
DEV = "cuda"


def randn(*shape, dtype=F32, seed=0):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed + 1000 * len(shape) + sum(shape))
    return torch.randn(shape, generator=gen, device=DEV).to(dtype)


def starts(lens):
    return torch.tensor([0, *lens], dtype=torch.int32, device=DEV).cumsum(0, dtype=torch.int32)


def check(q, k, v, out, lse, q_lens, k_lens, k_at, some, grads=None, dout=None):
    """The sequences `some`, of q_lens queries one after another and k_lens keys from k_at on."""
    q_at = starts(q_lens).tolist()
    for i in some:
        rows, keys = slice(q_at[i], q_at[i] + q_lens[i]), slice(k_at[i], k_at[i] + k_lens[i])
        want, tol = attend(q[rows], k[keys], v[keys], 1 / math.sqrt(q.shape[2]), True, None if dout is None else dout[rows])
        close(out[rows], want["out"], tol["out"], ("out", i))
        close(lse[rows], want["lse"], tol["lse"], ("lse", i))
        if grads is not None:
            for name, t, at in zip(("dq", "dk", "dv"), grads, (rows, keys, keys)):
                close(t[at], want[name], tol[name], (name, i))


@TYPES
@pytest.mark.parametrize("heads,kv_heads,d", [(4, 4, 64), (8, 2, 128)])
def test_hundreds_of_short_sequences(heads, kv_heads, d, dtype):
    lens = [1 + k * 37 % 17 for k in range(400)]
    lens[123] = 700
    n, at = sum(lens), starts(lens)
    qkv = randn(n, heads + 2 * kv_heads, d, dtype=dtype)
    q, k, v = qkv.split([heads, kv_heads, kv_heads], 1)
    dout = randn(n, heads, d, dtype=dtype, seed=1)
    out, lse = cq.attention(q, k, v, q_starts=at, k_starts=at)
    grads = cq.attention_grad(dout, q, k, v, out, lse, q_starts=at, k_starts=at)
    check(q, k, v, out, lse, lens, lens, at.tolist(), [0, 1, 2, 63, 64, 122, 123, 124, 399], grads, dout)


def test_thousands_of_short_sequences():
    """More tiles of rows than the grid would hold in several pieces each."""
    lens = [1 + k * 37 % 51 for k in range(5000)]
    n, at = sum(lens), starts(lens)
    q, k, v = (randn(n, 32, 8, dtype=BF16, seed=s) for s in range(3))
    out, lse = cq.attention(q, k, v, q_starts=at, k_starts=at)
    assert torch.isfinite(out).all() and torch.isfinite(lse).all()
    check(q, k, v, out, lse, lens, lens, at.tolist(), [0, 1, 77, 2500, 4998, 4999])


@TYPES
@pytest.mark.parametrize("heads,kv_heads,d", [(8, 2, 64), (16, 4, 128)])
def test_ragged_caches_in_both_forms(heads, kv_heads, d, dtype):
    """A token each over caches of very different lengths, by the parts of one
    tensor and by starts, in order and not: the same keys give the same results within their bounds."""
    cap, lens = 6000, [6000, 1, 0, 2047, 2048, 2049, 4097, 100, 65, 5999]
    b = len(lens)
    q = randn(b, heads, d, dtype=dtype)
    k, v = randn(b * cap, kv_heads, d, dtype=dtype, seed=1), randn(b * cap, kv_heads, d, dtype=dtype, seed=2)
    order = [3, 0, 9, 1, 8, 2, 7, 4, 6, 5]  # of the parts
    k_lens = torch.tensor(lens, dtype=torch.int32, device=DEV)
    for at, where in (([i * cap for i in range(b)], dict(sequences=b)), ([i * cap for i in order], dict(sequences=b)),
                      ([i * cap for i in order], dict(q_starts=starts([1] * b)))):
        if at[0]:
            where["k_starts"] = torch.tensor(at, dtype=torch.int32, device=DEV)
        out, lse = cq.attention(q, k, v, k_lens=k_lens, **where)
        check(q, k, v, out, lse, [1] * b, lens, at, range(b))


@TYPES
def test_one_long_sequence_among_single_tokens(dtype):
    """The long one has most of the keys, which the mean does not show."""
    lens = [9000] + [1 + k % 90 for k in range(70)]
    q_lens = [3] + [1] * 70
    at = starts(lens)[:-1]
    q = randn(sum(q_lens), 8, 128, dtype=dtype)
    k, v = randn(sum(lens), 2, 128, dtype=dtype, seed=1), randn(sum(lens), 2, 128, dtype=dtype, seed=2)
    out, lse = cq.attention(q, k, v, q_starts=starts(q_lens), k_starts=at, k_lens=torch.tensor(lens, dtype=torch.int32, device=DEV))
    check(q, k, v, out, lse, q_lens, lens, at.tolist(), range(0, 71, 7))


@TYPES
def test_a_long_prompt_among_single_tokens(dtype):
    heads, kv_heads, d = 16, 4, 64
    lens = [1] * 200 + [2500] + [1] * 200
    n, at = sum(lens), starts(lens)
    q, k, v = (randn(n, h, d, dtype=dtype, seed=s) for s, h in enumerate((heads, kv_heads, kv_heads)))
    out, lse = cq.attention(q, k, v, q_starts=at, k_starts=at)
    check(q, k, v, out, lse, lens, lens, at.tolist(), [0, 1, 199, 200, 201, 400])


def test_what_rides_along_leaves_a_long_prompt_as_it_is():
    """bf16: the same bits for a long prompt whether 10 or 400 single tokens are in
    its batch, as the same kernel takes it however low the mean length is."""
    heads, kv_heads, d, long = 16, 4, 64, 2500
    q, k, v = (randn(long + 400, h, d, dtype=BF16, seed=s) for s, h in enumerate((heads, kv_heads, kv_heads)))
    results = []
    for single in (10, 60, 200, 400):
        at = starts([long] + [1] * single)
        out, lse = cq.attention(q[:long + single], k[:long + single], v[:long + single], q_starts=at, k_starts=at)
        results.append((out[:long], lse[:long]))
    for out, lse in results[1:]:
        assert torch.equal(out, results[0][0]) and torch.equal(lse, results[0][1])


@TYPES
def test_a_captured_call_follows_starts_and_lengths(dtype):
    """The grid and the workspace come from the sizes; how a tile's keys are cut
    from what the arrays hold when the graph is replayed."""
    b, rows_k = 12, 20000
    q = randn(b, 8, 128, dtype=dtype)
    k, v = randn(rows_k, 2, 128, dtype=dtype, seed=1), randn(rows_k, 2, 128, dtype=dtype, seed=2)
    k_at, k_lens = (torch.zeros(b, dtype=torch.int32, device=DEV) for _ in range(2))
    where = dict(q_starts=starts([1] * b), k_starts=k_at, k_lens=k_lens)
    cq.attention(q, k, v, **where)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = cq.attention(q, k, v, **where)
    for lens in ([1600] * b, [18000] + [100] * (b - 1), [3, 0] * (b // 2), [1, 9000, 0, 5, 700, 64, 65, 2048, 33, 31, 4000, 128]):
        at = starts(lens)[:-1]
        k_at.copy_(at)
        k_lens.copy_(torch.tensor(lens, dtype=torch.int32))
        want = cq.attention(q, k, v, **where)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
        check(q, k, v, *got, [1] * b, lens, at.tolist(), range(b))
