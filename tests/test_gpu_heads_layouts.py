"""Keys and values interleaved in one cache, in every order of heads, rows and
the pair: no two of their values share memory, so the calls take them."""

import pytest
import torch

import rotated_codebook_bit_amd as cq

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16
TYPES = pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
DEV, ROWS, KVH, D = "cuda", 40, 2, 64
AXES = {"rows": ROWS, "heads": KVH, "pair": 2}
ORDERS = [("rows", "heads", "pair"), ("rows", "pair", "heads"), ("heads", "rows", "pair"), ("heads", "pair", "rows"), ("pair", "rows", "heads"),
          ("pair", "heads", "rows")]


def randn(*shape, dtype=F32, seed=0):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed + sum(shape))
    return torch.randn(shape, generator=gen, device=DEV).to(dtype)


def pair_of(order, dtype):
    """Two [rows, heads, D] tensors that lie in one, whose axes come in `order`."""
    whole = torch.full((*(AXES[a] for a in order), D), 7.0, dtype=dtype, device=DEV)
    first = whole.permute(order.index("pair"), order.index("rows"), order.index("heads"), 3)
    return whole, first[0], first[1]


@TYPES
@pytest.mark.parametrize("order", ORDERS, ids=["_".join(o) for o in ORDERS])
def test_a_cache_of_keys_and_values(order, dtype):
    q, k, v = randn(9, 4, D, dtype=dtype), randn(9, KVH, D, dtype=dtype, seed=1), randn(9, KVH, D, dtype=dtype, seed=2)
    positions, freqs = torch.arange(9, device=DEV), 100.0 ** (-torch.arange(D // 2, device=DEV) / (D // 2))
    slots = torch.tensor([3, 39, 0, 17, 5, 6, 8, 30, 11], device=DEV)
    whole, k_cache, v_cache = pair_of(order, dtype)
    cq.qk_norm_rope(q, k, positions, freqs, v=v, slots=slots, k_out=k_cache, v_out=v_cache)
    _, k_plain, v_plain = cq.qk_norm_rope(q, k, positions, freqs, v=v)
    want_k, want_v = (torch.full((ROWS, KVH, D), 7.0, dtype=dtype, device=DEV) for _ in range(2))
    want_k[slots], want_v[slots] = k_plain, v_plain
    assert torch.equal(k_cache, want_k) and torch.equal(v_cache, want_v)
    a, _ = cq.attention(q, k_cache, v_cache)
    b, _ = cq.attention(q, want_k, want_v)
    assert torch.equal(a, b)


@TYPES
@pytest.mark.parametrize("order", ORDERS, ids=["_".join(o) for o in ORDERS])
def test_gradients_of_keys_and_values(order, dtype):
    q, k, v, dout = (randn(ROWS, h, D, dtype=dtype, seed=s) for s, h in enumerate((4, KVH, KVH, 4)))
    out, lse = cq.attention(q, k, v)
    whole, dk, dv = pair_of(order, dtype)
    cq.attention_grad(dout, q, k, v, out, lse, dk=dk, dv=dv)
    for a, b in zip((dk, dv), cq.attention_grad(dout, q, k, v, out, lse)[1:]):
        assert torch.equal(a, b)


@pytest.mark.parametrize("order", ORDERS[2:4], ids=["_".join(o) for o in ORDERS[2:4]])
def test_pairs_that_share_memory_are_refused(order):
    q, k, v, dout = (randn(ROWS, h, D, seed=s) for s, h in enumerate((4, KVH, KVH, 4)))
    out, lse = cq.attention(q, k, v)
    whole, dk, dv = pair_of(order, F32)
    flat = whole.flatten()
    touching = torch.as_strided(flat, dv.shape, dv.stride(), dk.storage_offset() + D // 2)
    with pytest.raises(cq.CQError, match="overlap"):
        cq.attention_grad(dout, q, k, v, out, lse, dk=dk, dv=touching)
    if order[1] == "pair":  # keys' rows one further than their part
        touching = torch.as_strided(flat, dv.shape, dv.stride(), dk.storage_offset() + (ROWS - 1) * D)
        with pytest.raises(cq.CQError, match="overlap"):
            cq.attention_grad(dout, q, k, v, out, lse, dk=dk, dv=touching)
