"""The workspace of attention over a batch, on the CPU: the size function is
host-only.  It may not grow with the number of sequences, however the keys
are given, and no call of many short sequences may be refused."""

import ctypes

import pytest

import rotated_codebook_bit_amd as cq

try:
    L = cq.lib()
except ImportError:
    pytest.skip("libcq.so is not built", allow_module_level=True)

F32, BF16 = 0, 1
STARTS, LENS = 0x10000, 0x20000  # addresses, never touched
PER_ROW = {d: (d + 4) * 4 for d in (64, 128)}  # bytes of a row's share in one split


def workspace(n, rows_q, rows_k, dtype, heads, kv_heads, d, q_starts=True, k_starts=True, k_lens=False):
    seqs = cq.Sequences(n, rows_q, rows_k, STARTS if q_starts else None, STARTS if k_starts else None, LENS if k_lens else None, 4)
    out = ctypes.c_int64(-1)
    assert L.cq_attention_workspace(ctypes.byref(seqs), dtype, heads, kv_heads, d, ctypes.byref(out)) == 0, L.cq_last_error()
    return out.value


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("n,tokens", [(255, 8192), (257, 8192), (2100, 65536), (5000, 131072), (100000, 1 << 20)])
def test_packed_short_sequences_need_none(n, tokens, dtype):
    assert workspace(n, tokens, tokens, dtype, 32, 32, 128) == 0
    assert workspace(n, tokens, tokens, dtype, 32, 8, 64) == 0


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("n", [1, 2, 7, 16, 64, 150, 512, 4096])
@pytest.mark.parametrize("cap", [100, 1000, 8192, 70000])
def test_starts_of_a_cache_are_bounded(n, cap, dtype):
    """A token each over caches: by k_lens alone, by k_starts too, and as a pool
    of which the sequences use a part.  A grid of at most 16 rounds of 512 blocks
    and one more per tile of rows, each with its group's rows."""
    heads, kv_heads, d = 32, 8, 128
    bound = (16 * 512 + n * kv_heads) * (heads // kv_heads) * PER_ROW[d]
    for args in (dict(q_starts=False, k_starts=False, k_lens=True), dict(q_starts=False, k_lens=True), dict(k_lens=True)):
        assert 0 <= workspace(n, n, n * cap, dtype, heads, kv_heads, d, **args) <= bound, args


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("n,cap", [(1, 8192), (4, 2000), (64, 8192)])
def test_both_ways_to_say_a_cache_split_alike(n, cap, dtype):
    by_lens = workspace(n, n, n * cap, dtype, 32, 8, 128, q_starts=False, k_starts=False, k_lens=True)
    assert by_lens == workspace(n, n, n * cap, dtype, 32, 8, 128, q_starts=False, k_lens=True) > 0
