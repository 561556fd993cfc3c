"""Top tokens of rows with NaN that are read once more per top token, as more
values reach the floor than the list of candidates holds (2048)."""

import math

import pytest
import torch

import rotated_codebook_bit_amd as cq

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
@pytest.mark.parametrize("vocab", [2049, 9000, 140000])
def test_nan_at_token_0_of_a_row_past_the_list(vocab, dtype):
    logits = torch.full((4, vocab), math.nan, dtype=dtype, device=DEV)
    logits[1] = -math.inf
    logits[1, 0] = math.nan
    logits[2] = -math.inf
    logits[2, [0, 7, vocab - 1]] = torch.tensor([math.nan, 1.0, math.nan], dtype=dtype, device=DEV)
    logits[3] = 0.0
    r = cq.token_logprobs(logits, torch.zeros(4, dtype=torch.int64, device=DEV), 1.0, 4)
    assert r.top.tolist() == [[0, 1, 2, 3], [0, 1, 2, 3], [0, vocab - 1, 7, 1], [0, 1, 2, 3]]
    assert torch.isnan(r.top_logprob[:3]).all() and torch.isfinite(r.top_logprob[3]).all()
