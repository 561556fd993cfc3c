"""The embedding gradient of a short list into a table of 2^30 narrow rows and
more: the clearing blocks of the comparing kernel (one per 64 rows) would pass
a launch's 2^32 threads there, so the sort takes it."""

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover - CPU container
    pytest.skip("no GPU", allow_module_level=True)

import rotated_codebook_bit_amd as cq  # noqa: E402

DEV = "cuda"


@pytest.mark.parametrize("vocab", [(1 << 30) - 1024, (1 << 30) - 63, 1 << 30, (1 << 30) + 777])
@pytest.mark.parametrize("accumulate", [False, True])
def test_tall_table(vocab, accumulate):
    print(f"[gpu] embed_grad into {vocab} rows accumulate={accumulate}", flush=True)
    at = [0, 63, 64, vocab // 2, vocab - 65, vocab - 1, vocab - 1, vocab, -1, 1 << 40]
    tok = torch.tensor(at, device=DEV)
    d = torch.arange(1, len(at) + 1, device=DEV, dtype=torch.float32)[:, None]
    grad = torch.full((vocab, 1), 0.5 if accumulate else float("nan"), dtype=torch.bfloat16, device=DEV)
    cq.embed_grad(tok, d, vocab, 2.0, grad=grad, accumulate=accumulate)
    torch.cuda.synchronize()
    base = 0.5 if accumulate else 0.0
    want = {0: 2.0, 63: 4.0, 64: 6.0, vocab // 2: 8.0, vocab - 65: 10.0, vocab - 1: 26.0}
    for row, value in want.items():  # sums of small whole numbers: exact in bf16
        assert grad[row].item() == value + base, row
        grad[row] = base
    other = torch.count_nonzero(grad != base) if base else torch.count_nonzero(grad)
    assert other.item() == 0
