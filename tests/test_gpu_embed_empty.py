"""The embedding gradient of an empty token list: zeros for every row of the
table, whatever its size (past 2^20 rows the sort takes tiles, of which an
empty list has none), and nothing touched when accumulating."""

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover - CPU container
    pytest.skip("no GPU", allow_module_level=True)

import rotated_codebook_bit_amd as cq  # noqa: E402

DEV = "cuda"


@pytest.mark.parametrize("vocab", [1, 256, 1 << 20, (1 << 20) + 1, (1 << 24) + 3])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("index", [torch.int32, torch.int64])
def test_no_tokens(vocab, dtype, index):
    print(f"[gpu] embed_grad of no tokens, vocab={vocab} {dtype} {index}", flush=True)
    tok, dout = torch.empty(0, dtype=index, device=DEV), torch.empty(0, 3, device=DEV)
    grad = torch.full((vocab, 3), float("nan"), dtype=dtype, device=DEV)
    assert cq.embed_grad(tok, dout, vocab, 2.0, grad=grad) is grad
    torch.cuda.synchronize()
    assert torch.count_nonzero(grad) == 0
    ones = torch.ones(vocab, 3, dtype=dtype, device=DEV)
    cq.embed_grad(tok, dout, vocab, 2.0, grad=ones, accumulate=True)
    torch.cuda.synchronize()
    assert torch.equal(ones, torch.ones_like(ones))


def test_no_tokens_captured():
    print("[gpu] embed_grad of no tokens in a graph", flush=True)
    vocab = (1 << 20) + 5
    tok, dout = torch.empty(0, dtype=torch.int64, device=DEV), torch.empty(0, 2, device=DEV)
    grad = torch.empty(vocab, 2, device=DEV)
    cq.embed_grad(tok, dout, vocab, grad=grad)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        cq.embed_grad(tok, dout, vocab, grad=grad)
    for _ in range(3):
        grad.fill_(float("nan"))
        g.replay()
        torch.cuda.synchronize()
        assert torch.count_nonzero(grad) == 0
