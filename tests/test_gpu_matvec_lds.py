"""cq_dequant_matvec on rows that fill only part of a pass, after products that
left NaN in every compute unit's shared memory: lanes without columns must add
zeros whatever that memory held before."""

import zlib

import numpy as np
import pytest

from oracle import cq_oracle as O
from parity import check_matvec

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover - CPU container
    pytest.skip("no GPU", allow_module_level=True)

import rotated_codebook_bit_amd as cq  # noqa: E402

DEV = "cuda"


def stored(q, n_out):
    return (torch.from_numpy(q.packed.reshape(n_out, -1)).to(DEV),
            torch.from_numpy(q.norm16.view(np.int16)).to(DEV).view(torch.float16))


@pytest.mark.parametrize("g", [32, 64, 128, 256])
@pytest.mark.parametrize("bits", [2, 3, 4])
@pytest.mark.parametrize("batch", [1, 3])
@pytest.mark.parametrize("k", [256, 1280, 4352])
def test_partly_filled_pass_after_nan(g, bits, batch, k, levels32):
    print(f"[gpu] matvec after NaN: G={g} bits={bits} batch={batch} k={k}", flush=True)
    lv = levels32[bits]
    rng = np.random.default_rng(zlib.crc32(repr(("nan", g, bits, batch, k)).encode()))
    # Whole passes of NaN activations, rows enough for every compute unit.
    wide = O.quantize(rng.standard_normal((8, 4096)) * 0.02, bits, lv, g)
    p8, n8 = stored(wide, 8)
    rows = 4096
    bad = torch.full((batch, 4096), float("nan"), dtype=torch.float32, device=DEV)
    p, n = p8.repeat(rows // 8, 1), n8.reshape(8, -1).repeat(rows // 8, 1)
    n_out = 300
    q = O.quantize(rng.standard_normal((n_out, k)) * 0.02, bits, lv, g)
    w_hat = O.dequantize(q.packed, q.norm16, n_out, k, bits, lv, g)
    x = rng.standard_normal((batch, k)).astype(np.float32)
    qp, qn = stored(q, n_out)
    xd = torch.from_numpy(x).to(DEV)
    z = cq.dequant_matvec(p, n, rows, 4096, bits, lv, bad, group_size=g)
    y = cq.dequant_matvec(qp, qn, n_out, k, bits, lv, xd, group_size=g)
    torch.cuda.synchronize()
    assert torch.isnan(z).all()
    check_matvec(y.cpu().numpy(), x.astype(np.float64) @ w_hat.T, x, w_hat)
