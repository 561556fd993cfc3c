"""Calls whose rows take more than one launch (a launch counts its threads in
32 bits): what lies on either side of the cut equals a short call's result."""

import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover - CPU container
    pytest.skip("no GPU", allow_module_level=True)

import rotated_codebook_bit_amd as cq  # noqa: E402

DEV = "cuda"
ROWS = (1 << 26) + 6  # one wave per row, four waves per block of 256 threads
SPOTS = [0, 12345, (1 << 26) - 9, (1 << 26) - 1, 1 << 26, ROWS - 7, ROWS - 1]


def same(got, want):
    torch.cuda.synchronize()
    assert torch.equal(got, want)


def test_norm():
    print("[gpu] norm of 2^26 + 6 rows", flush=True)
    x = torch.randn(1 << 16, 8, device=DEV, dtype=torch.bfloat16).repeat(1025, 1)[:ROWS].contiguous()
    r = torch.ones_like(x)
    w = torch.rand(8, device=DEV)
    y, s = cq.add_rms_norm(x, r, w)
    for i in SPOTS:
        a, b = max(0, i - 3), min(ROWS, i + 4)
        y1, s1 = cq.add_rms_norm(x[a:b].clone(), r[a:b].clone(), w)
        same(y[a:b], y1)
        same(s[a:b], s1)


def test_norm_q8():
    print("[gpu] norm to 8 bits of 2^26 + 6 rows", flush=True)
    x = torch.randn(1 << 16, 32, device=DEV, dtype=torch.bfloat16).repeat(1025, 1)[:ROWS].contiguous()
    w = torch.rand(32, device=DEV)
    q, s, _ = cq.add_rms_norm_q8(x, None, w, group_size=32)
    for i in SPOTS:
        a, b = max(0, i - 3), min(ROWS, i + 4)
        q1, s1, _ = cq.add_rms_norm_q8(x[a:b].clone(), None, w, group_size=32)
        same(q[a:b], q1)
        same(s[a:b], s1)


@pytest.mark.parametrize("packed", [False, True])
def test_lookup(packed):
    print(f"[gpu] lookup of 2^26 + 6 tokens packed={packed}", flush=True)
    table = torch.randn(1000, 32, device=DEV)
    tok = torch.randint(0, 1000, (1 << 16,), device=DEV, dtype=torch.int32).repeat(1025)[:ROWS].contiguous()
    lv = np.array([-1.51, -0.4528, 0.4528, 1.51], np.float32)
    if packed:
        p, n = cq.quantize(table, 2, lv, group_size=32)

    def look(t):
        if packed:
            return cq.embed_packed(t, p, n, 1000, 32, 2, lv, 1.5, out_dtype=torch.bfloat16, group_size=32)
        return cq.embed(t, table, 1.5, out_dtype=torch.bfloat16)

    out = look(tok)
    for i in SPOTS:
        a, b = max(0, i - 3), min(ROWS, i + 4)
        same(out[a:b], look(tok[a:b].clone()))
