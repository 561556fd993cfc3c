"""The norm's gradient on rows whose magnitude is far from one: no factor of
the formula may leave float32 where the gradient itself is an ordinary number.
Rows of magnitude m have a reciprocal root of about 1 / m, whose cube leaves
float32 from m = 1e-13 down (infinite) and from 1e15 up (zero), while every
term of r u - h r (r mean(u h)) r stays near u / m.

Tolerances: the reciprocal root's error (32 2^-24, from the sum of squares of
at most 32 values per lane and 10 partial sums) enters three times, the dot
product's 42 additions and a few products once: (3 * 32 + 48) 2^-24 of the sum
of the terms' magnitudes.  A bf16 result adds half a unit in the last place of
an 8-bit significand, 2^-8 of the value.
"""

import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover - CPU container
    pytest.skip("no GPU", allow_module_level=True)

import rotated_codebook_bit_amd as cq  # noqa: E402

DEV = "cuda"
EPS = 2.0 ** -24
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


def host64(t):
    torch.cuda.synchronize()
    return t.double().cpu().numpy()


def check(rows, cols, magnitude, eps, kind, dsum):
    print(f"[gpu] norm_grad range rows={rows} cols={cols} {kind} magnitude={magnitude} eps={eps} dsum={dsum}", flush=True)
    rng = np.random.default_rng(rows + cols)

    def make(scale):
        return torch.from_numpy((rng.standard_normal((rows, cols)) * scale).astype(np.float32)).to(DEV, TYPES[kind])

    h, dy, ds = make(magnitude), make(1.0), make(1.0 / magnitude) if dsum else None
    w = torch.from_numpy((1 + 0.2 * rng.standard_normal(cols)).astype(np.float32)).to(DEV)
    dx, dw = cq.rms_norm_grad(dy, h, w, dsum=ds, eps=eps)
    h64, g64, w64, e64 = host64(h), host64(dy), host64(w), float(np.float32(eps))
    s64 = host64(ds) if dsum else np.zeros((rows, cols))
    r = 1 / np.sqrt((h64 * h64).mean(1, keepdims=True) + e64)
    u = w64 * g64
    hn = h64 * r
    want = s64 + r * (u - hn * (u * hn).mean(1, keepdims=True))
    tol = (3 * 32 + 48) * EPS * (np.abs(s64) + r * (np.abs(u) + np.abs(hn) * np.abs(u * hn).mean(1, keepdims=True)))
    if kind == "bf16":
        tol = tol + 2.0 ** -8 * (np.abs(want) + tol)
    got = host64(dx)
    assert np.isfinite(got).all()
    assert np.all(np.abs(got - want) <= tol), (np.abs(got - want) / tol).max()
    mass = np.abs(g64 * hn).sum(0)
    assert np.all(np.abs(host64(dw) - (g64 * hn).sum(0)) <= (rows + 64) * EPS * mass)


# Every kernel of the gradient: one wave per row, four waves, the wide one; whole pieces and single elements.
SHAPES = [(9, 64), (9, 65), (40, 512), (7, 1000), (7, 1001), (1100, 4096), (5, 8192), (5, 8193)]


@pytest.mark.parametrize("rows,cols", SHAPES)
@pytest.mark.parametrize("magnitude,eps", [(1e-13, 0.0), (1e-16, 0.0), (1e-15, 1e-30), (1e13, 1e-6), (1e16, 0.0)])
@pytest.mark.parametrize("kind,dsum", [("f32", False), ("bf16", True)])
def test_norm_grad_range(rows, cols, magnitude, eps, kind, dsum):
    check(rows, cols, magnitude, eps, kind, dsum)


def test_norm_grad_range_orthogonal_rows():
    """A dot product of exactly zero: the second term is zero, not infinity times zero."""
    print("[gpu] norm_grad range, orthogonal rows", flush=True)
    h = torch.tensor([[1e-14, 1e-14, -1e-14, -1e-14] * 16], device=DEV)
    dy = torch.tensor([[1.0, 1.0, 1.0, 1.0] * 16], device=DEV)
    dx, dw = cq.rms_norm_grad(dy, h, None, eps=0.0)
    torch.cuda.synchronize()
    # mean(h^2) = 1e-28 (float32's 1e-14 squared), r = 1e14: dx = r dy
    want = 1.0 / np.sqrt(float(h[0, 0]) ** 2)
    assert torch.all((dx.double() - want).abs() <= 64 * EPS * want)
    assert torch.all((dw.double().abs() - 1).abs() <= 64 * EPS)
