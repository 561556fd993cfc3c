"""The product of 8-bit rotated activations with a CQ matrix on the GPU against
float64 NumPy: every width, group size and output type, one batch row to
several tiles, ragged outputs, split k.  Each case prints its name before it
touches the GPU.

Tolerance per output: the 16-bit levels are off by at most delta = max |c -
scale (256 hi + lo)|, which costs delta * sum |q s| norm / sqrt(G); the sums
within a group are exact integers, converted (1 rounding) and added over ng
groups and at most 16 partial sums in float32: (ng + 20) 2^-24 of the sum of
magnitudes.  A bf16 result is the float32 one rounded once: bit-exact.
"""

import sys

import numpy as np
import pytest

from oracle import cq_oracle as O

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover - CPU container
    pytest.skip("no GPU", allow_module_level=True)

import rotated_codebook_bit_amd as cq  # noqa: E402

DEV = "cuda"
EPS = 2.0 ** -24
ALL_BITS = [O.TERNARY, 2, 3, 4]


def say(msg):
    print(f"[gpu] {msg}", flush=True)
    sys.stdout.flush()


def host64(t):
    torch.cuda.synchronize()
    return t.double().cpu().numpy()


def unpack(packed, bits, group):
    """Indices [..., G] of field storage, bit by bit."""
    sb = 2 if bits == O.TERNARY else bits
    b = np.unpackbits(packed, axis=-1, bitorder="little")
    b = b.reshape(*packed.shape[:-1], group, sb)
    return (b << np.arange(sb, dtype=np.uint8)).sum(-1)


def make(seed, n_out, k, bits, group, batch):
    rng = np.random.default_rng(seed)
    sb = 2 if bits == O.TERNARY else bits
    ng = k // group
    packed = rng.integers(0, 256, (n_out, ng, group * sb // 8), dtype=np.uint8)
    if bits == O.TERNARY:  # no field holds 3
        packed &= ~((packed & 0x55) << 1)
    norms = (0.2 * (1 + rng.random((n_out, ng)))).astype(np.float16)
    norms[0, 0] = 0.0
    q = rng.integers(-127, 128, (batch, k), dtype=np.int8)
    q[0, :2] = (-128, 127)
    scale = (0.01 * (1 + rng.random(batch))).astype(np.float32)
    return packed, norms, q, scale


def check(bits, group, n_out, k, batch, out, lv, seed=0):
    packed, norms, q, scale = make(seed + n_out + k + batch, n_out, k, bits, group, batch)
    table = cq.q8_levels(bits, lv)
    say(f"gemm_q8 bits={bits} G={group} n_out={n_out} k={k} batch={batch} {out}")
    dt = torch.bfloat16 if out == "bf16" else torch.float32
    dev = [torch.from_numpy(a).to(DEV) for a in (packed, norms, q, scale)]
    y = cq.dequant_gemm_q8(dev[0], dev[1], n_out, k, bits, table, dev[2], dev[3], group_size=group, out_dtype=dt)
    c = lv.astype(np.float64)[unpack(packed, bits, group)]
    nm = norms.astype(np.float64)[..., None] / np.sqrt(group)
    w = (c * nm).reshape(n_out, k)
    x = q.astype(np.float64) * scale.astype(np.float64)[:, None]
    ref = x @ w.T
    m = 256.0 * np.array(table.hi[:len(lv)]) + np.array(table.lo[:len(lv)])
    delta = np.abs(lv - table.scale * m).max() + EPS * np.abs(lv).max()
    assert delta <= 2.2e-5 * np.abs(lv).max()
    spread = np.abs(x) @ np.broadcast_to(nm, c.shape).reshape(n_out, k).T
    tol = delta * spread + (k // group + 20) * EPS * (np.abs(x) @ np.abs(w).T)
    y2 = cq.dequant_gemm_q8(dev[0], dev[1], n_out, k, bits, table, dev[2], dev[3], group_size=group, out_dtype=dt)
    assert torch.equal(y, y2)
    if out == "bf16":
        full = cq.dequant_gemm_q8(dev[0], dev[1], n_out, k, bits, table, dev[2], dev[3], group_size=group)
        assert y.dtype == torch.bfloat16 and torch.equal(y, full.to(torch.bfloat16))
        y = full
    err = np.abs(host64(y) - ref)
    assert y.shape == (batch, n_out) and np.all(err <= tol), (err / tol).max()


@pytest.mark.parametrize("bits", ALL_BITS)
@pytest.mark.parametrize("group", [32, 64, 128, 256])
@pytest.mark.parametrize("batch", [1, 17, 40, 64, 65, 130])
def test_gemm_q8_forms(bits, group, batch, levels32):
    check(bits, group, 150, 5 * group, batch, "f32", levels32[bits])
    check(bits, group, 33, 12 * group, batch, "bf16", levels32[bits])


@pytest.mark.parametrize("n_out", [1, 15, 16, 17, 127, 128, 129, 300])
@pytest.mark.parametrize("batch", [1, 3, 16, 32, 33, 48, 49, 96, 128, 129, 257])
def test_gemm_q8_sizes(n_out, batch, levels32):
    check(2, 128, n_out, 640, batch, "f32" if batch % 2 else "bf16", levels32[2])


@pytest.mark.parametrize("group,groups", [(32, 1), (32, 2), (32, 3), (32, 9), (64, 1), (64, 3), (128, 1), (128, 17), (256, 1),
                                          (256, 3)])
@pytest.mark.parametrize("batch", [1, 20, 70])
def test_gemm_q8_short_and_odd_k(group, groups, batch, levels32):
    for bits in (2, 3, 4):
        check(bits, group, 40, group * groups, batch, "f32", levels32[bits])


@pytest.mark.parametrize("bits,n_out,k,batch", [(2, 1100, 4096, 1), (4, 520, 11008, 37), (2, 260, 11008, 200), (3, 130, 8192, 65),
                                                (2, 2050, 2048, 300)])
def test_gemm_q8_large(bits, n_out, k, batch, levels32):
    check(bits, 128, n_out, k, batch, "f32", levels32[bits])


def test_gemm_q8_zero_and_nan_scales(levels32):
    packed, norms, q, scale = (torch.from_numpy(a).to(DEV) for a in make(1, 40, 256, 2, 128, 5))
    scale[1], scale[3] = 0.0, float("nan")
    say("gemm_q8 zero and NaN scales")
    y = cq.dequant_gemm_q8(packed, norms, 40, 256, 2, cq.q8_levels(2, levels32[2]), q, scale)
    assert torch.count_nonzero(y[1]) == 0 and torch.isnan(y[3]).all() and torch.isfinite(y[[0, 2, 4]]).all()
    say("gemm_q8 empty")
    e = cq.dequant_gemm_q8(packed[:, :0], norms[:, :0], 40, 0, 2, cq.q8_levels(2, levels32[2]), q[:, :0], scale,
                           out_dtype=torch.bfloat16)
    assert torch.count_nonzero(e) == 0 and e.shape == (5, 40)
    assert cq.dequant_gemm_q8(packed[:0], norms[:0], 0, 256, 2, cq.q8_levels(2, levels32[2]), q, scale).shape == (5, 0)


@pytest.mark.parametrize("bits", [2, 4])
@pytest.mark.parametrize("batch", [1, 100])
def test_norm_then_product(bits, batch, levels32):
    """norm -> 8 bits -> product against the float32 norm -> product: apart by
    at most half a step per activation."""
    rng = np.random.default_rng(batch)
    w = torch.from_numpy((rng.standard_normal((300, 512)) * 0.02).astype(np.float32)).to(DEV)
    packed, norms = cq.quantize(w, bits, levels32[bits])
    x, r = (torch.from_numpy(rng.standard_normal((batch, 512)).astype(np.float32)).to(DEV) for _ in range(2))
    g = torch.from_numpy((1 + 0.1 * rng.standard_normal(512)).astype(np.float32)).to(DEV)
    say(f"norm then product bits={bits} batch={batch}")
    q, s, h = cq.add_rms_norm_q8(x, r, g)
    y8 = cq.dequant_gemm_q8(packed, norms, 300, 512, bits, cq.q8_levels(bits, levels32[bits]), q, s)
    n, h2 = cq.add_rms_norm(x, r, g)
    w_hat = host64(cq.dequantize(packed, norms, 300, 512, bits, levels32[bits]))
    ref = host64(n) @ w_hat.T
    i = np.arange(128)
    had = (1.0 - 2.0 * np.array([[bin(a & b).count("1") & 1 for b in i] for a in i])) / np.sqrt(128)
    w_rot = (w_hat.reshape(300, 4, 128) @ had).reshape(300, 512)
    tol = 0.501 * host64(s)[:, None] * np.abs(w_rot).sum(1)[None] + 6e-5 * np.linalg.norm(host64(n), axis=1)[:, None] * np.linalg.norm(
        w_hat, axis=1)[None]
    assert torch.equal(h, h2) and np.all(np.abs(host64(y8) - ref) <= tol)


def test_gemm_q8_other_stream_and_graph(levels32):
    table = cq.q8_levels(2, levels32[2])
    for batch in (1, 90):
        packed, norms, q, scale = (torch.from_numpy(a).to(DEV) for a in make(2, 200, 4096, 2, 128, batch))
        args = (packed, norms, 200, 4096, 2, table, q, scale)
        s = torch.cuda.Stream()
        say(f"gemm_q8 streams batch={batch}")
        s.wait_stream(torch.cuda.current_stream())
        y1 = cq.dequant_gemm_q8(*args, stream=s)
        torch.cuda.current_stream().wait_stream(s)
        y = cq.dequant_gemm_q8(*args)
        torch.cuda.synchronize()
        assert torch.equal(y, y1)
        say(f"gemm_q8 graph batch={batch}")
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            y1 = cq.dequant_gemm_q8(*args)
        for _ in range(3):
            q.copy_(torch.randint(-127, 128, q.shape, device=DEV, dtype=torch.int8))
            g.replay()
            torch.cuda.synchronize()
            assert torch.equal(y1, cq.dequant_gemm_q8(*args))
