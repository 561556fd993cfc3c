"""The residual RMS norm (floating point and rotated 8-bit) and its gradient on
the GPU against float64 NumPy, over every width class of the kernels, both
types, odd widths, zero rows and values that are not finite.  Each case
prints its name before it touches the GPU.

Tolerances.  A row's sum of squares adds at most 32 values per lane and then
10 partial sums in float32, all of one sign: (32 + 10) 2^-24 relative, halved
by the root, plus the reciprocal root's own ulp and four products: TOL = 32 *
2^-24 relative covers it.  The rotation adds log2(G) roundings on the group's
sum of magnitudes.  A bf16 result is the float32 one rounded once: bit-exact,
or (the gradient) half a unit in the last place of an 8-bit significand,
HALF = 2^-8 of the value.
"""

import sys

import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover - CPU container
    pytest.skip("no GPU", allow_module_level=True)

import rotated_codebook_bit_amd as cq  # noqa: E402

DEV = "cuda"
EPS = 2.0 ** -24
TOL = 32 * EPS
HALF = 2.0 ** -8
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


def say(msg):
    print(f"[gpu] {msg}", flush=True)
    sys.stdout.flush()


def host64(t):
    torch.cuda.synchronize()
    return t.double().cpu().numpy()


def inputs(seed, rows, cols, kind, weight="f32"):
    rng = np.random.default_rng(seed)

    def make(scale):
        return torch.from_numpy((rng.standard_normal((rows, cols)) * scale).astype(np.float32)).to(DEV, TYPES[kind])

    w = None if weight is None else torch.from_numpy((1 + 0.2 * rng.standard_normal(cols)).astype(np.float32)).to(
        DEV, TYPES[weight])
    return make(1.0), make(2.0), w


def reference(x, r, w, eps):
    h = host64(x) + (0.0 if r is None else host64(r))
    rs = 1 / np.sqrt((h * h).mean(1, keepdims=True) + eps)
    return h, rs, h * rs * (1.0 if w is None else host64(w))


WIDTHS = [1, 7, 8, 64, 65, 255, 256, 512, 513, 1000, 1024, 1032, 2048, 2049, 4096, 4104, 8192, 8193, 16384, 16388, 32767,
          32768]


@pytest.mark.parametrize("cols", WIDTHS)
@pytest.mark.parametrize("kind,out,weight,residual", [("f32", "f32", "f32", True), ("bf16", "bf16", "bf16", True),
                                                      ("bf16", "f32", "f32", False), ("f32", "bf16", None, True)])
def test_norm(cols, kind, out, weight, residual):
    rows = 3 if cols > 4096 else 9
    x, r, w = inputs(cols, rows, cols, kind, weight)
    r = r if residual else None
    say(f"norm rows={rows} cols={cols} {kind}->{out} w={weight} residual={residual}")
    y, s = cq.add_rms_norm(x, r, w, 1e-5, out_dtype=TYPES[out])
    h, _, ref = reference(x, r, w, 1e-5)
    if out == "bf16":
        full, _ = cq.add_rms_norm(x, r, w, 1e-5, out_dtype=torch.float32)
        assert torch.equal(y, full.to(torch.bfloat16))
        y = full
    assert np.all(np.abs(host64(y) - ref) <= TOL * np.abs(ref))
    if residual:
        assert torch.equal(s, (x.float() + r.float()).to(TYPES[kind]))
    else:
        assert s is x


@pytest.mark.parametrize("rows,cols", [(1, 4096), (1023, 512), (1030, 2048), (2000, 1000), (1500, 4096)])
def test_norm_many_rows(rows, cols):
    x, r, w = inputs(rows, rows, cols, "bf16")
    say(f"norm rows={rows} cols={cols}")
    y, s = cq.add_rms_norm(x, r, w, out_dtype=torch.float32)
    _, _, ref = reference(x, r, w, 1e-6)
    assert np.all(np.abs(host64(y) - ref) <= TOL * np.abs(ref))
    # one row at a time, another split of the same row: near, and its sum equal
    y1, s1 = cq.add_rms_norm(x[5:6] if rows > 5 else x, r[5:6] if rows > 5 else r, w, out_dtype=torch.float32)
    i = 5 if rows > 5 else 0
    assert torch.equal(s1[0], s[i])
    assert np.all(np.abs(host64(y1)[0] - ref[i]) <= TOL * np.abs(ref[i]))


def test_norm_in_place_and_zero_rows():
    x, r, w = inputs(1, 40, 1024, "bf16")
    x[3], r[3] = 0, 0
    say("norm in place")
    y, s = cq.add_rms_norm(x, r, w)
    for target in ("x", "residual"):
        a, b = x.clone(), r.clone()
        y2, s2 = cq.add_rms_norm(a, b, w, sum_out=a if target == "x" else b)
        assert s2 is (a if target == "x" else b) and torch.equal(s2, s) and torch.equal(y2, y)
    assert torch.count_nonzero(y[3]) == 0
    y0, _ = cq.add_rms_norm(x, r, w, eps=0.0)  # 0 * rsqrt(0)
    assert torch.isnan(y0[3]).all() and torch.equal(y0[4], cq.add_rms_norm(x[4:5], r[4:5], w, eps=0.0)[0][0])


def hadamard(g):
    i = np.arange(g)
    return 1.0 - 2.0 * (np.array([[bin(a & b).count("1") & 1 for b in i] for a in i]))


Q8_WIDTHS = {32: [32, 96, 4096], 64: [64, 448, 2048], 128: [128, 512, 1152, 4096, 11008, 32768], 256: [256, 768, 8192]}


@pytest.mark.parametrize("group,cols", [(g, c) for g, cs in Q8_WIDTHS.items() for c in cs])
@pytest.mark.parametrize("kind,weight", [("f32", "bf16"), ("bf16", "f32")])
def test_norm_q8(group, cols, kind, weight):
    for rows in (1, 5, 1100) if cols <= 2048 else (1, 5):
        x, r, w = inputs(cols + rows, rows, cols, kind, weight)
        x[:, 0] += 30.0  # an outlier that the rotation spreads
        say(f"norm_q8 G={group} rows={rows} cols={cols} {kind}")
        q, s, h = cq.add_rms_norm_q8(x, r, w, 1e-6, group_size=group)
        _, _, y = reference(x, r, w, 1e-6)
        v = (y.reshape(rows, -1, group) @ hadamard(group)).reshape(rows, cols) / np.sqrt(group)
        mass = np.repeat(np.abs(y).reshape(rows, -1, group).sum(2), group, axis=1) / np.sqrt(group)
        tol = (np.log2(group) + 3) * EPS * mass + TOL * mass
        top = np.abs(v).max(1)
        s64, q64 = host64(s), host64(q)
        assert np.all(np.abs(s64 - top / 127) <= tol.max(1) / 127 + 4 * EPS * top)
        assert np.abs(q64).max() == 127
        # nearest multiple of the scale, up to the arithmetic's error
        assert np.all(np.abs(q64 * s64[:, None] - v) <= s64[:, None] * (0.5 + 127 * 4 * EPS) + tol)
        assert torch.equal(h, (x.float() + r.float()).to(TYPES[kind]))
        if rows == 1100:  # rows do not depend on each other's place
            q1, s1, _ = cq.add_rms_norm_q8(x[7:8], r[7:8], w, 1e-6, group_size=group)
            assert np.all(np.abs(host64(q1)[0] - q64[7]) <= 1)


def test_norm_q8_special_rows():
    x, _, w = inputs(3, 8, 512, "f32")
    x[0] = 0.0
    x[1, 100] = float("nan")
    x[2, 3] = float("inf")
    x[3] = 1e-30
    w2 = w.clone()
    say("norm_q8 special rows")
    q, s, h = cq.add_rms_norm_q8(x, None, w2, 1e-6)
    assert h is x
    assert s[0] == 0 and torch.count_nonzero(q[0]) == 0
    for i in (1, 2):
        assert torch.isnan(s[i]) and torch.count_nonzero(q[i]) == 0
    assert s[3] > 0 and q[3].abs().max() == 127  # small, but no underflow of the scale
    assert torch.isfinite(s[4:]).all()
    w2[7] = float("nan")
    q, s, _ = cq.add_rms_norm_q8(x[4:], None, w2, 1e-6)
    assert torch.isnan(s).all() and torch.count_nonzero(q) == 0
    q, s, _ = cq.add_rms_norm_q8(x[4:], None, torch.zeros_like(w), 1e-6)
    assert torch.count_nonzero(s) == 0 and torch.count_nonzero(q) == 0


def grad_reference(dout, h, dsum, w, eps):
    dy, h = host64(dout), host64(h)
    ww = 1.0 if w is None else host64(w)
    r = 1 / np.sqrt((h * h).mean(1, keepdims=True) + eps)
    u = ww * dy
    k = r ** 3 * (u * h).mean(1, keepdims=True)
    kmass = r ** 3 * np.abs(u * h).mean(1, keepdims=True)
    ds = 0.0 if dsum is None else host64(dsum)
    dx = ds + r * u - h * k
    mass = np.abs(ds) + np.abs(r * u) + np.abs(h) * kmass
    return dx, mass, (dy * h * r).sum(0), np.abs(dy * h * r).sum(0)


def check_grad(rows, cols, kind, weight, dsum, seed=0):
    h, dy, w = inputs(seed + rows + cols, rows, cols, kind, weight)
    ds = inputs(99, rows, cols, kind)[0] if dsum else None
    say(f"norm_grad rows={rows} cols={cols} {kind} w={weight} dsum={dsum}")
    dx, dw = cq.rms_norm_grad(dy, h, w, dsum=ds, eps=1e-5)
    rx, mass, rw, wmass = grad_reference(dy, h, ds, w, 1e-5)
    # three times the root's error (r^3) plus the dot product's 42 additions
    tol = (3 * 32 + 48) * EPS * mass
    if kind == "bf16":
        tol = tol + HALF * (np.abs(rx) + tol)
    assert np.all(np.abs(host64(dx) - rx) <= tol)
    assert np.all(np.abs(host64(dw) - rw) <= (rows + 64) * EPS * wmass)
    dx2, dw2 = cq.rms_norm_grad(dy, h, w, dsum=ds, eps=1e-5)
    assert torch.equal(dx, dx2) and torch.equal(dw, dw2)


@pytest.mark.parametrize("cols", WIDTHS)
@pytest.mark.parametrize("kind,weight,dsum", [("f32", "f32", True), ("bf16", "bf16", True), ("bf16", None, False)])
def test_norm_grad(cols, kind, weight, dsum):
    for rows in (1, 7):
        check_grad(rows, cols, kind, weight, dsum)


@pytest.mark.parametrize("rows,cols,kind", [(600, 64, "f32"), (3000, 64, "bf16"), (513, 1000, "f32"), (2100, 1024, "bf16"),
                                            (1100, 4096, "bf16"), (700, 2049, "bf16"), (530, 8193, "f32")])
def test_norm_grad_many_rows(rows, cols, kind):
    check_grad(rows, cols, kind, "f32", True)


def test_norm_grad_against_differences():
    """dx and dweight against central differences of the float64 formula."""
    rng = np.random.default_rng(2)
    h, dy, ds, w = (rng.standard_normal(s).astype(np.float32) for s in ((3, 10), (3, 10), (3, 10), (10,)))

    def loss(h, w):
        return (h / np.sqrt((h * h).mean(1, keepdims=True) + 1e-5) * w * dy + h * ds).sum()

    say("norm_grad differences")
    dx, dw = cq.rms_norm_grad(*(torch.from_numpy(a).to(DEV) for a in (dy, h, w)), dsum=torch.from_numpy(ds).to(DEV), eps=1e-5)
    step = 1e-5  # truncation step^2 and cancellation 2^-52 / step: below 1e-9 here
    for arr, got in ((h, host64(dx)), (w, host64(dw))):
        for i in np.ndindex(arr.shape):
            p, m = arr.astype(np.float64), arr.astype(np.float64)
            p[i] += step
            m[i] -= step
            diff = (loss(p, w) - loss(m, w) if arr is h else loss(h.astype(np.float64), p) - loss(h.astype(np.float64), m)) / (2 * step)
            assert abs(diff - got[i]) <= 1e-8 + 200 * EPS * 10


def test_norm_grad_in_place_and_empty():
    h, dy, w = inputs(4, 50, 256, "bf16")
    ds = inputs(5, 50, 256, "bf16")[0]
    say("norm_grad in place")
    dx, dw = cq.rms_norm_grad(dy, h, w, dsum=ds)
    dx2, dw2 = cq.rms_norm_grad(dy, h, w, dsum=ds, dx=ds)
    assert dx2 is ds and torch.equal(dx, dx2) and torch.equal(dw, dw2)
    _, dw0 = cq.rms_norm_grad(dy[:0], h[:0], w)
    assert torch.count_nonzero(dw0) == 0
    assert cq.add_rms_norm(h[:0], dy[:0], w)[0].shape == (0, 256)


def test_norm_other_stream_and_graph():
    x, r, w = inputs(6, 70, 4096, "bf16")
    dy = inputs(7, 70, 4096, "bf16")[0]
    s = torch.cuda.Stream()
    say("norm streams")
    s.wait_stream(torch.cuda.current_stream())
    q1, s1, h1 = cq.add_rms_norm_q8(x, r, w, stream=s)
    d1, w1 = cq.rms_norm_grad(dy, x, w, dsum=r, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    q, sc, h = cq.add_rms_norm_q8(x, r, w)
    d, dw = cq.rms_norm_grad(dy, x, w, dsum=r)
    torch.cuda.synchronize()
    assert torch.equal(q, q1) and torch.equal(sc, s1) and torch.equal(h, h1) and torch.equal(d, d1) and torch.equal(dw, w1)
    say("norm graph")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        q1, s1, h1 = cq.add_rms_norm_q8(x, r, w)
        d1, w1 = cq.rms_norm_grad(dy, x, w, dsum=r)
    for _ in range(3):
        x.normal_()
        dy.normal_()
        g.replay()
        torch.cuda.synchronize()
        q, sc, h = cq.add_rms_norm_q8(x, r, w)
        d, dw = cq.rms_norm_grad(dy, x, w, dsum=r)
        assert torch.equal(q, q1) and torch.equal(sc, s1) and torch.equal(h, h1) and torch.equal(d, d1) and torch.equal(dw, w1)


@pytest.mark.parametrize("rows,cols,kind", [(8195, 512, "f32"), (8195, 507, "f32"), (8195, 1016, "bf16"), (2050, 1024, "bf16"),
                                            (512, 8192, "bf16"), (515, 8192, "bf16"), (515, 4093, "f32")])
def test_norm_teams(rows, cols, kind):
    """Both sides of every choice of a row's team, by rows and by width."""
    x, r, w = inputs(rows + cols, rows, cols, kind)
    say(f"norm teams rows={rows} cols={cols} {kind}")
    y, s = cq.add_rms_norm(x, r, w, out_dtype=torch.float32)
    _, _, ref = reference(x, r, w, 1e-6)
    assert np.all(np.abs(host64(y) - ref) <= TOL * np.abs(ref))
    assert torch.equal(s, (x.float() + r.float()).to(TYPES[kind]))


@pytest.mark.parametrize("rows,cols,kind", [(2047, 1024, "bf16"), (2048, 1024, "bf16"), (512, 8192, "bf16"), (513, 8192, "bf16"),
                                            (2051, 512, "f32")])
def test_norm_q8_teams(rows, cols, kind):
    x, r, w = inputs(rows + cols, rows, cols, kind)
    say(f"norm_q8 teams rows={rows} cols={cols} {kind}")
    q, s, _ = cq.add_rms_norm_q8(x, r, w, 1e-6, group_size=128)
    _, _, y = reference(x, r, w, 1e-6)
    v = (y.reshape(rows, -1, 128) @ hadamard(128)).reshape(rows, cols) / np.sqrt(128)
    mass = np.repeat(np.abs(y).reshape(rows, -1, 128).sum(2), 128, axis=1) / np.sqrt(128)
    tol = (7 + 3) * EPS * mass + TOL * mass
    s64 = host64(s)
    assert np.all(np.abs(host64(q) * s64[:, None] - v) <= s64[:, None] * (0.5 + 127 * 4 * EPS) + tol)


@pytest.mark.parametrize("rows,cols,kind", [(1024, 4096, "f32"), (1025, 4096, "f32"), (1025, 3604, "f32"), (1024, 4096, "bf16"),
                                            (1025, 3608, "bf16"), (1025, 3601, "bf16"), (1025, 801, "bf16"), (90, 3601, "f32"),
                                            (600, 6001, "bf16")])
def test_norm_grad_teams(rows, cols, kind):
    check_grad(rows, cols, kind, "f32", True, seed=5)
