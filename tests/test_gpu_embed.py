"""The embedding lookup (dense and from CQ storage) and its gradient on the
GPU against float64 NumPy: every storage form and group size, odd widths, ids
outside the table, repeated tokens, and the sizes around the sort's and the
sums' internal boundaries.  Each case prints its name before it touches the
GPU.

Tolerances.  Dense lookup: one float32 product, rounded once: bit-exact.
Packed lookup: log2(G) butterfly additions and three products in float32 on
sums of at most G levels of magnitude cmax: |err| <= (log2 G + 4) 2^-24 scale
norm cmax.  Gradient: a float32 sum of c rows in a fixed order: |err| <=
(c + 2) 2^-24 scale sum |dout|.  A bf16 result is the float32 one rounded
once: bit-exact, or (where the float32 one is not at hand) half a unit in the
last place of an 8-bit significand, 2^-8 of the value.
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
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


def say(msg):
    print(f"[gpu] {msg}", flush=True)
    sys.stdout.flush()


def host64(t):
    torch.cuda.synchronize()
    return t.double().cpu().numpy()


def tokens_for(rng, n, vocab, index, outside=True):
    t = rng.integers(0, vocab, n)
    if outside and n > 3:
        t[1], t[n // 2], t[-1] = -1, vocab, vocab + 12345
    return t, torch.from_numpy(t.astype(np.int32 if index == 32 else np.int64)).to(DEV)


@pytest.mark.parametrize("src", ["f32", "bf16"])
@pytest.mark.parametrize("dst", ["f32", "bf16"])
@pytest.mark.parametrize("n,vocab,dim,index", [(1, 7, 1, 32), (5, 3, 4, 64), (37, 100, 8, 32), (64, 1000, 513, 64),
                                               (129, 50, 1000, 32), (33, 400, 4096, 64), (8, 1, 70, 64)])
def test_embed_dense(src, dst, n, vocab, dim, index):
    say(f"embed {src}->{dst} n={n} vocab={vocab} dim={dim} int{index}")
    rng = np.random.default_rng(n + dim)
    t, tok = tokens_for(rng, n, vocab, index)
    table = torch.from_numpy(rng.standard_normal((vocab, dim)).astype(np.float32)).to(DEV, TYPES[src])
    scale = 3.7
    out = cq.embed(tok, table, scale, out_dtype=TYPES[dst])
    inside = (t >= 0) & (t < vocab)
    ref = torch.zeros((n, dim), device=DEV)
    ref[torch.from_numpy(inside).to(DEV)] = table.float()[torch.from_numpy(t[inside]).to(DEV)] * np.float32(scale)
    assert out.shape == (n, dim) and out.dtype == TYPES[dst]
    assert torch.equal(out, ref.to(TYPES[dst]))


@pytest.mark.parametrize("bits", [O.TERNARY, cq.TERNARY_TRITS, 2, 3, 4])
@pytest.mark.parametrize("group", [32, 64, 128, 256])
@pytest.mark.parametrize("n,vocab,dim,dst,index", [(1, 5, 256, "f32", 64), (19, 33, 300, "f32", 32), (19, 33, 300, "bf16", 64),
                                                   (40, 20, 1000, "bf16", 32), (6, 9, 77, "f32", 64), (6, 9, 77, "bf16", 32),
                                                   (700, 64, 1024, "f32", 32), (700, 64, 1024, "bf16", 64)])
def test_embed_packed(bits, group, n, vocab, dim, dst, index, levels32):
    say(f"embed_packed bits={bits} G={group} n={n} vocab={vocab} dim={dim} {dst}")
    rng = np.random.default_rng(dim + group)
    lv = levels32[O.TERNARY if bits == cq.TERNARY_TRITS else bits]
    w = torch.from_numpy((rng.standard_normal((vocab, dim)) * 0.02).astype(np.float32)).to(DEV)
    packed, norms = cq.quantize(w, bits, lv, group_size=group)
    rows = host64(cq.dequantize(packed, norms, vocab, dim, bits, lv, group_size=group))
    t, tok = tokens_for(rng, n, vocab, index)
    scale = float(np.sqrt(dim))
    out = cq.embed_packed(tok, packed, norms, vocab, dim, bits, lv, scale, out_dtype=TYPES[dst], group_size=group)
    inside = (t >= 0) & (t < vocab)
    ref = np.zeros((n, dim))
    ref[inside] = rows[t[inside]] * scale
    # dequantize() itself is held to the oracle elsewhere; both sides round in float32.
    nm = np.zeros((n, dim))
    nm[inside] = np.repeat(host64(norms), group, axis=1)[:, :dim][t[inside]]
    tol = 2 * (np.log2(group) + 4) * EPS * scale * nm * np.abs(lv).max()
    assert out.shape == (n, dim) and out.dtype == TYPES[dst]
    if dst == "bf16":
        full = cq.embed_packed(tok, packed, norms, vocab, dim, bits, lv, scale, group_size=group)
        assert torch.equal(out, full.to(torch.bfloat16))
        out = full
    err = np.abs(host64(out) - ref)
    assert np.all(err <= tol), (err - tol).max()


def test_embed_packed_is_the_oracle(levels32):
    """Against the oracle's dequantization in float64 (ragged rows, 2 bits)."""
    rng = np.random.default_rng(0)
    w = rng.standard_normal((50, 1000)) * 0.02
    q = O.quantize(w, 2, levels32[2])
    ref = O.dequantize(q.packed, q.norm16, 50, 1000, 2, levels32[2])
    packed = torch.from_numpy(q.packed.reshape(50, -1)).to(DEV)
    norms = torch.from_numpy(q.norm16.view(np.int16)).to(DEV).view(torch.float16)
    tok = torch.arange(49, -1, -1, device=DEV)
    say("embed_packed oracle")
    out = host64(cq.embed_packed(tok, packed, norms, 50, 1000, 2, levels32[2]))
    nm = np.repeat(host64(norms).reshape(50, -1), 128, axis=1)[::-1, :1000]
    assert np.all(np.abs(out - ref[::-1]) <= 11 * EPS * nm * np.abs(levels32[2]).max())


def test_embed_packed_default_codebook_and_shape():
    w = torch.randn(30, 256, device=DEV)
    packed, norms = cq.quantize(w, 2, None)
    tok = torch.tensor([[3, 4], [29, 0]], device=DEV)
    say("embed_packed default levels")
    out = cq.embed_packed(tok, packed, norms, 30, 256, 2, None)
    assert out.shape == (2, 2, 256)
    assert torch.equal(out, cq.dequantize(packed, norms, 30, 256, 2, None)[tok])
    assert cq.embed(tok[:0], w).shape == (0, 2, 256)


def grad_case(seed, n, vocab, dim, kind, out, index, accumulate, tokens=None):
    rng = np.random.default_rng(seed)
    if tokens is None:
        t, tok = tokens_for(rng, n, vocab, index)
    else:
        t = tokens(rng)
        tok = torch.from_numpy(t.astype(np.int32 if index == 32 else np.int64)).to(DEV)
    d = torch.from_numpy(rng.standard_normal((n, dim)).astype(np.float32)).to(DEV, TYPES[kind])
    scale = 1.75
    old = torch.randn(vocab, dim, device=DEV).to(TYPES[out]) if accumulate else None
    say(f"embed_grad n={n} vocab={vocab} dim={dim} {kind}->{out} int{index} acc={accumulate}")
    g = cq.embed_grad(tok, d, vocab, scale, grad_dtype=TYPES[out], grad=None if old is None else old.clone(),
                      accumulate=accumulate)
    inside = (t >= 0) & (t < vocab)
    d64 = host64(d)
    ref, mass, count = np.zeros((vocab, dim)), np.zeros((vocab, dim)), np.zeros((vocab, 1))
    np.add.at(ref, t[inside], d64[inside] * scale)
    np.add.at(mass, t[inside], np.abs(d64[inside]) * scale)
    np.add.at(count, t[inside], 1.0)
    tol = (count + 2) * EPS * mass
    if accumulate:
        ref = ref + host64(old)
        tol = tol + EPS * np.abs(ref)
    if out == "bf16":
        tol = tol + 2.0 ** -8 * (np.abs(ref) + tol)
    err = np.abs(host64(g) - ref)
    assert np.all(err <= tol), (err - tol).max()
    if accumulate:  # rows of absent tokens are untouched
        absent = torch.from_numpy(count[:, 0] == 0).to(DEV)
        assert torch.equal(g[absent], old[absent])
    again = cq.embed_grad(tok, d, vocab, scale, grad_dtype=TYPES[out], grad=None if old is None else old.clone(),
                          accumulate=accumulate)
    assert torch.equal(g, again)


@pytest.mark.parametrize("n", [0, 1, 2, 63, 64, 65, 1023, 1024, 1025, 4097])
@pytest.mark.parametrize("vocab,dim,kind,out,index", [(300, 68, "f32", "f32", 64), (7, 33, "bf16", "f32", 32)])
def test_embed_grad_lengths(n, vocab, dim, kind, out, index):
    grad_case(n, n, vocab, dim, kind, out, index, False)


@pytest.mark.parametrize("vocab", [1, 2, 255, 256, 257, 65535, 65536, 70000])
def test_embed_grad_vocabularies(vocab):
    grad_case(vocab, 500, vocab, 12, "f32", "f32", 64, False)
    grad_case(vocab, 500, vocab, 12, "bf16", "bf16", 32, True)


@pytest.mark.parametrize("dim", [1, 3, 4, 255, 256, 260, 1000, 1028, 4096])
@pytest.mark.parametrize("kind,out", [("f32", "f32"), ("bf16", "f32"), ("bf16", "bf16")])
@pytest.mark.parametrize("accumulate", [False, True])
def test_embed_grad_widths(dim, kind, out, accumulate):
    grad_case(dim, 300, 90, dim, kind, out, 64, accumulate)


@pytest.mark.parametrize("n", [16384, 16385, 40000])
def test_embed_grad_many_tokens(n):
    # Half of the positions one token, a tail of rare ones, some outside.
    def skewed(rng):
        t = rng.integers(0, 5000, n)
        t[rng.random(n) < 0.5] = 77
        t[rng.random(n) < 0.1] = -1
        return t
    grad_case(n, n, 5000, 20, "f32", "f32", 64, False, skewed)
    grad_case(n, n, 5000, 21, "bf16", "f32", 32, True, skewed)


@pytest.mark.parametrize("n", [64, 65, 128, 129, 200, 1000])
def test_embed_grad_runs(n):
    # Runs that start, end and lie on the pieces' boundaries.
    grad_case(n, n, 10, 300, "f32", "f32", 64, False, lambda rng: np.full(n, 3))
    grad_case(n, n, 10, 300, "f32", "f32", 32, False, lambda rng: np.full(n, 9))
    grad_case(n, n, 10, 300, "f32", "f32", 64, True, lambda rng: np.sort(rng.integers(0, 3, n)))
    grad_case(n, n, 10, 300, "f32", "f32", 64, False, lambda rng: np.where(np.arange(n) < n // 3, 4, 5))
    grad_case(n, n, 10, 300, "f32", "f32", 64, False, lambda rng: np.full(n, -1))


def test_embed_grad_against_differences():
    """d/dW of sum(embed(t, W) * d) by differences of the forward: it is linear
    in W, so a step of 1 is exact up to float32 sums."""
    rng = np.random.default_rng(5)
    t = torch.from_numpy(rng.integers(0, 6, 40)).to(DEV)
    w = torch.from_numpy(rng.standard_normal((6, 5)).astype(np.float32)).to(DEV)
    d = torch.from_numpy(rng.standard_normal((40, 5)).astype(np.float32)).to(DEV)
    say("embed_grad differences")
    g = host64(cq.embed_grad(t, d, 6, 0.5))
    base = (host64(cq.embed(t, w, 0.5)) * host64(d)).sum()
    for v in range(6):
        for c in range(5):
            w2 = w.clone()
            w2[v, c] += 1.0
            diff = (host64(cq.embed(t, w2, 0.5)) * host64(d)).sum() - base
            # 40 products of float32-rounded values of magnitude up to about 5
            assert abs(diff - g[v, c]) <= 40 * 5 * 5 * 4 * EPS


def test_embed_other_stream_and_graph(levels32):
    w = torch.randn(64, 512, device=DEV) * 0.02
    packed, norms = cq.quantize(w, 4, levels32[4])
    tok = torch.randint(0, 64, (333,), device=DEV)
    d = torch.randn(333, 512, device=DEV)
    say("embed streams")
    out = cq.embed_packed(tok, packed, norms, 64, 512, 4, levels32[4])
    grad = cq.embed_grad(tok, d, 64)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    out2 = cq.embed_packed(tok, packed, norms, 64, 512, 4, levels32[4], stream=s)
    grad2 = cq.embed_grad(tok, d, 64, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    torch.cuda.synchronize()
    assert torch.equal(out, out2) and torch.equal(grad, grad2)
    say("embed graph")
    buf, gbuf = torch.empty_like(out), torch.empty_like(grad)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        cq.embed_packed(tok, packed, norms, 64, 512, 4, levels32[4], out=buf)
        cq.embed_grad(tok, d, 64, grad=gbuf)
    for i in range(3):
        tok.copy_(torch.randint(0, 64, (333,), device=DEV))
        d.normal_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(buf, cq.embed_packed(tok, packed, norms, 64, 512, 4, levels32[4]))
        assert torch.equal(gbuf, cq.embed_grad(tok, d, 64))


@pytest.mark.parametrize("n", [5000, 8192, 8193])
def test_embed_grad_one_block_sorts(n):
    grad_case(n, n, 300, 68, "f32", "f32", 64, False)


@pytest.mark.parametrize("bits", [0, O.TERNARY, cq.TERNARY_TRITS, 2, 3, 4])
@pytest.mark.parametrize("dim,dst", [(1000, "f32"), (1030, "f32"), (1032, "bf16"), (2051, "bf16")])
def test_embed_large_lookups(bits, dim, dst, levels32):
    """Lookups past 16 MiB (streaming stores, several units to a wave) equal
    the dequantized or dense rows."""
    say(f"embed large bits={bits} dim={dim} {dst}")
    rng = np.random.default_rng(dim + bits)
    n, vocab, group, scale = 8200, 60, 128, 2.5
    t, tok = tokens_for(rng, n, vocab, 64)
    w = torch.from_numpy((rng.standard_normal((vocab, dim)) * 0.02).astype(np.float32)).to(DEV)
    inside = torch.from_numpy((t >= 0) & (t < vocab)).to(DEV)
    at = torch.where(inside, tok, 0)
    if bits == 0:
        out = cq.embed(tok, w.to(TYPES[dst]), scale)
        ref = (w.to(TYPES[dst]).float()[at] * np.float32(scale) * inside[:, None]).to(TYPES[dst])
        assert torch.equal(out, ref)
        return
    lv = levels32[O.TERNARY if bits == cq.TERNARY_TRITS else bits]
    packed, norms = cq.quantize(w, bits, lv, group_size=group)
    rows = cq.dequantize(packed, norms, vocab, dim, bits, lv, group_size=group).double()
    ref = rows[at] * scale * inside[:, None]
    nm = norms.double().repeat_interleave(group, 1)[:, :dim][at] * inside[:, None]
    tol = 2 * (np.log2(group) + 4) * EPS * scale * float(np.abs(lv).max()) * nm
    out = cq.embed_packed(tok, packed, norms, vocab, dim, bits, lv, scale, out_dtype=TYPES[dst], group_size=group)
    if dst == "bf16":
        full = cq.embed_packed(tok, packed, norms, vocab, dim, bits, lv, scale, group_size=group)
        assert torch.equal(out, full.to(torch.bfloat16))
        out = full
    assert bool(((out.double() - ref).abs() <= tol).all())


@pytest.mark.parametrize("n,dim", [(2896, 256), (2897, 256), (2048, 512), (2049, 512), (1000, 4096), (724, 4096), (725, 4096),
                                   (90, 4099), (8, 33000), (3000, 33)])
@pytest.mark.parametrize("kind,out,accumulate", [("f32", "f32", False), ("bf16", "bf16", True)])
def test_embed_grad_scan_or_sort(n, dim, kind, out, accumulate):
    """Both sides of the choice between comparing all tokens and sorting them,
    tokens of one run to many (and a vocabulary past a clearing block's rows)."""
    def skewed(rng):
        t = np.minimum(rng.geometric(0.02, n) - 1, 129)
        t[0], t[n // 2] = -1, 131
        return t

    grad_case(n + dim, n, 131, dim, kind, out, 64, accumulate, tokens=skewed)


@pytest.mark.parametrize("n", [2900, 4097, 9000])
@pytest.mark.parametrize("distinct", [1, 2, 40])
def test_embed_grad_long_runs_sorted(n, distinct):
    grad_case(n, n, 50, 36, "f32", "f32", 32, False, tokens=lambda rng: rng.integers(0, distinct, n))


@pytest.mark.parametrize("vocab", [1 << 20, (1 << 20) + 1, 255, 511, 512])
@pytest.mark.parametrize("n", [3000, 5000, 12000])
def test_embed_grad_sorts_by_vocabulary(vocab, n):
    """Vocabularies at and past what one launch sorts, and at the ends of its ranges."""
    grad_case(n, n, vocab, 4, "f32", "f32", 64, False)
