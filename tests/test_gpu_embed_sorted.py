"""The embedding gradient by sorting (lists past 2896 tokens; shorter ones are
compared): runs laid against the pieces' borders for each of the three piece
sizes, every width class, every number of digit passes of the tiled sort, the
borders between the sorts' variants, graphs, side streams and workspaces full
of NaN.

Reference: float64 sums on the CPU.  Tolerance: a float32 sum of c rows is off
by at most (c + 2) 2^-24 scale sum |dout|, whatever its order; adding it to a
float32 gradient once more 2^-24 of the result; rounding to bf16 half a unit in
the last place of an 8-bit significand, 2^-8 of the value.
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


def need(n, vocab, dim):
    import ctypes
    out = ctypes.c_int64()
    assert cq.lib().cq_embed_grad_workspace(n, vocab, dim, ctypes.byref(out)) == 0
    return out.value


def check(name, tokens, vocab, dim, kind="f32", out="f32", accumulate=False, index=64):
    n = len(tokens)
    print(f"[gpu] embed_grad sorted: {name} n={n} vocab={vocab} dim={dim} {kind}->{out} int{index} acc={accumulate}", flush=True)
    gen = torch.Generator(device=DEV)
    gen.manual_seed(n + dim)
    tok = torch.from_numpy(np.asarray(tokens)).to(DEV, torch.int32 if index == 32 else torch.int64)
    d = torch.randn((n, dim), generator=gen, device=DEV).to(TYPES[kind])
    scale = 1.75
    old = torch.randn((vocab, dim), generator=gen, device=DEV).to(TYPES[out]) if accumulate else None
    # What the workspace and the gradient held before must not show.
    ws = torch.full((need(n, vocab, dim) // 4,), float("nan"), device=DEV)
    grad = old.clone() if accumulate else torch.full((vocab, dim), float("nan"), dtype=TYPES[out], device=DEV)
    cq.embed_grad(tok, d, vocab, scale, grad=grad, accumulate=accumulate, workspace=ws)
    torch.cuda.synchronize()
    # The tokens that occur, their rows' sums one run at a time.
    t64 = tok.cpu().numpy().astype(np.int64)
    order = np.argsort(t64, kind="stable")
    order = order[(t64[order] >= 0) & (t64[order] < vocab)]
    present = torch.zeros(vocab, dtype=torch.bool, device=DEV)
    if len(order):
        present_at, starts, count = np.unique(t64[order], return_index=True, return_counts=True)
        rows = d.cpu().double().numpy()[order] * scale
        ref = np.add.reduceat(rows, starts, axis=0)
        tol = ((count + 2) * EPS)[:, None] * np.add.reduceat(np.abs(rows, out=rows), starts, axis=0)
        at = torch.from_numpy(present_at).to(DEV)
        if accumulate:
            ref += old[at].cpu().double().numpy()
            tol += EPS * np.abs(ref)
        if out == "bf16":
            tol += 2.0 ** -8 * (np.abs(ref) + tol)
        err = np.abs(grad[at].cpu().double().numpy() - ref)
        assert np.all(err <= tol), (err - tol).max()
        present[at] = True
    if accumulate:
        assert torch.equal(grad[~present], old[~present])
    else:
        assert torch.count_nonzero(grad[~present]) == 0
    again = cq.embed_grad(tok, d, vocab, scale, grad_dtype=TYPES[out], grad=None if old is None else old.clone(),
                          accumulate=accumulate)
    assert torch.equal(grad, again)


def shuffled(lengths, first=0, seed=0):
    """Tokens first, first + 1, .. as often as `lengths` says, in random order."""
    t = np.repeat(first + np.arange(len(lengths)), lengths)
    return np.random.default_rng(seed).permutation(t)


PIECES = [(16, 3000), (16, 8192), (32, 9000), (32, 65536), (64, 65537), (64, 70000)]


def layouts(p, n):
    """Run lengths that start, end and span at the borders of pieces of p."""
    yield "whole pieces", [p] * 6 + [2 * p, 3 * p]
    yield "one off", [p - 1, 1, p + 1, p - 1, 2 * p - 1, 1, 2 * p + 1, p - 1, 1, p + 1]
    yield "from the middle", [p // 2, p, p // 2, p // 2, 2 * p, p // 2, p // 2 - 1, p + 1, p // 2 + 1, p + 2]
    yield "long ones", [5 * p, 3, 5 * p - 3, 7, 6 * p + 1, p, 4 * p - 8, 9 * p + 5, 1, 1]
    yield "singles", [1] * (3 * p + 1)
    yield "one long", [n - 2 * p - 1]
    yield "single then long", [1, n - 2 * p]
    yield "a piece, then long", [p, n - 2 * p - 1]


@pytest.mark.parametrize("piece,n", PIECES)
@pytest.mark.parametrize("tail", ["inside", "outside", "one"])
def test_runs_and_pieces(piece, n, tail):
    for name, lengths in layouts(piece, n):
        left = n - sum(lengths)
        vocab = 4000
        if tail == "inside":  # the rest in runs of one to twice a piece
            rest = np.random.default_rng(left).integers(1, 2 * piece, 2 * left // piece + 2)
            rest = rest[np.cumsum(rest) < left]
            lengths = lengths + list(rest) + [left - int(rest.sum())]
        elif tail == "one":
            lengths = lengths + [left]
        t = shuffled(lengths, seed=n)
        vocab = max(int(t.max()) + 1, 300)  # the last run is the table's last row, or rows without tokens follow
        t = np.concatenate([t, np.where(np.arange(n - len(t)) % 2, -1, vocab)])  # the rest, outside the table
        check(f"{name}, {tail}", np.random.default_rng(1).permutation(t), vocab, 12)


@pytest.mark.parametrize("n", [2897, 9001, 66001])
@pytest.mark.parametrize("token", [0, 7, 99, -1, 100])
def test_one_token(n, token):
    check("one token", np.full(n, token), 100, 20, "bf16", "f32")


@pytest.mark.parametrize("dim", [1, 3, 4, 68, 255, 256, 257, 260, 1000, 1028, 1029, 2051])
@pytest.mark.parametrize("kind,out,accumulate", [("f32", "f32", False), ("bf16", "f32", True), ("bf16", "bf16", False),
                                                 ("f32", "bf16", True)])
def test_widths(dim, kind, out, accumulate):
    for n in (3000, 9000):
        rng = np.random.default_rng(n + dim)
        t = np.minimum(rng.geometric(0.01, n) - 1, 420)
        t[::97] = -1
        check("widths", t, 400, dim, kind, out, accumulate, 32)


@pytest.mark.parametrize("dim", [4099, 8192])
def test_wide_rows(dim):
    rng = np.random.default_rng(dim)
    check("wide rows", rng.integers(-1, 60, 2900), 59, dim, "bf16", "f32")
    check("wide rows", rng.integers(-1, 60, 2900), 59, dim, "f32", "f32", True)


@pytest.mark.parametrize("vocab", [1, 200, 255, 256, 65535, 65536, (1 << 24) - 1, 1 << 24, (1 << 24) + 9])
@pytest.mark.parametrize("n", [16385, 18432, 18433, 66000])
def test_digit_passes(vocab, n):
    """One to four passes of the tiled sort, its tiles full or not."""
    rng = np.random.default_rng(vocab + n)
    t = rng.integers(0, vocab, n)
    t[rng.random(n) < 0.05] = -1
    t[rng.random(n) < 0.2] = vocab - 1
    t[0] = vocab + 5
    check("passes", t, vocab, 3 if vocab > 1 << 20 else 8)


@pytest.mark.parametrize("n,vocab,dim", [(2896, (1 << 20) + 1, 260), (128, 50, 131073), (17, 4, 29026 * 256 + 1),
                                         (16, 4, 32768 * 256 + 1)])
def test_short_lists_of_wide_rows(n, vocab, dim):
    """Short lists that the rows' width sends to a sort: more than 2^23
    comparisons over the row's slices of 256 columns."""
    assert n * n * -(-dim // 256) > 1 << 23
    t = np.random.default_rng(n).integers(0, vocab, n)
    t[n // 2:] = vocab - 1
    t[1] = -1
    check("wide rows", t, vocab, dim)


@pytest.mark.parametrize("vocab", [(1 << 18) - 1, 1 << 18, (1 << 18) + 1])
@pytest.mark.parametrize("n", [3000, 16384])
def test_ranges_or_tiles(vocab, n):
    """Both sides of the vocabulary past which tiles sort short lists too."""
    rng = np.random.default_rng(vocab + n)
    t = rng.integers(-1, vocab + 1, n)
    t[: n // 3] = vocab - 1
    check("ranges or tiles", t, vocab, 20, "bf16", "f32")
    check("ranges or tiles", t, vocab, 20, "f32", "bf16", True, 32)


@pytest.mark.parametrize("n", [4096, 4097, 8192, 8193, 16384, 16385, 65536, 65537, 200001])
def test_lengths(n):
    rng = np.random.default_rng(n)
    t = np.minimum(rng.geometric(0.002, n) - 1, 5000)
    check("lengths", t, 4990, 20)
    check("lengths", np.sort(t), 4990, 21, "bf16", "f32", True)


@pytest.mark.parametrize("n,vocab", [(3000, 500), (9000, 500), (17000, 500), (17000, (1 << 20) + 77), (66000, 70000)])
def test_graph_and_stream(n, vocab):
    print(f"[gpu] embed_grad sorted: graph and stream n={n} vocab={vocab}", flush=True)
    dim = 36
    gen = torch.Generator(device=DEV)
    gen.manual_seed(n)

    def draw():
        t = torch.randint(-1, vocab, (n,), generator=gen, device=DEV)
        return torch.where(torch.rand(n, generator=gen, device=DEV) < 0.3, 17, t)

    tok, d = draw(), torch.randn(n, dim, generator=gen, device=DEV)
    want = cq.embed_grad(tok, d, vocab)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = cq.embed_grad(tok, d, vocab, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    assert torch.equal(got, want)
    grad = torch.empty_like(want)
    ws = torch.empty(need(n, vocab, dim), dtype=torch.uint8, device=DEV)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        cq.embed_grad(tok, d, vocab, grad=grad, workspace=ws)
    for _ in range(3):
        tok.copy_(draw())
        d.normal_(generator=gen)
        ws.fill_(255)
        grad.fill_(float("nan"))
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(grad, cq.embed_grad(tok, d, vocab))
