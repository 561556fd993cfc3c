"""Timed cases of the operators around the CQ products: the embedding lookup
and its gradient, the residual addition with the root-mean-square norm (in
floating point, or rotated and held in 8 bits) and its gradient, and the
product of 8-bit activations with a CQ matrix.

``own`` selects what ``run`` calls: False, plain torch operations in float32;
True, the entry points of ``rotated_codebook_bit_amd``.

Sizes are those of the repository's workloads: the 32000 x 4096 embedding and
the 11008 x 4096 / 4096 x 11008 matrices of the 7B-shaped model, the 8192 x
512 embedding of the 45.5M-parameter set, and the 1000-column tensor whose
last group is partial.
"""

import functools
import math

import numpy as np
import torch

own = False

DEV = "cuda"
EPS = 1e-6
F32, BF16 = torch.float32, torch.bfloat16
TYPES = {"f32": F32, "bf16": BF16}

# Codebooks in N(0,1) units: the optimal Gaussian quantizers of J. Max (1960)
# for 4, 8 and 16 levels, and the three-level one.
_MAX = {2: (0.4528, 1.5104), 3: (0.2451, 0.7560, 1.3440, 2.1520),
        4: (0.1284, 0.3881, 0.6568, 0.9424, 1.2562, 1.6180, 2.0690, 2.7326)}
TERNARY, TRITS = 158, 159


def _levels(bits):
    if bits in (TERNARY, TRITS):
        return np.array([-1.2240064, 0.0, 1.2240064], np.float32)
    half = np.array(_MAX[bits], np.float32)
    return np.concatenate([-half[::-1], half])


# -- the cases --------------------------------------------------------------------

def listed():
    return [
        # One decode step's lookup of one token in the packed embedding.
        {"name": "embed_token", "op": "embed", "n": 1, "vocab": 32000, "dim": 4096, "bits": 2, "group": 128,
         "out": "f32", "index": 64},
        # A batch of prompts looked up in a 4-bit embedding.
        {"name": "embed_prompt", "op": "embed", "n": 8192, "vocab": 32000, "dim": 4096, "bits": 4, "group": 128,
         "out": "bf16", "index": 64},
        # A short training sequence on rows that end in a partial group.
        {"name": "embed_grad_short", "op": "embed_grad", "n": 777, "vocab": 8192, "dim": 1000, "type": "f32",
         "index": 32},
        # A training batch of the 7B-shaped model: a float32 gradient of the whole table from bf16 rows.
        {"name": "embed_grad_batch", "op": "embed_grad", "n": 16384, "vocab": 32000, "dim": 4096, "type": "bf16",
         "index": 64},
        # One decode step's norm in front of a quantized product.
        {"name": "norm_q8_token", "op": "norm_q8", "rows": 1, "cols": 4096, "type": "bf16", "group": 128},
        # The same for a batch of prompts.
        {"name": "norm_q8_prompt", "op": "norm_q8", "rows": 8192, "cols": 4096, "type": "bf16", "group": 128},
        # Training forward of the 45.5M-parameter set's width, float32.
        {"name": "norm_train", "op": "norm", "rows": 16384, "cols": 512, "type": "f32", "out": "f32"},
        # Gradient of a few rows of an odd width.
        {"name": "norm_grad_short", "op": "norm_grad", "rows": 300, "cols": 1000, "type": "f32"},
        # Gradient of a training batch.
        {"name": "norm_grad_batch", "op": "norm_grad", "rows": 8192, "cols": 4096, "type": "bf16"},
        # One decode step through an up projection.
        {"name": "product_token", "op": "product", "batch": 1, "n_out": 11008, "k": 4096, "bits": 2, "group": 128,
         "out": "f32"},
        # A short chunk of tokens through a 4-bit down projection.
        {"name": "product_chunk", "op": "product", "batch": 37, "n_out": 4096, "k": 11008, "bits": 4, "group": 128,
         "out": "bf16"},
        # A batch of prompts through an up projection.
        {"name": "product_prompt", "op": "product", "batch": 4096, "n_out": 11008, "k": 4096, "bits": 2,
         "group": 128, "out": "bf16"},
    ]


def draw(rng):
    def log(lo, hi):
        return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))

    op = rng.choice(["embed", "embed", "embed_grad", "norm_q8", "norm", "norm_grad", "product", "product"])
    kind, out = rng.choice(["f32", "bf16"]), rng.choice(["f32", "bf16"])
    group = rng.choice([32, 64, 128, 128, 256])
    if op == "embed":
        bits = rng.choice([0, TERNARY, TRITS, 2, 3, 4])  # 0: a table of floating-point rows
        return {"op": op, "n": log(1, 8192), "vocab": log(256, 32000), "dim": log(96, 4096), "bits": bits,
                "group": group, "out": out, "index": rng.choice([32, 64])}
    if op == "embed_grad":
        return {"op": op, "n": log(8, 16384), "vocab": log(256, 32000), "dim": log(96, 4096), "type": kind,
                "index": rng.choice([32, 64])}
    if op == "norm_q8":
        return {"op": op, "rows": log(1, 8192), "cols": group * max(1, log(256, 4096) // group), "type": kind,
                "group": group}
    if op == "norm":
        return {"op": op, "rows": log(1, 8192), "cols": log(96, 4096), "type": kind, "out": out}
    if op == "norm_grad":
        return {"op": op, "rows": log(16, 8192), "cols": log(96, 4096), "type": kind}
    return {"op": op, "batch": log(1, 4096), "n_out": log(96, 11008), "k": group * max(1, log(256, 4096) // group),
            "bits": rng.choice([TERNARY, 2, 3, 4]), "group": group, "out": out}


# -- inputs -------------------------------------------------------------------------

def _group_bytes(bits, group):
    return -(-group // 5) if bits == TRITS else group * (2 if bits == TERNARY else bits) // 8


def _pack(codes, bits):
    """codes: int32 [..., G] to the stored bytes [..., B]."""
    lead, g = codes.shape[:-1], codes.shape[-1]
    if bits == TRITS:
        nb = -(-g // 5)
        codes = torch.nn.functional.pad(codes, (0, 5 * nb - g)).view(*lead, nb, 5)
        return (codes * torch.tensor([1, 3, 9, 27, 81], device=codes.device, dtype=torch.int32)).sum(-1).to(torch.uint8)
    sb = 2 if bits == TERNARY else bits
    word = (codes.view(*lead, g // 8, 8) << (sb * torch.arange(8, device=codes.device, dtype=torch.int32))).sum(
        -1, dtype=torch.int64)  # eight indices are sb whole bytes
    return ((word[..., None] >> (8 * torch.arange(sb, device=codes.device))) & 255).to(torch.uint8).flatten(-2)


def _weights(gen, rows, cols, bits, group):
    """The stored form of a rows x cols matrix of N(0, 0.02^2) values: its
    rotated, normalised values are drawn and snapped to the levels."""
    ng = -(-cols // group)
    lv = torch.from_numpy(_levels(bits)).to(DEV)
    z = torch.randn((rows, ng, group), generator=gen, device=DEV)
    packed = _pack(torch.bucketize(z, (lv[1:] + lv[:-1]) / 2, out_int32=True), bits)
    spread = 1 + torch.randn((rows, ng), generator=gen, device=DEV) / math.sqrt(2 * group)
    return packed, (0.02 * math.sqrt(group) * spread).to(torch.float16)


def _tokens(gen, n, vocab, index, padding):
    """Token ids whose k-th most frequent one comes up about 1/k as often as
    the first; with `padding`, one position in a hundred holds -1."""
    u = torch.rand(n, generator=gen, device=DEV, dtype=torch.float64)
    rank = (torch.exp(u * math.log(vocab + 1)) - 1).long().clamp_(0, vocab - 1)
    ids = torch.randperm(vocab, generator=gen, device=DEV)[rank]
    if padding:
        ids[torch.rand(n, generator=gen, device=DEV) < 0.01] = -1
    return ids.to(torch.int32 if index == 32 else torch.int64)


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)

    def randn(*shape, dtype=F32, scale=1.0):
        return (torch.randn(shape, generator=gen, device=DEV) * scale).to(dtype)

    op, s = case["op"], {"case": dict(case)}
    if op == "embed":
        s["tokens"] = _tokens(gen, case["n"], case["vocab"], case["index"], False)
        s["scale"] = math.sqrt(case["dim"])
        if case["bits"]:
            s["levels"] = _levels(case["bits"])
            s["packed"], s["norms"] = _weights(gen, case["vocab"], case["dim"], case["bits"], case["group"])
        else:
            s["table"] = randn(case["vocab"], case["dim"], dtype=TYPES[case["out"]], scale=0.02)
    elif op == "embed_grad":
        s["tokens"] = _tokens(gen, case["n"], case["vocab"], case["index"], True)
        s["scale"] = math.sqrt(case["dim"])
        s["dout"] = randn(case["n"], case["dim"], dtype=TYPES[case["type"]], scale=1e-3)
    elif op in ("norm", "norm_q8"):
        kind, shape = TYPES[case["type"]], (case["rows"], case["cols"])
        s["x"], s["residual"] = randn(*shape, dtype=kind), randn(*shape, dtype=kind, scale=2.0)
        s["weight"] = 1 + randn(case["cols"], scale=0.1)
    elif op == "norm_grad":
        kind, shape = TYPES[case["type"]], (case["rows"], case["cols"])
        s["sum"] = randn(*shape, dtype=kind, scale=2.0)
        s["dout"], s["dsum"] = randn(*shape, dtype=kind, scale=1e-2), randn(*shape, dtype=kind, scale=1e-2)
        s["weight"] = 1 + randn(case["cols"], scale=0.1)
    else:
        s["levels"] = _levels(case["bits"])
        s["packed"], s["norms"] = _weights(gen, case["n_out"], case["k"], case["bits"], case["group"])
        x = randn(case["batch"], case["k"])
        s["scale"] = x.abs().amax(1) / 127
        s["q"] = torch.round(x / s["scale"][:, None]).to(torch.int8)
        if own:  # the codebook's 8-bit table, computed once per codebook
            import rotated_codebook_bit_amd as cq
            s["table"] = cq.q8_levels(case["bits"], s["levels"])
    return s


# -- the plain forms ----------------------------------------------------------------

def _hadamard(group):
    """The orthonormal Sylvester matrix, (-1)^popcount(i & j) / sqrt(G)."""
    i = torch.arange(group, device=DEV)
    v = i[:, None] & i
    v = v ^ (v >> 4)
    v = v ^ (v >> 2)
    v = (v ^ (v >> 1)) & 1
    return (1 - 2 * v).float() / math.sqrt(group)


def _codes(packed, bits, group):
    """Stored bytes [..., B] to indices [..., G]."""
    b = packed.to(torch.int32)
    if bits == TRITS:
        digits = b[..., None] // torch.tensor([1, 3, 9, 27, 81], device=DEV, dtype=torch.int32) % 3
        return digits.flatten(-2)[..., :group]
    if bits == 3:
        b = b.unflatten(-1, (group // 8, 3))
        word = b[..., 0] | (b[..., 1] << 8) | (b[..., 2] << 16)
        return ((word[..., None] >> (3 * torch.arange(8, device=DEV, dtype=torch.int32))) & 7).flatten(-2)
    sb = 2 if bits == TERNARY else bits
    return ((b[..., None] >> torch.arange(0, 8, sb, device=DEV, dtype=torch.int32)) & ((1 << sb) - 1)).flatten(-2)


def _rotated_rows(packed, norms, levels, bits, group):
    """norm / sqrt(G) * level of every element, [rows, groups, G]."""
    lv = torch.from_numpy(levels).to(DEV)
    return lv[_codes(packed, bits, group).long()] * (norms.float() / math.sqrt(group))[..., None]


def _plain(s):
    c, op = s["case"], s["case"]["op"]
    if op == "embed":
        ids = s["tokens"].long()
        if not c["bits"]:
            return {"out": (s["table"][ids].float() * s["scale"]).to(TYPES[c["out"]])}
        rows = _rotated_rows(s["packed"][ids], s["norms"][ids], s["levels"], c["bits"], c["group"])
        rows = rows @ _hadamard(c["group"])
        return {"out": (rows.flatten(1)[:, :c["dim"]] * s["scale"]).to(TYPES[c["out"]])}
    if op == "embed_grad":
        ids = s["tokens"].long()
        grad = torch.zeros((c["vocab"] + 1, c["dim"]), device=DEV)
        grad.index_add_(0, torch.where(ids < 0, c["vocab"], ids), s["dout"].float())
        return {"grad": grad[:c["vocab"]] * s["scale"]}
    if op in ("norm", "norm_q8"):
        h = s["x"].float() + s["residual"].float()
        y = h * torch.rsqrt((h * h).mean(1, keepdim=True) + EPS) * s["weight"]
        if op == "norm":
            return {"out": y.to(TYPES[c["out"]]), "sum": h.to(s["x"].dtype)}
        g = c["group"]
        y = (y.unflatten(1, (-1, g)) @ _hadamard(g)).flatten(1)
        scale = y.abs().amax(1) / 127
        q = torch.round(y / scale[:, None]).clamp_(-127, 127)
        return {"values": (q * scale[:, None]).to(BF16), "scale": scale, "sum": h.to(s["x"].dtype)}
    if op == "norm_grad":
        h, dy, w = s["sum"].float(), s["dout"].float(), s["weight"]
        r = torch.rsqrt((h * h).mean(1, keepdim=True) + EPS)
        wd = w * dy
        dx = s["dsum"].float() + r * wd - h * (r * r * r * (wd * h).mean(1, keepdim=True))
        return {"dx": dx.to(s["sum"].dtype), "dweight": (dy * h * r).sum(0)}
    w = _rotated_rows(s["packed"], s["norms"], s["levels"], c["bits"], c["group"]).flatten(1)
    y = (s["q"].float() @ w.t()) * s["scale"][:, None]
    return {"y": y.to(TYPES[c["out"]])}


# -- the framework's calls --------------------------------------------------------------

def _own(s):
    import rotated_codebook_bit_amd as cq

    c, op = s["case"], s["case"]["op"]
    if op == "embed":
        kind = TYPES[c["out"]]
        if not c["bits"]:
            return {"out": cq.embed(s["tokens"], s["table"], s["scale"], out_dtype=kind)}
        return {"out": cq.embed_packed(s["tokens"], s["packed"], s["norms"], c["vocab"], c["dim"], c["bits"], s["levels"],
                                       s["scale"], out_dtype=kind, group_size=c["group"])}
    if op == "embed_grad":
        return {"grad": cq.embed_grad(s["tokens"], s["dout"], c["vocab"], s["scale"], grad_dtype=F32)}
    if op == "norm":
        out, h = cq.add_rms_norm(s["x"], s["residual"], s["weight"], EPS, out_dtype=TYPES[c["out"]])
        return {"out": out, "sum": h}
    if op == "norm_q8":
        q, scale, h = cq.add_rms_norm_q8(s["x"], s["residual"], s["weight"], EPS, group_size=c["group"])
        values = torch.empty(q.shape, dtype=BF16, device=q.device)
        return {"values": torch.mul(q, scale[:, None], out=values), "scale": scale, "sum": h}
    if op == "norm_grad":
        dx, dweight = cq.rms_norm_grad(s["dout"], s["sum"], s["weight"], dsum=s["dsum"], eps=EPS)
        return {"dx": dx, "dweight": dweight}
    return {"y": cq.dequant_gemm_q8(s["packed"], s["norms"], c["n_out"], c["k"], c["bits"], s["table"], s["q"], s["scale"],
                                    group_size=c["group"], out_dtype=TYPES[c["out"]])}


def run(state):
    return _own(state) if own else _plain(state)


# -- work, and the definition in 64 bits ---------------------------------------------------

def work(case):
    c, op = case, case["op"]
    size = {"f32": 4, "bf16": 2}
    if op == "embed":
        elems, ng = c["n"] * c["dim"], c["n"] * -(-c["dim"] // c["group"])
        read = ng * (_group_bytes(c["bits"], c["group"]) + 2) if c["bits"] else elems * size[c["out"]]
        flops = elems * (math.log2(c["group"]) + 1 if c["bits"] else 1)
        return {"bytes": read + elems * size[c["out"]] + c["n"] * c["index"] // 8, "flops": flops}
    if op == "embed_grad":
        elems = c["n"] * c["dim"]
        return {"bytes": elems * size[c["type"]] + c["vocab"] * c["dim"] * 4 + c["n"] * c["index"] // 8, "flops": elems}
    elems = c["rows"] * c["cols"] if "rows" in c else 0
    if op == "norm":
        return {"bytes": elems * (3 * size[c["type"]] + size[c["out"]]) + 4 * c["cols"], "flops": 5 * elems}
    if op == "norm_q8":
        return {"bytes": elems * (3 * size[c["type"]] + 1) + 4 * c["cols"] + 4 * c["rows"],
                "flops": elems * (7 + math.log2(c["group"]))}
    if op == "norm_grad":
        return {"bytes": elems * 4 * size[c["type"]] + 8 * c["cols"], "flops": 11 * elems}
    b, n, k = c["batch"], c["n_out"], c["k"]
    weights = n * (k // c["group"]) * (_group_bytes(c["bits"], c["group"]) + 2)
    return {"bytes": weights + b * k + 4 * b + b * n * size[c["out"]], "flops": 2 * b * n * k}


def _signs64(group):
    """The +-1 Sylvester matrix as the Kronecker power of [[1, 1], [1, -1]]."""
    h = functools.reduce(np.kron, [np.array([[1.0, 1.0], [1.0, -1.0]])] * int(math.log2(group)))
    return torch.from_numpy(h).to(DEV)


def _stored64(packed, norms, levels, bits, group):
    """norm * level of every element in 64 bits, from the bytes bit by bit
    (digit by digit for the five-per-byte form)."""
    if bits == TRITS:
        digits = torch.stack([torch.div(packed.long(), 3 ** i, rounding_mode="floor") % 3 for i in range(5)], -1)
        index = digits.flatten(-2)[..., :group]
    else:
        sb = 2 if bits == TERNARY else bits
        bit = torch.stack([(packed >> j) & 1 for j in range(8)], -1).flatten(-2).unflatten(-1, (group, sb))
        index = sum(bit[..., j].long() << j for j in range(sb))
    table = torch.from_numpy(levels.astype(np.float64)).to(DEV)
    return torch.take(table, index) * norms.double()[..., None]


def exact(case, seed):
    s = prepare(case, seed)
    c, op = case, case["op"]
    if op == "embed":
        ids = s["tokens"].long()
        if not c["bits"]:
            return {"out": s["table"].double().index_select(0, ids) * s["scale"]}
        z = _stored64(s["packed"][ids], s["norms"][ids], s["levels"], c["bits"], c["group"])
        return {"out": (z @ _signs64(c["group"])).flatten(1)[:, :c["dim"]] * (s["scale"] / c["group"])}
    if op == "embed_grad":
        keep = s["tokens"] >= 0
        grad = torch.zeros((c["vocab"], c["dim"]), dtype=torch.float64, device=DEV)
        grad.index_add_(0, s["tokens"][keep].long(), s["dout"][keep].double() * s["scale"])
        return {"grad": grad}
    if op in ("norm", "norm_q8"):
        h = s["x"].double() + s["residual"].double()
        y = h / torch.sqrt(h.square().sum(1, keepdim=True) / c["cols"] + EPS) * s["weight"].double()
        if op == "norm":
            return {"out": y, "sum": h}
        y = (y.reshape(c["rows"], -1, c["group"]) @ _signs64(c["group"])).reshape(c["rows"], -1) / math.sqrt(c["group"])
        top = y.abs().max(1).values
        q = torch.round(127 * y / top[:, None])
        return {"values": q * top[:, None] / 127, "scale": top / 127, "sum": h}
    if op == "norm_grad":
        h, dy, w = s["sum"].double(), s["dout"].double(), s["weight"].double()
        n = h / torch.sqrt(h.square().sum(1, keepdim=True) / c["cols"] + EPS)
        r = 1 / torch.sqrt(h.square().sum(1, keepdim=True) / c["cols"] + EPS)
        dn = dy * w
        dx = s["dsum"].double() + r * (dn - n * (dn * n).sum(1, keepdim=True) / c["cols"])
        return {"dx": dx, "dweight": (dy * n).sum(0)}
    w = _stored64(s["packed"], s["norms"], s["levels"], c["bits"], c["group"]).flatten(1) / math.sqrt(c["group"])
    x = s["q"].double() * s["scale"].double()[:, None]
    return {"y": x @ w.t()}
