"""Timed cases of the operators of an attention block and of a model's end:
the norm of queries and keys per head with the position rotation, attention
over prompts and over a cache, and the log probabilities of given tokens, each
with its gradient.

``own`` selects what ``run`` calls: False, plain torch operations in float32;
True, the entry points of ``rotated_codebook_bit_amd``.

Head layouts and vocabularies are those of the repository's workloads: queries
of 512 and keys of 128 columns (8 and 2 heads of 64) and the 8192 tokens of the
45.5M-parameter set, the 4096 columns (32 heads of 128) and 32000 tokens of the
7B-shaped model, also with 8 key heads as generic grouped attention has them.
"""

import math
import random

import torch

own = False

DEV = "cuda"
EPS = 1e-6
F32, F64, BF16 = torch.float32, torch.float64, torch.bfloat16
TYPES = {"f32": F32, "bf16": BF16}
SIZE = {"f32": 4, "bf16": 2}


# -- the cases --------------------------------------------------------------------

def listed():
    return [
        # One decode step's queries and keys of the 7B-shaped model: the key and the value go to the cache.
        {"name": "rotate_token", "op": "rotate", "mode": "cache", "n": 1, "qh": 32, "kvh": 32, "d": 128, "rot": 128,
         "type": "bf16", "interleaved": False, "rows": 4096},
        # A chunk of prompts into the cache, grouped heads.
        {"name": "rotate_prompt", "op": "rotate", "mode": "cache", "n": 8192, "qh": 32, "kvh": 8, "d": 128, "rot": 128,
         "type": "bf16", "interleaved": False, "rows": 16384},
        # A training step of the 45.5M-parameter set's heads, forward and gradient, half of each head rotated.
        {"name": "rotate_train_short", "op": "rotate", "mode": "train", "n": 1000, "qh": 8, "kvh": 2, "d": 64, "rot": 32,
         "type": "f32", "interleaved": True},
        # The same of a training batch with grouped heads of 128.
        {"name": "rotate_train_batch", "op": "rotate", "mode": "train", "n": 8192, "qh": 32, "kvh": 8, "d": 128, "rot": 128,
         "type": "bf16", "interleaved": False},
        # One decode step of one long conversation.
        {"name": "attend_token", "op": "attend", "mode": "cache", "seqs": 1, "cap": 8192, "new": 1, "qh": 32, "kvh": 8,
         "d": 128, "type": "bf16", "mix": 1},
        # One decode step of many conversations of different lengths.
        {"name": "attend_tokens", "op": "attend", "mode": "cache", "seqs": 64, "cap": 8192, "new": 1, "qh": 32, "kvh": 8,
         "d": 128, "type": "bf16", "mix": 2},
        # Packed prompts of the 45.5M-parameter set, odd lengths, float32.
        {"name": "attend_packed", "op": "attend", "mode": "prompt", "seqs": 13, "n": 4001, "qh": 8, "kvh": 2, "d": 64,
         "type": "f32", "mix": 3},
        # One long prompt.
        {"name": "attend_prompt", "op": "attend", "mode": "prompt", "seqs": 1, "n": 8192, "qh": 32, "kvh": 8, "d": 128,
         "type": "bf16", "mix": 4},
        # A training batch of packed documents, forward and gradient.
        {"name": "attend_train", "op": "attend", "mode": "train", "seqs": 3, "n": 8192, "qh": 32, "kvh": 8, "d": 128,
         "type": "bf16", "mix": 5},
        # The scored token of one decode step with its alternatives.
        {"name": "score_token", "op": "score", "mode": "top", "rows": 1, "vocab": 32000, "type": "f32", "top": 5},
        # The scored tokens of a batch of prompts with their alternatives.
        {"name": "score_prompt", "op": "score", "mode": "top", "rows": 4096, "vocab": 32000, "type": "bf16", "top": 20},
        # The loss of a training batch, with an entropy term: forward and gradient of the logits.
        {"name": "score_train", "op": "score", "mode": "train", "rows": 4096, "vocab": 32000, "type": "bf16"},
    ]


def draw(rng):
    def log(lo, hi):
        return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))

    kind = rng.choice(["f32", "bf16", "bf16"])
    kvh = rng.choice([1, 2, 3, 4, 8])
    qh = min(32, kvh * rng.choice([1, 2, 4, 5, 8]))
    qh -= qh % kvh
    d = rng.choice([32, 64, 64, 80, 96, 128, 128])
    mix = rng.randrange(1 << 30)
    op = rng.choice(["rotate", "rotate", "attend", "attend", "attend", "score", "score"])
    if op == "rotate":
        case = {"op": op, "mode": rng.choice(["cache", "train"]), "n": log(1, 8192), "qh": qh, "kvh": kvh, "d": d,
                "rot": rng.choice([d, d, d // 2]), "type": kind, "interleaved": rng.choice([False, True])}
        if case["mode"] == "cache":
            case["rows"] = case["n"] + log(1, 8192)
        return case
    if op == "attend":
        mode = rng.choice(["cache", "prompt", "train"])
        if mode == "cache":
            seqs = log(1, 64)
            return {"op": op, "mode": mode, "seqs": seqs, "cap": log(16, 8192), "new": rng.choice([1, 1, 1, 2, 5]), "qh": qh,
                    "kvh": kvh, "d": d, "type": kind, "mix": mix}
        n = log(16, 6000 if mode == "prompt" else 3000)
        return {"op": op, "mode": mode, "seqs": min(log(1, 40), n), "n": n, "qh": qh, "kvh": kvh, "d": d, "type": kind,
                "mix": mix}
    rows, vocab = log(1, 4096), log(300, 32000)
    if rng.random() < 0.5:
        return {"op": op, "mode": "train", "rows": rows, "vocab": vocab, "type": kind}
    return {"op": op, "mode": "top", "rows": rows, "vocab": vocab, "type": kind, "top": rng.choice([0, 1, 5, 8, 20])}


def _lengths(case):
    """(new tokens, keys) of every sequence."""
    rng = random.Random(case["mix"])
    if case["mode"] == "cache":
        low = min(case["new"], case["cap"])
        return [(case["new"], case["cap"] if i == 0 else rng.randint(low, case["cap"])) for i in range(case["seqs"])]
    parts = [rng.expovariate(1.0) + 0.05 for _ in range(case["seqs"])]
    left = case["n"] - case["seqs"]
    lens = [1 + int(left * p / sum(parts)) for p in parts]
    lens[-1] += case["n"] - sum(lens)
    return [(m, m) for m in lens]


# -- inputs -------------------------------------------------------------------------

def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    kind, s = TYPES[case["type"]], {"case": dict(case)}

    def randn(*shape, dtype=F32, scale=1.0):
        return (torch.randn(shape, generator=gen, device=DEV) * scale).to(dtype)

    def whole(high, *shape, dtype=torch.int64):
        return torch.randint(0, high, shape, generator=gen, device=DEV, dtype=dtype)

    if case["op"] == "score":
        s["logits"] = randn(case["rows"], case["vocab"], dtype=kind, scale=2.5)
        s["tokens"] = whole(case["vocab"], case["rows"])
        s["scale"] = 0.8  # one over the temperature
        if case["mode"] == "train":
            s["tokens"][torch.rand(case["rows"], generator=gen, device=DEV) < 0.02] = -1  # padding
            s["dlogprob"] = torch.full((case["rows"],), -1.0 / case["rows"], device=DEV) * (1 + 0.1 * randn(case["rows"]))
            s["dentropy"] = torch.full((case["rows"],), -0.01 / case["rows"], device=DEV)
        return s
    qh, kvh, d = case["qh"], case["kvh"], case["d"]
    if case["op"] == "rotate":
        n = case["n"]
        s["qkv"] = randn(n, qh + 2 * kvh, d, dtype=kind)
        s["positions"] = whole(100000, 1) + torch.arange(n, device=DEV)
        half = case["rot"] // 2
        s["freqs"] = (10000.0 ** (-torch.arange(half, device=DEV, dtype=F64) / half)).float()
        s["qw"], s["kw"] = 1 + randn(d, scale=0.1), 1 + randn(d, scale=0.1)
        if case["mode"] == "cache":
            s["k_cache"], s["v_cache"] = randn(case["rows"], kvh, d, dtype=kind), randn(case["rows"], kvh, d, dtype=kind)
            s["slots"] = torch.randperm(case["rows"], generator=gen, device=DEV)[:n]
        else:
            s["dq"], s["dk"] = randn(n, qh, d, dtype=kind, scale=1e-2), randn(n, kvh, d, dtype=kind, scale=1e-2)
        return s
    lens = _lengths(case)
    s["scale"] = 1.0 / math.sqrt(d)
    if case["mode"] == "cache":
        b, cap = case["seqs"], case["cap"]
        s["q"] = randn(b * case["new"], qh, d, dtype=kind)
        s["k"], s["v"] = randn(b * cap, kvh, d, dtype=kind), randn(b * cap, kvh, d, dtype=kind)
        s["lens"] = torch.tensor([m for _, m in lens], dtype=torch.int32, device=DEV)
        return s
    starts = [0]
    for m, _ in lens:
        starts.append(starts[-1] + m)
    s["bounds"] = starts  # the same in the program's hands on the host
    s["starts"] = torch.tensor(starts, dtype=torch.int32, device=DEV)
    s["qkv"] = randn(case["n"], qh + 2 * kvh, d, dtype=kind)
    if case["mode"] == "train":
        s["dout"] = randn(case["n"], qh, d, dtype=kind, scale=1e-2)
    return s


def _split(s):
    """q, k and v as views of the fused projection's output."""
    c = s["case"]
    return s["qkv"].split([c["qh"], c["kvh"], c["kvh"]], dim=1)


# -- the plain forms ----------------------------------------------------------------

def _turn(x, cos, sin, rot, interleaved):
    """x [n, heads, d] with its first `rot` values turned by the angles."""
    cos, sin = cos[:, None], sin[:, None]
    if interleaved:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        turned = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    else:
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        turned = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    return torch.cat([turned, x[..., rot:]], -1)


def _plain_rotate(s):
    c = s["case"]
    kind = TYPES[c["type"]]
    q, k, v = _split(s)
    angle = s["positions"].double()[:, None] * s["freqs"].double()
    cos, sin = angle.cos().float(), angle.sin().float()

    def forward(x, w):
        x = x.float()
        y = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * w
        return _turn(y, cos, sin, c["rot"], c["interleaved"]).to(kind)

    def backward(dy, x, w):
        x, u = x.float(), _turn(dy.float(), cos, -sin, c["rot"], c["interleaved"])
        r = torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS)
        z = u * w
        dx = r * (z - x * (r * r) * (z * x).mean(-1, keepdim=True))
        return dx.to(kind), (u * x * r).sum((0, 1))

    if c["mode"] == "cache":
        s["k_cache"][s["slots"]] = forward(k, s["kw"])
        s["v_cache"][s["slots"]] = v
        return {"q": forward(q, s["qw"]), "k": s["k_cache"], "v": s["v_cache"]}
    dq, dqw = backward(s["dq"], q, s["qw"])
    dk, dkw = backward(s["dk"], k, s["kw"])
    return {"q": forward(q, s["qw"]), "k": forward(k, s["kw"]), "dq": dq, "dk": dk, "dqw": dqw, "dkw": dkw}


def _rows(x, kvh):
    """[n, heads, d] as [kvh, group * n, d] in float32."""
    n, h, d = x.shape
    return x.float().view(n, kvh, h // kvh, d).permute(1, 2, 0, 3).reshape(kvh, -1, d)


def _back(x, n):
    """[kvh, group * n, ...] as [n, heads, ...]."""
    kvh, gn = x.shape[:2]
    x = x.view(kvh, gn // n, n, *x.shape[2:])
    return x.permute(2, 0, 1, *range(3, x.dim())).flatten(1, 2)


def _plain_cache(s):
    """All sequences at once over the whole cache, masked by length."""
    c = s["case"]
    b, cap, new, kvh, d = c["seqs"], c["cap"], c["new"], c["kvh"], c["d"]
    g = c["qh"] // kvh
    q = s["q"].float().view(b, new, kvh, g, d).permute(0, 2, 3, 1, 4).reshape(b, kvh, g * new, d)
    k = s["k"].float().view(b, cap, kvh, d).permute(0, 2, 3, 1).contiguous()
    v = s["v"].float().view(b, cap, kvh, d).transpose(1, 2).contiguous()
    last = s["lens"].long()[:, None] - new + torch.arange(new, device=DEV)
    seen = torch.arange(cap, device=DEV) <= last[..., None]
    seen = seen[:, None, None].expand(b, 1, g, new, cap).reshape(b, 1, g * new, cap)
    x = (q @ k * s["scale"]).masked_fill(~seen, -math.inf)
    m = x.amax(-1, keepdim=True)
    p = torch.exp(x - m)
    total = p.sum(-1, keepdim=True)

    def out(t):
        return t.view(b, kvh, g, new, -1).permute(0, 3, 1, 2, 4).reshape(b * new, c["qh"], -1)

    return {"out": out(p @ v / total).to(s["q"].dtype), "lse": out(m + total.log()).squeeze(-1)}


def _plain_attend(s):
    c = s["case"]
    if c["mode"] == "cache":
        return _plain_cache(s)
    kvh, kind, train = c["kvh"], TYPES[c["type"]], c["mode"] == "train"
    parts = []
    for lo, hi in zip(s["bounds"], s["bounds"][1:]):
        n = hi - lo
        qkv = s["qkv"][lo:hi]
        q, k, v = (_rows(t, kvh) for t in qkv.split([c["qh"], kvh, kvh], dim=1))
        i = torch.arange(n, device=DEV)
        hidden = (i[None, :] > i[:, None]).repeat(c["qh"] // kvh, 1)
        x = (q @ k.transpose(1, 2) * s["scale"]).masked_fill_(hidden, -math.inf)
        m = x.amax(-1, keepdim=True)
        p = torch.exp(x - m)
        total = p.sum(-1, keepdim=True)
        p = p / total
        o = p @ v
        part = [_back(o, n).to(kind), _back(m + total.log(), n).squeeze(-1)]
        if train:
            do = _rows(s["dout"][lo:hi], kvh)
            ds = p * (do @ v.transpose(1, 2) - (do * o).sum(-1, keepdim=True)) * s["scale"]
            part += [_back(ds @ k, n).to(kind), _back(ds.transpose(1, 2) @ q, n).to(kind),
                     _back(p.transpose(1, 2) @ do, n).to(kind)]
        parts.append(part)
    return dict(zip(("out", "lse", "dq", "dk", "dv"), (torch.cat(t) for t in zip(*parts))))


def _plain_score(s):
    c, t = s["case"], s["tokens"]
    x = s["logits"].float() * s["scale"]
    m = x.amax(1, keepdim=True)
    e = torch.exp(x - m)
    total = e.sum(1, keepdim=True)
    lse = m + total.log()
    entropy = total.log() - (e * (x - m)).sum(1, keepdim=True) / total
    inside = t >= 0
    at = torch.where(inside, t, 0)[:, None]
    logprob = torch.where(inside, (x.gather(1, at) - lse)[:, 0], 0.0)
    out = {"logprob": logprob, "entropy": entropy[:, 0], "lse": lse[:, 0]}
    if c["mode"] == "top":
        order = torch.sort(s["logits"].float(), dim=1, descending=True, stable=True).indices[:, :c["top"]]
        out.update(top=order, top_logprob=x.gather(1, order) - lse)
        return out
    p = e / total
    g = torch.where(inside, s["dlogprob"], 0.0)[:, None]
    dx = -g * p - s["dentropy"][:, None] * p * (x - lse + entropy)
    dx.scatter_add_(1, at, g)
    out["dlogits"] = (dx * s["scale"]).to(s["logits"].dtype)
    return out


# -- the framework's calls --------------------------------------------------------------

def _own(s):
    import rotated_codebook_bit_amd as cq

    c = s["case"]
    if c["op"] == "rotate":
        q, k, v = _split(s)
        where = {"interleaved": c["interleaved"], "eps": EPS}
        if c["mode"] == "cache":
            out = cq.qk_norm_rope(q, k, s["positions"], s["freqs"], s["qw"], s["kw"], v=v, slots=s["slots"],
                                  k_out=s["k_cache"], v_out=s["v_cache"], **where)
            return {"q": out[0], "k": s["k_cache"], "v": s["v_cache"]}
        qo, ko = cq.qk_norm_rope(q, k, s["positions"], s["freqs"], s["qw"], s["kw"], **where)
        dq, dk, dqw, dkw = cq.qk_norm_rope_grad(s["dq"], s["dk"], q, k, s["positions"], s["freqs"], s["qw"], s["kw"], **where)
        return {"q": qo, "k": ko, "dq": dq, "dk": dk, "dqw": dqw, "dkw": dkw}
    if c["op"] == "attend":
        if c["mode"] == "cache":
            out, lse = cq.attention(s["q"], s["k"], s["v"], sequences=c["seqs"], k_lens=s["lens"], scale=s["scale"])
            return {"out": out, "lse": lse}
        q, k, v = _split(s)
        where = {"q_starts": s["starts"], "k_starts": s["starts"], "scale": s["scale"]}
        out, lse = cq.attention(q, k, v, **where)
        if c["mode"] == "prompt":
            return {"out": out, "lse": lse}
        dq, dk, dv = cq.attention_grad(s["dout"], q, k, v, out, lse, **where)
        return {"out": out, "lse": lse, "dq": dq, "dk": dk, "dv": dv}
    if c["mode"] == "top":
        r = cq.token_logprobs(s["logits"], s["tokens"], scale=s["scale"], top=c["top"])
        return {"logprob": r.logprob, "entropy": r.entropy, "lse": r.lse, "top": r.top, "top_logprob": r.top_logprob}
    r = cq.token_logprobs(s["logits"], s["tokens"], scale=s["scale"])
    dlogits = cq.token_logprobs_grad(s["logits"], s["tokens"], r.lse, s["dlogprob"], s["dentropy"], r.entropy,
                                     scale=s["scale"])
    return {"logprob": r.logprob, "entropy": r.entropy, "lse": r.lse, "dlogits": dlogits}


def run(state):
    if own:
        return _own(state)
    return {"rotate": _plain_rotate, "attend": _plain_attend, "score": _plain_score}[state["case"]["op"]](state)


# -- work, and the definition in 64 bits ---------------------------------------------------

def work(case):
    c, size = case, SIZE[case["type"]]
    if c["op"] == "score":
        elems = c["rows"] * c["vocab"]
        if c["mode"] == "top":
            return {"bytes": elems * size + c["rows"] * (20 + 12 * c["top"]), "flops": 6 * elems}
        return {"bytes": 2 * elems * size + c["rows"] * 28, "flops": 16 * elems}
    qh, kvh, d = c["qh"], c["kvh"], c["d"]
    if c["op"] == "rotate":
        q, kv = c["n"] * qh * d, c["n"] * kvh * d
        small = c["n"] * 8 + 8 * d + 2 * c["rot"]
        if c["mode"] == "cache":
            return {"bytes": 2 * (q + 2 * kv) * size + small, "flops": 8 * (q + kv)}
        return {"bytes": 4 * (q + kv) * size + small + 8 * d, "flops": 26 * (q + kv)}
    rows = keys = pairs = 0
    for m, n in _lengths(c):
        rows, keys = rows + m, keys + n
        pairs += m * n - m * (m - 1) // 2
    data = 2 * rows * qh * d * size + 2 * keys * kvh * d * size + 4 * rows * qh
    if c["mode"] == "train":
        return {"bytes": 2 * data, "flops": 14 * pairs * qh * d}
    return {"bytes": data, "flops": 4 * pairs * qh * d}


def _exact_rotate(s):
    c = s["case"]
    n, d, rot = c["n"], c["d"], c["rot"]
    q, k, v = (t.double() for t in _split(s))
    # The rotation as a complex product.
    turn = torch.polar(torch.ones((n, 1, rot // 2), dtype=F64, device=DEV),
                       (s["positions"].double()[:, None] * s["freqs"].double()[None])[:, None])
    if c["interleaved"]:
        first, second = torch.arange(0, rot, 2, device=DEV), torch.arange(1, rot, 2, device=DEV)
    else:
        first, second = torch.arange(rot // 2, device=DEV), torch.arange(rot // 2, rot, device=DEV)

    def forward(x, w):
        y = x / torch.sqrt(x.square().sum(-1, keepdim=True) / d + EPS) * w
        z = torch.complex(y[..., first], y[..., second]) * turn
        return y.index_copy(2, first, z.real).index_copy(2, second, z.imag)

    qw, kw = s["qw"].double(), s["kw"].double()
    if c["mode"] == "cache":
        kc, vc = s["k_cache"].double(), s["v_cache"].double()
        kc[s["slots"]] = forward(k, kw)
        vc[s["slots"]] = v
        return {"q": forward(q, qw), "k": kc, "v": vc}
    leaves = [t.requires_grad_() for t in (q, k, qw, kw)]
    with torch.enable_grad():
        qo, ko = forward(q, qw), forward(k, kw)
        grads = torch.autograd.grad([qo, ko], leaves, [s["dq"].double(), s["dk"].double()])
    return {"q": qo.detach(), "k": ko.detach(), "dq": grads[0], "dk": grads[1], "dqw": grads[2], "dkw": grads[3]}


def _exact_attend(s):
    c = s["case"]
    g, lens = c["qh"] // c["kvh"], _lengths(c)
    train = c["mode"] == "train"
    if c["mode"] == "cache":
        q, k, v = s["q"], s["k"], s["v"]
        spans = [(i * c["new"], m, i * c["cap"], n) for i, (m, n) in enumerate(lens)]
    else:
        q, k, v = _split(s)
        spans, at = [], 0
        for m, n in lens:
            spans.append((at, m, at, n))
            at += m
    out = {"out": torch.zeros(q.shape, dtype=F64, device=DEV), "lse": torch.zeros(q.shape[:2], dtype=F64, device=DEV)}
    if train:
        out.update(dq=torch.zeros(q.shape, dtype=F64, device=DEV), dk=torch.zeros(k.shape, dtype=F64, device=DEV),
                   dv=torch.zeros(k.shape, dtype=F64, device=DEV))
    for q0, m, k0, n in spans:
        future = torch.ones((m, n), dtype=torch.bool, device=DEV).triu(n - m + 1)
        for h in range(c["kvh"]):  # a group of heads at a time
            heads = slice(h * g, h * g + g)
            qs = q[q0:q0 + m, heads].double().transpose(0, 1).contiguous().requires_grad_(train)
            ks = k[k0:k0 + n, h].double().contiguous().requires_grad_(train)
            vs = v[k0:k0 + n, h].double().contiguous().requires_grad_(train)
            with torch.set_grad_enabled(train):
                x = (torch.matmul(qs, ks.t()) * s["scale"]).masked_fill(future, -math.inf)
                o = torch.matmul(torch.softmax(x, -1), vs)
            out["out"][q0:q0 + m, heads] = o.detach().transpose(0, 1)
            out["lse"][q0:q0 + m, heads] = torch.logsumexp(x.detach(), -1).t()
            if train:
                grads = torch.autograd.grad(o, [qs, ks, vs], s["dout"][q0:q0 + m, heads].double().transpose(0, 1))
                out["dq"][q0:q0 + m, heads] = grads[0].transpose(0, 1)
                out["dk"][k0:k0 + n, h], out["dv"][k0:k0 + n, h] = grads[1], grads[2]
    return out


def _exact_score(s):
    c, t = s["case"], s["tokens"]
    train = c["mode"] == "train"
    x = s["logits"].double().requires_grad_(train)
    with torch.set_grad_enabled(train):
        logp = torch.log_softmax(x * s["scale"], 1)
        entropy = -(logp.exp() * logp).sum(1)
        logprob = logp.gather(1, t.clamp(min=0)[:, None])[:, 0] * (t >= 0)
    lse = torch.logsumexp(x.detach() * s["scale"], 1)
    out = {"logprob": logprob.detach(), "entropy": entropy.detach(), "lse": lse}
    if train:
        loss = (logprob * s["dlogprob"].double()).sum() + (entropy * s["dentropy"].double()).sum()
        out["dlogits"], = torch.autograd.grad(loss, x)
        return out
    # Position in descending order: equal logits keep the order of their indices.
    left, tops = s["logits"].double(), []
    for _ in range(c["top"]):
        best = left.max(1, keepdim=True).values
        tops.append((left == best).int().argmax(1, keepdim=True))
        left.scatter_(1, tops[-1], -math.inf)
    out["top"] = torch.cat(tops, 1) if tops else torch.zeros((c["rows"], 0), dtype=torch.int64, device=DEV)
    out["top_logprob"] = logp.gather(1, out["top"])
    return out


def exact(case, seed):
    return {"rotate": _exact_rotate, "attend": _exact_attend, "score": _exact_score}[case["op"]](prepare(case, seed))
