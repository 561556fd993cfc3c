"""Argument checks and host-only calls of the operators of an attention block
and a model's end, on the CPU: every refusal comes before anything is
enqueued, so no GPU is needed; and the scan of their built code."""

import ctypes
import os

import pytest

import isa_scan as S
import rotated_codebook_bit_amd as cq

try:
    L = cq.lib()
except ImportError:
    pytest.skip("libcq.so is not built", allow_module_level=True)

NULL, ARG, ALIGN, UNSUPPORTED = -1, -2, -3, -4
A, B, C, D, E, F, G, H, I, J, K = (0x10000000 * i for i in range(1, 12))  # addresses far apart, never touched
BIG = 1 << 40
nan, inf = float("nan"), float("inf")


def heads(data, row=512, head=64):
    return ctypes.byref(cq.Heads(data, row, head))


def seqs(n=1, q=100, k=200, qs=None, ks=None, kl=None, ib=4):
    return ctypes.byref(cq.Sequences(n, q, k, qs, ks, kl, ib))


def replace(args, **changes):
    args = dict(args)
    args.update(changes)
    return list(args.values())


ROTATE = dict(q=heads(A), k=heads(B), v=heads(C), dt=0, n=10, qh=8, kvh=2, d=64, norm=1, qw=D, kw=D + 4096, wd=0, eps=1e-6, pos=E, pb=8,
              freqs=F, rot=64, inter=0, qo=heads(G), ko=heads(H), vo=heads(I), slots=J, sb=8, rows=50, stream=None)
ROTATE_GRAD = dict(dqo=heads(A), dko=heads(B), q=heads(C), k=heads(D), dt=1, n=10, qh=8, kvh=2, d=64, norm=1, qw=E, kw=E + 4096, wd=1,
                   eps=1e-6, pos=F, pb=4, freqs=F + 65536, rot=32, inter=1, dq=heads(G), dk=heads(H), dqw=I, dkw=I + 4096, ws=J, wb=BIG,
                   stream=None)
ATTEND = dict(q=heads(A), k=heads(B), v=heads(C), dt=0, seqs=seqs(), qh=8, kvh=2, d=64, causal=1, scale=0.125, out=heads(D), lse=E, ws=F,
              wb=BIG, stream=None)
ATTEND_GRAD = dict(dout=heads(A), q=heads(B), k=heads(C), v=heads(D), out=heads(E), lse=F, dt=1, seqs=seqs(), qh=8, kvh=2, d=64, causal=1,
                   scale=0.125, dq=heads(G), dk=heads(H), dv=heads(I), ws=J, wb=BIG, stream=None)
SCORE = dict(logits=A, dt=0, rows=10, vocab=1000, stride=1000, scale=1.0, tokens=B, tb=8, logprob=C, entropy=C + 4096, lse=C + 8192, top=5,
             ids=D, lps=E, stream=None)
SCORE_GRAD = dict(logits=A, dt=1, rows=10, vocab=1000, stride=1000, scale=1.0, tokens=B, tb=4, lse=C, dlogprob=D, dentropy=E, entropy=F,
                  dlogits=G, stride2=1000, stream=None)

REFUSALS = [
    (L.cq_qk_norm_rope, ROTATE, ARG, [
        dict(dt=2), dict(n=-1), dict(qh=0), dict(kvh=-1), dict(d=0), dict(norm=2), dict(inter=2), dict(wd=3), dict(eps=-1.0), dict(eps=nan),
        dict(rot=63), dict(rot=66), dict(rot=-2), dict(pb=2), dict(sb=3), dict(rows=-1), dict(norm=0), dict(q=heads(A, -512)),
        dict(qo=heads(G, 512, 0)), dict(qo=heads(G, 0)), dict(qo=heads(G, 256)), dict(ko=heads(H, 64)), dict(qo=heads(A, 1024)),
        dict(qo=heads(A + 16)), dict(qo=heads(H)), dict(ko=heads(B)), dict(vo=heads(C)), dict(ko=heads(J - 64)), dict(ko=heads(E - 32)),
        dict(qo=heads(F)), dict(qo=heads(D - 64))]),
    (L.cq_qk_norm_rope, ROTATE, NULL, [dict(q=None), dict(k=heads(None)), dict(v=None), dict(vo=None), dict(qo=None), dict(pos=None), dict(freqs=None)]),
    (L.cq_qk_norm_rope, ROTATE, ALIGN, [dict(q=heads(A + 8)), dict(k=heads(B, 514)), dict(ko=heads(H, 512, 66)), dict(pos=E + 4), dict(freqs=F + 2),
                                        dict(qw=D + 2), dict(slots=J + 4)]),
    (L.cq_qk_norm_rope, ROTATE, UNSUPPORTED, [dict(d=60), dict(d=264), dict(n=1 << 31), dict(qh=5000), dict(rows=1 << 31),
                                              dict(q=heads(A, (1 << 22) + 4)), dict(k=heads(B, 512, 1 << 60))]),
    (L.cq_qk_norm_rope_grad, ROTATE_GRAD, ARG, [dict(norm=0), dict(wb=100), dict(dqw=I + 4096), dict(dq=heads(C)), dict(dq=heads(A, 1024)),
                                                dict(dk=heads(G)), dict(dq=heads(J)), dict(dqw=C), dict(dqw=E), dict(ws=A), dict(ws=I),
                                                dict(dk=heads(H, 32)), dict(dq=heads(F))]),
    (L.cq_qk_norm_rope_grad, ROTATE_GRAD, NULL, [dict(dqo=None), dict(dko=None), dict(q=None), dict(k=None), dict(dq=None), dict(dk=None), dict(ws=None)]),
    (L.cq_qk_norm_rope_grad, ROTATE_GRAD, ALIGN, [dict(dqw=I + 2), dict(ws=J + 8), dict(dq=heads(G + 4)), dict(dqo=heads(A, 516))]),
    (L.cq_attention, ATTEND, ARG, [
        dict(dt=7), dict(qh=0), dict(qh=9), dict(causal=2), dict(scale=0.0), dict(scale=-1.0), dict(scale=inf), dict(scale=nan), dict(seqs=seqs(-1)),
        dict(seqs=seqs(3)), dict(seqs=seqs(1, -1)), dict(seqs=seqs(1, 100, -1)), dict(seqs=seqs(8, 100, 200)), dict(seqs=seqs(qs=G, ks=G, ib=2)),
        dict(out=heads(A)), dict(out=heads(B)), dict(out=heads(D, 64)), dict(lse=D), dict(lse=A), dict(seqs=seqs(qs=D + 64, ks=G)),
        dict(seqs=seqs(qs=G, ks=G, kl=E))]),
    (L.cq_attention, ATTEND, NULL, [dict(q=None), dict(k=None), dict(v=heads(None)), dict(out=None), dict(seqs=None)]),
    (L.cq_attention, ATTEND, ALIGN, [dict(q=heads(A + 4)), dict(v=heads(C, 510)), dict(lse=E + 2), dict(seqs=seqs(qs=G + 2, ks=G)),
                                     dict(seqs=seqs(kl=G + 4, ib=8))]),
    (L.cq_attention, ATTEND, UNSUPPORTED, [dict(d=36), dict(d=136), dict(qh=8192, kvh=1), dict(seqs=seqs(1, 1 << 31)), dict(k=heads(B, 1 << 23)),
                                           dict(seqs=seqs(1, (1 << 31) - 2), q=heads(1 << 44), out=heads(1 << 50), lse=1 << 55)]),
    (L.cq_attention_grad, ATTEND_GRAD, ARG, [dict(scale=0.0), dict(dq=heads(B)), dict(dk=heads(H), dv=heads(H)), dict(dq=heads(A)), dict(dv=heads(E)),
                                             dict(dq=heads(F)), dict(ws=A), dict(wb=64), dict(dk=heads(J)), dict(dv=heads(I, 128, 32))]),
    (L.cq_attention_grad, ATTEND_GRAD, NULL, [dict(dout=None), dict(q=None), dict(out=None), dict(lse=None), dict(dq=None), dict(dk=None), dict(dv=None),
                                              dict(ws=None), dict(seqs=None)]),
    (L.cq_attention_grad, ATTEND_GRAD, ALIGN, [dict(lse=F + 2), dict(ws=J + 8), dict(dk=heads(H, 516)), dict(dout=heads(A + 2))]),
    (L.cq_attention_grad, ATTEND_GRAD, UNSUPPORTED, [dict(d=136), dict(seqs=seqs(1, 100, 1 << 31))]),
    (L.cq_token_logprobs, SCORE, ARG, [dict(dt=2), dict(rows=-1), dict(vocab=-1), dict(stride=999), dict(scale=0.0), dict(scale=-1.0), dict(scale=nan),
                                       dict(top=-1), dict(top=6, vocab=5), dict(tb=1), dict(logprob=A), dict(lse=C), dict(ids=B), dict(lps=D), dict(entropy=B + 8)]),
    (L.cq_token_logprobs, SCORE, NULL, [dict(logits=None), dict(tokens=None), dict(ids=None), dict(lps=None)]),
    (L.cq_token_logprobs, SCORE, ALIGN, [dict(logits=A + 4), dict(tokens=B + 4), dict(lse=C + 8193), dict(ids=D + 4), dict(lps=E + 2)]),
    (L.cq_token_logprobs, SCORE, UNSUPPORTED, [dict(top=65), dict(vocab=1 << 29, stride=1 << 29), dict(rows=1 << 31), dict(rows=1 << 30, logits=1 << 46)]),
    (L.cq_token_logprobs_grad, SCORE_GRAD, ARG, [dict(tb=3), dict(stride2=999), dict(dlogits=A, stride2=1001), dict(dlogits=A + 16), dict(dlogits=B),
                                                 dict(dlogits=C), dict(dlogits=E), dict(scale=0.0)]),
    (L.cq_token_logprobs_grad, SCORE_GRAD, NULL, [dict(tokens=None), dict(lse=None), dict(dlogprob=None), dict(entropy=None), dict(dlogits=None)]),
    (L.cq_token_logprobs_grad, SCORE_GRAD, ALIGN, [dict(dlogits=G + 8), dict(tokens=B + 2), dict(dlogprob=D + 1)]),
    (L.cq_token_logprobs_grad, SCORE_GRAD, UNSUPPORTED, [dict(rows=1 << 30, logits=1 << 46, dlogits=1 << 54)]),
]


@pytest.mark.parametrize("func,base,status,changes", REFUSALS, ids=[f"{f.__name__}{s}" for f, _, s, _ in REFUSALS])
def test_refusals(func, base, status, changes):
    for c in changes:
        assert func(*replace(base, **c)) == status, (c, L.cq_last_error())
        assert L.cq_last_error()


def test_scales_past_a_power_of_two():
    # scale / log 2 has to be finite: 3e38 is a float32, 3e38 * 1.44 is not.
    for func, base in ((L.cq_attention, ATTEND), (L.cq_attention_grad, ATTEND_GRAD), (L.cq_token_logprobs, SCORE), (L.cq_token_logprobs_grad, SCORE_GRAD)):
        assert func(*replace(base, scale=3e38)) == ARG, func
    assert L.cq_token_logprobs(*replace(SCORE, scale=2.0**127, rows=0)) == 0


def test_empty_calls_succeed():
    assert L.cq_qk_norm_rope(*replace(ROTATE, n=0)) == 0
    assert L.cq_qk_norm_rope_grad(*replace(ROTATE_GRAD, n=0, dqw=None, dkw=None)) == 0
    assert L.cq_attention(*replace(ATTEND, seqs=seqs(0, 0, 0))) == 0
    assert L.cq_attention(*replace(ATTEND, seqs=seqs(4, 0, 200), q=None, out=None)) == 0
    assert L.cq_attention_grad(*replace(ATTEND_GRAD, seqs=seqs(3, 0, 0))) == 0
    assert L.cq_token_logprobs(*replace(SCORE, rows=0)) == 0
    assert L.cq_token_logprobs_grad(*replace(SCORE_GRAD, rows=0)) == 0
    assert L.cq_token_logprobs_grad(*replace(SCORE_GRAD, vocab=0)) == 0


def size(func, *args):
    out = ctypes.c_int64(-1)
    assert func(*args, ctypes.byref(out)) == 0
    return out.value


def test_workspace_sizes():
    assert size(L.cq_attention_workspace, seqs(1, 8192, 8192), 1, 32, 8, 128) == 0
    one = size(L.cq_attention_workspace, seqs(1, 1, 8192), 1, 32, 8, 128)
    assert 0 < one <= 64 * 32 * (128 + 4) * 4
    assert size(L.cq_attention_workspace, seqs(4, 0, 0), 1, 32, 8, 128) == 0
    assert size(L.cq_attention_grad_workspace, seqs(1, 100, 100), 0, 8, 2, 64) >= 2 * 100 * 8 * 4
    assert size(L.cq_qk_norm_rope_grad_workspace, 0, 8, 2, 64) == 0
    assert 0 < size(L.cq_qk_norm_rope_grad_workspace, 1 << 20, 8, 2, 64) <= 1024 * 2 * 64 * 4
    assert L.cq_attention_workspace(seqs(), 0, 8, 2, 64, None) == NULL
    assert L.cq_attention_workspace(seqs(3), 0, 8, 2, 64, ctypes.byref(ctypes.c_int64())) == ARG
    assert L.cq_qk_norm_rope_grad_workspace(1, 8, 2, 60, ctypes.byref(ctypes.c_int64())) == UNSUPPORTED


def test_parts_that_touch_are_refused():
    # Gradients into parts of one tensor, eight heads each, the second one head early.
    row = 3 * 8 * 64
    touching = dict(dq=heads(G, row), dk=heads(G + 7 * 64 * 2, row), dv=heads(G + 16 * 64 * 2, row))
    assert L.cq_attention_grad(*replace(dict(ATTEND_GRAD, kvh=8), **touching)) == ARG and b"overlap" in L.cq_last_error()
    touching = dict(dq=heads(G, row, 192), dk=heads(G + 56 * 2, row, 192), dv=heads(G + 128 * 2, row, 192))
    assert L.cq_attention_grad(*replace(dict(ATTEND_GRAD, kvh=8), **touching)) == ARG and b"overlap" in L.cq_last_error()


@pytest.mark.parametrize("name", ["rotate", "attention", "attention_grad", "logprobs"])
def test_no_lds_write_register_reuse(name):
    obj = os.path.join(S.BUILD, f"{name}.o")
    if not os.path.exists(obj) or not os.path.exists(f"{S.LLVM}/llvm-objdump"):
        pytest.skip("built objects or LLVM tools not present")
    funcs = S.disassemble(obj)
    assert funcs
    bad = {f: S.violations(lines)[:2] for f, lines in funcs.items() if S.violations(lines)}
    assert not bad, bad
    packed = {f for f, lines in funcs.items() for i in lines if i.startswith(("v_pk_add_f32", "v_pk_mul_f32", "v_pk_fma_f32"))}
    assert not packed
