"""Argument checks and host-only calls of the operators around the products
(embedding, norm, 8-bit product), on the CPU: every refusal comes before
anything is enqueued, so no GPU is needed."""

import ctypes
import os
import subprocess
import sys

import numpy as np
import pytest

import isa_scan as S
import rotated_codebook_bit_amd as cq

try:
    L = cq.lib()
except ImportError:
    pytest.skip("libcq.so is not built", allow_module_level=True)

NULL, ARG, ALIGN, UNSUPPORTED = -1, -2, -3, -4
A, B, C, D, E, F, G, H = (0x10000000 * i for i in range(1, 9))  # addresses far apart, never touched
BIG = 1 << 40


def replace(args, **changes):
    args = dict(args)
    args.update(changes)
    return list(args.values())


EMBED = dict(tokens=A, tb=8, n=4, table=B, td=0, vocab=10, dim=64, scale=1.0, out=C, od=0, stream=None)
PACKED = dict(tokens=A, tb=4, n=4, packed=B, norms=D, vocab=10, dim=64, bits=2, group=128, levels=None, nl=0, scale=1.0, out=C,
              od=1, stream=None)
EGRAD = dict(tokens=A, tb=8, n=100, dout=B, dd=0, vocab=10, dim=64, scale=1.0, acc=0, grad=C, gd=0, ws=D, wb=BIG, stream=None)
NORM = dict(x=A, r=B, dt=0, w=C, wd=0, rows=4, cols=64, eps=1e-6, sum=D, out=E, od=0, stream=None)
NORMQ = dict(x=A, r=B, dt=1, w=C, wd=1, rows=4, cols=256, group=128, eps=1e-6, sum=D, q=E, scale=F, stream=None)
NGRAD = dict(dout=A, sum=B, dsum=C, dt=0, w=D, wd=0, rows=40, cols=256, eps=1e-6, dx=E, dw=F, ws=G, wb=BIG, stream=None)
TABLE = cq.q8_levels(2)
GEMM = dict(packed=A, norms=B, n=32, k=256, bits=2, group=128, table=ctypes.byref(TABLE), q=C, scale=D, batch=4, y=E, yd=0, ws=F,
            wb=BIG, stream=None)

nan, inf = float("nan"), float("inf")
REFUSALS = [
    (L.cq_embed, EMBED, ARG, [dict(tb=2), dict(td=2), dict(od=-1), dict(n=-1), dict(vocab=-1), dict(dim=-1), dict(scale=nan),
                              dict(scale=inf), dict(out=B), dict(out=B + 2544), dict(out=A)]),
    (L.cq_embed, EMBED, NULL, [dict(tokens=None), dict(table=None), dict(out=None)]),
    (L.cq_embed, EMBED, ALIGN, [dict(tokens=A + 4), dict(table=B + 8), dict(out=C + 4)]),
    (L.cq_embed, EMBED, UNSUPPORTED, [dict(n=1 << 31), dict(vocab=1 << 31), dict(n=1 << 30, dim=1 << 20), dict(dim=1 << 40)]),
    (L.cq_embed_packed, PACKED, ARG, [dict(bits=5), dict(nl=3, levels=(ctypes.c_float * 4)(1, 2, 3, 4)), dict(tb=1), dict(od=7),
                                      dict(out=B), dict(out=D), dict(out=A)]),
    (L.cq_embed_packed, PACKED, NULL, [dict(tokens=None), dict(packed=None), dict(norms=None), dict(out=None)]),
    (L.cq_embed_packed, PACKED, ALIGN, [dict(tokens=A + 2), dict(packed=B + 8), dict(norms=D + 1), dict(out=C + 8)]),
    (L.cq_embed_packed, PACKED, UNSUPPORTED, [dict(group=16), dict(group=512), dict(n=1 << 31)]),
    (L.cq_embed_grad, EGRAD, ARG, [dict(acc=2), dict(dd=3), dict(gd=3), dict(wb=100), dict(grad=B), dict(ws=B), dict(ws=C),
                                   dict(ws=A), dict(scale=nan)]),
    (L.cq_embed_grad, EGRAD, NULL, [dict(tokens=None), dict(dout=None), dict(grad=None), dict(ws=None)]),
    (L.cq_embed_grad, EGRAD, ALIGN, [dict(tokens=A + 4), dict(dout=B + 4), dict(grad=C + 4), dict(ws=D + 4)]),
    (L.cq_add_rms_norm, NORM, ARG, [dict(dt=2), dict(wd=2), dict(od=2), dict(rows=-1), dict(cols=-1), dict(eps=-1.0), dict(eps=nan),
                                    dict(eps=inf), dict(out=A), dict(out=B), dict(out=C), dict(out=D), dict(sum=C),
                                    dict(sum=A + 16), dict(sum=B + 16)]),
    (L.cq_add_rms_norm, NORM, NULL, [dict(x=None), dict(out=None)]),
    (L.cq_add_rms_norm, NORM, ALIGN, [dict(x=A + 4), dict(r=B + 8), dict(w=C + 4), dict(sum=D + 4), dict(out=E + 4)]),
    (L.cq_add_rms_norm, NORM, UNSUPPORTED, [dict(cols=32769), dict(rows=1 << 31)]),
    (L.cq_add_rms_norm_q8, NORMQ, ARG, [dict(dt=5), dict(eps=-1.0), dict(q=A), dict(q=D), dict(scale=E), dict(scale=A), dict(scale=C)]),
    (L.cq_add_rms_norm_q8, NORMQ, NULL, [dict(x=None), dict(q=None), dict(scale=None)]),
    (L.cq_add_rms_norm_q8, NORMQ, ALIGN, [dict(q=E + 4), dict(scale=F + 2), dict(x=A + 2)]),
    (L.cq_add_rms_norm_q8, NORMQ, UNSUPPORTED, [dict(cols=200), dict(group=16), dict(group=0), dict(cols=1 << 16)]),
    (L.cq_rms_norm_grad, NGRAD, ARG, [dict(dt=2), dict(eps=nan), dict(dx=A), dict(dx=B), dict(dx=C + 16), dict(dx=D), dict(dx=F),
                                      dict(dw=A), dict(wb=10), dict(ws=A), dict(ws=E), dict(ws=F)]),
    (L.cq_rms_norm_grad, NGRAD, NULL, [dict(dout=None), dict(sum=None), dict(dx=None), dict(ws=None)]),
    (L.cq_rms_norm_grad, NGRAD, ALIGN, [dict(dout=A + 4), dict(dw=F + 4), dict(ws=G + 8), dict(dx=E + 2)]),
    (L.cq_rms_norm_grad, NGRAD, UNSUPPORTED, [dict(cols=40000)]),
    (L.cq_dequant_gemm_q8, GEMM, ARG, [dict(bits=7), dict(yd=2), dict(n=-1), dict(k=-128), dict(batch=0), dict(bits=4), dict(y=A),
                                       dict(y=B), dict(y=C), dict(y=D), dict(bits=cq.TERNARY)]),
    (L.cq_dequant_gemm_q8, GEMM, NULL, [dict(packed=None), dict(norms=None), dict(table=None), dict(q=None), dict(scale=None),
                                        dict(y=None)]),
    (L.cq_dequant_gemm_q8, GEMM, ALIGN, [dict(packed=A + 4), dict(norms=B + 1), dict(q=C + 8), dict(scale=D + 2), dict(y=E + 8)]),
    (L.cq_dequant_gemm_q8, GEMM, UNSUPPORTED, [dict(k=200), dict(group=16), dict(k=1 << 23), dict(bits=cq.TERNARY_TRITS),
                                               dict(n=1 << 31), dict(n=1 << 30, batch=1 << 30)]),
]


@pytest.mark.parametrize("func,base,status,changes", REFUSALS, ids=[f"{f.__name__}{s}" for f, _, s, _ in REFUSALS])
def test_refusals(func, base, status, changes):
    for c in changes:
        assert func(*replace(base, **c)) == status, (c, L.cq_last_error())
        assert L.cq_last_error()


def test_empty_calls_succeed():
    assert L.cq_embed(*replace(EMBED, n=0, tokens=None)) == 0
    assert L.cq_embed(*replace(EMBED, dim=0)) == 0
    assert L.cq_embed_packed(*replace(PACKED, n=0)) == 0
    assert L.cq_embed_grad(*replace(EGRAD, vocab=0)) == 0
    assert L.cq_embed_grad(*replace(EGRAD, dim=0)) == 0
    assert L.cq_embed_grad(*replace(EGRAD, n=0, acc=1)) == 0
    assert L.cq_add_rms_norm(*replace(NORM, rows=0)) == 0
    assert L.cq_add_rms_norm_q8(*replace(NORMQ, rows=0)) == 0
    assert L.cq_rms_norm_grad(*replace(NGRAD, rows=0, dw=None)) == 0
    assert L.cq_dequant_gemm_q8(*replace(GEMM, n=0)) == 0


def size(func, *args):
    out = ctypes.c_int64(-1)
    assert func(*args, ctypes.byref(out)) == 0
    return out.value


def test_workspace_sizes():
    assert size(L.cq_embed_grad_workspace, 0, 10, 10) == 0
    one, many = size(L.cq_embed_grad_workspace, 16384, 32000, 1), size(L.cq_embed_grad_workspace, 16385, 32000, 1)
    assert 2 * 4 * 16384 <= one < many
    assert size(L.cq_embed_grad_workspace, 1 << 20, 32000, 4096) < (1 << 20) * 4096 * 4  # below dout itself
    assert size(L.cq_rms_norm_grad_workspace, 1, 4096, 0) == 0
    assert size(L.cq_rms_norm_grad_workspace, 1 << 20, 4096, 1) <= 512 * 4096 * 4
    assert size(L.cq_dequant_gemm_q8_workspace, 11008, 4096, 1, 128) == 0
    assert L.cq_embed_grad_workspace(-1, 1, 1, ctypes.byref(ctypes.c_int64())) == ARG
    assert L.cq_rms_norm_grad_workspace(1, 1, 0, None) == NULL
    assert L.cq_dequant_gemm_q8_workspace(1, 100, 1, 128, ctypes.byref(ctypes.c_int64())) == UNSUPPORTED


@pytest.mark.parametrize("bits", [cq.TERNARY, cq.TERNARY_TRITS, 2, 3, 4])
def test_q8_levels_of_the_built_in_tables(bits):
    t = cq.q8_levels(bits)
    lv = cq.codebook(bits).astype(np.float64)
    m = 256.0 * np.array(t.hi[:len(lv)]) + np.array(t.lo[:len(lv)])
    assert t.n_levels == len(lv) and 24576 <= np.abs(m).max() <= 32639
    assert np.all(np.array(t.hi[len(lv):]) == 0) and np.all(np.array(t.lo[len(lv):]) == 0)
    assert np.abs(lv - t.scale * m).max() <= 2.1e-5 * np.abs(lv).max() * (1 + 1e-6)
    assert np.sqrt(((lv - t.scale * m) ** 2).mean()) <= 1e-5  # the search, not just the rounding (1.5e-5 at 16 levels)


def test_q8_levels_of_odd_tables():
    # one-sided, far from zero, tiny, huge: still within the bound
    for lv in ([0.5, 0.75, 1.0, 3.0], [-9.0, -8.5, -8.25, -8.0], [1e-30, 2e-30, 3e-30, 4e-30], [-1e30, 0.0, 1e20, 2e30]):
        t = cq.q8_levels(2, lv)
        m = 256.0 * np.array(t.hi[:4]) + np.array(t.lo[:4])
        a = np.array(lv, np.float32).astype(np.float64)
        assert np.abs(a - t.scale * m).max() <= 2.2e-5 * np.abs(a).max()
    with pytest.raises(cq.CQError):
        cq.q8_levels(2, [1, 2, 3])
    with pytest.raises(cq.CQError):
        cq.q8_levels(2, [1, 2, 3, nan])
    with pytest.raises(cq.CQError):
        cq.q8_levels(9)


def test_one_hip_runtime_whatever_is_imported_first():
    """A process that calls the library before it imports torch still has
    torch's HIP runtime only: two of them do not share streams or memory."""
    pytest.importorskip("torch")
    code = ("import rotated_codebook_bit_amd as cq; cq.q8_levels(2); import torch; "
            "print(len({l.split()[-1] for l in open('/proc/self/maps') if 'libamdhip64' in l}))")
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    out = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True, check=True).stdout
    assert int(out) <= 1


def test_binding_refuses_host_tensors():
    torch = pytest.importorskip("torch")
    t = torch.zeros(4, dtype=torch.int64)
    x = torch.zeros(4, 128)
    with pytest.raises(ValueError, match="CUDA"):
        cq.embed(t, x)
    with pytest.raises(TypeError, match="tokens"):
        cq.embed(t.to(torch.int16), x)
    with pytest.raises(TypeError, match="table"):
        cq.embed(t, x.half())
    with pytest.raises(ValueError, match="dout"):
        cq.embed_grad(t, x[:3], 5)
    with pytest.raises(ValueError, match="accumulate"):
        cq.embed_grad(t, x, 5, accumulate=True)
    with pytest.raises(ValueError, match="packed"):
        cq.embed_packed(t, torch.zeros(4, 1, 31, dtype=torch.uint8), torch.zeros(4, 1).half(), 4, 128, 2, None)
    with pytest.raises(ValueError, match="residual"):
        cq.add_rms_norm(x, x[:2])
    with pytest.raises(ValueError, match="weight"):
        cq.add_rms_norm(x, None, x[0, :5])
    with pytest.raises(ValueError, match="CUDA"):
        cq.add_rms_norm_q8(x)
    with pytest.raises(ValueError, match="dout"):
        cq.rms_norm_grad(x[:2], x)
    with pytest.raises(TypeError, match="table"):
        cq.dequant_gemm_q8(x, x, 4, 128, 2, None, x.to(torch.int8), x[:, 0])
    with pytest.raises(ValueError, match="scale"):
        cq.dequant_gemm_q8(x, x, 4, 128, 2, TABLE, x.to(torch.int8), x[:3, 0])


@pytest.mark.parametrize("name", ["embed", "norm", "gemm_q8"])
def test_no_lds_write_register_reuse(name):
    """As test_isa_lds_writes.py, for these kernels."""
    obj = os.path.join(S.BUILD, f"{name}.o")
    if not os.path.exists(obj) or not os.path.exists(f"{S.LLVM}/llvm-objdump"):
        pytest.skip("built objects or LLVM tools not present (run __graft_entry__.build())")
    funcs = S.disassemble(obj)
    assert funcs, "no device functions found"
    bad = {f: S.violations(lines)[:2] for f, lines in funcs.items() if S.violations(lines)}
    assert not bad, bad
