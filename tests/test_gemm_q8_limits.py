"""Sizes of the 8-bit product at a launch's 2^32 threads, on the CPU: what
would pass them is refused with CQ_ERR_UNSUPPORTED by the size function and by
the call, before anything is enqueued.  Up to 64 batch rows (32 at G = 256)
512 threads serve 16 outputs; past that 256 threads serve 128 x 128 values."""

import ctypes

import pytest

import rotated_codebook_bit_amd as cq

try:
    L = cq.lib()
except ImportError:
    pytest.skip("libcq.so is not built", allow_module_level=True)

OK, UNSUPPORTED = 0, -4
TABLE = cq.q8_levels(2)
FEW = (1 << 27) - 16  # outputs: 2^23 - 1 blocks of 512 threads
TILES = (1 << 24) - 1  # blocks of 256 threads

# n_out, k, batch, group
INSIDE = [(FEW, 128, 1, 128), (FEW, 32, 64, 32), (FEW, 256, 32, 256), ((1 << 27) - 1, 128, 65, 128), ((1 << 27) - 1, 256, 33, 256),
          (128, 32, TILES * 128, 32), (1, 128, TILES * 128, 128), (((1 << 20) - 1) * 128, 128, 128 * 16, 128), (0, 128, 1, 128)]
OUTSIDE = [(FEW + 1, 128, 1, 128), ((1 << 27) - 1, 32, 64, 32), (FEW + 1, 256, 32, 256), (1 << 27, 128, 65, 128),
           (128, 32, TILES * 128 + 1, 32), (1, 128, TILES * 128 + 1, 128), (129, 128, TILES * 64 + 1, 128),
           (TILES * 8, 128, 128 * 16, 128), ((1 << 27) - 1, 128, 1 << 20, 128)]


@pytest.mark.parametrize("n_out,k,batch,group", INSIDE)
def test_inside(n_out, k, batch, group):
    need = ctypes.c_int64(-1)
    assert L.cq_dequant_gemm_q8_workspace(n_out, k, batch, group, ctypes.byref(need)) == OK, L.cq_last_error()
    assert need.value >= 0


@pytest.mark.parametrize("n_out,k,batch,group", OUTSIDE)
def test_outside(n_out, k, batch, group):
    assert L.cq_dequant_gemm_q8_workspace(n_out, k, batch, group, ctypes.byref(ctypes.c_int64())) == UNSUPPORTED
    far = 1 << 44  # addresses far apart, never touched
    args = [far * i for i in range(1, 7)]
    assert L.cq_dequant_gemm_q8(args[0], args[1], n_out, k, 2, group, ctypes.byref(TABLE), args[2], args[3], batch, args[4], 0,
                                args[5], far - 1, None) == UNSUPPORTED
    assert b"grid" in L.cq_last_error() or b"2^27" in L.cq_last_error()
