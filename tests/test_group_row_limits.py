"""Rows in groups by the thousand million: the 32-bit row counts."""
import ctypes

import pytest
import torch

from fp4_precision_b200 import qfp4 as Q

P = 1 << 20  # an aligned address that a refused call never follows
MOST = (1 << 31) - 1024


@pytest.mark.parametrize("T,E", [(MOST + 1, 1), ((1 << 31) - 128, 1), (MOST - 2 * 127 + 127, 3)])
def test_more_rows_than_the_kernels_count_are_refused(T, E):
    from fp4_precision_b200 import build
    build.build()
    lib, seed, rec = Q.lib(), ctypes.byref(Q.make_seed()), Q.recipe("AMD_MXFP4_H")
    rows = Q.group_rows(T, E)
    assert MOST < rows < 1 << 31
    t = lambda rows, k: ctypes.byref(Q.TensorDesc(P, P, P, rows, k, Q.MXFP4, 0, 0, 0, 0))  # noqa: E731
    for axis in (Q.ROW, Q.COL):
        assert lib.qfp4_quantize_grouped(P, T, 64, 64, P, E, Q.MXFP4, Q.RTN, 0, axis, seed, None, t(0, 0), P, 1 << 20,
                                         None) == Q.ERR_INVALID_ARG
    assert lib.qfp4_gemm_grouped(t(rows, 128), t(128 * E, 128), P, E, T, P, 128, 0, None) == Q.ERR_INVALID_ARG
    assert lib.qfp4_gemm_grouped_wgrad(t(128, rows), t(128, rows), P, E, T, P, 1, 0, None) == Q.ERR_INVALID_ARG
    assert lib.qfp4_linear_grouped_fwd(P, P, P, P, E, T, 128, 128, ctypes.byref(rec), seed, None, P, 1 << 50,
                                       None) == Q.ERR_INVALID_ARG
    assert lib.qfp4_linear_grouped_bwd(P, P, P, P, P, P, E, T, 128, 128, ctypes.byref(rec), seed, P, 1 << 50,
                                       None) == Q.ERR_INVALID_ARG


@pytest.mark.gpu
def test_first_group_far_behind_the_first_row():
    """The first group's row and the rows to walk add up to more than 2^31."""
    T, C, last = 5 << 28, 16, 1000
    x = torch.empty((T, C), dtype=torch.bfloat16, device="cuda")
    x[-last:] = torch.randn((last, C), generator=torch.Generator().manual_seed(1)).bfloat16().cuda()
    cuts = torch.tensor([0, 300, last], dtype=torch.int32, device="cuda")
    assert T - last + T > 1 << 31
    q = Q.quantize_grouped(x, cuts + (T - last), Q.NVFP4, Q.RTN, Q.HAD_NONE, Q.ROW)
    want = Q.quantize_grouped(x[-last:], cuts, Q.NVFP4, Q.RTN, Q.HAD_NONE, Q.ROW)
    Q.status()
    assert torch.equal(q.tensor_scale, want.tensor_scale)
    for rows in (slice(0, 300), slice(384, 384 + last - 300)):
        assert torch.equal(q.codes[rows], want.codes[rows])
    # scale atoms of 128 rows, the groups' whole ones
    for rows in (slice(0, 256), slice(384, 1024)):
        s = slice(rows.start * 4, rows.stop * 4)
        assert torch.equal(q.scales[s], want.scales[s])
    del x, q
    torch.cuda.empty_cache()  # 60 GB
