"""Groups that end anywhere within a warp's 32 rows, and columns that end
anywhere within its 128: the epilogues' ragged edges, where lanes of one warp do
different things between its collective loads from tensor memory."""
import numpy as np
import pytest
import torch

import helpers
import oracle as O
from fp4_precision_b200 import qfp4 as Q
from test_gpu_grouped import cpu, operands, padded, starts, within

pytestmark = pytest.mark.gpu

SIZES = [*range(1, 34), 63, 64, 65, 95, 97, 127, 128, 129, 159, 161, 255, 257, 300]


@pytest.mark.parametrize("pair", ["0", "1"])
@pytest.mark.parametrize("N", [8, 136, 200, 416])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_every_tail(monkeypatch, pair, N, dtype):
    monkeypatch.setenv("QFP4_GEMM_PAIR", pair)
    E, K = len(SIZES), 128
    off = np.concatenate(([0], np.cumsum(SIZES)))
    T = int(off[-1])
    offsets = torch.tensor(off, dtype=torch.int32, device="cuda")
    xp = padded(cpu((T, K), 1), SIZES, off, T)
    (A, B), (a, b) = operands(Q.NVFP4, Q.HAD_NONE, xp, Q.ROW, cpu((N, E * K), 2, 0.1), Q.ROW)
    out, guard = helpers.guarded_matrix(T, N, dtype, "cuda")
    out.fill_(-5)
    Q.gemm_grouped(A, B, offsets, T, out=out)
    Q.status()
    helpers.assert_guards_intact(guard)
    p = starts(SIZES)
    parts = [(a[p[e]:p[e] + m], b[:, e * K:(e + 1) * K]) for e, m in enumerate(SIZES)]
    ref = np.concatenate([x @ w.T for x, w in parts])
    bound = np.concatenate([O.GEMM_REL_BOUND * (np.abs(x) @ np.abs(w).T) for x, w in parts])
    within(out, ref, bound, dtype == torch.bfloat16)
