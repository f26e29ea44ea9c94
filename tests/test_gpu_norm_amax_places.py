"""The amax that the RMSNorm returns, where one known entry decides it: in every
part of the kernel's walk (first and last rows and columns, a row of a CTA's or
a warp's second turn, a thread's second chunk). Against the oracle's rotation."""
import numpy as np
import pytest
import torch

import oracle as O
from fp4_precision_b200 import qfp4 as Q

pytestmark = pytest.mark.gpu

ROT, STREAM = 0x1234_5678_9ABC, 3
HADS = [Q.HAD_NONE, Q.HAD_DET16, Q.HAD_DET32, Q.HAD_RAND16, Q.HAD_RAND32]

# At most 888 CTAs walk the rows (six on each of 148 SMs), four rows each where a row is one warp's; so rows from 3552
# (C <= 512; 1024 with a 32-point rotation) and from 1024 (more columns) on are a later turn. From 8192 columns on, one
# CTA an SM, and columns past the first half are a thread's second chunk.
PLACES = [(4000, 256, 0, 0), (4000, 256, 3, 255), (4000, 256, 3700, 100), (4000, 256, 3999, 255),
          (3700, 528, 2, 527), (3700, 528, 1500, 511), (3700, 528, 3699, 0),
          (1300, 1536, 1, 1535), (1300, 1536, 1299, 700),
          (400, 8208, 0, 8207), (400, 8208, 399, 4600), (400, 8208, 200, 4608), (320, 16384, 319, 16383),
          (320, 16384, 149, 8192), (1, 4096, 0, 4095)]


@pytest.mark.parametrize("R,C,row,col", PLACES)
def test_one_entry_decides(R, C, row, col):
    g = torch.Generator().manual_seed(R + C + row)
    x = torch.randn((R, C), generator=g).bfloat16()
    x[row] = 0
    x[row, col] = 1  # the norm makes it sqrt(C): sqrt(C) / 4 or more after a rotation
    w = (1 + 0.1 * torch.randn(C, generator=g)).bfloat16()
    xd, wd = x.cuda(), w.cuda()
    for had in HADS:
        n = {Q.HAD_NONE: 1, Q.HAD_DET16: 16, Q.HAD_RAND16: 16}.get(had, 32)
        if C % n:
            continue
        y, _, _, amax = Q.rmsnorm_fwd(xd, wd, 1e-5, had=had, seed=Q.make_seed(ROT, 7, STREAM, 4), want_amax=True)
        v = np.abs(O.rotate(y.cpu(), had, O.ROW, ROT, STREAM))
        best = v.max()
        if n == 1 or C >= 1024:  # the entry, or its rotation group, decides
            at = slice(col // n * n, col // n * n + n)
            assert v[row, at].max() == best
            v[row, at] = 0
            assert v.max() < best
        assert amax.item() == best
    Q.status()
