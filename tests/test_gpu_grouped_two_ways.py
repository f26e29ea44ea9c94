"""dY of the grouped layer quantized along its rows and along the tokens from one
read, with every rotation along the rows and along the tokens: the backward pass
with both gradients rounded to nearest, against the oracle and in the
bounds-checked build."""
import dataclasses
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

import helpers
import oracle as O
from fp4_precision_b200 import qfp4 as Q
from test_gpu_grouped import ROT, SRS, cpu, layer_reference, split, within

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HADS = [Q.HAD_NONE, Q.HAD_DET16, Q.HAD_DET32, Q.HAD_RAND16, Q.HAD_RAND32]
FORMATS = [Q.NVFP4, Q.MXFP4, Q.MXFP4_RU]
N, K = 256, 128


def inputs(name):
    sizes, off, T, offsets = split(name)
    return sizes, off, T, offsets, cpu((T, K), 7), cpu((len(sizes), N, K), 8, 0.05), cpu((T, N), 9, 1e-3)


def recipe(q, fmt, had_row, had_col):
    rec = q.recipe("NVIDIA_NVFP4")
    for c, had in ((rec.dgrad, had_row), (rec.wgrad, had_col)):
        c.fmt, c.had, c.rnd_a, c.rnd_b = fmt, had, q.RTN, q.RTN
    return rec


@pytest.mark.parametrize("name", ["outside", "skewed"])
@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("had_row", HADS)
def test_backward(name, fmt, had_row):
    sizes, off, T, offsets, x, w, dy = inputs(name)
    X, W, dY = x.cuda(), w.cuda(), dy.cuda()
    inside = slice(int(off[0]), int(off[-1]))
    dY[:inside.start], dY[inside.stop:] = float("nan"), float("nan")  # rows of no group are not read
    for had_col in HADS:
        dX, dW = Q.linear_grouped_bwd(dY, X, W, offsets, recipe(Q, fmt, had_row, had_col), Q.make_seed(ROT, SRS))
        Q.status()
        r = O.preset("NVIDIA_NVFP4")
        r = O.Recipe(r.fprop, *(dataclasses.replace(c, fmt=fmt, had=had, rnd_a=O.RTN, rnd_b=O.RTN)
                                for c, had in ((r.dgrad, had_row), (r.wgrad, had_col))))
        _, dx, dw = layer_reference(dy, x, w, sizes, off, T, r)
        within(dX[inside], dx[0][inside], dx[1][inside], True)
        within(dW, dw[0], dw[1], False)


def run_cases(q):
    out = {}
    for name in ("outside", "ragged"):
        sizes, off, T, offsets, x, w, dy = inputs(name)
        inside = slice(int(off[0]), int(off[-1]))
        for fmt in FORMATS:
            for hr in HADS:
                for hc in HADS:
                    dX, dW = q.linear_grouped_bwd(dy.cuda(), x.cuda(), w.cuda(), offsets, recipe(q, fmt, hr, hc),
                                                  q.make_seed(ROT, SRS))
                    q.status()
                    out[f"{name}.{fmt}.{hr}.{hc}.x"] = dX[inside].contiguous().view(torch.int16).cpu().numpy()
                    out[f"{name}.{fmt}.{hr}.{hc}.w"] = dW.view(torch.int32).cpu().numpy()
    return out


CHILD = r"""
import sys
sys.path[:0] = [{root!r}, {tests!r}]
import numpy as np
from fp4_precision_b200 import qfp4 as Q
import test_gpu_grouped_two_ways as t
np.savez({path!r}, **t.run_cases(Q))
"""


def test_checked_build_agrees():
    path = os.path.join(helpers.scratch_dir("two_ways_"), "out.npz")
    code = CHILD.format(root=ROOT, tests=os.path.dirname(os.path.abspath(__file__)), path=path)
    subprocess.run([sys.executable, "-c", code], env=dict(os.environ, QFP4_BOUNDS_CHECK="1"), check=True, timeout=600)
    want, got = run_cases(Q), np.load(path)
    assert set(got.files) == set(want)
    for name in want:
        assert np.array_equal(got[name], want[name]), name
