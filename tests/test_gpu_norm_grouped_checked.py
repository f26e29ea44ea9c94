"""The RMSNorm and grouped entry points in the bounds-checked build (every
kernel store address checked against its buffer): no store is out of bounds and
the results are those of the normal build, byte for byte. And every one of them
opens an NVTX range of its name."""
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

import helpers

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def run_cases(Q, dev):
    """Every output of a fixed set of calls, as named uint8 arrays (status checked after each)."""
    out = {}
    g = torch.Generator().manual_seed(7)

    def rnd(*shape):
        return torch.randn(shape, generator=g).bfloat16().to(dev)

    def keep(name, *ts):
        Q.status()
        for i, t in enumerate(ts):
            if t is not None:
                out[f"{name}.{i}"] = t.detach().contiguous().view(torch.uint8).cpu().numpy().ravel()

    seed = Q.make_seed(11, 12, 3, 4)
    for R, C in ((1, 32), (131, 512), (130, 1056), (77, 2080), (3, 16384)):
        x, r, w, dy = rnd(R, C), rnd(R, C), rnd(C), rnd(R, C)
        wide = rnd(R, C + 8)[:, 8:]  # rows that are not 32-byte aligned
        for had in (Q.HAD_NONE, Q.HAD_RAND16, Q.HAD_DET32):
            keep(f"norm{R}.{C}.{had}", *Q.rmsnorm_fwd(x, w, 1e-5, res=wide, had=had, seed=seed, want_amax=True))
            y, h, rstd, q = Q.rmsnorm_quantize(x, w, 1e-5, res=r, had=had, seed=seed)
            keep(f"normq{R}.{C}.{had}", y, h, rstd, q.codes, q.scales[:Q.scales_bytes(Q.MXFP4, R, C)])
        keep(f"bwd{R}.{C}", *Q.rmsnorm_bwd(dy, h, w, rstd, dh=r))
    for sizes in ([5, 0, 128, 129, 1, 300], [0, 700], [1] * 200):
        E, N, K = len(sizes), 128 if len(sizes) > 9 else 384, 128 if len(sizes) > 9 else 256
        off = torch.tensor([0, *np.cumsum(sizes)], dtype=torch.int32, device=dev)
        T = sum(sizes)
        X, W, dY = rnd(T, K), rnd(E, N, K), rnd(T, N)
        for name in Q.PRESETS:
            rec = Q.recipe(name)
            keep(f"layer{E}{name}", Q.linear_grouped_fwd(X, W, off, rec, seed),
                 *Q.linear_grouped_bwd(dY, X, W, off, rec, seed))
        for axis in (Q.ROW, Q.COL):
            Tp = Q.group_rows(T, E)
            q = Q.empty_qtensor(Q.MXFP4, *((Tp, K) if axis == Q.ROW else (K, Tp)), dev)
            q.codes.zero_(), q.scales.zero_()
            Q.quantize_grouped(X, off, Q.MXFP4, Q.SR, Q.HAD_RAND32, axis, seed, out=q)
            keep(f"q{E}{axis}", q.codes, q.scales)
        rec = Q.recipe("NVIDIA_NVFP4")
        rec.dgrad.rnd_a = rec.wgrad.rnd_a = Q.RTN
        rec.y_dtype = rec.dx_dtype = Q.OUT_F32
        rec.dw_accumulate = 1
        keep(f"rtn{E}", Q.linear_grouped_fwd(X, W, off, rec, seed),
             *Q.linear_grouped_bwd(dY, X, W, off, rec, seed, dW=torch.ones((E, N, K), device=dev)))
    return out


CHILD = r"""
import os, sys
sys.path[:0] = [{root!r}, {tests!r}]
import numpy as np, torch
from fp4_precision_b200 import qfp4 as Q
import test_gpu_norm_grouped_checked as t
np.savez({path!r}, **t.run_cases(Q, torch.device("cuda", 0)))
"""


def test_checked_build_agrees():
    from fp4_precision_b200 import qfp4 as Q
    d = helpers.scratch_dir("checked_")
    path = os.path.join(d, "out.npz")
    code = CHILD.format(root=ROOT, tests=os.path.dirname(os.path.abspath(__file__)), path=path)
    subprocess.run([sys.executable, "-c", code], env=dict(os.environ, QFP4_BOUNDS_CHECK="1"), check=True, timeout=600)
    want = run_cases(Q, torch.device("cuda", 0))
    got = np.load(path)
    assert set(got.files) == set(want)
    for name in want:
        assert np.array_equal(got[name], want[name]), name


NVTX_CHILD = r"""
import sys, torch
sys.path[:0] = [{root!r}, {tests!r}]
from fp4_precision_b200 import qfp4 as Q
import test_gpu_norm_grouped_checked as t
t.run_cases(Q, torch.device("cuda", 0))
A = Q.quantize(torch.ones((128, 128), dtype=torch.bfloat16, device="cuda"), Q.MXFP4, Q.RTN, Q.HAD_NONE, Q.ROW)
off = torch.tensor([0, 1], dtype=torch.int32, device="cuda")
Q.gemm_grouped(A, A, off, 1)
Q.gemm_grouped_wgrad(A, A, off, 1)
Q.status()
"""


def test_entry_points_open_named_ranges():
    d = helpers.scratch_dir("nvtx_")
    lib, log = os.path.join(d, "libnvtx_record.so"), os.path.join(d, "nvtx.log")
    subprocess.check_call(["gcc", "-shared", "-fPIC", "-O1", "-I", "/usr/local/cuda/include",
                           os.path.join(ROOT, "tests", "nvtx_record.c"), "-o", lib])
    code = NVTX_CHILD.format(root=ROOT, tests=os.path.dirname(os.path.abspath(__file__)))
    subprocess.run([sys.executable, "-c", code], env=dict(os.environ, NVTX_INJECTION64_PATH=lib, QFP4_NVTX_LOG=log),
                   check=True, timeout=600)
    lines = open(log).read().splitlines()
    names = {line[5:] for line in lines if line.startswith("push ")}
    assert lines.count("pop") == sum(line.startswith("push ") for line in lines)
    for n in ("rmsnorm_fwd", "rmsnorm_quantize", "rmsnorm_bwd", "quantize_grouped", "gemm_grouped", "gemm_grouped_wgrad",
              "linear_grouped_fwd", "linear_grouped_bwd"):
        assert "qfp4_" + n in names, n
