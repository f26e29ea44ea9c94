"""What the RMSNorm and grouped calls of the binding refuse before they reach the
library: buffers and streams that are not the tensors' GPU's. Tensors here only
say that they are on a GPU, so this runs without one."""
from types import SimpleNamespace

import pytest
import torch

from fp4_precision_b200 import qfp4 as Q

T, E, N, K, R, C = 100, 3, 128, 128, 4, 64  # 384 rows of the padded layout


class OnGpu0(torch.Tensor):
    def get_device(self):
        return 0


class OnGpu1(torch.Tensor):
    def get_device(self):
        return 1


def gpu(*shape, dtype=torch.bfloat16, cls=OnGpu0):
    return torch.zeros(shape, dtype=dtype).as_subclass(cls)


@pytest.fixture(autouse=True)
def calls(monkeypatch):
    """The names of the library's calls that were reached."""
    from fp4_precision_b200 import build
    build.build()
    reached = []
    monkeypatch.setattr(Q, "_go", lambda fn, what, i, *args: reached.append(what))
    return reached


X, W, X0, DY = gpu(T, K), gpu(E, N, K), gpu(R, C), gpu(T, N)
OFF = gpu(E + 1, dtype=torch.int32)
SEED = Q.make_seed()


def vector(n):
    return gpu(n, dtype=torch.float32)


WITH_WORKSPACE = {
    "rmsnorm_fwd": lambda **k: Q.rmsnorm_fwd(X0, gpu(C), 1e-5, want_amax=True, **k),
    "rmsnorm_bwd": lambda **k: Q.rmsnorm_bwd(X0, X0, gpu(C), vector(R), **k),
    "quantize_grouped": lambda **k: Q.quantize_grouped(X, OFF, Q.NVFP4, Q.RTN, Q.HAD_NONE, Q.ROW, **k),
    "linear_grouped_fwd": lambda **k: Q.linear_grouped_fwd(X, W, OFF, Q.recipe("QUARTET2_NVFP4"), SEED, **k),
    "linear_grouped_bwd": lambda **k: Q.linear_grouped_bwd(DY, X, W, OFF, Q.recipe("QUARTET2_NVFP4"), SEED, **k),
}
BYTES = 1 << 20
BAD_WORKSPACES = {
    "on the CPU": torch.zeros(BYTES, dtype=torch.uint8),
    "on another GPU": gpu(BYTES, dtype=torch.uint8, cls=OnGpu1),
    "one byte for all": gpu(1, dtype=torch.uint8).expand(BYTES),
    "every other byte": gpu(2 * BYTES, dtype=torch.uint8)[::2],
}


@pytest.mark.parametrize("name", WITH_WORKSPACE)
def test_workspaces(calls, name):
    for bad in BAD_WORKSPACES.values():
        with pytest.raises(AssertionError, match="workspace"):
            WITH_WORKSPACE[name](workspace=bad)
    assert not calls
    WITH_WORKSPACE[name](workspace=gpu(BYTES, dtype=torch.uint8))
    WITH_WORKSPACE[name](workspace=None)
    assert calls == 2 * ["qfp4_" + name]


def operand(fmt, rows, k, **other):
    """Buffers for a rows x k operand, or with `other` ones in their place."""
    parts = dict(codes=gpu(rows, k // 2, dtype=torch.uint8), scales=gpu(Q.scales_bytes(fmt, rows, k), dtype=torch.uint8),
                 tensor_scale=gpu(1, dtype=torch.float32))
    named = Q.TensorDesc(*(t.data_ptr() for t in {**parts, **other}.values()))
    return Q.QTensor(**{**parts, **other}, desc=named)


@pytest.mark.parametrize("name,fmt,rows,k,less,call", [
    ("rmsnorm_quantize", Q.MXFP4, R, C, R - 1, lambda q: Q.rmsnorm_quantize(X0, gpu(C), 1e-5, out=q)),
    ("quantize_grouped", Q.NVFP4, 384, K, T, lambda q: Q.quantize_grouped(X, OFF, Q.NVFP4, Q.RTN, 0, Q.ROW, out=q)),
    ("quantize_grouped", Q.MXFP4, K, 384, K - 1, lambda q: Q.quantize_grouped(X, OFF, Q.MXFP4, Q.RTN, 0, Q.COL, out=q)),
])
def test_operand_buffers(calls, name, fmt, rows, k, less, call):
    """Buffers that are too small (x's own rows, say, in place of the padded layout's) or not on the tensors' GPU."""
    good = operand(fmt, rows, k)
    bad = [operand(fmt, rows, k, codes=gpu(less, k // 2, dtype=torch.uint8)),
           operand(fmt, rows, k, scales=gpu(good.scales.numel() - 1, dtype=torch.uint8)),
           operand(fmt, rows, k, tensor_scale=gpu(0, dtype=torch.float32)),
           operand(fmt, rows, k, codes=torch.zeros((rows, k // 2), dtype=torch.uint8)),
           operand(fmt, rows, k, scales=gpu(good.scales.numel(), dtype=torch.uint8, cls=OnGpu1)),
           operand(fmt, rows, k, codes=gpu(rows, k, dtype=torch.uint8)[:, ::2]),
           Q.QTensor(good.codes.clone(), good.scales, good.tensor_scale, good.desc)]
    for q in bad:
        with pytest.raises(AssertionError):
            call(q)
    assert not calls
    assert call(good) is good or call(good)[3] is good
    assert calls[0] == "qfp4_" + name


def quantized(rows, k):
    q = operand(Q.NVFP4, rows, k)
    q.desc.rows, q.desc.k = rows, k
    return q


STREAMED = WITH_WORKSPACE | {
    "rmsnorm_quantize": lambda **k: Q.rmsnorm_quantize(w=gpu(C), x=X0, eps=1e-5, **k),
    "gemm_grouped": lambda **k: Q.gemm_grouped(quantized(384, K), quantized(E * N, K), OFF, T, **k),
    "gemm_grouped_wgrad": lambda **k: Q.gemm_grouped_wgrad(quantized(N, 384), quantized(K, 384), OFF, T, **k),
}


@pytest.mark.parametrize("name", STREAMED)
def test_streams(calls, name):
    """A stream of another GPU than the tensors' would not be the one that the call runs on."""
    def stream(i):
        return SimpleNamespace(device=torch.device("cuda", i))
    with pytest.raises(AssertionError, match="stream"):
        STREAMED[name](stream=stream(1))
    assert not calls
    STREAMED[name](stream=stream(0))
    STREAMED[name](stream=None)
    assert calls == 2 * ["qfp4_" + name]
