"""What the RMSNorm and grouped calls of the binding refuse before they reach the
library: buffers and streams that are not the tensors' GPU's. Tensors here only
say that they are on a GPU, so this runs without one."""
import pytest
import torch

from fp4_precision_b200 import qfp4 as Q

T, E, N, K, R, C = 40, 3, 128, 128, 4, 64


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
