"""What the RMSNorm and the grouped entry points refuse, before anything reaches
a device (these run without a GPU), and their host-side sizes."""
import ctypes

import pytest

from fp4_precision_b200 import qfp4 as Q

P = 1 << 20          # an aligned address that a refused call never follows
ODD = P + 2
SEED = Q.make_seed()


@pytest.fixture(scope="module")
def lib():
    from fp4_precision_b200 import build
    build.build()
    return Q.lib()


def tensor(rows, k, fmt=Q.NVFP4, codes=P, scales=P, ts=P, had=0, rot=0):
    return Q.TensorDesc(codes, scales, ts, rows, k, fmt, had, rot, 0, 0)


def norm_fwd(lib, **kw):
    a = dict(x=P, ldx=64, res=None, ldres=0, w=P, R=4, C=64, eps=1e-5, h=None, ldh=0, y=P, ldy=64, rstd=P, had=0,
             seed=ctypes.byref(SEED), amax=P, ws=P, wsb=1 << 20)
    a.update(kw)
    return lib.qfp4_rmsnorm_fwd(*a.values(), None)


@pytest.mark.parametrize("kw,want", [
    (dict(R=-1), Q.ERR_INVALID_ARG), (dict(R=1 << 31), Q.ERR_INVALID_ARG),
    (dict(C=0), Q.ERR_INVALID_ARG), (dict(C=8), Q.ERR_INVALID_ARG), (dict(C=72, ldx=72, ldy=72), Q.ERR_INVALID_ARG),
    (dict(C=16400, ldx=16400, ldy=16400), Q.ERR_INVALID_ARG),
    (dict(ldx=48), Q.ERR_INVALID_ARG), (dict(ldx=68), Q.ERR_MISALIGNED), (dict(x=ODD), Q.ERR_MISALIGNED),
    (dict(x=None), Q.ERR_INVALID_ARG), (dict(w=None), Q.ERR_INVALID_ARG), (dict(w=ODD), Q.ERR_MISALIGNED),
    (dict(y=None), Q.ERR_INVALID_ARG), (dict(ldy=56), Q.ERR_INVALID_ARG), (dict(rstd=None), Q.ERR_INVALID_ARG),
    (dict(res=P, ldres=64), Q.ERR_INVALID_ARG), (dict(res=P, ldres=64, h=ODD, ldh=64), Q.ERR_MISALIGNED),
    (dict(h=P, ldh=64), Q.ERR_INVALID_ARG),  # y's place
    (dict(eps=-1.0), Q.ERR_INVALID_ARG), (dict(eps=float("nan")), Q.ERR_INVALID_ARG),
    (dict(eps=float("inf")), Q.ERR_INVALID_ARG),
    (dict(had=5), Q.ERR_INVALID_ARG), (dict(had=-1), Q.ERR_INVALID_ARG),
    (dict(had=Q.HAD_DET32, C=48, ldx=48, ldy=48), Q.ERR_INVALID_ARG),
    (dict(had=Q.HAD_RAND16, seed=None), Q.ERR_INVALID_ARG),
    (dict(had=Q.HAD_RAND16, seed=ctypes.byref(Q.make_seed(rot_stream=1 << 28))), Q.ERR_INVALID_ARG),
    (dict(ws=None), Q.ERR_WORKSPACE), (dict(wsb=100), Q.ERR_WORKSPACE), (dict(ws=ODD), Q.ERR_MISALIGNED),
])
def test_rmsnorm_fwd_refuses(lib, kw, want):
    assert norm_fwd(lib, **kw) == want


@pytest.mark.parametrize("kw,want", [
    (dict(fmt=Q.NVFP4), Q.ERR_INVALID_ARG), (dict(fmt=9), Q.ERR_INVALID_ARG),
    (dict(C=48, ldx=48, ldy=48), Q.ERR_INVALID_ARG), (dict(out=None), Q.ERR_INVALID_ARG),
    (dict(out=ctypes.byref(tensor(0, 0, codes=0))), Q.ERR_INVALID_ARG),
    (dict(out=ctypes.byref(tensor(0, 0, scales=ODD))), Q.ERR_MISALIGNED),
    (dict(out=ctypes.byref(tensor(0, 0, ts=0))), Q.ERR_INVALID_ARG),
])
def test_rmsnorm_quantize_refuses(lib, kw, want):
    a = dict(x=P, ldx=64, res=None, ldres=0, w=P, R=4, C=64, eps=1e-5, h=None, ldh=0, y=P, ldy=64, rstd=P,
             fmt=Q.MXFP4, had=0, seed=None, out=ctypes.byref(tensor(0, 0)))
    a.update(kw)
    assert lib.qfp4_rmsnorm_quantize(*a.values(), None) == want


@pytest.mark.parametrize("kw,want", [
    (dict(R=-1), Q.ERR_INVALID_ARG), (dict(C=24), Q.ERR_INVALID_ARG), (dict(dy=None), Q.ERR_INVALID_ARG),
    (dict(lddy=60), Q.ERR_INVALID_ARG), (dict(lddy=68), Q.ERR_MISALIGNED), (dict(h=None), Q.ERR_INVALID_ARG),
    (dict(dh=ODD), Q.ERR_MISALIGNED), (dict(dx=None), Q.ERR_INVALID_ARG), (dict(dw=None), Q.ERR_INVALID_ARG),
    (dict(rstd=None), Q.ERR_INVALID_ARG), (dict(acc=2), Q.ERR_INVALID_ARG), (dict(ws=None), Q.ERR_WORKSPACE),
    (dict(wsb=100), Q.ERR_WORKSPACE), (dict(ws=ODD), Q.ERR_MISALIGNED),
])
def test_rmsnorm_bwd_refuses(lib, kw, want):
    a = dict(dy=P, lddy=64, h=P, ldh=64, w=P, rstd=P, dh=P, lddh=64, R=4, C=64, dx=P, lddx=64, dw=P, acc=0, ws=P,
             wsb=1 << 20)
    a.update(kw)
    assert lib.qfp4_rmsnorm_bwd(*a.values(), None) == want


def test_group_rows(lib):
    """The padded layout holds every split of T rows into E groups, and is a multiple of 128."""
    assert [Q.group_rows(*a) for a in ((0, 5), (-1, 5), (5, 0), (5, 257))] == [0, -1, -1, -1]
    for T in (1, 2, 127, 128, 129, 1000, 4097):
        for E in (1, 2, 7, 256):
            rows = Q.group_rows(T, E)
            assert rows % 128 == 0
            # the worst split: one row in each of the groups but the last
            used = min(E, T)
            worst = max(128 * (g - 1) + (T - (g - 1) + 127) // 128 * 128 for g in range(1, used + 1))
            assert rows >= worst, (T, E)


def test_grouped_sizes(lib):
    rec = Q.recipe("QUARTET2_NVFP4")
    T, E, N, K = 1000, 5, 256, 384
    Tp = Q.group_rows(T, E)
    fwd = Q.linear_grouped_workspace_bytes(False, T, E, N, K, rec)
    bwd = Q.linear_grouped_workspace_bytes(True, T, E, N, K, rec)
    assert fwd >= Q.codes_bytes(Tp, K) + Q.codes_bytes(E * N, K)
    assert bwd >= 2 * Q.codes_bytes(Tp, N) + Q.codes_bytes(K, E * N) + Q.codes_bytes(K, Tp)
    assert lib.qfp4_rmsnorm_bwd_workspace_bytes(0, 64) == 0
    assert lib.qfp4_rmsnorm_bwd_workspace_bytes(1, 64) >= 256


@pytest.mark.parametrize("kw,want", [
    (dict(E=0), Q.ERR_INVALID_ARG), (dict(E=257), Q.ERR_INVALID_ARG), (dict(off=None), Q.ERR_INVALID_ARG),
    (dict(off=ODD), Q.ERR_MISALIGNED), (dict(T=-1), Q.ERR_INVALID_ARG), (dict(x=None), Q.ERR_INVALID_ARG),
    (dict(x=ODD), Q.ERR_MISALIGNED), (dict(ld=60), Q.ERR_INVALID_ARG), (dict(ld=68), Q.ERR_MISALIGNED),
    (dict(fmt=4), Q.ERR_INVALID_ARG), (dict(rnd=3), Q.ERR_INVALID_ARG), (dict(had=7), Q.ERR_INVALID_ARG),
    (dict(axis=2), Q.ERR_INVALID_ARG), (dict(C=40), Q.ERR_INVALID_ARG),
    (dict(axis=1, C=44), Q.ERR_INVALID_ARG), (dict(seed=None), Q.ERR_INVALID_ARG), (dict(out=None), Q.ERR_INVALID_ARG),
    (dict(out=ctypes.byref(tensor(0, 0, codes=ODD))), Q.ERR_MISALIGNED),
    (dict(ws=None), Q.ERR_WORKSPACE), (dict(wsb=4095), Q.ERR_WORKSPACE), (dict(ws=ODD), Q.ERR_MISALIGNED),
])
def test_quantize_grouped_refuses(lib, kw, want):
    a = dict(x=P, T=100, C=64, ld=64, off=P, E=3, fmt=Q.NVFP4, rnd=Q.RTN, had=0, axis=Q.ROW, seed=ctypes.byref(SEED),
             amax=None, out=ctypes.byref(tensor(0, 0)), ws=P, wsb=1 << 30)
    a.update(kw)
    assert lib.qfp4_quantize_grouped(*a.values(), None) == want


ROWS = 384  # of the padded layout of 100 rows in 3 groups


@pytest.mark.parametrize("kw,want", [
    (dict(A=None), Q.ERR_INVALID_ARG), (dict(A=ctypes.byref(tensor(256, 128))), Q.ERR_INVALID_ARG),
    (dict(A=ctypes.byref(tensor(ROWS, 96))), Q.ERR_INVALID_ARG),
    (dict(A=ctypes.byref(tensor(ROWS, 128, fmt=Q.MXFP4))), Q.ERR_INVALID_ARG),
    (dict(A=ctypes.byref(tensor(ROWS, 128, had=1))), Q.ERR_INVALID_ARG),
    (dict(A=ctypes.byref(tensor(ROWS, 128, codes=ODD))), Q.ERR_MISALIGNED),
    (dict(B=ctypes.byref(tensor(385, 128))), Q.ERR_INVALID_ARG),     # not a multiple of the groups
    (dict(B=ctypes.byref(tensor(3 * 64, 128))), Q.ERR_INVALID_ARG),  # 64 rows each
    (dict(B=ctypes.byref(tensor(256, 256))), Q.ERR_INVALID_ARG),     # neither K nor E K
    (dict(A=ctypes.byref(tensor(ROWS, 64)), B=ctypes.byref(tensor(128, 192))), Q.ERR_INVALID_ARG),
    (dict(B=ctypes.byref(tensor(100, 384))), Q.ERR_INVALID_ARG),     # 100 columns
    (dict(D=None), Q.ERR_INVALID_ARG), (dict(D=ODD), Q.ERR_MISALIGNED), (dict(ldd=100), Q.ERR_INVALID_ARG),
    (dict(ldd=132), Q.ERR_MISALIGNED), (dict(dt=2), Q.ERR_INVALID_ARG), (dict(off=None), Q.ERR_INVALID_ARG),
    (dict(E=300), Q.ERR_INVALID_ARG),
])
def test_gemm_grouped_refuses(lib, kw, want):
    assert Q.group_rows(100, 3) == ROWS
    a = dict(A=ctypes.byref(tensor(ROWS, 128)), B=ctypes.byref(tensor(384, 128)), off=P, E=3, T=100, D=P, ldd=128, dt=0)
    a.update(kw)
    assert lib.qfp4_gemm_grouped(*a.values(), None) == want


@pytest.mark.parametrize("kw,want", [
    (dict(A=ctypes.byref(tensor(100, ROWS))), Q.ERR_INVALID_ARG), (dict(A=ctypes.byref(tensor(128, 128))), Q.ERR_INVALID_ARG),
    (dict(B=ctypes.byref(tensor(100, ROWS))), Q.ERR_INVALID_ARG), (dict(B=ctypes.byref(tensor(128, 512))), Q.ERR_INVALID_ARG),
    (dict(B=None), Q.ERR_INVALID_ARG), (dict(D=None), Q.ERR_INVALID_ARG), (dict(D=ODD), Q.ERR_MISALIGNED),
    (dict(dt=0, acc=1), Q.ERR_INVALID_ARG), (dict(acc=2), Q.ERR_INVALID_ARG), (dict(dt=5), Q.ERR_INVALID_ARG),
    (dict(T=-5), Q.ERR_INVALID_ARG),
])
def test_gemm_grouped_wgrad_refuses(lib, kw, want):
    a = dict(A=ctypes.byref(tensor(128, ROWS)), B=ctypes.byref(tensor(128, ROWS)), off=P, E=3, T=100, D=P, dt=1, acc=0)
    a.update(kw)
    assert lib.qfp4_gemm_grouped_wgrad(*a.values(), None) == want


@pytest.mark.parametrize("kw,want", [
    (dict(E=0), Q.ERR_INVALID_ARG), (dict(N=64), Q.ERR_INVALID_ARG), (dict(K=192), Q.ERR_INVALID_ARG),
    (dict(N=0), Q.ERR_INVALID_ARG), (dict(rec=None), Q.ERR_INVALID_ARG), (dict(seed=None), Q.ERR_INVALID_ARG),
    (dict(X=None), Q.ERR_INVALID_ARG), (dict(W=None), Q.ERR_INVALID_ARG), (dict(Y=ODD), Q.ERR_MISALIGNED),
    (dict(off=None), Q.ERR_INVALID_ARG), (dict(wsb=1000), Q.ERR_WORKSPACE), (dict(ws=ODD), Q.ERR_MISALIGNED),
])
def test_linear_grouped_refuses(lib, kw, want):
    rec = Q.recipe("AMD_MXFP4_H")
    a = dict(X=P, W=P, Y=P, off=P, E=3, T=100, N=128, K=128, rec=ctypes.byref(rec), seed=ctypes.byref(SEED), am=None,
             ws=P, wsb=1 << 30)
    a.update(kw)
    assert lib.qfp4_linear_grouped_fwd(*a.values(), None) == want
    b = dict(dY=a["Y"], X=a["X"], W=a["W"], dX=P, dW=P, **{k: a[k] for k in ("off", "E", "T", "N", "K", "rec", "seed", "ws",
                                                                             "wsb")})
    assert lib.qfp4_linear_grouped_bwd(*b.values(), None) == want
    if not kw.keys() - {"N", "K"}:
        return
    bad = Q.recipe("AMD_MXFP4_H")
    bad.wgrad.had = 9
    a["rec"] = ctypes.byref(bad)
    assert lib.qfp4_linear_grouped_fwd(*a.values(), None) != Q.OK
