"""RMSNorm with the residual's addition: forward (values, tensor amax, MXFP4
quantization) against its definition bit for bit, backward against the
formula in 64 bits and against differences, and the uses that a program makes
of them (in place, strided, captured, on another stream, before an FP4 layer)."""
import numpy as np
import pytest
import torch

import helpers
from fp4_precision_b200 import qfp4 as Q

pytestmark = pytest.mark.gpu

EPS = 1e-5
HALF_BF16 = torch.finfo(torch.bfloat16).eps / 2
HALF_F32 = 2.0 ** -24
SEED = Q.make_seed(0x1234_5678_9ABC, 7, 3, 4)

SHAPES = [(5, 8208), (9, 528), (3, 16368), (1, 16), (1, 4096), (3, 48), (5, 1024), (7, 1040), (129, 768), (130, 2048), (1000, 1536), (4, 16384), (257, 5120)]


def draw(shape, seed, std=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(shape, generator=g, device="cuda") * std).bfloat16()


def inputs(R, C, seed=0):
    x, res = draw((R, C), seed), draw((R, C), seed + 1, 3.0)
    if R > 2:
        x[1], res[1] = 0, 0            # a row of zeros
        x[2, 0] = 2.0 ** 60            # a square past fp32's range
    return x, res, (1 + 0.2 * draw((C,), seed + 2).float()).bfloat16()


def definition(x, res, w, eps=EPS):
    h = x if res is None else (x.float() + res.float()).bfloat16()
    e = float(np.float32(eps))
    rstd = (1 / (h.double().square().sum(1) / h.shape[1] + e).sqrt()).float()
    return (h.float() * rstd[:, None] * w.float()).bfloat16(), h, rstd


def same(a, b):
    return torch.equal(a.view(torch.int16) if a.dtype == torch.bfloat16 else a.view(torch.int32),
                       b.view(torch.int16) if b.dtype == torch.bfloat16 else b.view(torch.int32))


@pytest.mark.parametrize("R,C", SHAPES)
@pytest.mark.parametrize("with_res", [True, False])
def test_forward_is_the_definition(R, C, with_res):
    x, res, w = inputs(R, C)
    res = res if with_res else None
    y, h, rstd, amax = Q.rmsnorm_fwd(x, w, EPS, res=res)
    Q.status()
    want_y, want_h, want_rstd = definition(x, res, w)
    assert amax is None
    assert same(h, want_h) and (with_res or h is x)
    # a root that lies within an fp64 rounding of two fp32 neighbours' middle may fall to either
    assert torch.all((rstd - want_rstd).abs() <= 2 * HALF_F32 * want_rstd)
    assert same(y, (h.float() * rstd[:, None] * w.float()).bfloat16())
    assert (rstd != want_rstd).sum() <= 1 and same(y[rstd == want_rstd], want_y[rstd == want_rstd])


HADS = [Q.HAD_NONE, Q.HAD_DET16, Q.HAD_DET32, Q.HAD_RAND16, Q.HAD_RAND32]


@pytest.mark.parametrize("had", HADS)
@pytest.mark.parametrize("R,C", [(1, 32), (1, 4096), (7, 96), (300, 1024), (129, 1056), (1000, 1536), (3, 16384), (5, 8208)])
def test_amax_is_that_of_y(R, C, had):
    if had in (Q.HAD_DET32, Q.HAD_RAND32) and C % 32:
        pytest.skip("not a multiple of the rotation")
    x, res, w = inputs(R, C, 5)
    y, _, _, amax = Q.rmsnorm_fwd(x, w, EPS, res=res, had=had, seed=SEED, want_amax=True)
    assert same(amax, Q.amax(y, had, Q.ROW, SEED))
    Q.status()


@pytest.mark.parametrize("had", HADS)
@pytest.mark.parametrize("fmt", [Q.MXFP4, Q.MXFP4_RU])
@pytest.mark.parametrize("R,C", [(1, 32), (5, 96), (127, 1024), (128, 1056), (300, 2080), (3, 16384)])
def test_quantized_output_is_that_of_y(R, C, fmt, had):
    x, res, w = inputs(R, C, 6)
    want_y, want_h, want_rstd, _ = Q.rmsnorm_fwd(x, w, EPS, res=res)
    want = Q.quantize(want_y, fmt, Q.RTN, had, Q.ROW, SEED)
    q, guards = helpers.guarded_qtensor(Q, fmt, R, C, x.device)
    y, h, rstd, _ = Q.rmsnorm_quantize(x, w, EPS, res=res, fmt=fmt, had=had, seed=SEED, out=q)
    helpers.assert_guards_intact(*guards)
    assert same(y, want_y) and same(h, want_h) and same(rstd, want_rstd)
    assert torch.equal(q.codes, want.codes) and q.tensor_scale.item() == 1.0
    n = Q.scales_bytes(fmt, R, C)
    assert torch.equal(q.scales[:n], want.scales[:n])
    for f, _ in Q.TensorDesc._fields_[3:]:
        assert getattr(q.desc, f) == getattr(want.desc, f), f
    # without y, and so without h and the residual
    none, h2, _, q2 = Q.rmsnorm_quantize(want_h, w, EPS, fmt=fmt, had=had, seed=SEED, want_y=False)
    assert none is None and h2 is want_h and torch.equal(q2.codes, want.codes)
    Q.status()


def gradients64(dy, h, w, rstd, dh):
    dy, h, w, r = dy.double(), h.double(), w.double(), rstd.double()[:, None]
    g, hr = dy * w, h * r
    c = (g * hr).mean(1, keepdim=True)
    dx = r * (g - hr * c) + (0 if dh is None else dh.double())
    # magnitudes that the fp32 roundings are relative to
    size = r * (g.abs() + hr.abs() * (g * hr).abs().mean(1, keepdim=True)) + (0 if dh is None else dh.double().abs())
    return dx, size, (dy * hr).sum(0), (dy * hr).abs().sum(0)


@pytest.mark.parametrize("R,C", SHAPES + [(2500, 2048), (1300, 512)])
@pytest.mark.parametrize("with_dh", [True, False])
def test_backward_is_the_formula(R, C, with_dh):
    x, res, w = inputs(R, C, 11)
    if R > 2:
        x[2, 0] = 100.0
    dy, dh = draw((R, C), 20, 1e-3), draw((R, C), 21, 1e-3) if with_dh else None
    _, h, rstd, _ = Q.rmsnorm_fwd(x, w, EPS, res=res)
    dx, dw = Q.rmsnorm_bwd(dy, h, w, rstd, dh=dh)
    Q.status()
    want, size, want_w, size_w = gradients64(dy, h, w, rstd, dh)
    # dx: fp32 roundings (32 terms per thread one after the other, 5 shuffles, at most 16 warps, and the products: under
    # 64 in a chain), and the result's to bf16
    assert torch.all((dx.double() - want).abs() <= HALF_BF16 * want.abs() * 1.01 + 64 * HALF_F32 * size)
    # dw: at most R additions and two products in a chain
    assert torch.all((dw.double() - want_w).abs() <= (R + 16) * HALF_F32 * size_w)


def test_backward_against_differences():
    """The gradient of sum(y * dy) + sum(h * dh) along a direction, by the forward formula in 64 bits."""
    R, C = 33, 320
    x, res, w = inputs(R, C, 31)
    x[2, 0] = 1.0
    dy, dh = draw((R, C), 32), draw((R, C), 33)
    _, h, rstd, _ = Q.rmsnorm_fwd(x, w, EPS, res=res)
    dx, dw = Q.rmsnorm_bwd(dy, h, w, rstd, dh=dh)
    v, vw = draw((R, C), 34).double(), draw((C,), 35).double()

    def f(t):
        hh, ww = h.double() + t * v, w.double() + t * vw
        y = hh / (hh.square().mean(1, keepdim=True) + EPS).sqrt() * ww
        return (y * dy.double()).sum() + (hh * dh.double()).sum()

    # Richardson step of two central differences: an error of order t^4, and fp64 cancellation below 1e-9 of the sum;
    # a row of zeros has rstd = eps^-1/2, so t stays well below eps^1/2
    t = 1e-5
    d1, d2 = (f(t) - f(-t)) / (2 * t), (f(2 * t) - f(-2 * t)) / (4 * t)
    want = (4 * d1 - d2) / 3
    got = (dx.double() * v).sum() + (dw.double() * vw).sum()
    # dx is rounded to bf16: half a step of each entry times its direction
    tol = (HALF_BF16 * dx.double().abs() * v.abs()).sum() + 1e-5 * (dw.double() * vw).abs().sum()
    assert abs(got - want) <= tol


@pytest.mark.parametrize("C", [512, 1536])
def test_weight_gradient_accumulates(C):
    R = 700
    x, _, w = inputs(R, C, 41)
    dy = draw((R, C), 42)
    _, h, rstd, _ = Q.rmsnorm_fwd(x, w, EPS)
    _, dw = Q.rmsnorm_bwd(dy, h, w, rstd)
    held = draw((C,), 43).float()
    got = held.clone()
    Q.rmsnorm_bwd(dy, h, w, rstd, dw=got, accumulate=True)
    assert same(got, held + dw)
    with pytest.raises(ValueError):
        Q.rmsnorm_bwd(dy, h, w, rstd, accumulate=True)


def test_no_rows():
    x, w = torch.empty((0, 64), dtype=torch.bfloat16, device="cuda"), draw((64,), 1)
    y, h, rstd, amax = Q.rmsnorm_fwd(x, w, EPS, res=x, had=Q.HAD_DET16, want_amax=True)
    assert y.shape == (0, 64) and amax.item() == 0
    q = Q.rmsnorm_quantize(x, w, EPS)[3]
    assert q.rows == 0 and q.tensor_scale.item() == 1
    dw = torch.full((64,), 3.0, device="cuda")
    Q.rmsnorm_bwd(y, x, w, rstd, dw=dw, accumulate=True)
    assert torch.all(dw == 3)
    Q.rmsnorm_bwd(y, x, w, rstd, dw=dw)
    assert torch.all(dw == 0)
    Q.status()


@pytest.mark.parametrize("C", [256, 2048])
def test_strides_in_place_and_guards(C):
    """Operands that are slices of wider buffers; outputs in the inputs' place; nothing else is touched."""
    R, wide = 131, C + 40
    xs, rs = draw((R, wide), 51), draw((R, wide), 52)
    x, res, w = xs[:, 8:8 + C], rs[:, 16:16 + C], draw((C,), 53)
    want_y, want_h, want_rstd, want_amax = Q.rmsnorm_fwd(x.contiguous(), w, EPS, res=res.contiguous(), had=Q.HAD_DET16,
                                                         want_amax=True)
    out, guard = helpers.guarded_matrix(R, wide, torch.bfloat16, x.device)
    out.fill_(7)
    before = xs.clone()
    y, h, rstd, amax = Q.rmsnorm_fwd(x, w, EPS, res=res, y=out[:, 24:24 + C], h=x, had=Q.HAD_DET16, want_amax=True)
    assert same(y.contiguous(), want_y) and same(x.contiguous(), want_h) and same(rstd, want_rstd)
    assert same(amax, want_amax)
    assert torch.all(out[:, :24] == 7) and torch.all(out[:, 24 + C:] == 7)
    assert same(xs[:, :8].contiguous(), before[:, :8].contiguous())
    assert same(xs[:, 8 + C:].contiguous(), before[:, 8 + C:].contiguous())
    want = Q.rmsnorm_fwd(res.contiguous(), w, EPS)[0]
    Q.rmsnorm_fwd(res, w, EPS, y=res)  # y over x
    assert same(res.contiguous(), want)
    dy, dh = draw((R, wide), 54)[:, :C], draw((R, C), 55)
    want_dx, want_dw = Q.rmsnorm_bwd(dy.contiguous(), want_h, w, rstd, dh=dh)
    dx, dw = Q.rmsnorm_bwd(dy, x, w, rstd, dh=dh, dx=dh)
    assert same(dx, want_dx) and same(dw, want_dw) and dx is dh
    dx, dw = Q.rmsnorm_bwd(dy, x, w, rstd, dx=dy)
    assert same(dw, want_dw)
    helpers.assert_guards_intact(guard)
    Q.status()


def test_special_values():
    """Infinities and NaN stay in their rows; a row of zeros with eps gives zeros."""
    x, w = draw((6, 64), 61), torch.ones(64, dtype=torch.bfloat16, device="cuda")
    x[0] = 0
    x[1, 3] = float("inf")
    x[2, 5] = float("nan")
    x[3] = 3e38
    y, _, rstd, _ = Q.rmsnorm_fwd(x, w, EPS)
    assert torch.all(y[0] == 0)
    assert rstd[1] == 0 and torch.isnan(y[1, 3]) and torch.all(y[1, 4:] == 0)
    assert torch.all(torch.isnan(y[2]))
    assert torch.all((y[3].float() - 1).abs() <= 2 * HALF_BF16)
    assert torch.all(torch.isfinite(y[4:]))
    Q.status()


def test_repeats_streams_and_graph():
    """The same bits at every call; on another stream; two calls at once; captured and replayed on other data."""
    R, C = 777, 2048
    x, res, w = inputs(R, C, 71)
    dy = draw((R, C), 72)
    first = Q.rmsnorm_fwd(x, w, EPS, res=res, had=Q.HAD_RAND16, seed=SEED, want_amax=True)
    grads = Q.rmsnorm_bwd(dy, first[1], w, first[2])
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    outs = []
    for s in (s1, s2, s1):
        outs.append((Q.rmsnorm_fwd(x, w, EPS, res=res, had=Q.HAD_RAND16, seed=SEED, want_amax=True, stream=s),
                     Q.rmsnorm_bwd(dy, first[1], w, first[2], stream=s)))
    torch.cuda.synchronize()
    for f, g in outs:
        assert all(same(a, b) for a, b in zip(f, first)) and all(same(a, b) for a, b in zip(g, grads))
    graph = torch.cuda.CUDAGraph()
    xs, rs = x.clone(), res.clone()
    with torch.cuda.graph(graph):
        y, h, rstd, amax = Q.rmsnorm_fwd(xs, w, EPS, res=rs, had=Q.HAD_RAND16, seed=SEED, want_amax=True)
        dx, dw = Q.rmsnorm_bwd(dy, h, w, rstd)
        q = Q.rmsnorm_quantize(xs, w, EPS, res=rs)[3]
    for k in (0, 3):
        xs.copy_(draw((R, C), 73 + k))
        graph.replay()
        want = Q.rmsnorm_fwd(xs, w, EPS, res=rs, had=Q.HAD_RAND16, seed=SEED, want_amax=True)
        assert all(same(a, b) for a, b in zip((y, h, rstd, amax), want))
        assert all(same(a, b) for a, b in zip((dx, dw), Q.rmsnorm_bwd(dy, want[1], w, want[2])))
        assert torch.equal(q.codes, Q.quantize(want[0], Q.MXFP4, Q.RTN, Q.HAD_NONE, Q.ROW).codes)
    Q.status()


def test_before_an_fp4_layer():
    """norm -> FP4 linear: the norm's amax in the chained call, and its MXFP4 output in the GEMM, give what the
    separate calls give; gradients flow through both functions."""
    M, K, N = 384, 512, 256
    x, res = draw((M, K), 81), draw((M, K), 82)
    w, W = (1 + 0.1 * draw((K,), 83).float()).bfloat16(), draw((N, K), 84, 0.05)
    rec, seed = Q.recipe("QUARTET2_NVFP4"), Q.make_seed(rot=5, sr=6)
    had = rec.fprop.had
    y, h, rstd, amax = Q.rmsnorm_fwd(x, w, EPS, res=res, had=had, seed=Q.make_seed(rot=5), want_amax=True)
    Y, _ = Q.linear_fwd_chain(y, W, rec, seed, x_amax=amax, want_y_amax=False)
    assert same(Y, Q.linear_fwd(y, W, rec, seed))
    q = Q.rmsnorm_quantize(x, w, EPS, res=res)[3]
    B = Q.quantize(W, Q.MXFP4, Q.RTN, Q.HAD_NONE, Q.ROW)
    assert same(Q.gemm(q, B), Q.gemm(Q.quantize(y, Q.MXFP4, Q.RTN, Q.HAD_NONE, Q.ROW), B))
    leaves = [t.detach().clone().requires_grad_() for t in (x, res, w, W)]
    yy, hh = Q.RmsNorm.apply(leaves[0].view(2, M // 2, K), leaves[1].view(2, M // 2, K), leaves[2], EPS)
    out = Q.Fp4Linear.apply(yy.view(M, K), leaves[3], rec, seed)
    dY, dh = draw((M, N), 85, 1e-2), draw((M, K), 86, 1e-2)
    torch.autograd.backward([out, hh], [dY, dh.view(2, M // 2, K)])
    dy, dW = Q.linear_bwd(dY, y, W, rec, seed)
    dx, dw = Q.rmsnorm_bwd(dy, h, w, rstd, dh=dh)
    assert same(leaves[0].grad, dx) and same(leaves[1].grad, dx)
    assert same(leaves[2].grad, dw.bfloat16()) and same(leaves[3].grad, dW.bfloat16())
    a = x.clone().requires_grad_()
    yy, hh = Q.RmsNorm.apply(a, None, w, EPS)   # no residual, and nothing flows back through h
    yy.backward(dy)
    _, h1, r1, _ = Q.rmsnorm_fwd(x, w, EPS)
    assert same(a.grad, Q.rmsnorm_bwd(dy, h1, w, r1)[0])
    b, c = x.clone().requires_grad_(), res.clone().requires_grad_()
    _, hh = Q.RmsNorm.apply(b, c, w, EPS)       # and through h alone
    hh.backward(dh)
    assert same(b.grad, dh) and same(c.grad, dh)
    Q.status()


def test_offsets_past_32_bits():
    """A matrix of more than 2^31 elements: its last rows."""
    R, C = 135_000, 16384
    x = torch.zeros((R, C), dtype=torch.bfloat16, device="cuda")
    w = draw((C,), 91)
    x[-3:] = draw((3, C), 92)
    y, _, rstd, _ = Q.rmsnorm_fwd(x, w, EPS, y=torch.empty_like(x))
    want = Q.rmsnorm_fwd(x[-3:].clone(), w, EPS)
    assert same(y[-3:], want[0]) and same(rstd[-3:], want[2]) and not y[:2].any()
    dx, _ = Q.rmsnorm_bwd(y, x, w, rstd, dx=y)
    assert same(dx[-3:], Q.rmsnorm_bwd(want[0], x[-3:].clone(), w, want[2])[0])
    Q.status()
