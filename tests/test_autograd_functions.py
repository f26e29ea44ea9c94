"""What the autograd functions promise around their kernels: outputs that a
program may change, inputs of any strides, first derivatives only. On the CPU
the kernels' calls are replaced by their formulas, so that the functions
themselves run here; on a GPU they are the real ones."""
import pytest
import torch

from fp4_precision_b200 import qfp4 as Q

EPS = 1e-5
DEVICES = ["cpu", pytest.param("cuda", marks=pytest.mark.gpu)]


def usable(m):
    """What the RMSNorm calls ask of a matrix's strides (include/qfp4.h)."""
    assert m.dim() == 2 and m.stride(1) == 1 and m.stride(0) >= m.shape[1] and m.stride(0) % 8 == 0
    assert m.data_ptr() % 16 == 0
    return m


def norm_fwd(x, w, eps, res=None, y=None, h=None, **_):
    y, h = (torch.empty_like(x) if t is None else t for t in (y, h))
    usable(x), usable(y), usable(h), usable(w.view(1, -1))
    v = (x.float() + (0 if res is None else usable(res).float())).bfloat16()
    rstd = (v.float().square().mean(1) + eps).rsqrt()
    h.copy_(v)
    y.copy_((v.float() * rstd[:, None] * w.float()).bfloat16())
    return y, h, rstd, None


def norm_bwd(dy, h, w, rstd, dh=None, dx=None, **_):
    g, hr = usable(dy).float() * w.float(), usable(h).float() * rstd[:, None]
    d = rstd[:, None] * (g - hr * (g * hr).mean(1, keepdim=True)) + (0 if dh is None else usable(dh).float())
    dx = torch.empty_like(dy) if dx is None else dx
    usable(dx).copy_(d.bfloat16())
    return dx, (dy.float() * hr).sum(0)


def grouped_fwd(X, W, offsets, rec, seed, Y=None, **_):
    for e, (a, b) in enumerate(zip(offsets.tolist(), offsets.tolist()[1:])):
        Y[a:b] = X[a:b] @ W[e].T
    return Y


def grouped_bwd(dY, X, W, offsets, rec, seed, dX=None, **_):
    dW = torch.zeros(W.shape)
    for e, (a, b) in enumerate(zip(offsets.tolist(), offsets.tolist()[1:])):
        dX[a:b] = dY[a:b] @ W[e]
        dW[e] = (dY[a:b].T @ X[a:b]).float()
    return dX, dW


@pytest.fixture(autouse=True)
def formulas(request, monkeypatch):
    if request.node.callspec.params["dev"] == "cpu":
        monkeypatch.setattr(Q, "rmsnorm_fwd", norm_fwd)
        monkeypatch.setattr(Q, "rmsnorm_bwd", norm_bwd)
        monkeypatch.setattr(Q, "linear_fwd", lambda X, W, *_: X @ W.T)
        monkeypatch.setattr(Q, "linear_bwd", lambda dY, X, W, *_: (dY @ W, (dY.T @ X).float()))
        monkeypatch.setattr(Q, "linear_grouped_fwd", grouped_fwd)
        monkeypatch.setattr(Q, "linear_grouped_bwd", grouped_bwd)


def draw(dev, *shape, seed=0):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(shape, generator=g).bfloat16().to(dev)


def norm_inputs(dev, R=6, C=32):
    return [draw(dev, R, C, seed=s).requires_grad_() for s in (1, 2)] + [draw(dev, C, seed=3).requires_grad_()]


@pytest.mark.parametrize("dev", DEVICES)
@pytest.mark.parametrize("with_res", [True, False])
def test_norm_output_may_be_changed_in_place(dev, with_res):
    """y scaled in place (a dropout, say): the gradients are those of the scaled y; h's change is refused backward."""
    x, r, w = norm_inputs(dev)
    r = r if with_res else None
    leaves = [t for t in (x, r, w) if t is not None]
    dy = draw(dev, *x.shape, seed=4)
    want = torch.autograd.grad(Q.RmsNorm.apply(x, r, w, EPS)[0], leaves, 2 * dy)
    y, h = Q.RmsNorm.apply(x, r, w, EPS)
    got = torch.autograd.grad(y.mul_(2), leaves, dy)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    y, h = Q.RmsNorm.apply(x, r, w, EPS)
    h.add_(1)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.backward(dy)


def grouped_inputs(dev, T=5, E=2, N=128, K=128):
    offsets = torch.tensor([0, 3, T], dtype=torch.int32, device=dev)
    return draw(dev, T, K, seed=5).requires_grad_(), draw(dev, E, N, K, seed=6).requires_grad_(), offsets


def norm_of_x(dev):
    x, r, w = norm_inputs(dev)
    return Q.RmsNorm.apply(x, r, w, EPS)[0], (x, r, w)


def norm_and_stream(dev):
    x, r, w = norm_inputs(dev)
    y, h = Q.RmsNorm.apply(x, r, w, EPS)
    return y.float() + h.float(), (x, r, w)


def norm_alone(dev):
    x, _, w = norm_inputs(dev)
    return Q.RmsNorm.apply(x, None, w, EPS)[0], (x, w)


def experts(dev):
    X, W, offsets = grouped_inputs(dev)
    return Q.Fp4GroupedLinear.apply(X, W, offsets, Q.recipe("AMD_MXFP4_H"), Q.make_seed()), (X, W)


def layer(dev):
    X, W = (draw(dev, 128, 128, seed=s).requires_grad_() for s in (7, 8))
    return Q.Fp4Linear.apply(X, W, Q.recipe("AMD_MXFP4_H"), Q.make_seed()), (X, W)


@pytest.mark.parametrize("dev", DEVICES)
@pytest.mark.parametrize("f", [norm_of_x, norm_and_stream, norm_alone, experts, layer])
def test_second_derivatives_are_refused(dev, f):
    """A penalty on the gradient, beside a path that has a second derivative: an error, where the function's part would
    be missing from the sum. A gradient made with create_graph=True has the values of one made without."""
    out, leaves = f(dev)
    want = torch.autograd.grad(out.float().sum(), leaves)
    out, leaves = f(dev)
    grads = torch.autograd.grad(out.float().sum(), leaves, create_graph=True)
    assert all(torch.equal(a, b) for a, b in zip(grads, want))
    for g, t in zip(grads, leaves):
        with pytest.raises(RuntimeError, match="first derivatives only"):
            torch.autograd.grad(g.float().square().sum() + t.float().square().sum(), t, retain_graph=True)
    if dev == "cuda":
        Q.status()


def apart(t, at):
    """t's values where each lies `at` elements behind the one before it."""
    held = torch.zeros(t.numel() * at, dtype=t.dtype, device=t.device)
    return held.as_strided(t.shape, (t.shape[1] * at, at)).copy_(t)


ORDERS = {
    "transposed": lambda t: t.t().contiguous().t(),
    "every other element": lambda t: apart(t, 2),
    "rows 20 bytes further apart": lambda t: torch.cat((t, t[:, :10]), 1)[:, :t.shape[1]],
    "an odd address": lambda t: torch.cat((t[:1, :1].flatten(), t.flatten()))[1:].view(t.shape),
    "one row for all": lambda t: t[:1].expand(t.shape),
    "a slice": lambda t: torch.cat((t, t), 1)[:, t.shape[1]:],
}


@pytest.mark.parametrize("dev", DEVICES)
@pytest.mark.parametrize("order", ORDERS)
def test_norm_takes_any_strides(dev, order):
    """x, the residual, the weight and both gradients in other orders: what contiguous ones give."""
    lay = ORDERS[order]
    x, r, dy, dh = (lay(draw(dev, 6, 32, seed=s)) for s in (11, 12, 13, 14))
    w = draw(dev, 32, 3, seed=15)[:, 1]

    def run(*ts):
        a, b, c, *gs = (t.detach() for t in ts)
        leaves = [t.requires_grad_() for t in (a, b, c)]
        out = Q.RmsNorm.apply(*leaves, EPS)
        return (*out, *torch.autograd.grad(out, leaves, gs))

    got, want = run(x, r, w, dy, dh), run(*(t.contiguous().clone() for t in (x, r, w, dy, dh)))
    assert all(a.is_contiguous() and torch.equal(a, b) for a, b in zip(got, want))
    if dev == "cuda":
        Q.status()
