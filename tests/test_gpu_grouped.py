"""The FP4 linear layer over groups of rows (the experts of a mixture) against
the oracle: its quantizations of the padded rows, its products in 64 bits per
group, the layer forward and backward, and the uses a program makes of them."""
import dataclasses

import numpy as np
import pytest
import torch

import helpers
import oracle as O
from fp4_precision_b200 import qfp4 as Q

pytestmark = pytest.mark.gpu

ROT, SRS = 0x1111_2222_3333_4444, 0x5555_6666_7777_8888

# group sizes, rows before the first group, rows behind the last
SPLITS = {
    "ragged": ([5, 0, 128, 129, 1, 300, 127], 0, 0),
    "one": ([333], 0, 0),
    "one row": ([0, 1, 0], 0, 0),
    "outside": ([64, 200, 31], 3, 9),
    "none": ([0, 0, 0, 0], 2, 2),
    "skewed": ([0, 0, 700, 1], 0, 0),
    "many": ([(i * 7) % 5 for i in range(256)], 1, 1),
}


def cpu(shape, seed, std=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * std).bfloat16()


def split(name):
    sizes, before, behind = SPLITS[name]
    off = np.concatenate(([0], np.cumsum(sizes))) + before
    return sizes, off, int(off[-1]) + behind, torch.tensor(off, dtype=torch.int32, device="cuda")


def starts(sizes):
    whole = [(m + 127) // 128 * 128 for m in sizes]
    return np.concatenate(([0], np.cumsum(whole))).astype(int)


def padded(x, sizes, off, T):
    """The padded layout, built row by row."""
    xp = torch.zeros((Q.group_rows(T, len(sizes)), x.shape[1]), dtype=x.dtype)
    p = starts(sizes)
    for e, m in enumerate(sizes):
        xp[p[e]:p[e] + m] = x[off[e]:off[e] + m]
    return xp


def within(got, ref, bound, bf16_out):
    g = got.double().cpu().numpy()
    tol = bound + (2.0 ** -8 * np.abs(ref) if bf16_out else 0.0)
    bad = np.abs(g - ref) > tol
    assert not bad.any(), f"{bad.sum()} of {bad.size} out of bound"


@pytest.mark.parametrize("name", SPLITS)
@pytest.mark.parametrize("fmt", [Q.NVFP4, Q.MXFP4, Q.MXFP4_RU])
@pytest.mark.parametrize("rnd", [Q.RTN, Q.SR, Q.QUARTET2])
@pytest.mark.parametrize("had,axis", [(Q.HAD_NONE, Q.ROW), (Q.HAD_RAND16, Q.ROW), (Q.HAD_NONE, Q.COL),
                                      (Q.HAD_RAND16, Q.COL), (Q.HAD_DET32, Q.COL)])
def test_quantize_is_that_of_the_padded_rows(name, fmt, rnd, had, axis):
    sizes, off, T, offsets = split(name)
    C = 160
    x = cpu((T, C), 1)
    xd = torch.full((T, C + 24), float("nan"), dtype=torch.bfloat16, device="cuda")  # a slice of a wider matrix
    xd[:, 16:16 + C] = x.cuda()
    for r in (*range(off[0]), *range(off[-1], T)):
        xd[r] = float("nan")  # rows of no group are not read
    Tp = Q.group_rows(T, len(sizes))
    rows, k = (Tp, C) if axis == Q.ROW else (C, Tp)
    q, guards = helpers.guarded_qtensor(Q, fmt, rows, k, "cuda")
    seed = Q.make_seed(ROT, SRS, 3, 5)
    Q.quantize_grouped(xd[:, 16:16 + C], offsets, fmt, rnd, had, axis, seed, out=q)
    Q.status()
    helpers.assert_guards_intact(*guards)
    want = O.quantize(padded(x, sizes, off, T), fmt, rnd, had, axis, ROT, 3, SRS, 5)
    nb = Q.BLOCK[fmt]
    codes, flat = helpers.to_numpy_u8(q.codes), helpers.to_numpy_u8(q.scales)
    own = np.ones(rows, dtype=bool)
    if axis == Q.ROW:  # rows that are no group's are left as they were
        own[:] = False
        for p, m in zip(starts(sizes), sizes):
            own[p:p + m] = True
        kb4 = (k // nb + 3) // 4 * 4
        every = flat[helpers.atom_offset(rows, k // nb, np.arange(rows)[:, None], np.arange(kb4)[None, :])]
        assert np.all(codes[~own] == helpers.GUARD_PATTERN) and np.all(every[~own] == helpers.GUARD_PATTERN)
        assert not every[own][:, k // nb:].any()
    else:
        assert helpers.padding_is_zero(flat, rows, k, nb)
    assert np.array_equal(codes[own], want.codes[own])
    assert np.array_equal(helpers.unswizzle_scales(flat, rows, k, nb)[own], want.scales[own])
    assert q.tensor_scale.item() == np.float32(want.g)
    assert (q.rows, q.k, q.desc.had) == (rows, k, had)


def operands(fmt, had, A, axis_a, B, axis_b, rot=ROT):
    """Quantized on both sides: (device, oracle) of two bf16 CPU matrices."""
    seed = Q.make_seed(rot, 0)
    dev = [Q.quantize(t.cuda(), fmt, Q.RTN, had, ax, seed) for t, ax in ((A, axis_a), (B, axis_b))]
    ora = [O.quantize(t, fmt, Q.RTN, had, ax, rot, 0) for t, ax in ((A, axis_a), (B, axis_b))]
    return dev, [O.dequantize(t) for t in ora]


@pytest.mark.parametrize("name", SPLITS)
@pytest.mark.parametrize("fmt", [Q.NVFP4, Q.MXFP4])
@pytest.mark.parametrize("form", ["rows", "k"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_gemm_is_the_product_of_each_group(name, fmt, form, dtype):
    sizes, off, T, offsets = split(name)
    E, N, K = len(sizes), 384 if len(sizes) < 100 else 128, 128 if len(sizes) > 100 else 384
    x = cpu((T, K), 2)
    xp = padded(x, sizes, off, T)
    W = cpu((E * N, K), 3, 0.1) if form == "rows" else cpu((N, E * K), 3, 0.1)
    (A, B), (a, b) = operands(fmt, Q.HAD_RAND16, xp, Q.ROW, W, Q.ROW)
    ld = N + 24  # and every row's rest stays as it was
    out, guard = helpers.guarded_matrix(T, ld, dtype, "cuda")
    out.fill_(-5)
    Q.gemm_grouped(A, B, offsets, T, out=out[:, :N])
    Q.status()
    helpers.assert_guards_intact(guard)
    p = starts(sizes)
    ref = np.full((T, N), -5.0)
    bound = np.zeros((T, N))
    for e, m in enumerate(sizes):
        be = b[e * N:(e + 1) * N] if form == "rows" else b[:, e * K:(e + 1) * K]
        ae = a[p[e]:p[e] + m]
        ref[off[e]:off[e] + m] = ae @ be.T
        bound[off[e]:off[e] + m] = O.GEMM_REL_BOUND * (np.abs(ae) @ np.abs(be).T)
    within(out[:, :N], ref, bound, dtype == torch.bfloat16)
    assert torch.all(out[:, N:] == -5)
    outside = [r for r in range(T) if r < off[0] or r >= off[-1]]
    assert torch.all(out[outside] == -5)


@pytest.mark.parametrize("pair", ["0", "1"])
@pytest.mark.parametrize("name", ["ragged", "skewed", "outside", "none"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_both_gemm_kernels_give_the_same(monkeypatch, pair, name, dtype):
    """The CTA-pair and the single-CTA kernel, whichever the group sizes choose."""
    sizes, off, T, offsets = split(name)
    E, N, K = len(sizes), 384, 320
    xp = padded(cpu((T, K), 51), sizes, off, T).cuda()
    A = Q.quantize(xp, Q.NVFP4, Q.RTN, Q.HAD_NONE, Q.ROW)
    B = Q.quantize(cpu((E * N, K), 52).cuda(), Q.NVFP4, Q.RTN, Q.HAD_NONE, Q.ROW)
    want = Q.gemm_grouped(A, B, offsets, T, out=torch.zeros((T, N), dtype=torch.float32, device="cuda"))
    monkeypatch.setenv("QFP4_GEMM_PAIR", pair)
    got = Q.gemm_grouped(A, B, offsets, T, out=torch.zeros((T, N), dtype=dtype, device="cuda"))
    Q.status()
    assert torch.all((got.float() - want).abs() <= (2.0 ** -8 if dtype == torch.bfloat16 else 2.0 ** -20) * want.abs()
                     + 2.0 ** -20 * want.norm(dim=1, keepdim=True))


@pytest.mark.parametrize("pair", ["0", "1"])
@pytest.mark.parametrize("T,N,K", [(1, 8, 64), (200, 72, 192), (129, 264, 64), (300, 1000, 448)])
@pytest.mark.parametrize("fmt", [Q.NVFP4, Q.MXFP4])
def test_gemm_of_one_group_with_odd_sizes(monkeypatch, pair, T, N, K, fmt):
    """One group: N a multiple of 8, K of 64."""
    monkeypatch.setenv("QFP4_GEMM_PAIR", pair)
    off = torch.tensor([0, T], dtype=torch.int32, device="cuda")
    x, w = cpu((T, K), 53), cpu((N, K), 54)
    xp = padded(x, [T], [0, T], T)
    (A, B), (a, b) = operands(fmt, Q.HAD_NONE, xp, Q.ROW, w, Q.ROW)
    for dtype in (torch.bfloat16, torch.float32):
        out, guard = helpers.guarded_matrix(T, N, dtype, "cuda")
        Q.gemm_grouped(A, B, off, T, out=out)
        Q.status()
        helpers.assert_guards_intact(guard)
        within(out, a[:T] @ b.T, O.GEMM_REL_BOUND * (np.abs(a[:T]) @ np.abs(b).T), dtype == torch.bfloat16)


@pytest.mark.parametrize("C", [8, 40, 200, 1032])
@pytest.mark.parametrize("had", [Q.HAD_NONE, Q.HAD_DET16, Q.HAD_DET32])
def test_quantize_along_tokens_with_odd_widths(C, had):
    sizes, off, T, offsets = split("ragged")
    x = cpu((T, C), 55)
    for fmt in (Q.NVFP4, Q.MXFP4):
        q = Q.quantize_grouped(x.cuda(), offsets, fmt, Q.RTN, had, Q.COL)
        want = O.quantize(padded(x, sizes, off, T), fmt, O.RTN, had, O.COL)
        assert np.array_equal(helpers.to_numpy_u8(q.codes), want.codes)
        flat = helpers.to_numpy_u8(q.scales)
        assert np.array_equal(helpers.unswizzle_scales(flat, C, q.k, Q.BLOCK[fmt]), want.scales)
    Q.status()


@pytest.mark.parametrize("name", SPLITS)
@pytest.mark.parametrize("fmt", [Q.NVFP4, Q.MXFP4])
@pytest.mark.parametrize("kind", ["f32", "bf16", "add"])
def test_wgrad_is_the_product_over_each_group(name, fmt, kind):
    sizes, off, T, offsets = split(name)
    E, M, N = len(sizes), 384 if len(sizes) < 100 else 128, 264 if len(sizes) < 100 else 40
    dy, x = cpu((T, M), 4), cpu((T, N), 5)
    (A, B), (a, b) = operands(fmt, Q.HAD_DET32, padded(dy, sizes, off, T), Q.COL, padded(x, sizes, off, T), Q.COL)
    dtype = torch.bfloat16 if kind == "bf16" else torch.float32
    flat, guard = helpers.guarded_matrix(E * M, N, dtype, "cuda")
    out = flat.view(E, M, N)
    held = cpu((E, M, N), 6).double().numpy() if kind == "add" else np.zeros((E, M, N))
    out.copy_(torch.tensor(held) if kind == "add" else torch.full((E, M, N), float("nan")))
    Q.gemm_grouped_wgrad(A, B, offsets, T, out=out, accumulate=kind == "add")
    Q.status()
    helpers.assert_guards_intact(guard)
    p = starts(sizes)
    ref, bound = held.copy(), np.zeros_like(held)
    for e in range(E):
        ae, be = a[:, p[e]:p[e + 1]], b[:, p[e]:p[e + 1]]
        prod = ae @ be.T
        ref[e] += prod
        bound[e] = O.GEMM_REL_BOUND * (np.abs(ae) @ np.abs(be).T) + (2.0 ** -24 * np.abs(ref[e]) if kind == "add" else 0)
    within(out, ref, bound, kind == "bf16")


def layer_reference(dy, x, w, sizes, off, T, r):
    """Oracle of the layer over the padded rows: (value, bound) of Y, dX and dW."""
    E, N, K = w.shape
    flat = w.reshape(E * N, K)
    xp, dyp = padded(x, sizes, off, T), padded(dy, sizes, off, T)
    c, d, g = r.fprop, r.dgrad, r.wgrad
    q = lambda t, cfg, rnd, ax, gemm, op: O.dequantize(  # noqa: E731
        O.quantize(t, cfg.fmt, rnd, cfg.had, ax, ROT, gemm, SRS, op))
    a, b = q(xp, c, c.rnd_a, O.ROW, 0, 0), q(flat, c, c.rnd_b, O.ROW, 0, 1)
    ad, bd = q(dyp, d, d.rnd_a, O.ROW, 1, 2), q(flat, d, d.rnd_b, O.COL, 1, 3)
    aw, bw = q(dyp, g, g.rnd_a, O.COL, 2, 4), q(xp, g, g.rnd_b, O.COL, 2, 5)
    y, dx, dw = np.zeros((2, T, N)), np.zeros((2, T, K)), np.zeros((2, E, N, K))
    p = starts(sizes)
    for e, m in enumerate(sizes):
        rows, pr = slice(off[e], off[e] + m), slice(p[e], p[e] + m)
        for i, f in enumerate((lambda t: t, np.abs)):
            s = O.GEMM_REL_BOUND if i else 1.0
            y[i, rows] = s * (f(a[pr]) @ f(b[e * N:(e + 1) * N]).T)
            dx[i, rows] = s * (f(ad[pr]) @ f(bd[:, e * N:(e + 1) * N]).T)
            dw[i, e] = s * (f(aw[:, p[e]:p[e + 1]]) @ f(bw[:, p[e]:p[e + 1]]).T)
    return y, dx, dw


@pytest.mark.parametrize("name", ["ragged", "one", "outside", "none", "skewed"])
@pytest.mark.parametrize("preset", ["QUARTET2_NVFP4", "NVIDIA_NVFP4", "AMD_MXFP4_H"])
def test_layer_forward_and_backward(name, preset):
    sizes, off, T, offsets = split(name)
    E, N, K = len(sizes), 256, 384
    x, w, dy = cpu((T, K), 7), cpu((E, N, K), 8, 0.05), cpu((T, N), 9, 1e-3)
    rec, seed = Q.recipe(preset), Q.make_seed(ROT, SRS)
    X, W, dY = x.cuda(), w.cuda(), dy.cuda()
    Y = torch.full((T, N), -3.0, dtype=torch.bfloat16, device="cuda")
    dX = torch.full((T, K), -3.0, dtype=torch.bfloat16, device="cuda")
    Q.linear_grouped_fwd(X, W, offsets, rec, seed, Y=Y)
    _, dW = Q.linear_grouped_bwd(dY, X, W, offsets, rec, seed, dX=dX)
    Q.status()
    y, dx, dw = layer_reference(dy, x, w, sizes, off, T, O.preset(preset))
    inside = slice(int(off[0]), int(off[-1]))
    within(Y[inside], y[0][inside], y[1][inside], True)
    within(dX[inside], dx[0][inside], dx[1][inside], True)
    within(dW, dw[0], dw[1], False)
    for t in (Y, dX):
        assert torch.all(t[:int(off[0])] == -3) and torch.all(t[int(off[-1]):] == -3)


@pytest.mark.parametrize("had", [Q.HAD_NONE, Q.HAD_DET16, Q.HAD_DET32])
def test_layer_round_to_nearest_backward(had):
    """dY's two quantizations from one read, dW added to what it holds, outputs in fp32."""
    sizes, off, T, offsets = split("ragged")
    E, N, K = len(sizes), 128, 256
    x, w, dy = cpu((T, K), 17), cpu((E, N, K), 18, 0.05), cpu((T, N), 19, 1e-3)
    rec, r = Q.recipe("NVIDIA_NVFP4"), O.preset("NVIDIA_NVFP4")
    rec.dgrad.rnd_a = rec.wgrad.rnd_a = Q.RTN
    rec.wgrad.had = had
    rec.y_dtype = rec.dx_dtype = Q.OUT_F32
    rec.dw_accumulate = 1
    r = O.Recipe(r.fprop, dataclasses.replace(r.dgrad, rnd_a=O.RTN), dataclasses.replace(r.wgrad, rnd_a=O.RTN, had=had))
    seed = Q.make_seed(ROT, SRS)
    held = cpu((E, N, K), 20, 1e-3).float()
    dW = held.cuda()
    Y = Q.linear_grouped_fwd(x.cuda(), w.cuda(), offsets, rec, seed)
    dX, _ = Q.linear_grouped_bwd(dy.cuda(), x.cuda(), w.cuda(), offsets, rec, seed, dW=dW)
    Q.status()
    y, dx, dw = layer_reference(dy, x, w, sizes, off, T, r)
    assert Y.dtype == dX.dtype == torch.float32
    within(Y, y[0], y[1], False)
    within(dX, dx[0], dx[1], False)
    ref = dw[0] + held.double().numpy()
    within(dW, ref, dw[1] + 2.0 ** -24 * np.abs(ref), False)
    with pytest.raises(ValueError):
        Q.linear_grouped_bwd(dy.cuda(), x.cuda(), w.cuda(), offsets, rec, seed)


def test_one_group_is_the_dense_layer():
    T, N, K = 512, 256, 384
    X, W, dY = cpu((T, K), 21).cuda(), cpu((N, K), 22, 0.05).cuda(), cpu((T, N), 23, 1e-3).cuda()
    off = torch.tensor([0, T], dtype=torch.int32, device="cuda")
    seed = Q.make_seed(3, 4)
    for preset in Q.PRESETS:
        rec = Q.recipe(preset)
        assert torch.equal(Q.linear_grouped_fwd(X, W[None], off, rec, seed), Q.linear_fwd(X, W, rec, seed))
        for a, b in zip(Q.linear_grouped_bwd(dY, X, W[None], off, rec, seed), Q.linear_bwd(dY, X, W, rec, seed)):
            assert torch.equal(a.view(b.shape), b)
    Q.status()


def test_no_rows_at_all():
    X = torch.empty((0, 128), dtype=torch.bfloat16, device="cuda")
    W = cpu((2, 256, 128), 24).cuda()
    off = torch.zeros(3, dtype=torch.int32, device="cuda")
    rec, seed = Q.recipe("QUARTET2_NVFP4"), Q.make_seed()
    Y = Q.linear_grouped_fwd(X, W, off, rec, seed)
    assert Y.shape == (0, 256)
    dX, dW = Q.linear_grouped_bwd(Y, X, W, off, rec, seed)
    assert dX.shape == (0, 128) and not dW.any()
    q = Q.quantize_grouped(X, off, Q.NVFP4, Q.RTN, Q.HAD_NONE, Q.ROW)
    B = Q.quantize(W.view(512, 128), Q.NVFP4, Q.RTN, Q.HAD_NONE, Q.ROW)
    assert Q.gemm_grouped(q, B, off, 0).shape == (0, 256)
    Q.status()


@pytest.mark.parametrize("bad", [[0, 5, 4, 10], [-1, 2, 3, 4], [0, 3, 9, 101], [200, 0, 0, 0]])
def test_bad_offsets_are_reported_and_nothing_is_touched(bad):
    T, E, N, K = 100, 3, 128, 128
    X, W = cpu((T, K), 25).cuda(), cpu((E, N, K), 26).cuda()
    good = torch.tensor([0, 30, 60, 100], dtype=torch.int32, device="cuda")
    off = torch.tensor(bad, dtype=torch.int32, device="cuda")
    rec, seed = Q.recipe("AMD_MXFP4_H"), Q.make_seed()
    Y, guard = helpers.guarded_matrix(T, N, torch.bfloat16, "cuda")
    Y.fill_(2)
    Q.linear_grouped_fwd(X, W, off, rec, seed, Y=Y)
    with pytest.raises(Q.QFP4Error) as e:
        Q.status()
    assert e.value.status == Q.ERR_OFFSETS and "offsets" in str(e.value)
    helpers.assert_guards_intact(guard)
    assert torch.all(Y == 2)
    dX, dW = Q.linear_grouped_bwd(Y, X, W, off, rec, seed, dX=Y.clone())
    with pytest.raises(Q.QFP4Error):
        Q.status()
    assert torch.all(dX == 2) and not dW.any()
    Q.linear_grouped_fwd(X, W, good, rec, seed, Y=Y)  # the next call is not affected
    Q.status()
    assert not torch.all(Y == 2)


def test_amax_from_the_norm():
    """norm -> experts: the norm's amax, taken before the rows are sorted by expert, in place of the layer's own."""
    T, E, N, K = 300, 4, 256, 512
    g = torch.Generator().manual_seed(27)
    to = torch.randint(0, E, (T,), generator=g)
    order = torch.argsort(to).cuda()
    off = torch.tensor(np.concatenate(([0], np.cumsum(np.bincount(to, minlength=E)))), dtype=torch.int32, device="cuda")
    x, w = cpu((T, K), 28).cuda(), (1 + 0.1 * cpu((K,), 29).float()).bfloat16().cuda()
    W = cpu((E, N, K), 30, 0.05).cuda()
    rec, seed = Q.recipe("QUARTET2_NVFP4"), Q.make_seed(8, 9)
    y, _, _, amax = Q.rmsnorm_fwd(x, w, 1e-5, had=rec.fprop.had, seed=Q.make_seed(8), want_amax=True)
    rows = y[order]
    assert torch.equal(Q.linear_grouped_fwd(rows, W, off, rec, seed, x_amax=amax),
                       Q.linear_grouped_fwd(rows, W, off, rec, seed))
    Q.status()


def test_autograd_streams_and_graph():
    sizes, off, T, offsets = split("outside")
    E, N, K = len(sizes), 128, 256
    X, W, dY = cpu((T, K), 31).cuda(), cpu((E, N, K), 32, 0.05).cuda(), cpu((T, N), 33, 1e-2).cuda()
    rec, seed = Q.recipe("NVIDIA_NVFP4"), Q.make_seed(1, 2)
    a, b = X.clone().requires_grad_(), W.clone().requires_grad_()
    Y = Q.Fp4GroupedLinear.apply(a, b, offsets, rec, seed)
    Y.backward(dY)
    ins = slice(int(off[0]), int(off[-1]))
    want = Q.linear_grouped_fwd(X, W, offsets, rec, seed)
    dX, dW = Q.linear_grouped_bwd(dY, X, W, offsets, rec, seed)
    assert torch.equal(Y[ins], want[ins]) and torch.equal(a.grad[ins], dX[ins]) and torch.equal(b.grad, dW.bfloat16())
    for t in (Y, a.grad):
        assert not t[:int(off[0])].any() and not t[int(off[-1]):].any()
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    got = [Q.linear_grouped_bwd(dY, X, W, offsets, rec, seed, stream=s) for s in (s1, s2)]
    torch.cuda.synchronize()
    for gx, gw in got:
        assert torch.equal(gx[ins], dX[ins]) and torch.equal(gw, dW)
    # captured once, replayed with other offsets (outputs from outside the graph, whose own memory is reused within it:
    # rows of no group keep what was there)
    o = offsets.clone()
    y, gx, gw = torch.empty_like(want), torch.empty_like(dX), torch.empty_like(dW)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        Q.linear_grouped_fwd(X, W, o, rec, seed, Y=y)
        Q.linear_grouped_bwd(dY, X, W, o, rec, seed, dX=gx, dW=gw)
    for cuts in ([0, 0, 299, 300], [0, 100, 200, 307]):
        o.copy_(torch.tensor(cuts, dtype=torch.int32))
        y.zero_(), gx.zero_()
        graph.replay()
        want = Q.linear_grouped_fwd(X, W, o, rec, seed, Y=torch.zeros_like(y))
        wx, ww = Q.linear_grouped_bwd(dY, X, W, o, rec, seed, dX=torch.zeros_like(gx))
        assert torch.equal(y, want) and torch.equal(gx, wx) and torch.equal(gw, ww)
    Q.status()


@pytest.mark.parametrize("T,E,N,K", [(1, 64, 1024, 512), (4099, 8, 512, 256), (3, 256, 128, 128), (2500, 3, 4224, 128)])
def test_larger_and_smallest(T, E, N, K):
    """Many tiles per CTA, few rows among many experts: against each expert's dense product."""
    g = torch.Generator().manual_seed(T)
    cuts = torch.sort(torch.randint(0, T + 1, (E - 1,), generator=g))[0].tolist()
    off = [0, *cuts, T]
    offsets = torch.tensor(off, dtype=torch.int32, device="cuda")
    X, W = cpu((T, K), 41).cuda(), cpu((E * N, K), 42, 0.05).cuda()
    for fmt in (Q.NVFP4, Q.MXFP4):
        A = Q.quantize_grouped(X, offsets, fmt, Q.RTN, Q.HAD_NONE, Q.ROW)
        B = Q.quantize(W, fmt, Q.RTN, Q.HAD_NONE, Q.ROW)
        Y = Q.gemm_grouped(A, B, offsets, T)
        amax = Q.amax(X) if fmt == Q.NVFP4 else None
        dense = Q.gemm(Q.quantize(X, fmt, Q.RTN, Q.HAD_NONE, Q.ROW, amax_in=amax), B, torch.float32)
        for e in range(E):
            r = slice(off[e], off[e + 1])
            want = dense[r, e * N:(e + 1) * N]
            # both sum the same products, each within 2^-18 of the sum of magnitudes; here compared with the row's norm
            tol = 2.0 ** -8 * want.abs() + 2.0 ** -16 * want.norm(dim=1, keepdim=True)
            assert torch.all((Y[r].float() - want).abs() <= tol)
    Q.status()


def test_training_step_captured():
    """norm -> experts, forward and backward through the autograd functions, captured and replayed on other data."""
    T, E, N, K = 256, 3, 256, 512
    off = torch.tensor([0, 100, 100, T], dtype=torch.int32, device="cuda")
    x, r = (cpu((T, K), s).cuda().requires_grad_() for s in (71, 72))
    w, W = torch.ones(K, dtype=torch.bfloat16, device="cuda").requires_grad_(), cpu((E, N, K), 73, 0.05).cuda().requires_grad_()
    dY, dh = cpu((T, N), 74).cuda(), cpu((T, K), 75).cuda()
    rec, seed = Q.recipe("QUARTET2_NVFP4"), Q.make_seed(1, 2)

    def step():
        y, h = Q.RmsNorm.apply(x, r, w, 1e-5)
        return torch.autograd.grad((Q.Fp4GroupedLinear.apply(y, W, off, rec, seed), h), (x, r, w, W), (dY, dh))

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for s in (76, 77):
        with torch.no_grad():
            x.copy_(cpu((T, K), s))
        graph.replay()
        held = [t.clone() for t in got]
        assert all(torch.equal(a, b) for a, b in zip(held, step()))
    Q.status()


def test_offsets_past_32_bits():
    """Inputs and outputs of more than 2^31 elements: their last rows, columns and groups against the dense calls."""
    T, C = 140_000, 16384
    cut = 69_999
    off = torch.tensor([0, cut, T], dtype=torch.int32, device="cuda")
    x = torch.zeros((T, C), dtype=torch.bfloat16, device="cuda")
    x[-200:] = cpu((200, C), 61).cuda()
    amax = torch.full((1,), 6.0, device="cuda")
    p = (cut + 127) // 128 * 128
    q = Q.quantize_grouped(x, off, Q.NVFP4, Q.SR, Q.HAD_DET16, Q.ROW, amax_in=amax)
    q0 = Q.quantize(torch.cat((torch.zeros((p, C), dtype=torch.bfloat16, device="cuda"), x[cut:])), Q.NVFP4, Q.SR,
                    Q.HAD_DET16, Q.ROW, amax_in=amax)
    assert torch.equal(q.codes[p:p + T - cut], q0.codes[p:]) and not q.codes[:cut].any()
    del q, q0
    q = Q.quantize_grouped(x, off, Q.MXFP4, Q.RTN, Q.HAD_DET32, Q.COL)
    first = (T - cut) // 128 * 128 - 128  # of the second group's rows: its last whole segment and the rest
    rest = T - cut - first
    want = Q.quantize_grouped(x[cut + first:], torch.tensor([0, rest], dtype=torch.int32, device="cuda"), Q.MXFP4, Q.RTN,
                              Q.HAD_DET32, Q.COL)
    k0, n = p + first, (rest + 127) // 128 * 128
    assert torch.equal(q.codes[:, k0 // 2:(k0 + n) // 2], want.codes[:, :n // 2]) and want.codes.any()
    assert not q.codes[:, :k0 // 2 - 64].any()
    del q, want, x
    # D of T x N
    T, N, K = 70_000, 33_024, 128
    off = torch.tensor([0, 65_000, T], dtype=torch.int32, device="cuda")
    X, W = cpu((T, K), 62).cuda(), cpu((2 * N, K), 63).cuda()
    A = Q.quantize_grouped(X, off, Q.MXFP4, Q.RTN, Q.HAD_NONE, Q.ROW)
    B = Q.quantize(W, Q.MXFP4, Q.RTN, Q.HAD_NONE, Q.ROW)
    Y = Q.gemm_grouped(A, B, off, T)
    d = Q.gemm(Q.quantize(X[-300:].contiguous(), Q.MXFP4, Q.RTN, Q.HAD_NONE, Q.ROW),
               Q.quantize(W[N:].contiguous(), Q.MXFP4, Q.RTN, Q.HAD_NONE, Q.ROW))
    assert torch.equal(Y[-300:], d)
    del Y, d, A, B
    # dW of E x M x N
    E, M, N, T = 8, 16384, 16640, 300
    off = torch.tensor([0, 10, 20, 30, 40, 50, 60, 70, T], dtype=torch.int32, device="cuda")
    dy, X = cpu((T, M), 64).cuda(), cpu((T, N), 65).cuda()
    A, B = (Q.quantize_grouped(t, off, Q.MXFP4, Q.RTN, Q.HAD_DET32, Q.COL) for t in (dy, X))
    dW = Q.gemm_grouped_wgrad(A, B, off, T)
    o1 = torch.tensor([0, T - 70], dtype=torch.int32, device="cuda")
    a, b = (Q.quantize_grouped(t[70:].contiguous(), o1, Q.MXFP4, Q.RTN, Q.HAD_DET32, Q.COL) for t in (dy, X))
    assert torch.equal(dW[-1], Q.gemm_grouped_wgrad(a, b, o1, T - 70)[0])
    Q.status()
