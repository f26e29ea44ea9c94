"""Infinities, NaN and values next to bf16's largest, in inputs and weights: what
the RMSNorm's amax and MXFP4 output and the grouped quantizers make of them is
what the calls that they stand for make of y and of the padded rows, byte for
byte."""
import pytest
import torch

from fp4_precision_b200 import qfp4 as Q
from test_gpu_grouped import cpu, padded, split, starts

pytestmark = pytest.mark.gpu

INF, NAN = float("inf"), float("nan")
HADS = [Q.HAD_NONE, Q.HAD_DET16, Q.HAD_DET32, Q.HAD_RAND16, Q.HAD_RAND32]
SEED = Q.make_seed(1, 2, 3, 4)


def same(a, b):
    return torch.equal(a.contiguous().view(torch.uint8), b.contiguous().view(torch.uint8))


NORM_KINDS = {
    "infinite weights": lambda x, w: (w[5:6].fill_(INF), w[w.numel() // 2:].fill_(-INF)),
    "a group of infinite weights": lambda x, w: w[:32].fill_(INF),
    "the largest weights": lambda x, w: w.fill_(3.3e38),
    "NaN": lambda x, w: (x[3, 7:8].fill_(NAN), x[9, -1:].fill_(NAN)),
    "infinite inputs": lambda x, w: (x[3, 7:8].fill_(INF), x[4].fill_(INF)),
    "nothing but NaN": lambda x, w: x.fill_(NAN),
}


@pytest.mark.parametrize("kind", NORM_KINDS)
@pytest.mark.parametrize("R,C", [(40, 96), (40, 512), (40, 1056), (40, 2048), (20, 16384)])
def test_norm(kind, R, C):
    x, w = cpu((R, C), 1).cuda(), cpu((C,), 2).cuda()
    NORM_KINDS[kind](x, w)
    for had in HADS:
        y, _, _, amax = Q.rmsnorm_fwd(x, w, 1e-5, had=had, seed=SEED, want_amax=True)
        assert same(amax, Q.amax(y, had, Q.ROW, SEED)), had
        for fmt in (Q.MXFP4, Q.MXFP4_RU):
            q = Q.rmsnorm_quantize(x, w, 1e-5, fmt=fmt, had=had, seed=SEED)[3]
            want = Q.quantize(y, fmt, Q.RTN, had, Q.ROW, SEED)
            n = Q.scales_bytes(fmt, R, C)
            assert same(q.codes, want.codes) and same(q.scales[:n], want.scales[:n]), (had, fmt)
    Q.status()


GROUP_KINDS = {
    "NaN": lambda x, first, last: (x[first + 5, 3:4].fill_(NAN), x[last, -1:].fill_(NAN)),
    "infinities": lambda x, first, last: (x[first + 5, 3:4].fill_(INF), x[last, -1:].fill_(-INF)),
    "a run of infinities": lambda x, first, last: x[first + 5, :40].fill_(INF),
    "the largest": lambda x, first, last: x[first + 5].fill_(3.3e38),
}


@pytest.mark.parametrize("kind", GROUP_KINDS)
@pytest.mark.parametrize("name", ["ragged", "outside"])
def test_grouped_quantizers(kind, name):
    sizes, off, T, offsets = split(name)
    x = cpu((T, 160), 3)
    GROUP_KINDS[kind](x, int(off[0]), int(off[-1]) - 1)
    xp, p = padded(x, sizes, off, T).cuda(), starts(sizes)
    own = torch.cat([torch.arange(p[e], p[e] + m) for e, m in enumerate(sizes)]).cuda()
    for fmt in (Q.NVFP4, Q.MXFP4, Q.MXFP4_RU):
        for rnd in (Q.RTN, Q.SR, Q.QUARTET2):
            for had in HADS:
                for axis in (Q.ROW, Q.COL):
                    q = Q.quantize_grouped(x.cuda(), offsets, fmt, rnd, had, axis, SEED)
                    want = Q.quantize(xp, fmt, rnd, had, axis, SEED)
                    assert same(q.tensor_scale, want.tensor_scale), (fmt, rnd, had, axis)
                    if axis == Q.ROW:  # (rows of no group are not written)
                        assert same(q.codes[own], want.codes[own]), (fmt, rnd, had)
                    else:
                        n = Q.scales_bytes(fmt, q.rows, q.k)
                        assert same(q.codes, want.codes) and same(q.scales[:n], want.scales[:n]), (fmt, rnd, had)
    Q.status()
