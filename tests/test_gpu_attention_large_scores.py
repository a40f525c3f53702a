"""Attention of large finite scores: one key takes all, and nothing overflows."""
import math

import pytest
import torch

import exact_sum_gemm_gb300 as dg

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16
U = 2.0 ** -24


def one_hot_scores(lq, lk, dim, size, dt, seed=0):
    """q, k, v, do, the key of each query's largest score, and that score.

    k_j = the 16 digits (+-1/16 in 16 columns) of a code, q_i = a code times size (1 + m / 128), m of 0 .. 127:
    the product of equal codes is that factor, of others at most 7/8 of it (a digit and more differ).  All are
    exact in both types, and the sums exact in f32.
    """
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    code = torch.stack([((torch.arange(lk, device="cuda") >> b) & 1) * 2 - 1 for b in range(16)], 1).float()
    best = torch.randint(0, lk, (lq,), generator=g, device="cuda")
    q, k = torch.zeros(1, lq, 1, dim, device="cuda"), torch.zeros(1, lk, 1, dim, device="cuda")
    k[0, :, 0, :16] = code / 16
    top = size * (1 + torch.randint(0, 128, (lq,), generator=g, device="cuda") / 128)
    q[0, :, 0, :16] = code[best] * top[:, None]
    v = torch.randn(1, lk, 1, dim, generator=g, device="cuda")
    do = torch.randn(1, lq, 1, dim, generator=g, device="cuda")
    return q.to(dt), k.to(dt), v.to(dt), do.to(dt), best, top.double()


SIZES = [2.0 ** e for e in (8, 14, 20, 24, 28, 30, 31, 33, 40, 60, 100)]


@pytest.mark.parametrize("dt", [F32, BF16])
@pytest.mark.parametrize("dim,lq,lk", [(64, 40, 300), (64, 300, 300), (128, 300, 300), (96, 130, 70), (128, 33, 50)])
@pytest.mark.parametrize("size", SIZES)
@pytest.mark.parametrize("scale", [1.0, 0.3])
def test_forward(size, scale, dim, lq, lk, dt):
    q, k, v, do, best, top = one_hot_scores(lq, lk, dim, size, dt)
    o, lse = dg.det_attention_forward(q, k, v, scale=scale)
    # the next score is size / 8 less, or 2^8 0.3 / 8 > 9: at most 2^-13 of the probability with 16 like it
    want = v[0, best, 0].double()
    close = 16 * math.exp(-size * scale / 8)
    assert o.isfinite().all()
    unit = 2.0 ** -8 if dt == BF16 else 2.0 ** -22
    assert ((o[0, :, 0].double() - want).abs() <= unit * want.abs() + 2 * close * 6).all()
    # lse: five roundings of the score, and the other keys' share
    assert ((lse[0, 0].double() - top * scale).abs() <= 5 * U * top * scale + close + 1e-6).all()
    # the negative scores: the smallest product takes all
    o2, _ = dg.det_attention_forward(q, -k, v, scale=-scale)
    assert torch.equal(o2, o)


@pytest.mark.parametrize("dt", [F32, BF16])
@pytest.mark.parametrize("dim,lq,lk", [(64, 40, 300), (64, 300, 300), (128, 300, 300), (96, 130, 70), (128, 33, 50)])
@pytest.mark.parametrize("size", SIZES)
def test_backward(size, dim, lq, lk, dt):
    """No probability above 1: dv is at most the sum of |do| of the queries, whatever the scores' rounding."""
    q, k, v, do, best, top = one_hot_scores(lq, lk, dim, size, dt, seed=1)
    most = torch.zeros(lk, dim, dtype=torch.float64, device="cuda")
    most.index_add_(0, best, do[0, :, 0].double().abs())
    want = torch.zeros(lk, dim, dtype=torch.float64, device="cuda")
    want.index_add_(0, best, do[0, :, 0].double())
    for i in range(8):
        scale = 0.3 + 0.037 * i
        o, lse = dg.det_attention_forward(q, k, v, scale=scale)
        dq, dk, dv = dg.det_attention_backward(do, q, k, v, o, lse, scale=scale)
        for name, t in (("dq", dq), ("dk", dk), ("dv", dv)):
            assert t.isfinite().all(), (name, scale)
        others = 16 * lq * math.exp(-size * scale / 8) * 6
        assert (dv[0, :, 0].double().abs() <= most * (1 + 2.0 ** -7) + others).all(), scale
        # while the rounding of the scores is small, the gradient itself: six roundings of 2 size * scale in
        # the exponent
        if size <= 2.0 ** 14:
            off = 12 * U * size * scale + (2.0 ** -7 if dt == BF16 else 2.0 ** -20)
            assert ((dv[0, :, 0].double() - want).abs() <= off * most + others).all(), scale
