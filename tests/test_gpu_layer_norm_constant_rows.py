"""Layer norm backward of constant rows of large values: what lies past a row's end adds nothing."""
import pytest
import torch

import exact_sum_gemm_gb300 as dg
from training_ref import assert_within

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16


# With mean = x, xhat = 0 and dx = rstd (g - mean(g)).
@pytest.mark.parametrize("dt", [F32, BF16])
@pytest.mark.parametrize("value", [1.0, 2.0 ** 100, -2.0 ** 118])
@pytest.mark.parametrize("width", [3, 4, 8, 16, 64, 512, 520, 1024, 4096, 8192, 16384, 20000])
@pytest.mark.parametrize("rows", [2, 70])
def test_constant_rows(rows, width, value, dt):
    g = torch.Generator(device="cuda")
    g.manual_seed(width)
    x = torch.full((rows, width), value, device="cuda", dtype=dt)
    w = torch.randn(width, generator=g, device="cuda").to(dt)
    dy = torch.randn(rows, width, generator=g, device="cuda").to(dt)
    mean = torch.full((rows,), value, device="cuda")
    rstd = torch.full((rows,), 1e6, device="cuda")           # of eps = 1e-12
    # f32: the product, the sum of `width` terms (their mean magnitude is below 1) in at most 90 steps,
    # two roundings of the difference and of the result; the result's own rounding
    unit = 2.0 ** -8 if dt == BF16 else 2.0 ** -23
    for given in (True, False):                              # with the sums over rows, without
        param = w if given else None
        dx, dw, db = dg.det_layer_norm_backward(dy, x, mean, rstd, param, param)
        gw = dy.double() * (w.double() if given else 1.0)
        want = 1e6 * (gw - gw.mean(1, keepdim=True))
        assert dx.isfinite().all()
        assert_within(dx, want, 1e6 * 2.0 ** -24 * (4 * gw.abs() + 100) + unit * want.abs(), "dx")
        if given:
            assert not dw.any()
            total = dy.double().sum(0)
            assert_within(db, total, 2.0 ** -24 * 130 * dy.double().abs().sum(0) + unit * total.abs(), "dbias")
