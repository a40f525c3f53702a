"""Layer norm of many rows against its 64-bit definition: every kernel, with several rows to a block."""
import pytest
import torch

import exact_sum_gemm_gb300 as dg
from training_ref import assert_within, layer_norm

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16


def rand(*shape, seed=0, std=1.0, dtype=F32):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return (torch.randn(*shape, generator=g, device="cuda") * std).to(dtype)


# More than 64 rows, as the backward pass of fewer is another kernel.  Blocks have a second row, and the
# ring a second turn, from 2432 rows of up to 512 columns on, 912 of up to 2048, 456 of up to 4096 and 304
# of more (152 of more than 8192).  Odd widths put rows off 16 bytes.
@pytest.mark.parametrize("types", [(F32, F32), (BF16, BF16), (BF16, F32)])
@pytest.mark.parametrize("rows,width", [
    (65, 500), (5000, 40), (8000, 512), (8000, 333),
    (65, 513), (4000, 1000), (4000, 513), (3000, 2048),
    (65, 2049), (1500, 2056), (2000, 4096), (1500, 4095),
    (65, 4097), (400, 4104), (1500, 5001), (1500, 8192),
    (65, 8193), (400, 8200), (400, 12289), (1500, 16384), (700, 16383),
    (65, 16385), (400, 16392), (700, 20001)])
def test_many_rows(rows, width, types):
    dt, wdt = types
    x = rand(rows, width, seed=1, std=2.0, dtype=dt) + 0.5
    w, b = 1 + rand(width, seed=2, std=0.3, dtype=wdt), rand(width, seed=3, dtype=wdt)
    dy = rand(rows, width, seed=4, dtype=dt)
    y, mean, rstd = dg.det_layer_norm_forward(x, w, b)
    dx, dw, db = dg.det_layer_norm_backward(dy, x, mean, rstd, w, b)
    want = layer_norm(x, w, b, 1e-5, dy)
    got = {"y": y, "mean": mean, "rstd": rstd, "dx": dx, "dweight": dw, "dbias": db}
    for name, t in got.items():
        assert_within(t, *want[name], name)
    # the last rows alone, and without parameters' gradients: the same bits
    part = dg.det_layer_norm_backward(dy[-9:], x[-9:], mean[-9:], rstd[-9:], w, b)[0]
    assert torch.equal(part, dx[-9:])
    assert torch.equal(dg.det_layer_norm_forward(x[-9:], w, b)[0], y[-9:])


@pytest.mark.parametrize("dt", [F32, BF16])
@pytest.mark.parametrize("rows,width", [(65, 300), (3000, 2048), (1500, 4096), (1500, 5001), (400, 16384)])
def test_many_rows_without_parameters(rows, width, dt):
    x, dy = rand(rows, width, seed=5, dtype=dt), rand(rows, width, seed=6, dtype=dt)
    y, mean, rstd = dg.det_layer_norm_forward(x)
    dx, dw, db = dg.det_layer_norm_backward(dy, x, mean, rstd)
    want = layer_norm(x, None, None, 1e-5, dy)
    assert dw is None and db is None
    assert_within(y, *want["y"], "y")
    assert_within(dx, *want["dx"], "dx")
    # a bias alone takes the kernel that sums over rows
    dx2, _, db = dg.det_layer_norm_backward(dy, x, mean, rstd, None, torch.zeros(width, device="cuda", dtype=dt))
    assert torch.equal(dx2, dx)
    total = dy.double().sum(0)
    steps = rows // 152 + 120
    assert_within(db, total, steps * 2.0 ** -24 * dy.double().abs().sum(0) + (2.0 ** -8 if dt == BF16 else 2.0 ** -23)
                  * total.abs(), "dbias")


def test_strided_rows():
    """Rows of a wider matrix, several to a block, aligned and not: the contiguous call's bits."""
    for dt in (F32, BF16):
        wide, dwide = rand(1200, 5200, seed=7, dtype=dt), rand(1200, 5200, seed=8, dtype=dt)
        w = rand(5000, seed=9, dtype=dt)
        for start in (0, 8, 1):
            x, dy = wide[:, start:start + 5000], dwide[:, start:start + 5000]
            got, want = [], []
            for out, a, g in ((got, x, dy), (want, x.contiguous(), dy.contiguous())):
                y, mean, rstd = dg.det_layer_norm_forward(a, w, w)
                out += [y, mean, rstd, *dg.det_layer_norm_backward(g, a, mean, rstd, w, w)]
            for a, b in zip(got, want):
                assert torch.equal(a, b), (dt, start)
