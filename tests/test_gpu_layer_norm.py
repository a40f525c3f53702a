"""Layer norm against its 64-bit definition: sizes, types, layouts, gradients, refusals."""
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


def run(x, w, b, dy, eps=1e-5):
    y, mean, rstd = dg.det_layer_norm_forward(x, w, b, eps)
    dx, dw, db = dg.det_layer_norm_backward(dy, x, mean, rstd, w, b)
    return {"y": y, "mean": mean, "rstd": rstd, "dx": dx, "dweight": dw, "dbias": db}


def check(x, w, b, dy, eps=1e-5):
    got = run(x, w, b, dy, eps)
    want = layer_norm(x, w, b, eps, dy)
    for name, t in got.items():
        if t is not None:
            assert_within(t, *want[name], name)
    return got


# widths on both sides of every kernel's limit: a warp per row up to 512
# columns, a block up to 16384, then the re-reading kernels; odd ones start rows
# off 16 bytes
@pytest.mark.parametrize("width", [1, 2, 3, 7, 8, 31, 64, 127, 128, 129, 256, 257, 511, 512, 513,
                                   1000, 1024, 1025, 2047, 2048, 2049, 4095, 4096, 4097, 5001, 8192,
                                   8193, 16383, 16384, 16385, 32768, 32771])
@pytest.mark.parametrize("types", [(F32, F32), (BF16, BF16), (BF16, F32)])
def test_widths(width, types):
    dt, wdt = types
    rows = 13
    x = rand(rows, width, seed=1, std=2.0, dtype=dt) + 0.5
    w, b = 1 + rand(width, seed=2, std=0.3, dtype=wdt), rand(width, seed=3, dtype=wdt)
    check(x, w, b, rand(rows, width, seed=4, dtype=dt))


@pytest.mark.parametrize("rows", [1, 2, 9, 151, 152, 153, 609, 5000])
@pytest.mark.parametrize("width", [40, 700, 3001])
def test_row_counts(rows, width):
    x = rand(rows, width, seed=5)
    check(x, rand(width, seed=6), rand(width, seed=7), rand(rows, width, seed=8))


@pytest.mark.parametrize("dt", [F32, BF16])
def test_without_parameters_and_single_gradients(dt):
    x, dy = rand(37, 300, seed=9, dtype=dt), rand(37, 300, seed=10, dtype=dt)
    got = check(x, None, None, dy)
    assert got["dweight"] is None and got["dbias"] is None
    w = rand(300, seed=11, dtype=dt)
    full = run(x, w, w, dy)
    y, mean, rstd = dg.det_layer_norm_forward(x, w, w)
    dx, dw, db = dg.det_layer_norm_backward(dy, x, mean, rstd, w, None)
    assert db is None and torch.equal(dx, full["dx"]) and torch.equal(dw, full["dweight"])
    dx, dw, db = dg.det_layer_norm_backward(dy, x, mean, rstd, w, w, need_dx=False)
    assert dx is None and torch.equal(dw, full["dweight"]) and torch.equal(db, full["dbias"])


@pytest.mark.parametrize("dt", [F32, BF16])
def test_strides_and_offsets(dt):
    """Column slices (rows off 16 bytes, a wide stride), transposed and expanded inputs."""
    wide, dwide = rand(20, 1200, seed=12, dtype=dt), rand(20, 1200, seed=13, dtype=dt)
    w, b = rand(1001, seed=14, dtype=dt)[1:], rand(1003, seed=15, dtype=dt)[3:]
    for start in (0, 1, 3, 8):
        x, dy = wide[:, start:start + 1000], dwide[:, start:start + 1000]
        got = check(x, w, b, dy)
        plain = run(x.contiguous(), w.clone(), b.clone(), dy.contiguous())
        for name in got:                          # the same bits wherever a row starts
            assert torch.equal(got[name], plain[name]), (name, start)
    check(wide.t(), rand(20, seed=16, dtype=dt), None, dwide.t())
    check(wide[:1].expand(5, 1200), None, rand(1200, seed=17, dtype=dt), dwide[:5])
    x3 = wide.reshape(4, 5, 1200).transpose(0, 1)
    check(x3, rand(1200, seed=18, dtype=dt), None, dwide.reshape(5, 4, 1200))


def test_rows_do_not_depend_on_other_rows_and_calls_repeat():
    x, dy = rand(700, 1536, seed=19), rand(700, 1536, seed=20)
    w, b = rand(1536, seed=21), rand(1536, seed=22)
    first = run(x, w, b, dy)
    again = run(x, w, b, dy)
    for name in first:
        assert torch.equal(first[name], again[name]), name
    part = run(x[333:340], w, b, dy[333:340])
    for name in ("y", "mean", "rstd", "dx"):
        assert torch.equal(part[name], first[name][333:340]), name


def test_values():
    """Constant rows, a large mean, huge and tiny values, non-finite rows stay in their row."""
    x = rand(8, 600, seed=23)
    x[0] = 3.0
    x[1] = 0.0
    x[2] += 4096.0
    x[3] *= 1e15
    x[4] *= 1e-15
    w, b, dy = rand(600, seed=24), rand(600, seed=25), rand(8, 600, seed=26)
    check(x, w, b, dy)
    bad = x.clone()
    bad[5, 17] = float("nan")
    bad[6, 599] = float("inf")
    y, mean, rstd = dg.det_layer_norm_forward(bad, w, b)
    clean, _, _ = dg.det_layer_norm_forward(x, w, b)
    keep = [0, 1, 2, 3, 4, 7]
    assert torch.equal(y[keep], clean[keep]) and y[5].isnan().all() and y[6].isnan().all()
    dx, dw, _ = dg.det_layer_norm_backward(dy, bad, mean, rstd, w)
    assert dx[keep].isfinite().all() and dx[5].isnan().all() and dw.isnan().all()


def test_no_rows():
    x, w = rand(0, 33), rand(33, seed=27)
    y, mean, rstd = dg.det_layer_norm_forward(x, w, w)
    assert y.shape == (0, 33) and mean.shape == (0,)
    dx, dw, db = dg.det_layer_norm_backward(x, x, mean, rstd, w, w)
    assert dx.shape == (0, 33) and not dw.any() and not db.any()


def test_gradient_against_differences():
    x, w, b = rand(6, 200, seed=28), 1 + rand(200, seed=29, std=0.2), rand(200, seed=30)
    dy = rand(6, 200, seed=31)
    got = run(x, w, b, dy)
    loss = lambda x, w, b: float((dg.det_layer_norm_forward(x, w, b)[0].double() * dy).sum())  # noqa: E731
    # central difference over 2^-6: off by the third derivative over 6 times
    # 2^-12 of a step of unit size, and by 1200 roundings of about 2^-24 x 4 over 2^-5
    step = 2.0 ** -6
    for name, i in (("dx", 0), ("dweight", 1), ("dbias", 2)):
        args = [x, w, b]
        v = rand(*args[i].shape, seed=32 + i)
        up, down = list(args), list(args)
        up[i], down[i] = args[i] + step * v, args[i] - step * v
        slope = (loss(*up) - loss(*down)) / (2 * step)
        dot = float((got[name].double() * v).sum())
        assert abs(slope - dot) <= 4e-3 * float(got[name].double().norm()) * float(v.norm()) / v.numel() ** 0.5 + 4e-3


def test_autograd_and_module():
    layer = dg.DetLayerNorm(96, device="cuda")
    with torch.no_grad():
        layer.weight.copy_(1 + rand(96, seed=35))
    x = rand(3, 5, 96, seed=36).requires_grad_(True)
    dy = rand(3, 5, 96, seed=37)
    y = layer(x)
    y.backward(dy)
    want = layer_norm(x.detach(), layer.weight.detach(), layer.bias.detach(), 1e-5, dy)
    assert_within(y.detach(), *want["y"], "y")
    for t, name in ((x.grad, "dx"), (layer.weight.grad, "dweight"), (layer.bias.grad, "dbias")):
        assert_within(t, *want[name], name)
    plain = dg.DetLayerNorm(96, bias=False, device="cuda")
    plain(x).sum().backward()
    assert plain.weight.grad is not None
    with pytest.raises(ValueError, match="last dim"):
        layer(rand(3, 95))


def test_other_stream():
    x, w = rand(2000, 4096, seed=38), rand(4096, seed=39)
    want = dg.det_layer_norm_forward(x, w)[0]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        x2 = x * 1.0
        got = dg.det_layer_norm_forward(x2, w)[0]
    side.synchronize()
    assert torch.equal(got, want)


def test_refusals():
    x, w = rand(4, 8), rand(8)
    y, mean, rstd = dg.det_layer_norm_forward(x, w)
    for call, match in [
            (lambda: dg.det_layer_norm_forward(x.half()), "float32 or bfloat16"),
            (lambda: dg.det_layer_norm_forward(x.cpu()), "CUDA"),
            (lambda: dg.det_layer_norm_forward(x, w[:7]), "shape"),
            (lambda: dg.det_layer_norm_forward(x, w.to(BF16)), "bfloat16 for a float32"),
            (lambda: dg.det_layer_norm_forward(x.to(BF16), w, w.to(BF16)), "share"),
            (lambda: dg.det_layer_norm_forward(x, w, w.cpu()), "CUDA"),
            (lambda: dg.det_layer_norm_forward(x, eps=-1.0), "eps"),
            (lambda: dg.det_layer_norm_forward(x, eps=float("nan")), "eps"),
            (lambda: dg.det_layer_norm_forward(x[:, :0]), "last axis"),
            (lambda: dg.det_layer_norm_backward(x[:3], x, mean, rstd), "dy"),
            (lambda: dg.det_layer_norm_backward(x.to(BF16), x, mean, rstd), "dy"),
            (lambda: dg.det_layer_norm_backward(x, x, mean[:3], rstd), "mean"),
            (lambda: dg.det_layer_norm_backward(x, x, mean, rstd.double()), "rstd")]:
        with pytest.raises(ValueError, match=match):
            call()
