"""Token log probabilities of large finite logits and large gradients, against the 64-bit definition."""
import math

import pytest
import torch

import exact_sum_gemm_gb300 as dg
from training_ref import assert_within, token_logprobs

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16
VOCAB = 40000                                               # five f32 or three bf16 segments


def make(rows, dt, seed=0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    x = (torch.randn(rows, VOCAB, generator=g, device="cuda") * 2.5).to(dt)
    t = torch.randint(0, VOCAB, (rows,), generator=g, device="cuda")
    dlp = torch.randn(rows, generator=g, device="cuda")
    dh = torch.randn(rows, generator=g, device="cuda") * 0.1
    return x, t, dlp, dh


def check(x, t, g, h, top=4):
    lp, entropy, stats, tlp, tt = dg.det_token_logprobs_forward(x, t, top=top)
    dx = dg.det_token_logprobs_backward(g, h, x, t, entropy, stats)
    want = token_logprobs(x, t, top, g, h)
    assert torch.equal(tt, want["top_tokens"][0])
    for name, v in (("logprobs", lp), ("entropy", entropy), ("top_logprobs", tlp), ("dlogits", dx)):
        assert v.isfinite().all(), name
        assert_within(v, *want[name], name)


@pytest.mark.parametrize("dt", [F32, BF16])
@pytest.mark.parametrize("size", [1e3, 1e6, 2.0 ** 20, 1.1e6, 1e8, 1e9, 3e9, 5e9, 1e10, 1e12, 1e20, 0.99e30, 1.01e30])
def test_large_logits(size, dt):
    """What is used as a mask or a boost, over a whole row, a whole segment, all but one, one alone."""
    x, t, g, h = make(12, dt)
    x[0] = -size
    x[1] = size
    x[2, :16384] = -size                                    # the first segments
    x[3, 16384:] = -size
    x[4, 1:] = -size
    x[5, :-1] = -size
    x[6, 20000] = size
    x[7, 0], x[7, 39999] = size, -size
    x[8, ::2] = -size
    x[9, 8192:16384] = size
    x[10] = -size
    x[10, 777] = -size * 2
    x[11] = size
    x[11, 777] = size * 2
    t[4], t[6], t[11] = 0, 20000, 777
    check(x, t, g, h)


@pytest.mark.parametrize("dt", [F32, BF16])
@pytest.mark.parametrize("level", [-2.0 ** 20, -1e6, -3e5, 1e4, 2.0 ** 20, 1.2e6, 2.0 ** 23])
def test_logits_around_a_large_level(level, dt):
    """Every logit next to a level whose rounding is felt: differences of a few spacings."""
    x, t, g, h = make(6, dt, seed=1)
    check((x.to(F32) + level).to(dt), t, g, h)


@pytest.mark.parametrize("dt", [F32, BF16])
def test_large_entropy_gradients(dt):
    """-inf logits have no gradient, however large the gradient of the entropy is."""
    x, t, g, h = make(4, dt, seed=2)
    x[0, ::3] = -math.inf
    x[1, 5:] = torch.finfo(dt).min
    x[2, 100:] = -1e10
    h = torch.full_like(h, 1e12)
    t[0], t[1], t[2] = 1, 2, 3
    lp, entropy, stats, _, _ = dg.det_token_logprobs_forward(x, t)
    dx = dg.det_token_logprobs_backward(g, h, x, t, entropy, stats)
    assert dx.isfinite().all()
    assert not dx[0, ::3].any() and not dx[1, 5:].any() and not dx[2, 100:].any()
    assert_within(dx, *token_logprobs(x, t, 0, g, h)["dlogits"], "dlogits")
