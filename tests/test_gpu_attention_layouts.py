"""Attention on tensors that TMA does not read, over several turns of the loaders' rings."""
import math

import pytest
import torch

import exact_sum_gemm_gb300 as dg
from training_ref import assert_within, attention

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16


def make(batch, lq, lk, hq, hkv, dim, dt, seed=0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    new = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    return ((new(batch, lq, hq, dim) * 1.2).to(dt), (new(batch, lk, hkv, dim) * 1.2).to(dt),
            new(batch, lk, hkv, dim).to(dt), new(batch, lq, hq, dim).to(dt))


def run(q, k, v, do, **kw):
    o, lse = dg.det_attention_forward(q, k, v, **kw)
    dq, dk, dv = dg.det_attention_backward(do, q, k, v, o, lse, **kw)
    return {"o": o, "lse": lse, "dq": dq, "dk": dk, "dv": dv}


def odd(x):
    """The same values, two (bf16) or four (f32) bytes off a 16-byte boundary."""
    return torch.cat([x.reshape(-1)[:1], x.reshape(-1)])[1:].view(x.shape)


def wide(x):
    """The same values in rows that are farther apart: aligned pieces, but strides off 16 bytes."""
    pad = torch.zeros(*x.shape[:3], x.shape[3] + 2, dtype=x.dtype, device=x.device)
    pad[..., :x.shape[3]] = x
    return pad[..., :x.shape[3]]


def assert_same(got, want, what):
    for name in want:
        a, b = got[name], want[name]
        assert torch.equal(a.isnan(), b.isnan()), (what, name)
        assert torch.equal(a.nan_to_num(0, math.inf, -math.inf), b.nan_to_num(0, math.inf, -math.inf)), (what, name)


# forward's ring turns after 256 keys, backward's after 384 queries or keys; with shared heads a key
# block's steps go on with the next head's queries
@pytest.mark.parametrize("layout", [odd, wide])
@pytest.mark.parametrize("lq,lk,hq,hkv,dim,causal,lengths", [
    (900, 900, 4, 1, 64, True, None), (900, 900, 6, 2, 128, True, None), (520, 1300, 4, 2, 80, False, [1300, 777]),
    (1300, 520, 3, 1, 64, True, [520, 300]), (700, 700, 4, 4, 128, True, [1, 650]), (700, 700, 2, 1, 96, False, [0, 513])])
def test_long_rows_without_tensor_maps(lq, lk, hq, hkv, dim, causal, lengths, layout):
    args = make(2, lq, lk, hq, hkv, dim, BF16, seed=lq + dim)
    if lengths is not None:
        lengths = torch.tensor(lengths, dtype=torch.int32, device="cuda")
    want = run(*args, causal=causal, k_lengths=lengths)
    assert_same(run(*(layout(x) for x in args), causal=causal, k_lengths=lengths), want, layout.__name__)
    # one tensor alone decides for all
    for i in range(4):
        mixed = [layout(x) if i == j else x for j, x in enumerate(args)]
        assert_same(run(*mixed, causal=causal, k_lengths=lengths), want, i)


# (no head dimension that is no multiple of 8 has a tensor map)
@pytest.mark.parametrize("dt", [F32, BF16])
@pytest.mark.parametrize("dim", [33, 71, 100, 127])
def test_long_rows_of_odd_head_dims(dim, dt):
    q, k, v, do = make(1, 800, 800, 4, 2, dim, dt, seed=dim)
    got = run(q, k, v, do, causal=True)
    want = attention(q, k, v, do=do, causal=True)
    for name, t in got.items():
        assert_within(t, *want[name], name)


@pytest.mark.parametrize("dt", [F32, BF16])
@pytest.mark.parametrize("dim", [64, 128])
def test_expanded_heads_and_lengths(dim, dt):
    """A stride of 0 over heads, and gradients of one value for every row."""
    q, k, v, do = make(2, 700, 700, 4, 4, dim, dt, seed=5)
    k1, v1 = k[:, :, :1].expand(-1, -1, 4, -1), v[:, :, :1].expand(-1, -1, 4, -1)
    ones = torch.ones(1, device="cuda", dtype=dt).expand(do.shape)
    lengths = torch.tensor([700, 450], dtype=torch.int32, device="cuda")
    want = run(q, k1.contiguous(), v1.contiguous(), ones.contiguous(), causal=True, k_lengths=lengths)
    assert_same(run(q, k1, v1, ones, causal=True, k_lengths=lengths), want, "expanded")


@pytest.mark.parametrize("dim,hq,hkv", [(64, 2, 2), (64, 4, 1), (128, 4, 2)])
@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
def test_masks_hide_without_tensor_maps(bad, dim, hq, hkv):
    """Non-finite values that a mask hides, or shows to some: the bits of the aligned call."""
    q, k, v, do = make(2, 600, 600, hq, hkv, dim, BF16, seed=2)
    lengths = torch.tensor([410, 600], dtype=torch.int32, device="cuda")
    clean = run(odd(q), odd(k), odd(v), odd(do), causal=True, k_lengths=lengths)
    places = {"past the length": {1: (0, slice(410, 600)), 2: (0, slice(410, 600))},
              "a key": {1: (1, 450)}, "a value": {2: (1, 450, 0, 3)}, "a query": {0: (1, 470)},
              "a gradient": {3: (1, 470)}, "an early key": {1: (1, 20)}, "the last query": {0: (1, 599), 3: (1, 599)}}
    for what, where in places.items():
        args = [x.clone() for x in (q, k, v, do)]
        for i, at in where.items():
            args[i][at] = bad
        want = run(*args, causal=True, k_lengths=lengths)
        got = run(*(odd(x) for x in args), causal=True, k_lengths=lengths)
        assert_same(got, want, what)
        for name in clean:                       # the other entry never sees it
            assert torch.equal(got[name][0], clean[name][0]), (what, name)
        if what == "past the length":
            assert_same(got, clean, what)
        if what in ("a key", "a value"):
            for name in ("o", "dq"):
                assert torch.equal(got[name][1, :450], clean[name][1, :450]), (what, name)
        if what in ("a query", "a gradient"):
            for name in ("dk", "dv"):
                assert torch.equal(got[name][1, 471:], clean[name][1, 471:]), (what, name)


@pytest.mark.parametrize("dim", [64, 128])
def test_masks_hide_in_strided_f32(dim):
    q, k, v, do = make(2, 300, 300, 4, 2, dim, F32, seed=3)
    lengths = torch.tensor([210, 300], dtype=torch.int32, device="cuda")
    k[0, 210:], v[0, 210:], k[1, 150], do[1, 170] = math.nan, math.inf, -math.inf, math.nan
    want = run(q, k, v, do, causal=True, k_lengths=lengths)
    assert want["o"][0].isfinite().all() and want["dk"][0].isfinite().all()
    for layout in (odd, wide):
        assert_same(run(*(layout(x) for x in (q, k, v, do)), causal=True, k_lengths=lengths), want, layout.__name__)
