"""The training operators in CUDA graphs, on several streams and from several threads."""
import threading

import pytest
import torch

import exact_sum_gemm_gb300 as dg

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16


def operator(name, dt):
    """(inputs, forward -> tuple of outputs, backward(inputs, outputs) -> tuple of gradients)"""
    g = torch.Generator(device="cuda")
    g.manual_seed(7)
    new = lambda *s: torch.randn(*s, generator=g, device="cuda").to(dt)  # noqa: E731
    if name == "layer_norm":
        return ((new(900, 1500), new(1500), new(1500), new(900, 1500)),
                lambda x, w, b, dy: dg.det_layer_norm_forward(x, w, b),
                lambda x, w, b, dy, y, m, r: dg.det_layer_norm_backward(dy, x, m, r, w, b))
    if name == "attention":
        lengths = torch.tensor([300, 155], dtype=torch.int32, device="cuda")
        kw = dict(causal=True, k_lengths=lengths)
        return ((new(2, 300, 4, 64), new(2, 300, 2, 64), new(2, 300, 2, 64), new(2, 300, 4, 64)),
                lambda q, k, v, do: dg.det_attention_forward(q, k, v, **kw),
                lambda q, k, v, do, o, lse: dg.det_attention_backward(do, q, k, v, o, lse, **kw))
    if name == "attention_wide":
        return ((new(2, 200, 4, 96), new(2, 200, 2, 96), new(2, 200, 2, 96), new(2, 200, 4, 96)),
                lambda q, k, v, do: dg.det_attention_forward(q, k, v),
                lambda q, k, v, do, o, lse: dg.det_attention_backward(do, q, k, v, o, lse))
    tokens = torch.randint(0, 20001, (130,), generator=g, device="cuda")
    return ((new(130, 20001), new(130).float(), new(130).float()),
            lambda x, a, b: dg.det_token_logprobs_forward(x, tokens, top=5),
            lambda x, a, b, lp, h, s, tl, tt: (dg.det_token_logprobs_backward(a, b, x, tokens, h, s),))


def step(inputs, forward, backward):
    outputs = forward(*inputs)
    return tuple(outputs) + tuple(backward(*inputs, *outputs))


def same(got, want):
    return all(torch.equal(a, b) for a, b in zip(got, want, strict=True))


CASES = [(n, dt) for n in ("layer_norm", "attention", "attention_wide", "logprobs") for dt in (F32, BF16)]


@pytest.mark.parametrize("name,dt", CASES)
def test_graph(name, dt):
    """Captured once, replayed on new values in the same places."""
    inputs, forward, backward = operator(name, dt)
    want = [t.clone() for t in step(inputs, forward, backward)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(inputs, forward, backward)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step(inputs, forward, backward)
    for _ in range(2):
        for t in got:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert same(got, want)
    inputs[0].mul_(0.5)
    graph.replay()
    torch.cuda.synchronize()
    assert same(got, step(inputs, forward, backward))
    assert not same(got, want)


@pytest.mark.parametrize("name,dt", CASES)
def test_backward_on_another_stream(name, dt):
    inputs, forward, backward = operator(name, dt)
    want = step(inputs, forward, backward)
    torch.cuda.synchronize()
    first, second = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(3):
        with torch.cuda.stream(first):
            outputs = forward(*inputs)
        second.wait_stream(first)
        with torch.cuda.stream(second):
            grads = backward(*inputs, *outputs)
        first.wait_stream(second)                 # (the outputs belong to the first)
        torch.cuda.synchronize()
        assert same(tuple(outputs) + tuple(grads), want)


@pytest.mark.parametrize("dt", [F32, BF16])
def test_threads(dt):
    """Every operator from a thread of its own, each on its stream, at once."""
    cases = [operator(n, dt) for n in ("layer_norm", "attention", "attention_wide", "logprobs")]
    wants = [step(*c) for c in cases]
    torch.cuda.synchronize()
    wrong = []

    def work(case, want):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                for _ in range(10):
                    got = step(*case)
                    torch.cuda.current_stream().synchronize()
                    if not same(got, want):
                        wrong.append("bits")
        except Exception as e:  # noqa: BLE001
            wrong.append(repr(e))
    threads = [threading.Thread(target=work, args=(c, w)) for c, w in zip(cases * 2, wants * 2, strict=True)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong
    assert dg.device_status() == "ok"
