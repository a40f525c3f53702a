"""Token log probabilities backward: more rows than 2^15 times the largest grid dimension."""
import pytest
import torch

import exact_sum_gemm_gb300 as dg

pytestmark = pytest.mark.gpu


def test_two_billion_rows():
    rows = (1 << 15) * 65535 + 1
    if torch.cuda.mem_get_info()[0] < 100 << 30:
        pytest.skip("needs 60 GB")
    x = torch.zeros(rows, 1, dtype=torch.bfloat16, device="cuda")
    tokens = torch.zeros(rows, dtype=torch.int64, device="cuda")
    entropy, g = torch.zeros(rows, device="cuda"), torch.ones(rows, device="cuda")
    stats = torch.tensor([[0.0, 2.0]], device="cuda").repeat(rows, 1)       # p = 1 / 2
    dx = dg.det_token_logprobs_backward(g, None, x, tokens, entropy, stats)
    low, high = float(dx.min()), float(dx.max())
    del x, tokens, entropy, g, stats, dx
    torch.cuda.empty_cache()
    assert low == 0.5 and high == 0.5
