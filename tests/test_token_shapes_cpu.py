"""det_token_logprobs: the tokens' shape is the logits' without the vocabulary."""
import pytest
import torch

import exact_sum_gemm_gb300 as dg


@pytest.mark.parametrize("shape", [(3, 2), (6,), (1, 6), (2, 3, 1), ()])
def test_tokens_of_another_shape_are_refused(shape):
    logits = torch.zeros(2, 3, 10)
    with pytest.raises(ValueError, match="tokens must have shape"):
        dg.det_token_logprobs(logits, torch.zeros(shape, dtype=torch.int64))


def test_logits_without_a_vocabulary_are_refused():
    with pytest.raises(ValueError, match="logits"):
        dg.det_token_logprobs(torch.zeros(()), torch.zeros((), dtype=torch.int64))
    with pytest.raises(ValueError, match="logits"):
        dg.det_token_logprobs(torch.zeros(3, 0), torch.zeros(3, dtype=torch.int64))
